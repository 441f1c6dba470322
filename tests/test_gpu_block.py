"""The operators around the Linear together, as a transformer block runs them,
and under the conditions of a serving program: captured into graphs, on several
streams at once, back to back without a wait, in place, beyond 2^31 elements.

Tolerances: an E4M3 code of y with scale s is off by half a step, 2^-4 |y|, or
s 2^-10 where the code is subnormal, and the quotient y / s by 2 ulp (1e-6 |y|);
the norm itself by far less (1e-4 (1 + |y|), see the norm's own tests).  The
Linear and the rotation are checked from their actual inputs with the bounds of
their own tests.  Everything else here is the same bits.
"""
import threading

import pytest
import torch

import int8_w8a8_quantized_b200 as tfq
from int8_w8a8_quantized_b200 import build
from test_gpu_lora import check as check_lora
from test_gpu_lora import e4m3
from test_gpu_lora import problem as lora_problem
from test_gpu_rope import check as check_rope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def norm64(x, weight, bias, offset, eps=1e-6):
    x = x.double()
    x = (x - x.mean(1, keepdim=True)) * torch.rsqrt(x.var(1, unbiased=False, keepdim=True) + eps)
    return x * (weight + offset) + bias


class Block:
    """Adaptive norm -> Q/K/V projection with adapters -> rotary positions, G samples of M / G tokens."""

    def __init__(self, M, G, K=512, H=4, D=64, R=16, n=5, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed + M)
        self.g, self.M, self.G, self.K, self.H, self.D = g, M, G, K, H, D
        N = 3 * H * D
        w = (0.05 * torch.randn((N, K), generator=g, device="cuda")).bfloat16()
        self.W_q, self.s_w = tfq.tfq_quant_weight_per_channel(w)
        self.bias = torch.randn(N, generator=g, device="cuda").bfloat16()
        self.A = (torch.randn((n, R, K), generator=g, device="cuda") / K ** 0.5).bfloat16()
        self.Bs = tfq.tfq_lora_fold(torch.randn((n, N, R), generator=g, device="cuda").bfloat16(), None, self.s_w)
        self.adapter = torch.randint(-1, n, (M,), generator=g, device="cuda", dtype=torch.int32)
        self.scale = 0.3 * torch.randn((G, K), generator=g, device="cuda")
        self.shift = 0.3 * torch.randn((G, K), generator=g, device="cuda")
        self.inv, self.axis = tfq.rope_axes_frequencies([16, 24, 24])
        self.pos = torch.randint(0, 500, (M, 3), generator=g, device="cuda", dtype=torch.int32)
        self.x = torch.empty((M, K), device="cuda", dtype=torch.bfloat16)
        self.new_input()

    def new_input(self):
        self.x.copy_(torch.randn((self.M, self.K), generator=self.g, device="cuda") * 2 + 0.5)

    def project(self):
        y = tfq.tfq_layer_norm(self.x, self.scale, self.shift, weight_offset=1.0)
        codes, s = tfq.tfq_layer_norm_quant_fp8(self.x, self.scale, self.shift, weight_offset=1.0)
        p = dict(A_q=codes, s_a=s, W_q=self.W_q, s_w=self.s_w, x=y, lora_A=self.A, lora_Bs=self.Bs,
                 adapter=self.adapter, bias=self.bias)
        return p, tfq.tfq_scaled_fp8_linear_lora(**p)

    def heads(self, qkv):
        return qkv.view(self.M, 3, self.H, self.D).unbind(1)

    def rotate(self, qkv, inverse=False):
        q, k, v = self.heads(qkv)
        tfq.tfq_rope_axes(q, k, self.pos, self.inv, self.axis, inverse=inverse, q_out=q, k_out=k)
        return q, k, v

    def run(self):
        return torch.stack([t.contiguous() for t in self.rotate(self.project()[1])])


@pytest.mark.parametrize("M,G", [(1, 1), (6, 3), (96, 2), (700, 4)])
def test_a_block(M, G):
    blk = Block(M, G)
    p, qkv = blk.project()
    y = norm64(blk.x, blk.scale.double().repeat_interleave(M // G, 0), blk.shift.double().repeat_interleave(M // G, 0), 1.0)
    s = p["s_a"].double()[:, None]
    tol = 1e-4 * (1 + y.abs())
    assert ((e4m3(p["A_q"]) * s - y).abs() <= torch.maximum(y.abs() * (2.0 ** -4 + 1e-6), s * 2.0 ** -10) + 1.1 * tol).all()
    assert ((p["x"].double() - y).abs() <= y.abs() * 2.0 ** -8 + 1.1 * tol).all()
    check_lora(p, qkv)
    before = qkv.clone()
    q, k, v = blk.rotate(qkv)
    for got, was in ((q, blk.heads(before)[0]), (k, blk.heads(before)[1])):
        check_rope(got, was, blk.pos, blk.inv, blk.axis, "interleaved", False)
    assert torch.equal(v, blk.heads(before)[2])  # in place, and nothing but queries and keys
    # the two Linears of the public surface are these calls
    a = tfq.w8a8_norm_linear(blk.x, blk.scale, blk.shift, blk.W_q, blk.s_w, blk.bias, weight_offset=1.0)
    assert torch.equal(a, tfq.tfq_scaled_fp8_linear(p["A_q"], p["s_a"], blk.W_q, blk.s_w, blk.bias))
    b = tfq.w8a8_lora_linear(p["x"], blk.W_q, blk.s_w, blk.A, blk.Bs, blk.adapter, blk.bias)
    p["A_q"], p["s_a"] = tfq.tfq_quant_act_fp8_per_token(p["x"])
    assert torch.equal(b, tfq.tfq_scaled_fp8_linear_lora(**p))


def test_training_run():
    """Gradients through rotation and norm: the inverse rotation feeds the norm's backward, against 64 bits."""
    M, H, D = 130, 3, 32
    K = H * D
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((M, K), generator=g, device="cuda")
    w, b = (torch.randn(K, generator=g, device="cuda") for _ in range(2))
    up = torch.randn((M, H, D), generator=g, device="cuda")
    pos = torch.randint(0, 90, (M, 2), generator=g, device="cuda")
    inv, axis = tfq.rope_axes_frequencies([16, 16])
    y, mean, rstd = tfq.tfq_layer_norm(x, w, b, stats=True)
    out, _ = tfq.tfq_rope_axes(y.view(M, H, D), None, pos, inv, axis)
    dy, _ = tfq.tfq_rope_axes(up, None, pos, inv, axis, inverse=True)
    dx, dw, db = tfq.tfq_layer_norm_backward(dy.reshape(M, K), x, w, mean, rstd)
    x6, w6, b6 = (t.double().requires_grad_() for t in (x, w, b))
    y6 = norm64(x6, w6, b6, 0.0).view(M, H, D)
    ang = (pos.double()[:, axis.long().cuda()] * inv.cuda())[:, None]
    a, c = y6[..., 0::2], y6[..., 1::2]
    out6 = torch.stack((a * ang.cos() - c * ang.sin(), a * ang.sin() + c * ang.cos()), -1).flatten(-2)
    out6.backward(up.double())
    # fp32 throughout: some hundred roundings of 2^-24 and the table's 4.4e-7, on sums of up to M terms of size 10
    for got, want, terms in ((out, out6, 1), (dx, x6.grad, 1), (dw, w6.grad, M), (db, b6.grad, M)):
        assert ((got.double() - want).abs() <= 1e-5 * 10 * terms).all()


@pytest.mark.parametrize("M,G", [(1, 1), (16, 2), (700, 4)])
def test_captured_and_replayed(M, G):
    blk = Block(M, G)
    dy = torch.randn((M, blk.K), generator=blk.g, device="cuda").bfloat16()

    def step():
        y, mean, rstd = tfq.tfq_layer_norm(blk.x, blk.scale, blk.shift, weight_offset=1.0, stats=True)
        return (blk.run(), y) + tfq.tfq_layer_norm_backward(dy, blk.x, blk.scale, mean, rstd, weight_offset=1.0)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs, each with workspaces of its own from its pool
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        graphs.append((graph, got))
    for i in range(4):
        blk.new_input()
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = step()
        for _, got in graphs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams_at_once():
    """Calls that overlap, each with a workspace of its own."""
    blocks = [Block(900, 3, seed=1), Block(40, 2, seed=2), Block(300, 1, seed=3)]
    want = [b.run() for b in blocks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    outs = [[] for _ in blocks]
    for _ in range(8):
        for b, s, o in zip(blocks, streams, outs):
            with torch.cuda.stream(s):
                o.append(b.run())
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, got) for got in o)


def test_stream_argument():
    """stream= (a torch stream or its handle): the call waits for that stream's work and for no other."""
    blk = Block(64, 1)
    p, want = blk.project()
    dy = torch.randn_like(blk.x)
    y, mean, rstd = tfq.tfq_layer_norm(blk.x, blk.scale[0], stats=True)
    grads = tfq.tfq_layer_norm_backward(dy, blk.x, blk.scale[0], mean, rstd)
    rot = tfq.tfq_rope_axes(blk.x.view(64, 8, 64), None, blk.pos, blk.inv, blk.axis)[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        x = torch.zeros_like(blk.x)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(10_000_000)  # the input arrives late, on that stream
            x.copy_(blk.x)
        y2, mean2, rstd2 = tfq.tfq_layer_norm(x, blk.scale[0], stats=True, stream=handle)
        codes, sa = tfq.tfq_layer_norm_quant_fp8(x, blk.scale, blk.shift, weight_offset=1.0, stream=handle)
        grads2 = tfq.tfq_layer_norm_backward(dy, x, blk.scale[0], mean2, rstd2, stream=handle)
        rot2 = tfq.tfq_rope_axes(x.view(64, 8, 64), None, blk.pos, blk.inv, blk.axis, stream=handle)[0]
        out = tfq.tfq_scaled_fp8_linear_lora(**dict(p, A_q=codes, s_a=sa), stream=handle)
        s.synchronize()
        for a, b in zip((y2, mean2, rstd2, *grads2, rot2, out), (y, mean, rstd, *grads, rot, want)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("K", [48, 512, 1536])
def test_back_to_back(K):
    """A long chain in which every call reads what the one before wrote, without
    a wait, against the same chain with a wait behind every call."""
    M = 333
    g = torch.Generator(device="cuda").manual_seed(K)
    x0 = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    w = torch.randn(K, generator=g, device="cuda").bfloat16()
    W_q, s_w = tfq.tfq_quant_weight_per_channel((torch.randn((K, K), generator=g, device="cuda") / K ** 0.5).bfloat16())
    A = (torch.randn((3, 16, K), generator=g, device="cuda") / K ** 0.5).bfloat16()
    Bs = tfq.tfq_lora_fold(torch.randn((3, K, 16), generator=g, device="cuda").bfloat16(), None, s_w)
    idx = torch.randint(-1, 3, (M,), generator=g, device="cuda", dtype=torch.int32)
    pos = torch.randint(0, 100, (M, 1), generator=g, device="cuda", dtype=torch.int32)
    inv, axis = tfq.rope_axes_frequencies([16])
    few = M // 8

    def chain(wait):
        x = x0
        for i in range(12):
            y, mean, rstd = wait(tfq.tfq_layer_norm(x, w, stats=True))
            dx, dw, db = wait(tfq.tfq_layer_norm_backward(x, y, w, mean, rstd))
            codes, s = wait(tfq.tfq_layer_norm_quant_fp8(dx, dw, db))
            rows = M if i % 2 else few  # both of the adapters' paths
            z = wait(tfq.tfq_scaled_fp8_linear_lora(codes[:rows], s[:rows], W_q, s_w, dx[:rows], A, Bs, idx[:rows]))
            z, _ = wait(tfq.tfq_rope_axes(z.view(rows, -1, 16), None, pos[:rows], inv, axis))
            x = torch.cat((z.view(rows, K), y[rows:])) if rows < M else z.view(rows, K)
        return x

    def waiting(v):
        torch.cuda.synchronize()
        return v

    want = chain(waiting)
    for _ in range(3):
        assert torch.equal(chain(lambda v: v).view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(40, 33), (500, 96), (70, 400), (300, 1001), (9, 5120), (5000, 1536), (5000, 5120),
                                 (12, 10400), (6, 20000)])
def test_norm_in_place(M, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    x = torch.randn((M, K), generator=g, device="cuda").to(dtype)
    w = torch.randn(K, generator=g, device="cuda").to(dtype)
    want = tfq.tfq_layer_norm(x, w)
    assert tfq.tfq_layer_norm(x, w, y=x) is x
    assert torch.equal(x, want)


def test_one_workspace_for_calls_in_turn():
    """Calls of one stream may share a workspace, whatever their sizes."""
    cases = [(700, 24, 4), (3, 8, 9), (130, 64, 2), (100, 16, 70)]
    ps = [lora_problem(M, 264, 272, R, n, "any", True) for M, R, n in cases]
    want = [tfq.tfq_scaled_fp8_linear_lora(**p) for p in ps]
    ws = torch.empty(max(tfq.tfq_scaled_fp8_linear_lora_workspace_bytes(M, R) for M, R, _ in cases), device="cuda",
                     dtype=torch.uint8)
    got = [[tfq.tfq_scaled_fp8_linear_lora(**p, workspace=ws) for p in ps] for _ in range(5)]
    assert all(torch.equal(a, b) for turn in got for a, b in zip(turn, want))


def test_beyond_2_31_elements():
    """The last rows of tensors past 2^31 elements, against the same rows alone."""
    M, K = 425_000, 5120
    x = torch.zeros((M, K), device="cuda", dtype=torch.bfloat16)
    tail = slice(M - 300, M)
    g = torch.Generator(device="cuda").manual_seed(9)
    x[tail] = torch.randn((300, K), generator=g, device="cuda").bfloat16()
    w = torch.randn(K, generator=g, device="cuda").bfloat16()
    y, mean, rstd = tfq.tfq_layer_norm(x, w, stats=True)
    want = tfq.tfq_layer_norm(x[tail], w)
    # another kernel takes 300 rows: a bf16 step apart at most
    assert ((y[tail].double() - want.double()).abs() <= want.double().abs() * 2.0 ** -7 + 1e-6).all()
    assert (y[:200] == 0).all()
    q, s = tfq.tfq_layer_norm_quant_fp8(x, w)
    q1, s1 = tfq.tfq_layer_norm_quant_fp8(x[tail], w)
    d, d1 = e4m3(q[tail]) * s[tail].double()[:, None], e4m3(q1) * s1.double()[:, None]
    assert ((d - d1).abs() <= d1.abs() * 2.0 ** -3 + s1.double()[:, None] * 2.0 ** -9).all()
    del q, d
    dx, dw, db = tfq.tfq_layer_norm_backward(y, x, w, mean, rstd)
    dx1, dw1, db1 = tfq.tfq_layer_norm_backward(y[tail], x[tail], w, mean[tail].contiguous(), rstd[tail].contiguous())
    assert torch.equal(dx[tail], dx1)  # a row's gradient does not depend on the others
    # sums of 300 rows (the others add zeros) in another order, then a bf16 rounding of each
    for a, b, terms in ((dw, dw1, (y[tail].double() * norm64(x[tail], 1.0, 0.0, 0.0)).abs().sum(0)),
                        (db, db1, y[tail].double().abs().sum(0))):
        assert ((a.double() - b.double()).abs() <= b.double().abs() * 2.0 ** -7 + 1e-4 * terms).all()
    del dx, y
    pos = torch.arange(M, device="cuda", dtype=torch.int32)[:, None]
    inv, axis = tfq.rope_axes_frequencies([128])
    out, _ = tfq.tfq_rope_axes(x.view(M, 40, 128), None, pos, inv, axis)
    want, _ = tfq.tfq_rope_axes(x[tail].view(300, 40, 128), None, pos[tail], inv, axis)
    assert torch.equal(out[tail], want)
    del out
    # adapters: x past 2^31 elements, rows of one adapter at the end
    W_q, s_w = tfq.tfq_quant_weight_per_channel(torch.randn((8, K), generator=g, device="cuda").bfloat16())
    A = (torch.randn((2, 8, K), generator=g, device="cuda") / K ** 0.5).bfloat16()
    Bs = tfq.tfq_lora_fold(torch.randn((2, 8, 8), generator=g, device="cuda").bfloat16(), None, s_w)
    idx = torch.zeros(M, device="cuda", dtype=torch.int32)
    idx[tail] = torch.randint(-1, 2, (300,), generator=g, device="cuda", dtype=torch.int32)
    A_q, s_a = tfq.tfq_quant_act_fp8_per_token(x)
    y = tfq.tfq_scaled_fp8_linear_lora(A_q, s_a, W_q, s_w, x, A, Bs, idx)
    check_lora(dict(A_q=A_q[tail], s_a=s_a[tail], W_q=W_q, s_w=s_w, x=x[tail], lora_A=A, lora_Bs=Bs, adapter=idx[tail],
                    bias=None), y[tail])


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("K,N", [(8192, 64), (64, 8192)])
def test_factors_beyond_2_31_elements(M, K, N):
    n, R = 4200, 64
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    A_q, s_a = tfq.tfq_quant_act_fp8_per_token(x)
    W_q, s_w = tfq.tfq_quant_weight_per_channel((torch.randn((N, K), generator=g, device="cuda") / K ** 0.5).bfloat16())
    A = torch.empty((n, R, K), device="cuda", dtype=torch.bfloat16).normal_(0, K ** -0.5, generator=g)
    B = torch.empty((n, N, R), device="cuda", dtype=torch.bfloat16).normal_(0, 1, generator=g)
    Bs = tfq.tfq_lora_fold(B, None, s_w, out=B)
    idx = torch.tensor([n - 1, 4100, 0, -1, n - 2], device="cuda", dtype=torch.int32).repeat(M // 5)
    y = tfq.tfq_scaled_fp8_linear_lora(A_q, s_a, W_q, s_w, x, A, Bs, idx)
    check_lora(dict(A_q=A_q, s_a=s_a, W_q=W_q, s_w=s_w, x=x, lora_A=A, lora_Bs=Bs, adapter=idx, bias=None), y)


def test_fold_never_stores_inf_or_nan():
    B = torch.tensor([[[float("inf")] * 8, [float("-inf")] * 8, [float("nan")] * 8, [1e30] * 8, [-1e30] * 8, [0.0] * 8,
                       [2.0] * 8, [-0.5] * 8]], device="cuda").bfloat16()
    Bs = tfq.tfq_lora_fold(B, torch.tensor([3.0], device="cuda"), torch.full((8,), 1e-20, device="cuda"))
    big = torch.finfo(torch.bfloat16).max
    want = torch.tensor([big, -big, big, big, -big, 0.0, 6e20, -1.5e20], device="cuda")
    assert torch.equal(Bs[0], want.bfloat16()[:, None].expand(8, 8))


@pytest.mark.parametrize("M,K", [(7, 96), (60, 1001), (33, 1536), (5000, 1536), (3, 20000)])
def test_bias_without_weight(M, K):
    """A missing weight multiplies by 1, whatever its offset; groups come from the bias."""
    g = torch.Generator(device="cuda").manual_seed(K)
    G = 3 if M % 3 == 0 else 1
    x = torch.randn((M, K), generator=g, device="cuda")
    b = torch.randn((G, K), generator=g, device="cuda")
    y = tfq.tfq_layer_norm(x, None, b, weight_offset=5.0)
    want = tfq.tfq_layer_norm(x, torch.ones_like(b), b)
    assert torch.equal(y, want)
    if K % 16 == 0:
        q, s = tfq.tfq_layer_norm_quant_fp8(x, None, b, weight_offset=5.0)
        q1, s1 = tfq.tfq_layer_norm_quant_fp8(x, torch.ones_like(b), b)
        assert torch.equal(q, q1) and torch.equal(s, s1)


def test_refusals_on_the_gpu():
    x = torch.zeros((4, 32), device="cuda")
    w = torch.zeros(32, device="cuda")
    with pytest.raises(TypeError):
        tfq.tfq_layer_norm(x, 1.0)
    with pytest.raises(ValueError):
        tfq.tfq_layer_norm(x, w[:16])
    with pytest.raises(ValueError):
        tfq.tfq_layer_norm(x, w, stream=torch.cuda.current_stream(), y=x[:2])
    with pytest.raises(ValueError):
        tfq.tfq_layer_norm(x.cpu(), w)
    with pytest.raises(ValueError):
        tfq.tfq_layer_norm(x, w.cpu())


@pytest.mark.parametrize("M", [30, 300, 700])
@pytest.mark.parametrize("N,K,R", [(8, 16, 8), (264, 16, 64), (8, 144, 24), (24, 48, 256)])
def test_adapters_at_the_smallest_sizes(M, N, K, R):
    p = lora_problem(M, N, K, R, 3, "any", True)
    check_lora(p, tfq.tfq_scaled_fp8_linear_lora(**p))


def test_host_threads_at_once():
    """Calls from several host threads, a stream each."""
    blocks = [Block(m, 1, seed=m) for m in (700, 33, 300, 1)]
    want = [b.run() for b in blocks]
    torch.cuda.synchronize()
    outs = [[] for _ in blocks]

    def work(b, o):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                o.append(b.run())
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(b, o)) for b, o in zip(blocks, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for w, o in zip(want, outs):
        assert len(o) == 10 and all(torch.equal(w, got) for got in o)


def test_stream_zero_is_the_default_stream():
    """stream=0: behind the default stream's work, and in front of what it gets next."""
    blk = Block(64, 1)
    want = tfq.tfq_layer_norm(blk.x, blk.scale[0])
    x = torch.zeros_like(blk.x)
    torch.cuda.synchronize()
    torch.cuda._sleep(10_000_000)
    x.copy_(blk.x)  # late
    with torch.cuda.stream(torch.cuda.Stream()):
        y = tfq.tfq_layer_norm(x, blk.scale[0], stream=0)
    x.zero_()
    got = y.clone()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("call", ["lora", "norm"])
def test_linears_keep_their_codes_on_the_stream_argument(call, monkeypatch):
    """stream=: the codes between the two kernels are allocated and freed on that
    stream, so that no other stream gets their memory while the GEMM still reads it."""
    from int8_w8a8_quantized_b200 import _block

    blk = Block(64, 1)
    p, _ = blk.project()
    name = "tfq_quant_act_fp8_per_token" if call == "lora" else "tfq_layer_norm_quant_fp8"
    quantize, seen = getattr(_block, name), []

    def spied(*args, **kwargs):
        codes, s = quantize(*args, **kwargs)
        seen.append((codes.data_ptr(), torch.cuda.current_stream()))
        return codes, s

    monkeypatch.setattr(_block, name, spied)

    def run(stream=None):
        if call == "lora":
            return _block.w8a8_lora_linear(p["x"], blk.W_q, blk.s_w, blk.A, blk.Bs, blk.adapter, blk.bias, stream=stream)
        return _block.w8a8_norm_linear(blk.x, blk.scale, blk.shift, blk.W_q, blk.s_w, blk.bias, weight_offset=1.0,
                                       stream=stream)

    want = run()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (s, s.cuda_stream):
        with torch.cuda.stream(s):
            torch.cuda._sleep(10_000_000)
        got = run(handle)
        at, stream = seen[-1]
        assert stream.cuda_stream == s.cuda_stream
        taken = [torch.full((64, 512), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert at not in [t.data_ptr() for t in taken]
        s.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("call", ["fp8", "int8", "mxfp8", "one call"])
def test_plain_linears_keep_their_buffers_on_the_stream_argument(call, monkeypatch):
    """The same for the Linears without adapters or norm: codes and workspaces belong to stream=."""
    from int8_w8a8_quantized_b200 import _capi

    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((600, 512), generator=g, device="cuda").bfloat16()
    w = torch.randn((264, 512), generator=g, device="cuda").bfloat16()
    fp8, i8, mx = tfq.tfq_quant_weight_per_channel(w), tfq.tfq_quant_weight_per_channel(w, "int8"), tfq.tfq_quant_mxfp8(w)
    run, kernel = {"fp8": (lambda s=None: tfq.w8a8_linear(x, *fp8, stream=s), "tfq_quant_act_fp8_per_token"),
                   "int8": (lambda s=None: tfq.w8a8_int8_linear(x, *i8, stream=s), "tfq_quant_act_int8_per_token"),
                   "mxfp8": (lambda s=None: tfq.mxfp8_linear(x, *mx, stream=s), "tfq_quant_mxfp8"),
                   "one call": (lambda s=None: tfq.tfq_quant_scaled_fp8_linear(x, *fp8, stream=s)[0],
                                "tfq_quant_scaled_fp8_linear")}[call]
    want = run()
    enter, seen = getattr(_capi.load_library(), kernel), []

    def spied(*args):
        seen.append((torch.cuda.current_stream().cuda_stream, args[-1]))
        return enter(*args)

    monkeypatch.setattr(_capi.raw, kernel, spied, raising=False)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream, handle in ((s, s.cuda_stream), (s.cuda_stream, s.cuda_stream), (0, 0)):
        got = run(stream)
        assert seen[-1] == (handle, handle)  # where the buffers are allocated, and where the kernel runs
        torch.cuda.synchronize()
        assert torch.equal(got, want)
