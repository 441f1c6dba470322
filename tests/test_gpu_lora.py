"""The scaled FP8 Linear with low-rank adapters on the GPU, against the formula
in 64 bits (the codes' exact products, lora_Bs as the call is given it).

Tolerance: that of the scaled GEMM (2^-7 |y| + 1e-3 rms(y)), which covers the
fp32 sum over K and the output's rounding, plus the adapters': the rank-R
intermediate is rounded to bf16 (half a step: 2^-8 relative) and carries the
rounding of an fp32 sum of K products (K 2^-24 of the sum of their magnitudes).
"""
import pytest
import torch

import int8_w8a8_quantized_b200 as tfq
from int8_w8a8_quantized_b200 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def problem(M, N, K, R, n, order, bias, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + M + N + K + R)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    w = (0.05 * torch.randn((N, K), generator=g, device="cuda")).bfloat16()
    A_q, s_a = tfq.tfq_quant_act_fp8_per_token(x)
    W_q, s_w = tfq.tfq_quant_weight_per_channel(w)
    A = (torch.randn((n, R, K), generator=g, device="cuda") / K ** 0.5).bfloat16()
    B = torch.randn((n, N, R), generator=g, device="cuda").bfloat16()
    scaling = torch.rand(n, generator=g, device="cuda") + 0.5
    if order == "runs":
        idx = torch.sort(torch.randint(-1, n, (M,), generator=g, device="cuda")).values
    elif order == "any":
        idx = torch.randint(-1, n, (M,), generator=g, device="cuda")
    elif order == "none":
        idx = torch.full((M,), -1, device="cuda")
    elif order == "wild":  # values outside [0, n) mean no adapter
        idx = torch.randint(-3, n + 3, (M,), generator=g, device="cuda")
        idx[::5], idx[1::7] = -2 ** 31, 2 ** 31 - 1
    else:
        idx = torch.full((M,), n - 1, device="cuda")
    b = torch.randn(N, generator=g, device="cuda").bfloat16() if bias else None
    return dict(A_q=A_q, s_a=s_a, W_q=W_q, s_w=s_w, x=x, lora_A=A, lora_Bs=tfq.tfq_lora_fold(B, scaling, s_w),
                adapter=idx.to(torch.int32), bias=b)


def e4m3(q):
    return q.view(torch.float8_e4m3fn).double()


def check(p, y):
    base = (e4m3(p["A_q"]) * p["s_a"].double()[:, None]) @ (e4m3(p["W_q"]) * p["s_w"].double()[:, None]).t()
    if p["bias"] is not None:
        base = base + p["bias"].double()
    n, K = p["lora_A"].shape[0], p["x"].shape[1]
    ref, tol = base.clone(), torch.zeros_like(base)
    for a in range(n):
        rows = torch.nonzero(p["adapter"] == a).flatten()
        if rows.numel() == 0:
            continue
        x, A = p["x"][rows].double(), p["lora_A"][a].double()
        B = p["lora_Bs"][a].double() * p["s_w"].double()[:, None]
        t = x @ A.t()
        ref[rows] += t @ B.t()
        tol[rows] = (t.abs() * 2.0 ** -8 + (K * 2.0 ** -24) * (x.abs() @ A.abs().t())) @ B.abs().t() * 1.01
    tol += 2.0 ** -7 * ref.abs() + 1e-3 * ref.square().mean().sqrt()
    err = (y.double() - ref).abs()
    assert torch.isfinite(y).all()
    assert (err <= tol).all(), f"worst error / tolerance {float((err / tol).max()):.3f}"


CASES = [  # M, N, K, R, adapters
    (1, 8, 16, 8, 1), (1, 5120, 5120, 16, 3), (2, 136, 144, 24, 2), (7, 264, 1040, 32, 7), (16, 512, 256, 64, 40),
    (64, 1024, 2064, 16, 64), (65, 1000, 528, 40, 5), (128, 256, 512, 128, 3), (129, 264, 272, 8, 200),
    (300, 520, 1024, 256, 4), (511, 328, 784, 72, 6), (512, 256, 512, 64, 2), (600, 1032, 528, 16, 9),
    (1025, 776, 2064, 64, 33), (2500, 520, 1040, 200, 5), (4111, 264, 272, 24, 100),
    (9000, 2056, 272, 24, 6), (5000, 4104, 784, 72, 3), (33, 24, 16, 8, 2), (48, 13824, 512, 256, 5),
    (1300, 64, 144, 8, 1000), (70, 72, 4096, 256, 3), (513, 328, 2064, 248, 70),
    (700, 264, 528, 32, 9), (1025, 520, 272, 8, 33), (100, 1032, 784, 64, 20), (128, 264, 528, 24, 30),
    (3000, 2056, 528, 16, 3), (129, 264, 144, 48, 9),
]


@pytest.mark.parametrize("order", ["runs", "any", "one"])
@pytest.mark.parametrize("M,N,K,R,n", CASES)
def test_lora(M, N, K, R, n, order):
    p = problem(M, N, K, R, n, order, bias=bool(M % 2))
    out = torch.full((M * N + 64,), 3.0, device="cuda", dtype=torch.bfloat16)
    y = tfq.tfq_scaled_fp8_linear_lora(**p, out=out[:M * N].view(M, N))
    tfq.tfq_device_error()
    assert (out[M * N:] == 3).all()
    check(p, y)


@pytest.mark.parametrize("M", [5, 200, 700])
def test_rows_without_an_adapter(M):
    """No adapter: the plain Linear's value; indexes outside [0, n) of any size read nothing."""
    p = problem(M, 264, 272, 16, 3, "none", True)
    y = tfq.tfq_scaled_fp8_linear_lora(**p)
    check(p, y)
    p = problem(M, 264, 272, 16, 3, "wild", True)
    check(p, tfq.tfq_scaled_fp8_linear_lora(**p))


def test_no_adapters_is_the_plain_linear():
    p = problem(300, 264, 272, 16, 3, "any", True)
    want = tfq.tfq_scaled_fp8_linear(p["A_q"], p["s_a"], p["W_q"], p["s_w"], p["bias"])
    p["lora_A"], p["lora_Bs"] = p["lora_A"][:0], p["lora_Bs"][:0]
    assert torch.equal(tfq.tfq_scaled_fp8_linear_lora(**p), want)


def test_stale_workspace_and_rows_of_other_calls():
    """The workspace's contents mean nothing: NaN everywhere before the call, and the same bits after."""
    for M in (3, 130, 777):
        p = problem(M, 264, 528, 24, 4, "any", False)
        n = tfq.tfq_scaled_fp8_linear_lora_workspace_bytes(M, 24)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        y = tfq.tfq_scaled_fp8_linear_lora(**p, workspace=ws)
        check(p, y)
        again = tfq.tfq_scaled_fp8_linear_lora(**p, workspace=ws)
        assert torch.equal(y, again)


def test_zero_rows_and_channels():
    """All-zero activations (scale at its floor) and all-zero weight channels: only bias and adapters are left."""
    p = problem(140, 264, 272, 16, 2, "one", True)
    x = p["x"].clone()
    x[::3] = 0
    p["x"] = x
    p["A_q"], p["s_a"] = tfq.tfq_quant_act_fp8_per_token(x)
    y = tfq.tfq_scaled_fp8_linear_lora(**p)
    check(p, y)
    assert torch.equal(y[0], p["bias"])


def test_fold():
    g = torch.Generator(device="cuda").manual_seed(0)
    for n, N, R in ((1, 1, 1), (3, 40, 7), (5, 264, 64)):
        B = torch.randn((n, N, R), generator=g, device="cuda").bfloat16()
        s = torch.rand(n, generator=g, device="cuda") + 0.5
        w = torch.rand(N, generator=g, device="cuda") * 1e-3 + 1e-5
        got = tfq.tfq_lora_fold(B, s, w)
        want = ((B.float() * s[:, None, None]) / w[None, :, None]).bfloat16()
        assert torch.equal(got, want)
        assert torch.equal(tfq.tfq_lora_fold(B, None, w), (B.float() / w[None, :, None]).bfloat16())
        tfq.tfq_lora_fold(B, s, w, out=B)
        assert torch.equal(B, want)


def test_refused_calls():
    p = problem(4, 16, 32, 8, 2, "any", False)
    for k, v in (("x", p["x"].float()), ("x", p["x"][:3]), ("lora_A", p["lora_A"][:, :, :16]),
                 ("lora_Bs", p["lora_Bs"][:1]), ("adapter", p["adapter"].long()), ("adapter", p["adapter"][:2]),
                 ("s_a", p["s_a"].cpu()), ("A_q", p["A_q"].to(torch.int8))):
        with pytest.raises((TypeError, ValueError)):
            tfq.tfq_scaled_fp8_linear_lora(**{**p, k: v})
    with pytest.raises(ValueError, match="workspace"):
        tfq.tfq_scaled_fp8_linear_lora(**p, workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))
    p = problem(4, 16, 32, 16, 2, "any", False)
    with pytest.raises(tfq.TfqError):
        tfq.tfq_scaled_fp8_linear_lora(**{**p, "lora_A": p["lora_A"][:, :12].contiguous(),
                                          "lora_Bs": p["lora_Bs"][..., :12].contiguous()})


@pytest.mark.parametrize("M", [20, 200, 600])
def test_a_broken_adapter_stays_with_its_own_rows(M):
    """An adapter folded from NaN and inf: rows of other adapters in the same tile keep their values."""
    p = problem(M, 264, 528, 16, 4, "any", False)
    clean = tfq.tfq_scaled_fp8_linear_lora(**p)
    B = torch.randn(4, 264, 16, device="cuda").bfloat16()
    B[2, ::3], B[2, 1::3] = float("nan"), float("inf")
    bad = p["lora_Bs"].clone()
    bad[2] = tfq.tfq_lora_fold(B, None, p["s_w"])[2]
    assert torch.isfinite(bad).all()
    y = tfq.tfq_scaled_fp8_linear_lora(**{**p, "lora_Bs": bad})
    others = p["adapter"] != 2
    assert torch.equal(y[others], clean[others])
    x = p["x"].clone()
    x[7, 3] = float("nan")  # a row's own NaN stays in that row
    y = tfq.tfq_scaled_fp8_linear_lora(**{**p, "x": x})
    rows = torch.arange(M, device="cuda") != 7
    assert torch.equal(y[rows], clean[rows])


def bare_rows(M, n, order):
    """Rows without an adapter (-1) between the others': of M rows, n adapters."""
    i = torch.arange(M, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(M + n)
    some = torch.rand(M, generator=g, device="cuda")
    if order == "every second":
        idx = torch.where(i % 2 == 0, i * n // M, -1)
    elif order == "some":
        idx = torch.where(some < 0.9, i * n // M, -1)
    elif order == "single":  # runs cut by single rows
        idx = torch.where(some < 0.98, i * n // M, -1)
    elif order == "falling":  # the adapters decrease, a bare row in front of each change
        idx = n - 1 - i * n // M
        idx[1:][idx[1:] != idx[:-1]] = -1
    else:  # decreasing and increasing in turn, bare rows in front of every decrease
        idx = torch.where(i % 4 == 3, -1, (i % 4) * (n - 1) // 2)
    return idx.to(torch.int32)


@pytest.mark.parametrize("order", ["every second", "some", "single", "falling", "saw"])
@pytest.mark.parametrize("M,n,R", [(140, 1, 16), (140, 3, 64), (513, 1, 64), (700, 2, 24), (2500, 1, 8), (2500, 5, 128),
                                   (1300, 1100, 16)])
def test_rows_without_an_adapter_between_others(M, n, R, order):
    p = problem(M, 264, 528, R, n, "one", True)
    p["adapter"] = bare_rows(M, n, order)
    check(p, tfq.tfq_scaled_fp8_linear_lora(**p))


@pytest.mark.parametrize("order", ["every second", "some"])
@pytest.mark.parametrize("M", [256, 9472])
def test_rows_without_an_adapter_do_not_cut_the_others_apart(M, order):
    """Rows without an adapter scattered among the rows of one: the call takes at most twice as long
    as with the adapter on every row (it took 4 to 17 times as long when each of them began an item)."""
    p = problem(M, 1024, 5120, 64, 1, "one", False)
    whole = p["adapter"]

    def us(adapter):
        out = torch.empty((M, 1024), dtype=torch.bfloat16, device="cuda")
        best = float("inf")
        for _ in range(5):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            for _ in range(10):
                tfq.tfq_scaled_fp8_linear_lora(**{**p, "adapter": adapter}, out=out)
            end.record()
            end.synchronize()
            best = min(best, start.elapsed_time(end) * 100)
        return best

    us(whole)  # warm
    assert us(bare_rows(M, 1, order)) <= 2 * us(whole)


@pytest.mark.parametrize("M", [20, 100, 140, 700])
def test_zero_channels(M):
    """All-zero weight channels (scale at its floor, so that lora_Bs is some 1e15 there) and all-zero rows: the
    channels hold bias and adapters, the rows the bias alone."""
    p = problem(M, 264, 272, 16, 3, "any", True)
    g = torch.Generator(device="cuda").manual_seed(M)
    w = (0.05 * torch.randn((264, 272), generator=g, device="cuda")).bfloat16()
    w[::5] = 0
    p["W_q"], p["s_w"] = tfq.tfq_quant_weight_per_channel(w)
    assert (p["s_w"][::5] < 1e-14).all()
    p["lora_Bs"] = tfq.tfq_lora_fold(torch.randn((3, 264, 16), generator=g, device="cuda").bfloat16(), None, p["s_w"])
    x = p["x"].clone()
    x[::3] = 0
    p["x"] = x
    p["A_q"], p["s_a"] = tfq.tfq_quant_act_fp8_per_token(x)
    y = tfq.tfq_scaled_fp8_linear_lora(**p)
    check(p, y)
    assert torch.equal(y[::3], p["bias"].expand(len(range(0, M, 3)), -1))
    bare = p["adapter"] < 0
    assert torch.equal(y[bare][:, ::5], p["bias"][::5].expand(int(bare.sum()), -1))


@pytest.mark.parametrize("M", [9, 300])
def test_ranks_padded_with_zeros(M):
    """Adapters of ranks 4, 8 and 12 as rank 16: zeros behind their own rows of both factors."""
    p = problem(M, 264, 272, 16, 3, "any", True)
    for a, rank in enumerate((4, 8, 12)):
        p["lora_A"][a, rank:] = 0
        p["lora_Bs"][a, :, rank:] = 0
    y = tfq.tfq_scaled_fp8_linear_lora(**p)
    check(p, y)
    junk = {**p, "lora_Bs": p["lora_Bs"].clone()}
    for a, rank in enumerate((4, 8, 12)):  # the first factor's zeros alone are enough
        junk["lora_Bs"][a, :, rank:] = 7.0
    assert torch.equal(tfq.tfq_scaled_fp8_linear_lora(**junk), y)


@pytest.mark.parametrize("M,K,R,order", [(40, 64, 16, "any"), (200, 64, 16, "one"), (300, 64, 8, "any"), (300, 512, 24, "any"),
                                         (300, 64, 64, "runs"), (2500, 128, 16, "any"), (2500, 512, 72, "runs"),
                                         (600, 64, 256, "any"), (5000, 16, 32, "any"), (40000, 48, 40, "runs")])
def test_the_first_product_keeps_16_bits_for_a_short_sum(M, K, R, order):
    """Adapters alone (all weight codes 0, s_w 1), K up to 512: the output is off by half a bf16 step and
        |Bs| (2^-17 |t| + 2 K 2^-24 |x| |A| + 4 R 2^-24 |t|),
    the lower half's rounding (2^-18) and two fp32 sums whose additions are off by a whole step at most.
    (t in bf16 alone would be off by 2^-9 of every term.)"""
    N, n = 264, 3
    p = problem(M, N, K, R, n, order, False)
    g = torch.Generator(device="cuda").manual_seed(R)
    p["W_q"], p["s_w"] = torch.zeros_like(p["W_q"]), torch.ones_like(p["s_w"])
    p["lora_Bs"] = torch.randn((n, N, R), generator=g, device="cuda").bfloat16()
    y = tfq.tfq_scaled_fp8_linear_lora(**p).double()
    tfq.tfq_device_error()
    for a in range(-1, n):
        rows = torch.nonzero(p["adapter"] == a).flatten()
        if a < 0:
            assert (y[rows] == 0).all()
            continue
        x, A, B = p["x"][rows].double(), p["lora_A"][a].double(), p["lora_Bs"][a].double()
        t = x @ A.t()
        want = t @ B.t()
        tol = ((2.0 ** -17 + 4 * R * 2.0 ** -24) * t.abs() + 2 * K * 2.0 ** -24 * (x.abs() @ A.abs().t())) @ B.abs().t()
        assert ((y[rows] - want).abs() <= tol + (want.abs() + tol) * 2.0 ** -8).all()


@pytest.mark.parametrize("M,n,order", [(100, 60, "any"), (300, 3, "runs"), (2000, 3, "one"), (2000, 64, "any")])
def test_the_error_against_a_32_bit_form(M, n, order):
    """Adapters alone, folded: the output's rounding and that of lora_Bs have the same rms, so the error is
    sqrt(2) times that of the products in 32 bits, rounded once (1.02: their sampling).  A bf16 t would make it
    sqrt(3) times."""
    N, K, R = 2000, 64, 32
    p = problem(M, N, K, R, n, order, False)
    g = torch.Generator(device="cuda").manual_seed(n)
    B = torch.randn((n, N, R), generator=g, device="cuda").bfloat16()
    scaling = torch.rand(n, generator=g, device="cuda") + 0.5
    p["W_q"], p["s_w"] = torch.zeros_like(p["W_q"]), torch.rand(N, generator=g, device="cuda") + 0.5
    p["lora_Bs"] = tfq.tfq_lora_fold(B, scaling, p["s_w"])
    want = torch.zeros((M, N), dtype=torch.float64, device="cuda")
    for a in range(n):
        rows = torch.nonzero(p["adapter"] == a).flatten()
        want[rows] = (p["x"][rows].double() @ p["lora_A"][a].double().t() @ B[a].double().t()) * float(scaling[a])
    error = lambda y: float((y.double() - want).norm())  # noqa: E731
    assert error(tfq.tfq_scaled_fp8_linear_lora(**p)) <= 1.02 * 2 ** 0.5 * error(want.float().bfloat16())
