"""Rotary positions with several axes on the GPU, against the formula in 64 bits.

Tolerance.  The angle's fraction of a turn is rounded to fp32 (2^-25 of a turn
at most, 1.9e-7 rad) and sincospi is good to 2 ulp (2.4e-7 at 1): the table is
off by at most 4.4e-7.  The rotation adds 2 roundings of each product and the
output half a step of its type:
    |err| <= (|a| + |b|) (4.4e-7 + 2 * 2^-24) + half_step(out).
"""
import math

import pytest
import torch

import int8_w8a8_quantized_b200 as tfq
from int8_w8a8_quantized_b200 import build

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def half_step(v, dtype):
    return v.abs() * (torch.finfo(dtype).eps / 2) + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -150)


def check(out, x, pos, inv, axis, pairing, inverse):
    P = inv.shape[0]
    ang = pos.double().cuda()[:, axis.long().cuda()] * inv.cuda()
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None] * (-1 if inverse else 1)
    f = x.double()
    first, second = ((slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if pairing == "interleaved"
                     else (slice(0, P), slice(P, 2 * P)))
    a, b = f[..., first], f[..., second]
    tol = (a.abs() + b.abs()) * (4.4e-7 + 2 * 2.0 ** -24)
    for got, want in ((out[..., first], a * c - b * s), (out[..., second], a * s + b * c)):
        assert ((got.double() - want).abs() <= tol + half_step(want.abs() + tol, out.dtype)).all()
    assert torch.equal(out[..., 2 * P:], x[..., 2 * P:])


CASES = [  # M, H, Hk, D, dims
    (1, 1, 1, 2, (2,)), (3, 2, 1, 8, (4, 4)), (7, 16, 2, 80, (16, 24, 24)), (33, 40, 40, 128, (44, 42, 42)),
    (130, 28, 4, 128, (32, 48, 48)), (5, 3, 3, 96, (96,)), (65, 8, 8, 256, (64, 64, 64, 64)), (9, 4, 1, 72, (10, 14, 6)),
    (1000, 1, 1, 16, (4, 4, 4)), (2, 300, 7, 64, (16, 24, 24)), (4, 5, 0, 7, (2, 4)), (513, 2, 2, 32, (8, 0, 16)),
]


@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,H,Hk,D,dims", CASES)
def test_rope(M, H, Hk, D, dims, dtype, pairing):
    g = torch.Generator(device="cuda").manual_seed(M + H + D)
    big = torch.randn((M, H + 2 * Hk, D), generator=g, device="cuda").to(DT[dtype])
    q, k = big[:, :H], big[:, H:H + Hk] if Hk else None
    pos = torch.randint(-1000, 1 << 20, (M, len(dims)), generator=g, device="cuda")
    pos = pos if M % 2 else pos.to(torch.int32)
    inv, axis = tfq.rope_axes_frequencies(dims, ladder="axis" if D % 3 else "shared")
    inverse = bool(M % 3 == 0)
    before = big.clone()
    qo, ko = tfq.tfq_rope_axes(q, k, pos, inv, axis, pairing=pairing, inverse=inverse)
    tfq.tfq_device_error()
    assert torch.equal(big, before)
    check(qo, q, pos, inv, axis, pairing, inverse)
    if Hk:
        check(ko, k, pos, inv, axis, pairing, inverse)
    # in place, inside the fused buffer: the same bits, the values behind the keys left as they were
    tfq.tfq_rope_axes(q, k, pos, inv, axis, pairing=pairing, inverse=inverse, q_out=q, k_out=k)
    assert torch.equal(q, qo)
    if Hk:
        assert torch.equal(k, ko)
        assert torch.equal(big[:, H + Hk:], before[:, H + Hk:])


@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
def test_layouts_and_guards(pairing):
    """[heads, tokens, D] storage, odd strides, transposed positions; nothing behind the outputs is written."""
    M, H, D = 19, 6, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    inv, axis = tfq.rope_axes_frequencies((16, 24, 24))
    pos = torch.randint(0, 500, (3, M), generator=g, device="cuda", dtype=torch.int32).t()
    for make in (lambda: torch.randn((H, M, D), generator=g, device="cuda").transpose(0, 1),
                 lambda: torch.randn((M, H, D + 3), generator=g, device="cuda")[..., :D],
                 lambda: torch.randn((M, H, D + 1), generator=g, device="cuda").bfloat16()[..., 1:],
                 lambda: torch.randn((M, 1, D), generator=g, device="cuda").expand(M, H, D)):
        q = make()
        out = torch.full((M, H + 1, D + 8), 5.0, device="cuda", dtype=q.dtype)
        qo, ko = tfq.tfq_rope_axes(q, None, pos, inv, axis, pairing=pairing, q_out=out[:, :H, :D])
        assert ko is None
        check(qo, q, pos, inv, axis, pairing, False)
        assert (out[:, H:] == 5).all() and (out[..., D:] == 5).all()


def test_inverse_is_the_gradient():
    """<R q, d> = <q, R^-1 d>, and the inverse undoes the rotation."""
    g = torch.Generator(device="cuda").manual_seed(1)
    q, d = (torch.randn((50, 4, 128), generator=g, device="cuda") for _ in range(2))
    pos = torch.randint(0, 100000, (50, 3), generator=g, device="cuda")
    inv, axis = tfq.rope_axes_frequencies((44, 42, 42))
    r, _ = tfq.tfq_rope_axes(q, None, pos, inv, axis)
    back, _ = tfq.tfq_rope_axes(r, None, pos, inv, axis, inverse=True)
    dq, _ = tfq.tfq_rope_axes(d, None, pos, inv, axis, inverse=True)
    assert ((back - q).abs() <= 3e-6 * (1 + q.abs().amax())).all()
    lhs, rhs = (r.double() * d.double()).sum((1, 2)), (q.double() * dq.double()).sum((1, 2))
    scale = q.double().norm(dim=(1, 2)) * d.double().norm(dim=(1, 2))
    assert ((lhs - rhs).abs() <= 4e-6 * scale).all()


def test_far_positions():
    """Positions where an fp32 angle has no fraction left."""
    pos = torch.tensor([[0], [1], [2 ** 24 + 1], [2 ** 31 - 1], [-2 ** 31], [10 ** 12 + 7]], device="cuda")
    inv, axis = tfq.rope_axes_frequencies((64,))
    q = torch.randn((6, 2, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(0))
    out, _ = tfq.tfq_rope_axes(q, None, pos, inv, axis)
    # both sides form pos * inv_freq in 64 bits: 2^-53 of 10^12 rad twice is 2.2e-4 rad, at the last row only
    check(out[:5], q[:5], pos[:5], inv, axis, "interleaved", False)
    assert math.isfinite(float(out.abs().sum()))
    assert ((out.norm(dim=2) - q.norm(dim=2)).abs() <= 1e-5).all()


def test_position_offsets_past_32_bits():
    """A row stride that takes the last rows past 2^31 elements."""
    M, D = 5, 64
    stride = (1 << 29) + 64
    buf = torch.empty((M - 1) * stride + 2 * D, device="cuda", dtype=torch.bfloat16)
    q = buf.as_strided((M, 2, D), (stride, D, 1))
    q.copy_(torch.randn((M, 2, D), device="cuda"))
    pos = torch.arange(M, device="cuda")[:, None].to(torch.int32)
    inv, axis = tfq.rope_axes_frequencies((D,))
    out, _ = tfq.tfq_rope_axes(q, None, pos, inv, axis)
    check(out, q, pos, inv, axis, "interleaved", False)


def test_refused_calls():
    q = torch.zeros(4, 2, 16, device="cuda")
    inv, axis = tfq.rope_axes_frequencies((8, 8))
    pos = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    for args in ((q, q.half(), pos, inv, axis), (q, None, pos.float(), inv, axis), (q, None, pos[:3], inv, axis),
                 (q, None, pos, inv.float(), axis), (q, None, pos, inv.cuda(), axis), (q, None, pos, inv, axis[:3]),
                 (q[0], None, pos, inv, axis), (q, q[:, :, :8], pos, inv, axis), (q.double(), None, pos, inv, axis),
                 (q.transpose(1, 2), None, pos, inv, axis)):
        with pytest.raises((TypeError, ValueError)):
            tfq.tfq_rope_axes(*args)
    with pytest.raises(ValueError):
        tfq.tfq_rope_axes(q, None, pos, inv, axis, pairing="other")
    with pytest.raises(ValueError, match="overlap"):
        tfq.tfq_rope_axes(q, None, pos, inv, axis, q_out=q[:1].expand(4, 2, 16))
    with pytest.raises(tfq.TfqError):
        tfq.tfq_rope_axes(q, None, pos[:, :1], inv, axis)  # an axis without a position
    with pytest.raises(tfq.TfqError):
        tfq.tfq_rope_axes(q[..., :8].contiguous(), None, pos, inv, axis)  # more pairs than the head has
    assert tfq.tfq_rope_axes(q[:0], None, pos[:0], inv, axis)[0].shape == (0, 2, 16)


@pytest.mark.parametrize("M", [1, 2, 147, 593, 1183, 1185, 2369, 4737])
@pytest.mark.parametrize("H,D,rot", [(3, 32, 4), (5, 256, 2), (1, 8, 8), (40, 64, 64)])
def test_tokens_dealt_to_the_ctas(M, H, D, rot):
    """Token counts around whole numbers of CTAs per SM, with few pairs and many."""
    g = torch.Generator(device="cuda").manual_seed(M + D)
    x = torch.randn((M, H, D), generator=g, device="cuda").bfloat16()
    pos = torch.randint(-50, 5000, (M, 1), generator=g, device="cuda")
    inv, axis = tfq.rope_axes_frequencies([rot])
    for pairing in ("interleaved", "halves"):
        out, _ = tfq.tfq_rope_axes(x, None, pos, inv, axis, pairing=pairing)
        check(out, x, pos, inv, axis, pairing, False)


def test_few_pairs_use_the_whole_gpu():
    """2000 tokens, 40 heads of 256: with one pair rotated the call takes at most eight times as long as with
    all 128 (its copied part goes by elements, the other by 16 bytes; on 8 CTAs it took over a hundred times as long)."""
    x = torch.randn((2000, 40, 256), device="cuda").bfloat16()
    pos = torch.arange(2000, device="cuda")[:, None]
    out = torch.empty_like(x)

    def us(rot):
        inv, axis = tfq.rope_axes_frequencies([rot])
        best = float("inf")
        for _ in range(5):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            for _ in range(10):
                tfq.tfq_rope_axes(x, None, pos, inv, axis, q_out=out)
            end.record()
            end.synchronize()
            best = min(best, start.elapsed_time(end) * 100)
        return best

    us(256)  # warm
    assert us(2) <= 8 * us(256)


@pytest.mark.parametrize("far", [100, 1 << 20])
@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
def test_fp32_is_as_exact_as_a_table_rounded_from_64_bits(far, pairing):
    """fp32: the rms error is that of the elementary form whose cos and sin are
    rounded from 64 bits.  That form has entries off by half a step (0.29 rms) and three
    roundings; the kernel's entries are off by up to a step, and it has two: at
    most 1.05 times the error.  (An angle rounded to fp32 alone gives 1.13 to 1.32.)"""
    M, H, D = 4000, 4, 128
    g = torch.Generator(device="cuda").manual_seed(far)
    x = torch.randn((M, H, D), generator=g, device="cuda")
    inv, axis = tfq.rope_axes_frequencies([44, 42, 42])
    pos = torch.randint(-100, far, (M, 3), generator=g, device="cuda")
    out, _ = tfq.tfq_rope_axes(x, None, pos, inv, axis, pairing=pairing)
    ang = (pos.double()[:, axis.long().cuda()] * inv.cuda())[:, None]

    def rotated(f, c, s):
        first, second = (slice(0, D, 2), slice(1, D, 2)) if pairing == "interleaved" else (slice(0, 64), slice(64, D))
        r = torch.empty_like(f)
        r[..., first], r[..., second] = f[..., first] * c - f[..., second] * s, f[..., first] * s + f[..., second] * c
        return r

    want = rotated(x.double(), ang.cos(), ang.sin())
    rms = lambda v: float((v.double() - want).square().mean().sqrt())  # noqa: E731
    assert rms(out) <= 1.05 * rms(rotated(x, ang.cos().float(), ang.sin().float()))
