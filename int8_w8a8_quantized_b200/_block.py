"""The operators around the W8A8 Linear of a transformer block (include/tfq.h):
layer norm (with its gradients, and straight to E4M3 codes), rotary positions
with several axes, and the scaled FP8 Linear with low-rank adapters.

Argument marshalling only, as in ``_capi``: every step runs in the CUDA
library, and there is no fallback.  ``stream`` (a torch stream or a
cudaStream_t as an integer) makes the call, and whatever it allocates, belong
to that stream; the default is torch's current stream of the tensors' device.
"""
from __future__ import annotations

import functools

import torch

from ._capi import (
    TFQ_DTYPE_BF16,
    TFQ_DTYPE_FP16,
    TFQ_DTYPE_FP32,
    TFQ_ROPE_HALVES,
    TFQ_ROPE_INTERLEAVED,
    _check,
    load_library,
    tfq_quant_act_fp8_per_token,
    tfq_scaled_fp8_linear,
)

_DTYPES = {torch.bfloat16: TFQ_DTYPE_BF16, torch.float16: TFQ_DTYPE_FP16, torch.float32: TFQ_DTYPE_FP32}
_PAIRINGS = {"interleaved": TFQ_ROPE_INTERLEAVED, "halves": TFQ_ROPE_HALVES}
_POSITIONS = {torch.int32: 0, torch.int64: 1}


def _as_stream(stream, device):
    if hasattr(stream, "cuda_stream"):
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the operands on {device}")
        return stream
    # 0 is the legacy default stream, as everywhere in the library (ExternalStream(0) would be some stream of torch's pool)
    return torch.cuda.ExternalStream(int(stream), device=device) if stream else torch.cuda.default_stream(device)


def _under(stream, operand, name="x"):
    """Makes `stream` the current one: what runs and what is allocated and freed in between belongs to it."""
    _operand(operand, name)
    return torch.cuda.stream(_as_stream(stream, operand.device))


def _streamed(fn):
    """Adds the ``stream`` argument: the call and its allocations run under that stream."""

    name = fn.__code__.co_varnames[0]  # an operand: its device is the stream's

    @functools.wraps(fn)
    def call(*args, stream=None, **kwargs):
        if stream is None:
            return fn(*args, **kwargs)
        with _under(stream, args[0] if args else kwargs.get(name), name):
            return fn(*args, **kwargs)

    return call


def _operand(t, name, dtype=None, ndim=None, device=None):
    """Refuses what is not a CUDA tensor of this type, dimension and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the other operands on cuda:{device}")


def _dense(t, name, dtype, shape, device):
    """A contiguous operand of exactly this type and shape (a tuple)."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == device
            and t.is_contiguous()):
        return t  # the usual case, in as few steps as it takes: small calls are bound by them
    _operand(t, name, dtype, None, device)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _codes(t, name, device):
    """A matrix of E4M3 codes: uint8, or torch.float8_e4m3fn (the same bytes)."""
    _operand(t, name, None, 2, device)
    if t.dtype is not torch.uint8 and t.dtype is not torch.float8_e4m3fn:
        raise TypeError(f"{name} must be torch.uint8 or torch.float8_e4m3fn, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# Outputs are allocated in the cheapest form (a call with few rows is bound by such
# steps): empty_like takes 1.4 us, new_empty of an int 1.6, of a shape with a type 2 to 2.4.
def _like(t, dtype=None):
    """A new contiguous tensor of t's shape."""
    return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)


def _output(t, name, dtype, shape, like):
    if t is not None:
        return _dense(t, name, dtype, shape, like.get_device())
    if like.shape == shape:
        return _like(like, dtype)
    return like.new_empty(*shape, dtype=dtype)


def _workspace(t, need, like):
    if t is None:
        return like.new_empty(need, dtype=torch.uint8)
    _operand(t, "workspace", torch.uint8, 1, like.get_device())
    if t.numel() < need or not t.is_contiguous():
        raise ValueError(f"workspace must hold {need} contiguous bytes")
    return t


def _ptr(t):
    return None if t is None else t.data_ptr()


_functions = {}
_current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _function(name):
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(load_library(), name)
    return fn


def _call(name, device, *args):
    """Calls the C entry point on `device`'s current stream."""
    fn = _functions.get(name) or _function(name)
    if device == _current_device():
        st = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(device))
    if st:
        _check(st, name)


def _rows(t, name, dtype=None, device=None):
    """(row stride) of a matrix whose rows are contiguous."""
    _operand(t, name, dtype, 2, device)
    M, K = t.shape
    row, element = t.stride()
    if K > 1 and element != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if M <= 1:
        return K
    if row < K:
        raise ValueError(f"{name} must not have overlapping rows")
    return row


def _affine(weight, bias, x, K, device):
    """(groups, type) of a norm's weight and bias: [K], or [G, K] for G equal groups of rows."""
    given = weight if weight is not None else bias
    if given is None:
        return 1, x.dtype
    if not isinstance(given, torch.Tensor):
        raise TypeError("weight and bias must be torch.Tensors")
    if given.dtype is not x.dtype and given.dtype is not torch.float32:
        raise TypeError(f"weight and bias must be {x.dtype} or torch.float32, got {given.dtype}")
    groups = given.shape[0] if given.dim() == 2 else 1
    if groups < 1 or x.shape[0] % groups:
        raise ValueError(f"{x.shape[0]} rows do not make {groups} equal groups")
    shape = (groups, K) if given.dim() == 2 else (K,)
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _dense(t, name, given.dtype, shape, device)
    return groups, given.dtype


def _norm_type(x):
    dtype = _DTYPES.get(x.dtype)
    if dtype is None:
        raise TypeError(f"x must be bfloat16, float16 or float32, got {x.dtype}")
    return dtype


@_streamed
def tfq_layer_norm(x, weight=None, bias=None, eps: float = 1e-6, weight_offset: float = 0.0, stats: bool = False,
                   y=None):
    """Layer norm over the rows of x [M, K] (bf16, fp16 or fp32; rows may be
    strided): (x - mean) * rstd * (weight + weight_offset) + bias.  weight and
    bias: [K], or [G, K] for G equal groups of consecutive rows (an adaptive
    norm's scale, with weight_offset 1, and shift), of x's type or fp32, or None.
    Returns y, with stats=True (y, mean, rstd) (fp32 [M], what the gradient needs).
    y=x (contiguous) normalizes in place."""
    stride = _rows(x, "x")
    dtype = _norm_type(x)
    dev = x.get_device()
    M, K = x.shape
    groups, wdt = _affine(weight, bias, x, K, dev)
    y = _output(y, "y", x.dtype, (M, K), x)
    mean = rstd = None
    if stats:
        mean = x.new_empty(M, dtype=torch.float32)
        rstd = _like(mean)
    _call("tfq_layer_norm", dev, x.data_ptr(), stride, dtype, _ptr(weight), _ptr(bias), _DTYPES[wdt], weight_offset,
          M, K, groups, eps, y.data_ptr(), _ptr(mean), _ptr(rstd))
    return (y, mean, rstd) if stats else y


@_streamed
def tfq_layer_norm_quant_fp8(x, weight=None, bias=None, eps: float = 1e-6, weight_offset: float = 0.0,
                             qmax: float = 448.0, q=None, s=None):
    """tfq_layer_norm straight to the W8A8 Linear's input: (q uint8 [M, K] E4M3
    codes, s fp32 [M]) of the norm's fp32 rows, K a multiple of 16."""
    stride = _rows(x, "x")
    dtype = _norm_type(x)
    dev = x.get_device()
    M, K = x.shape
    groups, wdt = _affine(weight, bias, x, K, dev)
    q = _output(q, "q", torch.uint8, (M, K), x)
    s = _output(s, "s", torch.float32, (M,), x)
    _call("tfq_layer_norm_quant_fp8", dev, x.data_ptr(), stride, dtype, _ptr(weight), _ptr(bias), _DTYPES[wdt],
          weight_offset, M, K, groups, eps, qmax, q.data_ptr(), s.data_ptr())
    return q, s


def tfq_layer_norm_backward_workspace_bytes(M: int, K: int, groups: int = 1) -> int:
    """Bytes of the workspace tfq_layer_norm_backward needs for weight or bias gradients."""
    return _function("tfq_layer_norm_backward_workspace_bytes")(int(M), int(K), int(groups))


@_streamed
def tfq_layer_norm_backward(dy, x, weight, mean, rstd, weight_offset: float = 0.0, need_x: bool = True,
                            need_weight: bool = True, need_bias: bool = True, groups: int | None = None,
                            dweight_dtype=None, workspace=None):
    """The gradients (dx, dweight, dbias) of tfq_layer_norm at dy [M, K], from
    the forward's mean and rstd.  dweight and dbias have weight's shape and
    type; without a weight there is no dweight, and dbias is [K] (or [groups,
    K]) of dweight_dtype (x's type by default).  An unneeded gradient is None."""
    x_stride = _rows(x, "x")
    dtype = _norm_type(x)
    dev = x.get_device()
    dy_stride = _rows(dy, "dy", x.dtype, dev)
    M, K = x.shape
    if dy.shape != x.shape:
        raise ValueError("dy and x must have the same shape")
    _dense(mean, "mean", torch.float32, (M,), dev)
    _dense(rstd, "rstd", torch.float32, (M,), dev)
    if weight is not None:
        if groups is not None and groups != (weight.shape[0] if weight.dim() == 2 else 1):
            raise ValueError("groups differs from weight's")
        if dweight_dtype is not None and dweight_dtype is not weight.dtype:
            raise TypeError("dweight_dtype differs from weight's")
        groups, wdt = _affine(weight, None, x, K, dev)
    else:
        wdt = x.dtype if dweight_dtype is None else dweight_dtype
        if wdt is not x.dtype and wdt is not torch.float32:
            raise TypeError(f"dweight_dtype must be {x.dtype} or torch.float32")
        shape = (K,) if groups is None else (groups, K)
        groups = 1 if groups is None else groups
        if groups < 1 or M % groups:
            raise ValueError(f"{M} rows do not make {groups} equal groups")
        need_weight = False
    dx = _like(x) if need_x else None
    dw = _like(weight) if need_weight else None
    db = None
    if need_bias:
        db = x.new_empty(*shape, dtype=wdt) if weight is None else _like(weight)
    if need_weight or need_bias:
        workspace = _workspace(workspace, tfq_layer_norm_backward_workspace_bytes(M, K, groups), x)
    else:
        workspace = None
    _call("tfq_layer_norm_backward", dev, dy.data_ptr(), dy_stride, x.data_ptr(), x_stride, dtype, _ptr(weight),
          _DTYPES[wdt], weight_offset, mean.data_ptr(), rstd.data_ptr(), M, K, groups, _ptr(dx), _ptr(dw), _ptr(db),
          _ptr(workspace))
    return dx, dw, db


def rope_axes_frequencies(dims, theta: float = 10000.0, ladder: str = "axis"):
    """(inv_freq, axis) of tfq_rope_axes, CPU tensors: dims[a] channels of a head
    turn with axis a (even numbers; their sum is the rotated part).  ladder
    "axis": each axis has the frequencies theta^(-2 j / dims[a]); "shared": one
    ladder theta^(-2 i / sum(dims)) over all pairs, handed out to the axes in order."""
    dims = [int(d) for d in dims]
    if not dims or any(d < 0 or d % 2 for d in dims):
        raise ValueError("dims must be even")
    if ladder not in ("axis", "shared"):
        raise ValueError("ladder must be 'axis' or 'shared'")
    rot = sum(dims)
    inv, axis = [], []
    for a, d in enumerate(dims):
        for j in range(d // 2):
            inv.append(float(theta) ** (-2.0 * j / d if ladder == "axis" else -2.0 * len(inv) / rot))
            axis.append(a)
    return torch.tensor(inv, dtype=torch.float64), torch.tensor(axis, dtype=torch.int32)


def _heads(t, name, dtype, device, M, D):
    _operand(t, name, dtype, 3, device)
    if t.shape[0] != M or t.shape[2] != D:
        raise ValueError(f"{name} must be [{M}, heads, {D}], got {tuple(t.shape)}")
    if D > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have contiguous heads")


def _rope_output(out, name, like, device):
    if out is None:
        return _like(like)
    _heads(out, name, like.dtype, device, like.shape[0], like.shape[2])
    if out.shape[1] != like.shape[1]:
        raise ValueError(f"{name} must have {like.shape[1]} heads")
    M, H, D = out.shape  # its elements must be distinct places
    row, head = out.stride(0), out.stride(1)
    if out.numel() and not ((H <= 1 or head >= D) and (M <= 1 or row >= (H - 1) * head + D)
                            or (M <= 1 or row >= D) and (H <= 1 or head >= (M - 1) * row + D)):
        raise ValueError(f"{name} must not overlap itself")
    return out


@_streamed
def tfq_rope_axes(q, k, positions, inv_freq, axis, pairing: str = "interleaved", inverse: bool = False, q_out=None,
                  k_out=None):
    """Rotary positions with several axes on q [M, H, D] and k [M, Hk, D] (or
    None), bf16, fp16 or fp32, with any row and head strides (slices of a fused
    Q/K/V projection).  positions int32 or int64 [M, axes]; inv_freq fp64 and
    axis int32, CPU tensors with an entry per rotated pair
    (rope_axes_frequencies).  pairing "interleaved": pairs (2 i, 2 i + 1),
    "halves": (i, pairs + i).  inverse=True rotates back (the gradient).
    Returns (q_out, k_out); q_out=q, k_out=k rotates in place."""
    _operand(q, "q", None, 3)
    dtype = _DTYPES.get(q.dtype)
    if dtype is None:
        raise TypeError(f"q must be bfloat16, float16 or float32, got {q.dtype}")
    dev = q.get_device()
    M, H, D = q.shape
    _heads(q, "q", q.dtype, dev, M, D)
    if k is not None:
        _heads(k, "k", q.dtype, dev, M, D)
    _operand(positions, "positions", None, 2, dev)
    pos64 = _POSITIONS.get(positions.dtype)
    if pos64 is None:
        raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
    if positions.shape[0] != M:
        raise ValueError(f"positions must have {M} rows")
    for t, name, dt in ((inv_freq, "inv_freq", torch.float64), (axis, "axis", torch.int32)):
        if not isinstance(t, torch.Tensor) or t.is_cuda or t.dtype is not dt or t.dim() != 1 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous 1-D CPU tensor of {dt}")
    pairs = inv_freq.shape[0]
    if axis.shape[0] != pairs:
        raise ValueError("inv_freq and axis must have the same length")
    if pairing not in _PAIRINGS:
        raise ValueError("pairing must be 'interleaved' or 'halves'")
    q_out = _rope_output(q_out, "q_out", q, dev)
    kh = ko = None
    ks, kos, Hk = (0, 0), (0, 0), 0
    if k is not None:
        k_out = _rope_output(k_out, "k_out", k, dev)
        kh, ko, Hk = k.data_ptr(), k_out.data_ptr(), k.shape[1]
        ks, kos = k.stride(), k_out.stride()
    qs, qos = q.stride(), q_out.stride()
    ps = positions.stride()
    _call("tfq_rope_axes", dev, q.data_ptr(), qs[0], qs[1], H, q_out.data_ptr(), qos[0], qos[1], kh, ks[0], ks[1], Hk,
          ko, kos[0], kos[1], M, D, dtype, positions.data_ptr(), pos64, ps[0], ps[1], positions.shape[1], pairs,
          inv_freq.data_ptr(), axis.data_ptr(), _PAIRINGS[pairing], bool(inverse))
    return q_out, (k_out if k is not None else None)


@_streamed
def tfq_lora_fold(lora_B, scaling, s_w, out=None):
    """lora_B bf16 [n, N, R], scaling fp32 [n] or None, s_w fp32 [N] ->
    lora_Bs bf16 [n, N, R] = scaling * lora_B / s_w, what
    tfq_scaled_fp8_linear_lora takes; once per adapter and weight (out=lora_B
    folds in place)."""
    _operand(lora_B, "lora_B", torch.bfloat16, 3)
    dev = lora_B.get_device()
    n, N, R = lora_B.shape
    _dense(lora_B, "lora_B", torch.bfloat16, (n, N, R), dev)
    if scaling is not None:
        _dense(scaling, "scaling", torch.float32, (n,), dev)
    _dense(s_w, "s_w", torch.float32, (N,), dev)
    out = _output(out, "out", torch.bfloat16, (n, N, R), lora_B)
    _call("tfq_lora_fold", dev, lora_B.data_ptr(), _ptr(scaling), s_w.data_ptr(), n, N, R, out.data_ptr())
    return out


def tfq_scaled_fp8_linear_lora_workspace_bytes(M: int, R: int) -> int:
    """Bytes of the workspace tfq_scaled_fp8_linear_lora needs for M rows and rank R."""
    return _function("tfq_scaled_fp8_linear_lora_workspace_bytes")(int(M), int(R))


@_streamed
def tfq_scaled_fp8_linear_lora(A_q, s_a, W_q, s_w, x, lora_A, lora_Bs, adapter, bias=None, out=None, workspace=None):
    """tfq_scaled_fp8_linear with low-rank adapters beside it: out[m] +=
    scaling[a] lora_B[a] (lora_A[a] x[m]) for a = adapter[m] (int32 [M]; outside
    [0, n): none).  x bf16 [M, K]: the activations A_q was made from; lora_A
    bf16 [n, R, K]; lora_Bs bf16 [n, N, R] from tfq_lora_fold; R a multiple of 8
    (adapters of lower or unequal ranks: zeros behind their own rows of both)."""
    _codes(A_q, "A_q", None)
    dev = A_q.get_device()
    _codes(W_q, "W_q", dev)
    M, K = A_q.shape
    N = W_q.shape[0]
    if W_q.shape[1] != K:
        raise ValueError("A_q and W_q must have the same K")
    _dense(s_a, "s_a", torch.float32, (M,), dev)
    _dense(s_w, "s_w", torch.float32, (N,), dev)
    _dense(x, "x", torch.bfloat16, (M, K), dev)
    _operand(lora_A, "lora_A", torch.bfloat16, 3, dev)
    n, R, _ = lora_A.shape
    _dense(lora_A, "lora_A", torch.bfloat16, (n, R, K), dev)
    _dense(lora_Bs, "lora_Bs", torch.bfloat16, (n, N, R), dev)
    _dense(adapter, "adapter", torch.int32, (M,), dev)
    if bias is not None:
        _dense(bias, "bias", torch.bfloat16, (N,), dev)
    out = _output(out, "out", torch.bfloat16, (M, N), x)
    workspace = _workspace(workspace, tfq_scaled_fp8_linear_lora_workspace_bytes(M, R), x)
    _call("tfq_scaled_fp8_linear_lora", dev, A_q.data_ptr(), s_a.data_ptr(), W_q.data_ptr(), s_w.data_ptr(),
          _ptr(bias), M, N, K, x.data_ptr(), lora_A.data_ptr(), lora_Bs.data_ptr(), adapter.data_ptr(), n, R,
          out.data_ptr(), workspace.data_ptr())
    return out


def w8a8_lora_linear(x, W_q, s_w, lora_A, lora_Bs, adapter, bias=None, qmax: float = 448.0, stream=None):
    """w8a8_linear with low-rank adapters: per-token FP8 quantization of x, then
    the scaled GEMM with one adapter per row beside it."""
    if stream is not None:
        with _under(stream, x):
            return w8a8_lora_linear(x, W_q, s_w, lora_A, lora_Bs, adapter, bias, qmax)
    A_q, s_a = tfq_quant_act_fp8_per_token(x, qmax)
    return tfq_scaled_fp8_linear_lora(A_q, s_a, W_q, s_w, x, lora_A, lora_Bs, adapter, bias=bias)


def w8a8_norm_linear(x, norm_weight, norm_bias, W_q, s_w, bias=None, eps: float = 1e-6, weight_offset: float = 0.0,
                     qmax: float = 448.0, stream=None):
    """Layer norm (tfq_layer_norm's arguments) and the W8A8 Linear on it: the
    norm's rows go to E4M3 codes in one pass, then the scaled GEMM."""
    if stream is not None:
        with _under(stream, x):
            return w8a8_norm_linear(x, norm_weight, norm_bias, W_q, s_w, bias, eps, weight_offset, qmax)
    A_q, s_a = tfq_layer_norm_quant_fp8(x, norm_weight, norm_bias, eps=eps, weight_offset=weight_offset, qmax=qmax)
    return tfq_scaled_fp8_linear(A_q, s_a, W_q, s_w, bias)
