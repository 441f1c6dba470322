"""Host-side checks of the operators around the Linear (no GPU needed): every
bad call is refused before any device work, and the frequency tables of the
rotary positions are what their definition says."""
import ctypes
import os
import subprocess

import pytest
import torch

import int8_w8a8_quantized_b200 as tfq
from int8_w8a8_quantized_b200 import _capi, build

P = 0x10000  # a fake, aligned address: never dereferenced by a refused call
BF16, FP16, FP32 = _capi.TFQ_DTYPE_BF16, _capi.TFQ_DTYPE_FP16, _capi.TFQ_DTYPE_FP32
INVAL, UNSUP, OK = _capi.TFQ_EINVAL, _capi.TFQ_EUNSUPPORTED, _capi.TFQ_OK


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _capi.load_library()


NORM = dict(x=P, x_stride=64, dtype=BF16, w=P, b=P, w_dtype=BF16, offset=0.0, M=4, K=64, groups=1, eps=1e-6, y=P,
            mean=P, rstd=P)


@pytest.mark.parametrize("change,status", [
    (dict(M=-4), INVAL), (dict(K=-1), INVAL), (dict(dtype=0), INVAL), (dict(dtype=9), INVAL),
    (dict(w_dtype=FP16), INVAL), (dict(groups=0), INVAL), (dict(groups=3), INVAL), (dict(x_stride=63), INVAL),
    (dict(eps=-1e-6), INVAL), (dict(eps=float("nan")), INVAL), (dict(offset=float("inf")), INVAL),
    (dict(x=None), INVAL), (dict(y=None), INVAL), (dict(mean=None), INVAL), (dict(rstd=None), INVAL),
    (dict(x=P + 1), INVAL), (dict(w=P + 1), INVAL), (dict(b=P + 1), INVAL), (dict(y=P + 1), INVAL),
    (dict(mean=P + 2), INVAL), (dict(w_dtype=FP32, w=P + 2), INVAL),
    (dict(K=32769, x_stride=32769), UNSUP), (dict(M=1 << 31), UNSUP),
    (dict(M=1 << 27, groups=1 << 27), UNSUP),
    (dict(M=0, x=None, y=None), OK), (dict(K=0, x_stride=0, x=None, y=None), OK),
])
def test_layer_norm_refusals(lib, change, status):
    assert lib.tfq_layer_norm(*{**NORM, **change}.values(), None) == status
    if status != OK:
        assert _capi.last_error_message()


@pytest.mark.parametrize("change,status", [
    (dict(K=72, x_stride=72), INVAL), (dict(qmax=0.5), INVAL), (dict(qmax=449.0), INVAL),
    (dict(qmax=float("nan")), INVAL), (dict(q=None), INVAL), (dict(s=None), INVAL), (dict(q=P + 8), INVAL),
    (dict(s=P + 4), INVAL), (dict(groups=3), INVAL), (dict(x=None), INVAL), (dict(M=0, x=None, q=None, s=None), OK),
])
def test_layer_norm_quant_refusals(lib, change, status):
    a = {k: NORM[k] for k in ("x", "x_stride", "dtype", "w", "b", "w_dtype", "offset", "M", "K", "groups", "eps")}
    a.update(qmax=448.0, q=P, s=P)
    a.update(change)
    assert lib.tfq_layer_norm_quant_fp8(*a.values(), None) == status


BWD = dict(dy=P, dy_stride=64, x=P, x_stride=64, dtype=BF16, w=P, w_dtype=BF16, offset=0.0, mean=P, rstd=P, M=4, K=64,
           groups=1, dx=P, dw=P, db=P, ws=P)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), INVAL), (dict(dtype=7), INVAL), (dict(w_dtype=FP16), INVAL), (dict(groups=3), INVAL),
    (dict(dy_stride=63), INVAL), (dict(x_stride=63), INVAL), (dict(offset=float("nan")), INVAL),
    (dict(dy=None), INVAL), (dict(x=None), INVAL), (dict(mean=None), INVAL), (dict(rstd=None), INVAL),
    (dict(dy=P + 1), INVAL), (dict(dx=P + 1), INVAL), (dict(dw=P + 1), INVAL), (dict(db=P + 1), INVAL),
    (dict(rstd=P + 1), INVAL), (dict(ws=None), INVAL), (dict(ws=P + 8), INVAL), (dict(ws=None, dw=None), INVAL),
    (dict(K=40000, x_stride=40000, dy_stride=40000), UNSUP),
    (dict(dx=None, dw=None, db=None, dy=None, ws=None), OK), (dict(K=0, dy=None), OK),
])
def test_layer_norm_backward_refusals(lib, change, status):
    assert lib.tfq_layer_norm_backward(*{**BWD, **change}.values(), None) == status


def test_layer_norm_backward_workspace(lib):
    f = lib.tfq_layer_norm_backward_workspace_bytes
    assert f(0, 64, 1) == 0 and f(4, 0, 1) == 0 and f(4, 64, 3) == 0 and f(-4, 64, 1) == 0
    assert f(1, 64, 1) == 2 * 64 * 4
    for M, K, G in ((32760, 5120, 1), (7, 1001, 7), (4096, 16, 2), (75600, 8, 1), (65536, 32768, 1)):
        n = f(M, K, G)
        assert n % (2 * G * K * 4) == 0 and 0 < n <= 2 * 4 * K * max(G, min(M, 160 * 8 + G))


ROPE = dict(q=P, q_rs=512, q_hs=64, q_heads=8, qo=P, qo_rs=512, qo_hs=64, k=P, k_rs=128, k_hs=64, k_heads=2, ko=P,
            ko_rs=128, ko_hs=64, M=4, D=64, dtype=BF16, pos=P, pos64=0, p_rs=3, p_as=1, axes=3, pairs=3, inv=None,
            axis=None, pairing=0, inverse=0)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), INVAL), (dict(q_heads=-1), INVAL), (dict(D=-2), INVAL), (dict(dtype=1), INVAL),
    (dict(pairing=2), INVAL), (dict(pairs=0), INVAL), (dict(D=5), INVAL), (dict(axes=0), INVAL), (dict(axes=2), INVAL),
    (dict(q=None), INVAL), (dict(qo=None), INVAL), (dict(k=None), INVAL), (dict(ko=P + 1), INVAL),
    (dict(pos=None), INVAL), (dict(pos=P + 2), INVAL), (dict(pos=P + 4, pos64=1), INVAL), (dict(inv=0), INVAL),
    (dict(axis=0), INVAL), (dict(nan=True), INVAL), (dict(D=264), UNSUP), (dict(axes=256), UNSUP),
    (dict(q_heads=65537), UNSUP), (dict(q_heads=65536, k_heads=1), UNSUP), (dict(M=1 << 31), UNSUP),
    (dict(M=0, q=None, k=None, pos=None), OK), (dict(q_heads=0, k_heads=0, pos=None), OK),
])
def test_rope_refusals(lib, change, status):
    a = {**ROPE, **{k: v for k, v in change.items() if k in ROPE}}
    freqs = (ctypes.c_double * 3)(1.0, float("nan") if change.get("nan") else 0.5, 0.25)
    axis = (ctypes.c_int32 * 3)(0, 1, 2)
    a["inv"] = None if change.get("inv") == 0 else ctypes.cast(freqs, ctypes.c_void_p)
    a["axis"] = None if change.get("axis") == 0 else ctypes.cast(axis, ctypes.c_void_p)
    assert lib.tfq_rope_axes(*a.values(), None) == status


LORA = dict(A_q=P, s_a=P, W_q=P, s_w=P, bias=None, M=4, N=16, K=32, x=P, A=P, Bs=P, idx=P, n=2, R=8, out=P, ws=P)


@pytest.mark.parametrize("change,status", [
    (dict(K=24), INVAL), (dict(N=12), INVAL), (dict(M=-1), INVAL), (dict(A_q=None), INVAL), (dict(n=-1), INVAL),
    (dict(R=-8), INVAL), (dict(R=12), INVAL), (dict(R=264), UNSUP), (dict(n=1 << 28), UNSUP),
    (dict(n=(1 << 22) + 1), UNSUP), (dict(n=1 << 22, N=512), UNSUP), (dict(n=1 << 16, N=32768), UNSUP),
    (dict(x=None), INVAL), (dict(A=None), INVAL), (dict(Bs=None), INVAL), (dict(idx=None), INVAL),
    (dict(ws=None), INVAL), (dict(x=P + 8), INVAL), (dict(A=P + 8), INVAL), (dict(Bs=P + 2), INVAL),
    (dict(idx=P + 2), INVAL), (dict(ws=P + 4), INVAL), (dict(M=0, x=None), OK), (dict(N=0, Bs=None), OK),
])
def test_lora_refusals(lib, change, status):
    assert lib.tfq_scaled_fp8_linear_lora(*{**LORA, **change}.values(), None) == status


def test_lora_fold_refusals(lib):
    f = lib.tfq_lora_fold
    assert f(P, P, P, -1, 4, 8, P, None) == INVAL
    assert f(None, P, P, 1, 4, 8, P, None) == INVAL
    assert f(P, P, None, 1, 4, 8, P, None) == INVAL
    assert f(P, P, P, 1, 4, 8, None, None) == INVAL
    assert f(P + 1, P, P, 1, 4, 8, P, None) == INVAL
    assert f(P, P + 2, P, 1, 4, 8, P, None) == INVAL
    assert f(P, P, P, 1 << 31, 4, 8, P, None) == UNSUP
    assert f(None, None, None, 0, 4, 8, None, None) == OK


def test_lora_workspace_bytes(lib):
    f = lib.tfq_scaled_fp8_linear_lora_workspace_bytes
    assert f(0, 8) == 0 and f(4, 0) == 0 and f(-1, 8) == 0 and f(4, 512) == 0
    assert f(100, 16) >= 100 * 16 * 2


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU behaviour")
def test_valid_calls_without_gpu_fail_loudly(lib):
    bad = (_capi.TFQ_ECUDA, _capi.TFQ_EUNSUPPORTED)
    assert lib.tfq_layer_norm(*NORM.values(), None) in bad
    assert lib.tfq_layer_norm_backward(*BWD.values(), None) in bad
    assert lib.tfq_scaled_fp8_linear_lora(*LORA.values(), None) in bad


def test_python_layer_refuses_cpu_tensors():
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        tfq.tfq_layer_norm(x)
    with pytest.raises(ValueError, match="CUDA"):
        tfq.tfq_layer_norm_quant_fp8(x, stream=0)
    with pytest.raises(TypeError, match="torch.Tensor"):
        tfq.tfq_layer_norm([1.0])
    inv, axis = tfq.rope_axes_frequencies((8, 8))
    with pytest.raises(ValueError, match="CUDA"):
        tfq.tfq_rope_axes(x.view(4, 2, 16), None, torch.zeros(4, 2, dtype=torch.int32), inv, axis)
    with pytest.raises(ValueError, match="CUDA"):
        tfq.tfq_lora_fold(torch.zeros(1, 8, 8, dtype=torch.bfloat16), None, torch.ones(8))


def test_rope_axes_frequencies():
    inv, axis = tfq.rope_axes_frequencies((4, 6, 6), theta=100.0)
    assert axis.tolist() == [0, 0, 1, 1, 1, 2, 2, 2]
    want = [1.0, 100.0 ** -0.5] + 2 * [1.0, 100.0 ** (-1 / 3), 100.0 ** (-2 / 3)]
    assert torch.equal(inv, torch.tensor(want, dtype=torch.float64))
    inv, axis = tfq.rope_axes_frequencies((4, 0, 4), theta=16.0, ladder="shared")
    assert axis.tolist() == [0, 0, 2, 2]
    assert torch.allclose(inv, torch.tensor([1.0, 0.5, 0.25, 0.125], dtype=torch.float64), rtol=1e-15)
    for bad in ((), (3, 5), (-2, 4)):
        with pytest.raises(ValueError):
            tfq.rope_axes_frequencies(bad)
    with pytest.raises(ValueError):
        tfq.rope_axes_frequencies((4, 4), ladder="other")


def test_package_lists_the_operators():
    for name in ("tfq_layer_norm", "tfq_layer_norm_quant_fp8", "tfq_layer_norm_backward", "tfq_rope_axes",
                 "tfq_scaled_fp8_linear_lora", "tfq_lora_fold", "w8a8_lora_linear", "w8a8_norm_linear"):
        assert name in tfq.__all__ and name in dir(tfq) and callable(getattr(tfq, name))
    with pytest.raises(AttributeError):
        tfq.no_such_operator


def test_only_tensors_are_operands():
    x = torch.zeros((4, 32))
    for call in (lambda: tfq.tfq_layer_norm(x), lambda: tfq.tfq_layer_norm([1.0]), lambda: tfq.tfq_rope_axes(x, None, x, x, x),
                 lambda: tfq.tfq_lora_fold(x, None, x), lambda: tfq.tfq_layer_norm(x, stream=0)):
        with pytest.raises((TypeError, ValueError)):
            call()


def test_stream_zero_is_the_default_stream(monkeypatch):
    from int8_w8a8_quantized_b200 import _block

    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: ("default", device))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: (handle, device))
    assert _block._as_stream(0, "cuda:1") == ("default", "cuda:1")
    assert _block._as_stream(0x5000, "cuda:1") == (0x5000, "cuda:1")


def test_layer_norm_backward_fills_whole_waves(lib):
    """Groups that do not divide the GPU: no CTA beyond the last full wave.  The workspace holds
    two fp32 rows for each CTA of a device of 160 SMs; 5120 columns run two CTAs per SM at most, 1536
    columns six."""
    f = lib.tfq_layer_norm_backward_workspace_bytes
    for M, K, G, per_sm in ((32760, 5120, 3, 2), (32760, 5120, 5, 2), (32760, 5120, 7, 2), (32767, 1536, 7, 6)):
        ctas = f(M, K, G) // (2 * K * 4)
        assert ctas % G == 0 and 0.95 * 160 * per_sm <= ctas <= 160 * per_sm


def test_launch_attributes_are_set_once_behind_the_mutex(tmp_path):
    """Host threads at once (under the thread sanitizer), and no launch attribute set or looked up elsewhere."""
    exe = tmp_path / "once"
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc_path())), "include")
    here = os.path.dirname(os.path.abspath(__file__))
    for sanitizer in (["-fsanitize=thread"], []):
        subprocess.run(["g++", "-std=c++17", "-O1", *sanitizer, "-pthread", "-I", build.INCLUDE, "-I", build.CSRC, "-I", cuda,
                        os.path.join(here, "c", "once_per_device.cpp"), "-o", str(exe)], check=True)
        r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
        if "unexpected memory mapping" not in r.stderr:  # the sanitizer cannot run under some kernels' address layouts
            break
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
    for path in build.sources():
        with open(path) as f:
            for line in f:
                assert "attr_set" not in line or "once_per_device(" in line, (path, line)
