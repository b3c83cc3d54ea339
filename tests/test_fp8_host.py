"""Host-side checks of the FP8 entry points (no GPU): argument errors come back as statuses before
anything is launched, and the binding refuses what the kernels do not take."""
import ctypes

import pytest
import torch

from nvfp4_mixture_experts_w4a4_b200 import _lib as C
from nvfp4_mixture_experts_w4a4_b200 import build, ops


@pytest.fixture(scope="module")
def so():
    build.build()
    return C.lib()


def quantize(so, x=256, dtype=0, batch=1, rows=4, K=64, ldx=64, xb=0, tile=0, codes=256, ldc=64, cb=0, scale=256,
             lds=1, sb=0):
    return so.fp8_quantize(x, dtype, batch, rows, K, ldx, xb, tile, codes, ldc, cb, scale, lds, sb, None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), C.INVALID_ARG), (dict(tile=2), C.INVALID_ARG), (dict(rows=-1), C.INVALID_ARG),
    (dict(x=None), C.INVALID_ARG), (dict(codes=None), C.INVALID_ARG), (dict(scale=None), C.INVALID_ARG),
    (dict(ldx=63), C.INVALID_ARG), (dict(ldc=63), C.INVALID_ARG), (dict(K=129, ldx=129, ldc=129, lds=1), C.INVALID_ARG),
    (dict(xb=-1), C.INVALID_ARG), (dict(x=257), C.INVALID_ARG),
    (dict(rows=1 << 31), C.UNSUPPORTED_SHAPE), (dict(batch=1 << 16, rows=1 << 16), C.UNSUPPORTED_SHAPE),
    (dict(K=1 << 30, ldx=1 << 30, ldc=1 << 30, lds=1 << 23), C.UNSUPPORTED_SHAPE),
    (dict(rows=0), C.OK), (dict(batch=0), C.OK), (dict(K=0), C.OK),
])
def test_quantize_statuses(so, change, status):
    assert quantize(so, **change) == status


def gemm(so, A=256, lda=256, sa=256, lds_a=2, B=256, ldb=256, sb=256, lds_b=2, M=8, N=8, K=256, D=256, ldd=8, dt=0):
    return so.fp8_gemm(A, lda, sa, lds_a, B, ldb, sb, lds_b, M, N, K, D, ldd, dt, None)


@pytest.mark.parametrize("change,status", [
    (dict(dt=2), C.INVALID_ARG), (dict(M=-1), C.INVALID_ARG), (dict(A=None), C.INVALID_ARG),
    (dict(sb=None), C.INVALID_ARG), (dict(D=None), C.INVALID_ARG), (dict(D=257), C.INVALID_ARG),
    (dict(lda=240), C.INVALID_ARG), (dict(ldb=240), C.INVALID_ARG), (dict(ldd=7), C.INVALID_ARG),
    (dict(lds_a=1), C.INVALID_ARG), (dict(lds_b=1), C.INVALID_ARG),
    (dict(lda=260), C.UNSUPPORTED_SHAPE), (dict(ldb=264), C.UNSUPPORTED_SHAPE), (dict(A=264), C.UNSUPPORTED_SHAPE),
    (dict(B=264), C.UNSUPPORTED_SHAPE), (dict(K=0), C.UNSUPPORTED_SHAPE),
    (dict(M=1 << 31, N=1, ldd=1), C.UNSUPPORTED_SHAPE), (dict(lda=1 << 41), C.UNSUPPORTED_SHAPE),
    (dict(M=0), C.OK), (dict(N=0), C.OK),
])
def test_gemm_statuses(so, change, status):
    assert gemm(so, **change) == status


def desc(**change):
    d = C.Fp8MoeFfnDesc()
    base = dict(T=16, H=256, I=128, E=8, top_k=2, launch_mode=C.LAUNCH_AUTO, w13_codes=256, w13_scale=256,
                w2_codes=256, w2_scale=256)
    for name, value in {**base, **change}.items():
        setattr(d, name, value)
    return d


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), C.INVALID_ARG), (dict(H=100), C.UNSUPPORTED_SHAPE), (dict(H=0), C.UNSUPPORTED_SHAPE),
    (dict(I=24), C.UNSUPPORTED_SHAPE), (dict(E=1025), C.UNSUPPORTED_SHAPE), (dict(E=0), C.UNSUPPORTED_SHAPE),
    (dict(top_k=9), C.UNSUPPORTED_SHAPE), (dict(top_k=0), C.UNSUPPORTED_SHAPE),
    (dict(E=64, top_k=33), C.UNSUPPORTED_SHAPE), (dict(T=1 << 24), C.UNSUPPORTED_SHAPE),
    (dict(launch_mode=7), C.INVALID_ARG), (dict(launch_mode=C.LAUNCH_SINGLE, T=17), C.UNSUPPORTED_SHAPE),
    (dict(launch_mode=C.LAUNCH_SINGLE, H=16384), C.UNSUPPORTED_SHAPE),
])
def test_layer_statuses(so, change, status):
    d = desc(**change)
    assert so.fp8_moe_ffn_workspace_size(ctypes.byref(d)) == 0
    assert so.fp8_moe_ffn_forward(ctypes.byref(d), 256, 256, 256, 256, 1 << 40, None) == status
    assert so.nvfp4moe_last_error()


def test_layer_pointers_and_workspace(so):
    d = desc()
    need = so.fp8_moe_ffn_workspace_size(ctypes.byref(d))
    assert need > 0
    for args in ((None, 256, 256, 256), (256, None, 256, 256), (256, 256, None, 256), (256, 256, 256, None),
                 (264, 256, 256, 256), (256, 256, 264, 256), (256, 256, 256, 128)):
        assert so.fp8_moe_ffn_forward(ctypes.byref(d), *args, need, None) == C.INVALID_ARG
    assert so.fp8_moe_ffn_forward(ctypes.byref(desc(w2_scale=None)), 256, 256, 256, 256, need, None) == C.INVALID_ARG
    assert so.fp8_moe_ffn_forward(ctypes.byref(d), 256, 256, 256, 256, need - 1, None) == C.WORKSPACE_TOO_SMALL
    assert so.fp8_moe_ffn_forward(ctypes.byref(desc(T=0)), None, None, None, None, 0, None) == C.OK
    assert so.fp8_moe_ffn_forward(None, 256, 256, 256, 256, need, None) == C.INVALID_ARG


def test_binding_refuses():
    x = torch.zeros(4, 128)
    with pytest.raises(ValueError, match="CUDA"):
        ops.fp8_quantize(x)
    with pytest.raises(ValueError, match="bf16 or fp32"):
        ops.fp8_quantize(x.half())
    with pytest.raises(ValueError, match="rows, K"):
        ops.fp8_quantize(x[0])
    a, s = torch.zeros(4, 128, dtype=torch.float8_e4m3fn), torch.ones(4, 1)
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        ops.fp8_gemm(x, s, a, s[:1])
    with pytest.raises(ValueError, match="A must be"):
        ops.fp8_gemm(a, s, a[:, :64], s[:1])
    with pytest.raises(ValueError, match="A_scale"):
        ops.fp8_gemm(a, s[:3], a, s[:1])
    with pytest.raises(ValueError, match="B_scale"):
        ops.fp8_gemm(a, s, a, s)
    with pytest.raises(ValueError, match="bf16 or fp32"):
        ops.fp8_gemm(a, s, a, s[:1], out_dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.fp8_gemm(a, s, a, s[:1])
    w13, w2 = torch.zeros(2, 2, 32, 128, dtype=torch.uint8), torch.zeros(2, 128, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="w2_scale"):
        ops.FP8Experts(w13, torch.ones(2, 2, 1, 1), w2, torch.ones(2, 2, 1))
    with pytest.raises(ValueError, match="w13_codes"):
        ops.FP8Experts(w13[:, 0], torch.ones(2, 2, 1, 1), w2, torch.ones(2, 1, 1))
    with pytest.raises(ValueError, match="CUDA"):
        ops.FP8Experts(w13, torch.ones(2, 2, 1, 1), w2, torch.ones(2, 1, 1))


@pytest.mark.parametrize("change,status", [
    (dict(), C.INVALID_ARG), (dict(cb=4 * 64 - 1, sb=4), C.INVALID_ARG), (dict(cb=4 * 64, sb=3), C.INVALID_ARG),
    (dict(cb=4 * 64), C.INVALID_ARG), (dict(sb=4), C.INVALID_ARG), (dict(cb=63, ldc=128, sb=4), C.INVALID_ARG),
    (dict(cb=64, ldc=127, sb=4), C.INVALID_ARG), (dict(tile=1, cb=4 * 64), C.INVALID_ARG),
])
def test_outputs_of_a_batch_stay_apart(so, change, status):
    assert quantize(so, **{**dict(batch=2, xb=256), **change}) == status
    assert b"overlap" in so.nvfp4moe_last_error()


def stand_in(E, I, H):
    """Experts whose tensors are on the CPU (the class takes CUDA tensors alone)."""
    w, nI, nH = ops.FP8Experts.__new__(ops.FP8Experts), -(-I // 128), -(-H // 128)
    w.__dict__.update(E=E, I=I, H=H, w13_codes=torch.zeros(E, 2, I, H, dtype=torch.uint8),
                      w13_scale=torch.ones(E, 2, nI, nH), w2_codes=torch.zeros(E, H, I, dtype=torch.uint8),
                      w2_scale=torch.ones(E, nH, nI))
    return w


def test_layer_calls_follow_their_experts(so, monkeypatch):
    """A layer whose experts, top_k or launch are replaced calls the library with the sizes and workspace of the
    new ones (the calls are recorded here, not made)."""
    calls = []
    monkeypatch.setattr(ops, "_same_device", lambda *ts: torch.device("cpu"))
    monkeypatch.setattr(ops, "_call", lambda dev, fn, ref, x, lg, out, ws, n: calls.append((ref._obj, ws, n)))

    def call(layer, T):
        layer(torch.zeros(T, layer.w.H, dtype=torch.bfloat16), torch.zeros(T, layer.w.E))
        d, ws, n = calls[-1]
        return {f: getattr(d, f) for f, _ in d._fields_}, n

    first, second = stand_in(64, 256, 256), stand_in(8, 128, 528)
    layer = ops.FP8MoeFFN(first, 8)
    for T in (4, 40):
        assert call(layer, T)[0]["E"] == 64
    layer.w, layer.top_k = second, 2
    for T in (4, 40):
        d, n = call(layer, T)
        want, m = call(ops.FP8MoeFFN(second, 2), T)
        assert d == want and d["E"] == 8 and d["I"] == 128 and d["H"] == 528 and d["top_k"] == 2
        assert n >= so.fp8_moe_ffn_workspace_size(ctypes.byref(layer.desc(T)))
        assert d["w13_codes"] == second.w13_codes.data_ptr() and d["w2_scale"] == second.w2_scale.data_ptr()
    layer.launch = C.LAUNCH_MULTI
    assert call(layer, 4)[0]["launch_mode"] == C.LAUNCH_MULTI
    layer.top_k = 9
    with pytest.raises(C.Nvfp4MoeError, match="top_k"):
        call(layer, 4)
    with pytest.raises(ValueError, match="FP8Experts"):
        layer.w = object()
    with pytest.raises(AttributeError, match="size"):
        second.E = 64
