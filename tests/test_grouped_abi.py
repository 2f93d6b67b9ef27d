"""Host-side checks of the experts' operators that need no GPU: every bad
argument is refused before CUDA is touched, and calls without rows are no-ops."""
import ctypes

import pytest

from mixture_experts_layer_43_b200 import binding as B
from mixture_experts_layer_43_b200 import build as build_mod

P = 0x10000          # a well-aligned address that no refused call may touch


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return B.lib()


def _g(**kw):
    base = dict(rows=64, n_experts=8, d_in=64, d_out=128, dtype=B.MOE_DTYPE_BF16,
                out_dtype=B.MOE_DTYPE_BF16, accumulate=0, offsets=P, x_stride=64, y_stride=128)
    base.update(kw)
    return B.moe_grouped_t(**base)


BAD = [dict(rows=-1), dict(rows=(1 << 30) + 1), dict(n_experts=0), dict(n_experts=1025),
       dict(d_in=0), dict(d_in=60), dict(d_in=(1 << 20) + 8, x_stride=(1 << 20) + 8),
       dict(d_out=0), dict(d_out=124), dict(d_out=-8), dict(dtype=2), dict(dtype=4), dict(dtype=-1),
       dict(out_dtype=1), dict(out_dtype=3), dict(accumulate=2), dict(accumulate=-1),
       dict(accumulate=1), dict(x_stride=56), dict(x_stride=68), dict(y_stride=120),
       dict(y_stride=130), dict(x_stride=-64), dict(x_stride=1 << 40)]


@pytest.mark.parametrize("kw", BAD, ids=str)
def test_grouped_rejects_bad_descriptions(L, kw):
    g = _g(**kw)
    for f in (L.moe_grouped_gemm, L.moe_grouped_dgrad, L.moe_grouped_wgrad):
        assert f(ctypes.byref(g), P, P, P, None) == B.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [k for k in BAD if "dtype" not in k and "out_dtype" not in k] +
                         [dict(dtype=B.MOE_DTYPE_BF16), dict(out_dtype=B.MOE_DTYPE_I8), dict(d_in=72, x_stride=80),
                          dict(x_stride=72), dict(d_in=131072, x_stride=131072)], ids=str)
def test_i8_rejects_bad_descriptions(L, kw):
    g = _g(**{**dict(dtype=B.MOE_DTYPE_I8), **kw})
    assert L.moe_i8_grouped_gemm(ctypes.byref(g), P, P, P, P, P, None) == B.MOE_ERR_INVALID_ARG


def test_only_wgrad_in_32_bits_accumulates(L):
    g = _g(accumulate=1, out_dtype=B.MOE_DTYPE_F32)
    assert L.moe_grouped_gemm(ctypes.byref(g), P, P, P, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_grouped_dgrad(ctypes.byref(g), P, P, P, None) == B.MOE_ERR_INVALID_ARG


def test_grouped_rejects_bad_pointers(L):
    fs = (L.moe_grouped_gemm, L.moe_grouped_dgrad, L.moe_grouped_wgrad)
    for f in fs:
        assert f(None, P, P, P, None) == B.MOE_ERR_INVALID_ARG
        for i in range(3):
            for bad in (None, P + 8):
                ptr = [P, P, P]
                ptr[i] = bad
                assert f(ctypes.byref(_g()), *ptr, None) == B.MOE_ERR_INVALID_ARG
        for bad in (None, P + 2):
            assert f(ctypes.byref(_g(offsets=bad)), P, P, P, None) == B.MOE_ERR_INVALID_ARG
    g8 = _g(dtype=B.MOE_DTYPE_I8)
    assert L.moe_i8_grouped_gemm(None, P, P, P, P, P, None) == B.MOE_ERR_INVALID_ARG
    for i in range(5):
        for bad in (None, P + (2 if i in (1, 3) else 8)):
            ptr = [P] * 5
            ptr[i] = bad
            assert L.moe_i8_grouped_gemm(ctypes.byref(g8), *ptr, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_i8_grouped_gemm(ctypes.byref(_g(dtype=B.MOE_DTYPE_I8, offsets=None)), P, P, P, P, P,
                                 None) == B.MOE_ERR_INVALID_ARG


def test_calls_without_rows_do_nothing(L):
    g = _g(rows=0, offsets=None)
    assert L.moe_grouped_gemm(ctypes.byref(g), None, None, None, None) == B.MOE_OK
    assert L.moe_grouped_dgrad(ctypes.byref(g), None, None, None, None) == B.MOE_OK
    g = _g(rows=0, offsets=None, dtype=B.MOE_DTYPE_I8)
    assert L.moe_i8_grouped_gemm(ctypes.byref(g), None, None, None, None, None, None) == B.MOE_OK
    assert L.moe_i8_quantize(0, 8, 0, None, 8, None, 8, None, None) == B.MOE_OK
    assert L.moe_swiglu(0, 8, 0, None, None, 8, None, 8, None) == B.MOE_OK
    assert L.moe_swiglu_grad(0, 8, 0, None, 8, None, None, 8, None, None, 8, None) == B.MOE_OK
    assert L.moe_swiglu_i8(0, 8, 0, None, None, 8, None, 8, None, None) == B.MOE_OK
    # a weight gradient without rows still has its zeros to write
    assert L.moe_grouped_wgrad(ctypes.byref(_g(rows=0)), None, None, None, None) == B.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("rows,cols,dtype", [(-1, 64, 0), ((1 << 30) + 1, 64, 0), (4, 0, 0), (4, 60, 0),
                                             (4, (1 << 20) + 8, 0), (4, 64, 2), (4, 64, 3), (4, 64, -1)])
def test_rows_reject_bad_sizes(L, rows, cols, dtype):
    s = max(64, cols)
    assert L.moe_i8_quantize(rows, cols, dtype, P, s, P, s, P, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_swiglu(rows, cols, dtype, P, P, s, P, s, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_swiglu_grad(rows, cols, dtype, P, s, P, P, s, P, P, s, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_swiglu_i8(rows, cols, dtype, P, P, s, P, s, P, None) == B.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [56, 68, -64, 1 << 40])
def test_rows_reject_bad_strides(L, bad):
    I = B.MOE_ERR_INVALID_ARG
    assert L.moe_i8_quantize(4, 64, 0, P, bad, P, 64, P, None) == I
    assert L.moe_i8_quantize(4, 64, 0, P, 64, P, bad, P, None) == I
    assert L.moe_swiglu(4, 64, 0, P, P, bad, P, 64, None) == I
    assert L.moe_swiglu(4, 64, 0, P, P, 64, P, bad, None) == I
    assert L.moe_swiglu_grad(4, 64, 0, P, bad, P, P, 64, P, P, 64, None) == I
    assert L.moe_swiglu_grad(4, 64, 0, P, 64, P, P, bad, P, P, 64, None) == I
    assert L.moe_swiglu_grad(4, 64, 0, P, 64, P, P, 64, P, P, bad, None) == I
    assert L.moe_swiglu_i8(4, 64, 0, P, P, bad, P, 64, P, None) == I
    assert L.moe_swiglu_i8(4, 64, 0, P, P, 64, P, bad, P, None) == I


def test_rows_reject_bad_pointers(L):
    def each(n, call, loose=()):
        for i in range(n):
            for bad in (None, P + (2 if i in loose else 8)):
                ptr = [P] * n
                ptr[i] = bad
                assert call(*ptr) == B.MOE_ERR_INVALID_ARG

    each(3, lambda x, q, s: L.moe_i8_quantize(4, 64, 0, x, 64, q, 64, s, None), loose=(2,))
    each(3, lambda a, b, h: L.moe_swiglu(4, 64, 0, a, b, 64, h, 64, None))
    each(5, lambda d, a, b, p, q: L.moe_swiglu_grad(4, 64, 0, d, 64, a, b, 64, p, q, 64, None))
    each(4, lambda a, b, q, s: L.moe_swiglu_i8(4, 64, 0, a, b, 64, q, 64, s, None), loose=(3,))


def test_binding_raises_with_the_name(L):
    with pytest.raises(B.MoeError, match="moe_grouped_gemm"):
        B.moe_grouped_gemm(_g(d_in=60), P, P, P)
    with pytest.raises(B.MoeError, match="moe_swiglu_i8"):
        B.moe_swiglu_i8(4, 60, 0, P, P, 64, P, 64, P)
