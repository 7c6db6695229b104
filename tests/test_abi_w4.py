"""Host-side checks of the 4-bit weight entry points: bad arguments are refused before anything touches a GPU (fake
pointers, never dereferenced)."""
import ctypes
import math
import os

import pytest

from moe_expert_layer_amd import binding as B


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return B.lib()


def both(L, d, values=0x1000, codes=0x1000, scales=0x1000, zeros=0x1000):
    r = ctypes.byref(d) if d is not None else None
    return [L.moe_quantize_int4(r, values, codes, scales, zeros, None),
            L.moe_dequantize_int4(r, codes, scales, zeros, values, None)]


@pytest.mark.parametrize("field,value", [("rows", -1), ("rows", (1 << 30) + 1), ("k", 0), ("k", -64), ("k", 96),
                                         ("k", (1 << 20) + 64), ("group", 0), ("group", -32), ("group", 16),
                                         ("group", 48), ("group", 96), ("group", 160), ("group", 256), ("dtype", 3),
                                         ("dtype", -1), ("scale_dtype", 3), ("scale_dtype", -1), ("zeros", 2),
                                         ("zeros", -1), ("stride", 127), ("stride", -128), ("stride", (1 << 40) + 1)])
def test_quantize_descriptor(L, field, value):
    d = B.make_int4_desc(10, 128, 64, zeros=True)
    setattr(d, field, value)
    assert both(L, d) == [B.MOE_ERR_INVALID_DESC] * 2
    assert L.moe_last_error()


def test_quantize_pointers(L):
    d = B.make_int4_desc(10, 128, 64, zeros=True)
    assert both(L, None) == [B.MOE_ERR_NULL] * 2
    for bad in ("values", "codes", "scales", "zeros"):
        assert both(L, d, **{bad: None}) == [B.MOE_ERR_NULL] * 2
    assert both(L, B.make_int4_desc(10, 128, 64)) == [B.MOE_ERR_INVALID_DESC] * 2  # zero points that are not asked for
    assert both(L, d, values=0x1001) == both(L, d, codes=0x1008) == both(L, d, scales=0x1001) == [B.MOE_ERR_MISALIGNED] * 2
    assert both(L, B.make_int4_desc(10, 128, 64, dtype="f32", zeros=True), values=0x1002) == [B.MOE_ERR_MISALIGNED] * 2
    assert both(L, B.make_int4_desc(10, 128, 64, scale_dtype="f32", zeros=True), scales=0x1002) == [B.MOE_ERR_MISALIGNED] * 2
    assert both(L, B.make_int4_desc(0, 128, 64, zeros=True), None, None, None, None) == [B.MOE_OK] * 2


NAMES = ["a", "b", "scales", "zeros", "offsets", "c"]


def gemm(L, d, **kw):
    p = {n: 0x1000 for n in NAMES}
    p.update(kw)
    return L.moe_w4_gemm(ctypes.byref(d) if d is not None else None, *[p[n] for n in NAMES], None)


def desc(**kw):
    args = dict(rows=10, n=100, k=256, groups=4, zeros=True)
    args.update(kw)
    return B.make_w4_gemm_desc(**args)


@pytest.mark.parametrize("field,value", [("rows", -1), ("rows", (1 << 30) + 1), ("n", 0), ("n", (1 << 23) + 1), ("k", 0),
                                         ("k", 192), ("k", (1 << 20) + 128), ("groups", 0), ("groups", 1025),
                                         ("group_size", 0), ("group_size", 96), ("group_size", 512), ("weight_format", 2),
                                         ("weight_format", -1), ("weight_format", 1), ("scale_dtype", 3),
                                         ("scale_dtype", -1), ("zeros", 2), ("dtype", 2), ("dtype", 3), ("dtype", -1),
                                         ("out_dtype", 3), ("activation", 2), ("activation", -2), ("a_stride", 255),
                                         ("a_stride", -256), ("a_stride", (1 << 40) + 1), ("out_stride", 99),
                                         ("out_stride", (1 << 40) + 1)])
def test_gemm_descriptor(L, field, value):
    d = desc()
    setattr(d, field, value)
    assert gemm(L, d) == B.MOE_ERR_INVALID_DESC
    assert L.moe_last_error()


def test_gemm_too_many_weight_rows(L):
    assert gemm(L, desc(n=1 << 20, groups=1024)) == B.MOE_ERR_INVALID_DESC


@pytest.mark.parametrize("field,value", [("group_size", 64), ("group_size", 128), ("scale_dtype", 0), ("zeros", 1)])
def test_mxfp4_descriptor(L, field, value):
    d = desc(weight_format="mxfp4", group_size=32, scale_dtype="ue8m0", zeros=False)
    setattr(d, field, value)
    assert gemm(L, d) == B.MOE_ERR_INVALID_DESC


@pytest.mark.parametrize("field,value", [("act_clamp", 0.0), ("act_clamp", -1.0), ("act_clamp", math.nan),
                                         ("act_alpha", math.inf), ("act_up_bias", math.nan)])
def test_activation(L, field, value):
    d = desc(activation="swigluoai", activation_clamp=7.0)
    setattr(d, field, value)
    assert gemm(L, d) == B.MOE_ERR_INVALID_DESC


def test_gemm_pointers(L):
    d = desc()
    assert gemm(L, None) == B.MOE_ERR_NULL
    for n in NAMES:
        assert gemm(L, d, **{n: None}) == B.MOE_ERR_NULL
    assert gemm(L, desc(zeros=False)) == B.MOE_ERR_INVALID_DESC
    assert gemm(L, d, a=0x1001) == gemm(L, d, b=0x1008) == gemm(L, d, scales=0x1001) == B.MOE_ERR_MISALIGNED
    assert gemm(L, d, offsets=0x1002) == gemm(L, d, c=0x1001) == B.MOE_ERR_MISALIGNED
    assert gemm(L, desc(scale_dtype="f32"), scales=0x1002) == B.MOE_ERR_MISALIGNED
    assert gemm(L, desc(out_dtype="f32"), c=0x1002) == B.MOE_ERR_MISALIGNED
    assert gemm(L, desc(rows=0), **{n: None for n in NAMES}) == B.MOE_OK


def test_binding_wants_gpu_tensors():
    import torch
    v, u = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.uint8)
    s = torch.zeros(4, 1, dtype=torch.bfloat16)
    for call in (lambda: B.moe_quantize_int4(B.make_int4_desc(4, 128), v, u, s),
                 lambda: B.moe_dequantize_int4(B.make_int4_desc(4, 128), u, s, None, v),
                 lambda: B.moe_w4_gemm(B.make_w4_gemm_desc(4, 4, 128), v, u, s, None, None, v)):
        with pytest.raises(B.MoeError) as e:
            call()
        assert e.value.status == B.MOE_ERR_UNSUPPORTED
