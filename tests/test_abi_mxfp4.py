"""Host-side checks of the MXFP4 entry points: bad arguments are refused before anything touches a GPU (fake
pointers, never dereferenced)."""
import ctypes
import os

import pytest

from moe_expert_layer_amd import binding as B


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(B.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return B.lib()


def both(L, d, values=0x1000, codes=0x1000, sf=0x1000):
    r = ctypes.byref(d) if d is not None else None
    return [L.moe_quantize_mxfp4(r, values, codes, sf, None), L.moe_dequantize_mxfp4(r, codes, sf, values, None)]


@pytest.mark.parametrize("field,value", [("rows", -1), ("rows", (1 << 30) + 1), ("k", 0), ("k", 16), ("k", 100),
                                         ("k", (1 << 20) + 32), ("dtype", 3), ("dtype", -1), ("scale_layout", 2),
                                         ("stride", 63), ("stride", -64), ("stride", (1 << 40) + 1)])
def test_quantize_descriptor(L, field, value):
    d = B.make_mxfp4_desc(10, 64)
    setattr(d, field, value)
    assert both(L, d) == [B.MOE_ERR_INVALID_DESC] * 2
    assert L.moe_last_error()


def test_quantize_pointers(L):
    d = B.make_mxfp4_desc(10, 64)
    assert both(L, None) == [B.MOE_ERR_NULL] * 2
    for bad in ("values", "codes", "sf"):
        assert both(L, d, **{bad: None}) == [B.MOE_ERR_NULL] * 2
    assert both(L, d, values=0x1001) == [B.MOE_ERR_MISALIGNED] * 2
    assert both(L, d, codes=0x1008) == [B.MOE_ERR_MISALIGNED] * 2
    assert both(L, B.make_mxfp4_desc(10, 64, scale_layout="packed"), sf=0x1002) == [B.MOE_ERR_MISALIGNED] * 2
    assert both(L, B.make_mxfp4_desc(10, 64, dtype="f32"), values=0x1002) == [B.MOE_ERR_MISALIGNED] * 2
    assert both(L, B.make_mxfp4_desc(0, 64), None, None, None) == [B.MOE_OK] * 2


def gemm(L, d, *p):
    return L.moe_mxfp4_gemm(ctypes.byref(d) if d is not None else None, *(p or [0x1000] * 6), None)


@pytest.mark.parametrize("field,value", [("rows", -1), ("rows", (1 << 30) + 1), ("n", 0), ("n", (1 << 24) + 1), ("k", 0),
                                         ("k", 48), ("k", (1 << 20) + 32), ("groups", 0), ("groups", 1025),
                                         ("out_dtype", 3), ("a_scale_layout", 2), ("b_scale_layout", -1),
                                         ("variant", 99), ("variant", -2), ("out_stride", 99),
                                         ("out_stride", (1 << 40) + 1)])
def test_gemm_descriptor(L, field, value):
    d = B.make_mxfp4_gemm_desc(10, 100, 128, groups=4)
    setattr(d, field, value)
    assert gemm(L, d) == B.MOE_ERR_INVALID_DESC


def test_gemm_pointers(L):
    d = B.make_mxfp4_gemm_desc(10, 100, 128, groups=4)
    assert gemm(L, None) == B.MOE_ERR_NULL
    for i in range(6):
        p = [0x1000] * 6
        p[i] = None
        assert gemm(L, d, *p) == B.MOE_ERR_NULL
    for i, at in ((0, 0x1008), (1, 0x1002), (2, 0x1008), (3, 0x1002), (4, 0x1002), (5, 0x1001)):
        p = [0x1000] * 6
        p[i] = at
        assert gemm(L, d, *p) == B.MOE_ERR_MISALIGNED
    assert gemm(L, B.make_mxfp4_gemm_desc(0, 100, 128), *[None] * 6) == B.MOE_OK
    for kw in ({"a_scale_layout": "rows"}, {"b_scale_layout": "rows"}):  # a scale word would span two rows
        assert gemm(L, B.make_mxfp4_gemm_desc(10, 100, 160, **kw)) == B.MOE_ERR_UNSUPPORTED
    assert gemm(L, B.make_mxfp4_gemm_desc(10, 1 << 24, 128, groups=65)) == B.MOE_ERR_INVALID_DESC


def test_binding_wants_gpu_tensors():
    import torch
    v = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(B.MoeError) as e:
        B.moe_quantize_mxfp4(B.make_mxfp4_desc(4, 64), v, torch.zeros(4, 32, dtype=torch.uint8),
                             torch.zeros(4, 2, dtype=torch.uint8))
    assert e.value.status == B.MOE_ERR_UNSUPPORTED
