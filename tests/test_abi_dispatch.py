"""Host-side checks of the sort / dispatch / combine entry points: bad arguments are refused before
anything touches a GPU (fake pointers, never dereferenced)."""
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


def desc(**kw):
    args = dict(num_tokens=64, hidden=100, num_experts=8, topk=2)
    args.update(kw)
    return B.make_dispatch_desc(**args)


BAD = [("num_tokens", -1), ("hidden", 0), ("hidden", (1 << 20) + 1), ("num_experts", 0), ("num_experts", 1025),
       ("num_local", 0), ("num_local", 9), ("local_begin", -1), ("local_begin", 1), ("topk", 0), ("topk", 17),
       ("num_tokens", 1 << 30), ("num_tokens", (1 << 30) - (1 << 16) + 1), ("dtype", 4), ("dtype", -1), ("max_rows", -1), ("max_rows", 129), ("token_stride", 99),
       ("token_stride", -100), ("row_stride", 1), ("row_stride", (1 << 40) + 1)]


def calls(L, d, p, ws=0x100000):
    r = ctypes.byref(d)
    return [L.moe_sort_tokens(r, p, p, p, p, p, ws, 1 << 30, None), L.moe_dispatch(r, p, p, p, None),
            L.moe_dispatch_backward(r, p, p, p, None), L.moe_combine(r, p, p, p, p, None),
            L.moe_combine_backward(r, p, p, p, p, p, p, p, p, None)]


@pytest.mark.parametrize("field,value", BAD)
def test_bad_descriptor(L, field, value):
    d = desc()
    setattr(d, field, value)
    n = ctypes.c_size_t(0)
    assert L.moe_sort_workspace_size(ctypes.byref(d), ctypes.byref(n)) == B.MOE_ERR_INVALID_DESC
    assert L.moe_last_error()
    assert calls(L, d, 0x1000) == [B.MOE_ERR_INVALID_DESC] * 5


def test_null_and_misaligned(L):
    d = desc()
    assert L.moe_sort_workspace_size(None, None) == B.MOE_ERR_NULL
    assert L.moe_sort_workspace_size(ctypes.byref(d), None) == B.MOE_ERR_NULL
    assert calls(L, d, None) == [B.MOE_ERR_NULL] * 5
    assert calls(L, d, 0x1001) == [B.MOE_ERR_MISALIGNED] * 5
    r, p = ctypes.byref(d), 0x1000
    for i in range(6):  # each required pointer of the backward call by itself
        a = [p] * 6
        a[i] = None
        assert L.moe_combine_backward(r, *a, p, p, None) == B.MOE_ERR_NULL
    assert L.moe_combine_backward(r, p, p, p, p, p, p, None, p, None) == B.MOE_ERR_NULL  # dlogits without ids
    # odd addresses are fine for bytes, and only there
    d.dtype = B.MOE_DT_F32
    assert L.moe_dispatch(r, 0x1002, p, p, None) == B.MOE_ERR_MISALIGNED
    d.dtype = B.MOE_DT_U8
    assert L.moe_dispatch(r, 0x1001, 0x1002, 0x1003, None) == B.MOE_ERR_MISALIGNED  # the map


def test_bytes_are_not_summed(L):
    assert calls(L, desc(dtype="u8"), None)[2:] == [B.MOE_ERR_UNSUPPORTED] * 3


def test_sort_workspace(L):
    d = desc(num_tokens=5000, num_experts=300, topk=8, local_begin=7, num_local=200)
    need = B.moe_sort_workspace_size(d)
    chunks = (5000 * 8 + 1023) // 1024
    assert need % 256 == 0 and need >= 2 * chunks * 201 * 4 + 201 * 4
    r, p = ctypes.byref(d), 0x1000
    assert L.moe_sort_tokens(r, p, p, p, p, p, 0x100000, need - 1, None) == B.MOE_ERR_WORKSPACE
    assert L.moe_sort_tokens(r, p, p, p, p, p, None, need, None) == B.MOE_ERR_WORKSPACE
    assert L.moe_sort_tokens(r, p, p, p, p, p, 0x100010, need, None) == B.MOE_ERR_MISALIGNED


def test_no_tokens_is_a_noop(L):
    assert calls(L, desc(num_tokens=0), None) == [B.MOE_OK] * 5


def test_binding_wants_gpu_tensors():
    import torch
    d = desc(num_tokens=4, hidden=8)
    x, m = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int32)
    with pytest.raises(B.MoeError) as e:
        B.moe_dispatch(d, x, m, torch.zeros(8, 8, dtype=torch.bfloat16))
    assert e.value.status == B.MOE_ERR_UNSUPPORTED
