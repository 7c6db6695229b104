"""Host-side checks of the balance loss entry points: bad arguments are refused before anything touches a GPU (fake
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


def desc(**kw):
    args = dict(num_tokens=5000, num_experts=40, topk=3, num_seqs=4)
    args.update(kw)
    return B.make_balance_desc(**args)


NAMES = ["logits", "ids", "mask", "offsets", "counts", "tokens", "psum", "balance", "z"]
BACK = ["logits", "mask", "offsets", "counts", "tokens", "dbalance", "dz", "add", "dlogits"]


def forward(L, d, ws=0x100000, size=1 << 30, **kw):
    p = {n: 0x1000 for n in NAMES}
    p.update(kw)
    return L.moe_balance_loss(ctypes.byref(d) if d is not None else None, *[p[n] for n in NAMES], ws, size, None)


def backward(L, d, **kw):
    p = {n: 0x1000 for n in BACK}
    p.update(kw)
    return L.moe_balance_loss_backward(ctypes.byref(d) if d is not None else None, *[p[n] for n in BACK], None)


@pytest.mark.parametrize("field,value", [("num_tokens", -1), ("num_experts", 0), ("num_experts", 1025), ("topk", 0),
                                         ("topk", 17), ("num_tokens", 1 << 30), ("num_seqs", 0), ("num_seqs", 65537),
                                         ("dtype", 3), ("dtype", -1), ("score", 2), ("score", -1), ("logit_stride", 39),
                                         ("logit_stride", -40), ("grad_stride", 1), ("grad_stride", (1 << 40) + 1)])
def test_bad_descriptor(L, field, value):
    d = desc()
    setattr(d, field, value)
    n = ctypes.c_size_t(0)
    assert L.moe_balance_workspace_size(ctypes.byref(d), ctypes.byref(n)) == B.MOE_ERR_INVALID_DESC
    assert L.moe_last_error()
    assert forward(L, d) == backward(L, d) == B.MOE_ERR_INVALID_DESC


def test_pointers(L):
    d = desc()
    assert L.moe_balance_workspace_size(None, None) == B.MOE_ERR_NULL
    assert L.moe_balance_workspace_size(ctypes.byref(d), None) == B.MOE_ERR_NULL
    assert forward(L, None) == backward(L, None) == B.MOE_ERR_NULL
    for n in ("logits", "ids", "counts", "tokens", "psum", "balance", "offsets"):
        assert forward(L, d, **{n: None}) == B.MOE_ERR_NULL
    for n in ("logits", "counts", "tokens", "dbalance", "dlogits", "offsets"):
        assert backward(L, d, **{n: None}) == B.MOE_ERR_NULL
    for n in NAMES:
        if n != "mask":
            assert forward(L, d, **{n: 0x1002}) == B.MOE_ERR_MISALIGNED
    for n in BACK:
        if n != "mask":
            assert backward(L, d, **{n: 0x1002}) == B.MOE_ERR_MISALIGNED
    assert forward(L, desc(dtype="bf16"), logits=0x1001) == B.MOE_ERR_MISALIGNED


def test_z_goes_with_softmax(L):
    d = desc(score="sigmoid")
    assert forward(L, d) == backward(L, d) == B.MOE_ERR_UNSUPPORTED


def test_workspace(L):
    for kw in (dict(), dict(num_tokens=1), dict(num_tokens=1 << 20, num_experts=1024, num_seqs=65536)):
        d = desc(**kw)
        need = B.moe_balance_workspace_size(d)
        assert need % 256 == 0
        assert forward(L, d, ws=None, size=need) == B.MOE_ERR_WORKSPACE
        assert forward(L, d, ws=0x100010, size=need) == B.MOE_ERR_MISALIGNED
        if need:
            assert forward(L, d, size=need - 1) == B.MOE_ERR_WORKSPACE


def test_no_tokens_is_a_noop(L):
    d = desc(num_tokens=0)
    assert forward(L, d, None, 0, **{n: None for n in NAMES}) == B.MOE_OK
    assert backward(L, d, **{n: None for n in BACK}) == B.MOE_OK


def test_binding_wants_gpu_tensors():
    import torch
    d = desc(num_tokens=4, num_seqs=1)
    f, i = torch.zeros(4, 40), torch.zeros(160, dtype=torch.int32)
    with pytest.raises(B.MoeError) as e:
        B.moe_balance_loss(d, f, i, i, i, f, f, torch.zeros(256, dtype=torch.uint8))
    assert e.value.status == B.MOE_ERR_UNSUPPORTED
    with pytest.raises(B.MoeError) as e:
        B.moe_balance_loss_backward(d, f, i, i, f, f)
    assert e.value.status == B.MOE_ERR_UNSUPPORTED
