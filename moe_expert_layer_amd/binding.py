"""Thin ctypes binding over the C ABI in include/moe_expert_layer.h.

Argument marshalling only: every step of the layer runs in the HIP library.  Tensors
are torch device tensors (torch provides device memory and the current HIP stream);
the functions carry the C names.  If the shared library is missing or fails to load,
every call raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe_expert_layer.so")

MOE_OK, MOE_ERR_NULL, MOE_ERR_INVALID_DESC, MOE_ERR_MISALIGNED, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, \
    MOE_ERR_DEVICE = range(7)
MOE_ACT_SWIGLU, MOE_ACT_SWIGLU_OAI = 0, 1
MOE_W_FP8_E4M3_B128, MOE_W_MXFP4_E2M1_B32, MOE_W_FP8_E5M2_B128, MOE_W_BF16 = 0, 1, 2, 3
ACTIVATIONS = {"swiglu": MOE_ACT_SWIGLU, "swigluoai": MOE_ACT_SWIGLU_OAI}
MOE_SCALE_BLOCK, MOE_SCALE_TENSOR = 0, 1
MOE_SF_ROW_MAJOR, MOE_SF_PACKED_MN = 0, 1
SCALE_LAYOUTS = {"rows": MOE_SF_ROW_MAJOR, "packed": MOE_SF_PACKED_MN}
SCALINGS = {"block": MOE_SCALE_BLOCK, "tensor": MOE_SCALE_TENSOR}
WEIGHT_FORMATS = {"fp8": MOE_W_FP8_E4M3_B128, "mxfp4": MOE_W_MXFP4_E2M1_B32, "fp8e5m2": MOE_W_FP8_E5M2_B128, "bf16": MOE_W_BF16}


class MoeLayerDesc(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
        ("num_experts", ctypes.c_int32), ("local_begin", ctypes.c_int32), ("num_local", ctypes.c_int32),
        ("topk", ctypes.c_int32), ("weight_format", ctypes.c_int32), ("activation", ctypes.c_int32),
        ("act_clamp", ctypes.c_float), ("act_alpha", ctypes.c_float), ("act_up_bias", ctypes.c_float),
        ("variant", ctypes.c_int32), ("scale_mode", ctypes.c_int32), ("h_scale", ctypes.c_float),
        ("num_shared", ctypes.c_int32), ("scale_layout", ctypes.c_int32),
    ]


MOE_DT_BF16, MOE_DT_F16, MOE_DT_F32, MOE_DT_U8 = range(4)
DTYPES = {"bf16": MOE_DT_BF16, "f16": MOE_DT_F16, "f32": MOE_DT_F32, "u8": MOE_DT_U8}
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
MOE_W4_INT4, MOE_W4_MXFP4 = 0, 1
W4_FORMATS = {"int4": MOE_W4_INT4, "mxfp4": MOE_W4_MXFP4}


class MoeDispatchDesc(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("num_experts", ctypes.c_int32),
        ("local_begin", ctypes.c_int32), ("num_local", ctypes.c_int32), ("topk", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("max_rows", ctypes.c_int32), ("token_stride", ctypes.c_int64),
        ("row_stride", ctypes.c_int64),
    ]


class MoeMxfp4Desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("k", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale_layout", ctypes.c_int32), ("stride", ctypes.c_int64)]


class MoeMxfp4GemmDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("a_scale_layout", ctypes.c_int32), ("b_scale_layout", ctypes.c_int32),
                ("variant", ctypes.c_int32), ("out_stride", ctypes.c_int64)]


class MoeBalanceDesc(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("num_experts", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("num_seqs", ctypes.c_int32), ("dtype", ctypes.c_int32), ("score", ctypes.c_int32),
                ("logit_stride", ctypes.c_int64), ("grad_stride", ctypes.c_int64)]


class MoeInt4Desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("k", ctypes.c_int32), ("group", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int32), ("zeros", ctypes.c_int32), ("stride", ctypes.c_int64)]


class MoeW4GemmDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("weight_format", ctypes.c_int32), ("group_size", ctypes.c_int32), ("scale_dtype", ctypes.c_int32),
                ("zeros", ctypes.c_int32), ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("act_clamp", ctypes.c_float), ("act_alpha", ctypes.c_float),
                ("act_up_bias", ctypes.c_float), ("a_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64)]


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{status_str(status)}: {msg}")
        self.status = status


_lib = None


def lib():
    """The loaded C library (raises if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"HIP library not built: {LIB_PATH} (run __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        P, S, I32, VP = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p
        D = ctypes.POINTER(MoeLayerDesc)
        L.moe_abi_version.restype = ctypes.c_int
        L.moe_status_str.restype = ctypes.c_char_p
        L.moe_status_str.argtypes = [I32]
        L.moe_last_error.restype = ctypes.c_char_p
        L.moe_desc_defaults.restype = I32
        L.moe_desc_defaults.argtypes = [D]
        L.moe_workspace_size.restype = I32
        L.moe_workspace_size.argtypes = [D, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_route_permute.restype = I32
        L.moe_route_permute.argtypes = [D, P, P, P, P, P, P, P, P, S, VP]
        L.moe_grouped_fc1_swiglu.restype = I32
        L.moe_grouped_fc1_swiglu.argtypes = [D, P, P, P, P, P, P, P, P, P, S, VP]
        L.moe_grouped_fc2_combine.restype = I32
        L.moe_grouped_fc2_combine.argtypes = [D, P, P, P, P, P, P, P, P, P, P, S, VP]
        L.moe_layer.restype = I32
        L.moe_layer.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, S, VP]
        L.moe_static_scratch_bytes.restype = ctypes.c_size_t
        L.moe_static_scratch_bytes.argtypes = []
        L.moe_layer_static.restype = I32
        L.moe_layer_static.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, P, P, P, VP]
        L.moe_quantize_act.restype = I32
        L.moe_quantize_act.argtypes = [D, P, P, P, VP]
        L.moe_pack_scales.restype = I32
        L.moe_pack_scales.argtypes = [I32, I32, P, P, VP]
        L.moe_unpack_scales.restype = I32
        L.moe_unpack_scales.argtypes = [I32, I32, P, P, VP]
        DD = ctypes.POINTER(MoeDispatchDesc)
        for name, args in {
            "moe_sort_workspace_size": [DD, ctypes.POINTER(ctypes.c_size_t)],
            "moe_sort_tokens": [DD, P, P, P, P, P, P, S, VP],
            "moe_dispatch": [DD, P, P, P, VP],
            "moe_dispatch_backward": [DD, P, P, P, VP],
            "moe_combine": [DD, P, P, P, P, VP],
            "moe_combine_backward": [DD, P, P, P, P, P, P, P, P, VP],
            "moe_quantize_mxfp4": [ctypes.POINTER(MoeMxfp4Desc), P, P, P, VP],
            "moe_dequantize_mxfp4": [ctypes.POINTER(MoeMxfp4Desc), P, P, P, VP],
            "moe_mxfp4_gemm": [ctypes.POINTER(MoeMxfp4GemmDesc), P, P, P, P, P, P, VP],
            "moe_balance_workspace_size": [ctypes.POINTER(MoeBalanceDesc), ctypes.POINTER(ctypes.c_size_t)],
            "moe_balance_loss": [ctypes.POINTER(MoeBalanceDesc), P, P, P, P, P, P, P, P, P, P, S, VP],
            "moe_balance_loss_backward": [ctypes.POINTER(MoeBalanceDesc), P, P, P, P, P, P, P, P, P, VP],
            "moe_quantize_int4": [ctypes.POINTER(MoeInt4Desc), P, P, P, P, VP],
            "moe_dequantize_int4": [ctypes.POINTER(MoeInt4Desc), P, P, P, P, VP],
            "moe_w4_gemm": [ctypes.POINTER(MoeW4GemmDesc), P, P, P, P, P, P, VP],
        }.items():
            f = getattr(L, name)
            f.restype, f.argtypes = I32, args
        _lib = L
    return _lib


def status_str(st: int) -> str:
    return lib().moe_status_str(st).decode()


def _check(st: int):
    if st != MOE_OK:
        raise MoeError(st, lib().moe_last_error().decode())


def make_desc(num_tokens: int, hidden: int, inter: int, num_experts: int, topk: int, local_begin: int = 0,
              num_local: Optional[int] = None, weight_format: str = "fp8", activation: str = "swiglu",
              activation_clamp: Optional[float] = None, activation_alpha: float = 1.0,
              activation_up_bias: float = 0.0, variant: int = -1, scaling: str = "block",
              h_scale: float = 1.0, num_shared: int = 0, scale_layout: str = "rows") -> MoeLayerDesc:
    """Descriptor with the pages' keyword names (activation, activation_clamp/alpha/up_bias).

    weight_format: "fp8" (E4M3), "fp8e5m2", "mxfp4" or "bf16" (the whole layer in BF16);
    scaling: "block" (UE8M0 scale tensors) or "tensor" (float32 scales, static h_scale);
    num_shared: shared experts after the local ones in the weight tensors;
    scale_layout: "rows" (UE8M0 bytes [rows, groups]) or "packed" (int32 MN-major words) for x_sf / h_sf."""
    d = MoeLayerDesc()
    _check(lib().moe_desc_defaults(ctypes.byref(d)))
    d.num_tokens, d.hidden, d.inter = num_tokens, hidden, inter
    d.num_experts, d.topk = num_experts, topk
    d.local_begin = local_begin
    d.num_local = num_experts if num_local is None else num_local
    d.weight_format = WEIGHT_FORMATS[weight_format]
    d.activation = ACTIVATIONS[activation]
    d.act_clamp = math.inf if activation_clamp is None else activation_clamp
    d.act_alpha, d.act_up_bias = activation_alpha, activation_up_bias
    d.variant = variant
    d.scale_mode = SCALINGS[scaling]
    d.h_scale = h_scale
    d.num_shared = num_shared
    d.scale_layout = SCALE_LAYOUTS[scale_layout]
    return d


def desc_from_workload(w, variant: int = -1, scale_layout: str = "rows") -> MoeLayerDesc:
    return make_desc(w.tokens, w.hidden, w.inter, w.num_experts, w.topk, w.local_begin, w.num_local,
                     w.weight_format, w.activation, w.act_clamp, w.act_alpha, w.act_up_bias, variant,
                     getattr(w, "scaling", "block"), getattr(w, "h_scale", 1.0), getattr(w, "num_shared", 0),
                     scale_layout)


def moe_workspace_size(desc: MoeLayerDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_workspace_size(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def moe_route_permute(desc, logits, topk_ids, topk_w, counts, offsets, row_to_slot, slot_to_row, workspace,
                      stream=None):
    _check(lib().moe_route_permute(ctypes.byref(desc), _ptr(logits), _ptr(topk_ids), _ptr(topk_w), _ptr(counts),
                                   _ptr(offsets), _ptr(row_to_slot), _ptr(slot_to_row), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_grouped_fc1_swiglu(desc, x, x_sf, w1, w1_sf, offsets, row_to_slot, h, h_sf, workspace, stream=None):
    _check(lib().moe_grouped_fc1_swiglu(ctypes.byref(desc), _ptr(x), _ptr(x_sf), _ptr(w1), _ptr(w1_sf),
                                        _ptr(offsets), _ptr(row_to_slot), _ptr(h), _ptr(h_sf), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_grouped_fc2_combine(desc, h, h_sf, w2, w2_sf, offsets, row_to_slot, slot_to_row, topk_w, y, workspace,
                            stream=None):
    _check(lib().moe_grouped_fc2_combine(ctypes.byref(desc), _ptr(h), _ptr(h_sf), _ptr(w2), _ptr(w2_sf),
                                         _ptr(offsets), _ptr(row_to_slot), _ptr(slot_to_row), _ptr(topk_w), _ptr(y),
                                         _ptr(workspace), workspace.numel() * workspace.element_size(),
                                         _stream(stream)))


def moe_layer(desc, logits, x, x_sf, w1, w1_sf, w2, w2_sf, y, workspace, topk_ids=None, topk_w=None, counts=None,
              offsets=None, row_to_slot=None, slot_to_row=None, stream=None):
    _check(lib().moe_layer(ctypes.byref(desc), _ptr(logits), _ptr(x), _ptr(x_sf), _ptr(w1), _ptr(w1_sf), _ptr(w2),
                           _ptr(w2_sf), _ptr(y), _ptr(topk_ids), _ptr(topk_w), _ptr(counts), _ptr(offsets),
                           _ptr(row_to_slot), _ptr(slot_to_row), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_layer_static(desc, logits, x, x_sf, w1, w1_sf, w2, w2_sf, y, topk_ids=None, topk_w=None, counts=None,
                     offsets=None, row_to_slot=None, slot_to_row=None, stream=None):
    """moe_layer with the library's static scratch array instead of a workspace (allocates nothing)."""
    _check(lib().moe_layer_static(ctypes.byref(desc), _ptr(logits), _ptr(x), _ptr(x_sf), _ptr(w1), _ptr(w1_sf),
                                  _ptr(w2), _ptr(w2_sf), _ptr(y), _ptr(topk_ids), _ptr(topk_w), _ptr(counts),
                                  _ptr(offsets), _ptr(row_to_slot), _ptr(slot_to_row), _stream(stream)))


def moe_quantize_act(desc, x_bf16, x, x_sf, stream=None):
    """bf16 activations [T, H] (int16/uint16/bfloat16 tensor) -> E4M3 codes x [T, H] and UE8M0 x_sf [T, H/128]."""
    _check(lib().moe_quantize_act(ctypes.byref(desc), _ptr(x_bf16), _ptr(x), _ptr(x_sf), _stream(stream)))


def moe_pack_scales(rows, groups, sf, packed, stream=None):
    """UE8M0 bytes [rows, groups] -> packed int32 words [ceil(groups/4) * pad_up(rows, 4)] (MN-major)."""
    _check(lib().moe_pack_scales(rows, groups, _ptr(sf), _ptr(packed), _stream(stream)))


def moe_unpack_scales(rows, groups, packed, sf, stream=None):
    """Inverse of moe_pack_scales."""
    _check(lib().moe_unpack_scales(rows, groups, _ptr(packed), _ptr(sf), _stream(stream)))


def alloc_workspace(desc, device="cuda"):
    """A uint8 device tensor of moe_workspace_size(desc) bytes (torch allocations are 256-byte aligned)."""
    import torch
    return torch.empty(max(moe_workspace_size(desc), 256), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------------------------------
# operators beside the layer.  Their tensors carry their sizes, so these functions also check them
# against the descriptor (dtype, shape, row stride, device) before they hand out pointers, and run on
# the tensors' device whichever device is current.

def _refuse(status: int, msg: str):
    raise MoeError(status, msg)


def _rows_tensor(name, t, dtype, rows, cols, stride, dev, at_least=False):
    """A [rows, cols] tensor of dtype on device dev whose rows lie stride elements apart (at_least: it
    may have more rows)."""
    sh = t.shape
    if t.dtype is not dtype or t.get_device() != dev or len(sh) != 2 or sh[1] != cols or (
            sh[0] < rows if at_least else sh[0] != rows):
        _refuse_tensor(name, t, dtype, dev, f"({rows}, {cols})")
    st = t.stride()
    if (st[1] != 1 and cols > 1) or (st[0] != stride and rows > 1):
        _refuse(MOE_ERR_INVALID_DESC, f"{name} has strides {st}, not ({stride}, 1)")


def _array(name, t, dtype, n, dev):
    """A dense tensor of dtype with at least n elements on device dev."""
    if t.dtype is not dtype or t.get_device() != dev or t.numel() < n or not t.is_contiguous():
        _refuse_tensor(name, t, dtype, dev, f"{n} elements, contiguous")


def _refuse_tensor(name, t, dtype, dev, wanted):
    if t.dtype is not dtype:
        _refuse(MOE_ERR_INVALID_DESC, f"{name} is {t.dtype}, not {dtype}")
    if t.get_device() != dev:
        _refuse(MOE_ERR_UNSUPPORTED, f"{name} is not on the GPU of the other tensors")
    _refuse(MOE_ERR_INVALID_DESC, f"{name} has shape {tuple(t.shape)} and strides {t.stride()}, not {wanted}")


def _device_of(t) -> int:
    dev = t.get_device()
    if dev < 0:
        _refuse(MOE_ERR_UNSUPPORTED, "tensors must be on a GPU")
    return dev


class _Torch:
    """What the calls below need of torch, looked up once (torch is imported with the first call, not with this module)."""

    def __init__(self):
        import torch
        self.raw_stream, self.current = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        self.device = torch.cuda.device
        self.i32, self.f32, self.u8, self.bool = torch.int32, torch.float32, torch.uint8, torch.bool
        self.dtypes = {MOE_DT_BF16: torch.bfloat16, MOE_DT_F16: torch.float16, MOE_DT_F32: torch.float32,
                       MOE_DT_U8: torch.uint8}


_torch_names = None


def _torch() -> _Torch:
    global _torch_names
    if _torch_names is None:
        _torch_names = _Torch()
    return _torch_names


def _launch(fn, dev: int, stream, *args):
    """fn(*args, stream) with device dev current, on its current stream unless one is given."""
    T = _torch()
    if stream is None:
        raw = T.raw_stream(dev)
    else:
        if stream.device.index != dev:
            _refuse(MOE_ERR_UNSUPPORTED, f"stream of GPU {stream.device.index}, tensors on GPU {dev}")
        raw = stream.cuda_stream
    if T.current() == dev:
        st = fn(*args, raw)
    else:
        with T.device(dev):
            st = fn(*args, raw)
    if st:
        _check(st)


def _torch_dtype(dtype: int):
    t = _torch().dtypes.get(dtype)
    if t is None:
        _refuse(MOE_ERR_INVALID_DESC, f"dtype {dtype} unknown")
    return t


def make_dispatch_desc(num_tokens: int, hidden: int, num_experts: int, topk: int, local_begin: int = 0,
                       num_local: Optional[int] = None, dtype: str = "bf16", max_rows: int = 0, token_stride: int = 0,
                       row_stride: int = 0) -> MoeDispatchDesc:
    """Descriptor of tokens in expert order.  dtype: "bf16", "f16", "f32" or "u8" (bytes, moe_dispatch only);
    max_rows: rows of the expert-ordered tensors (0 = num_tokens * topk); strides in elements (0 = hidden)."""
    return MoeDispatchDesc(num_tokens, hidden, num_experts, local_begin,
                           num_experts - local_begin if num_local is None else num_local, topk, DTYPES[dtype],
                           max_rows, token_stride, row_stride)


def moe_sort_workspace_size(desc: MoeDispatchDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_sort_workspace_size(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def alloc_sort_workspace(desc: MoeDispatchDesc, device="cuda"):
    """A uint8 device tensor of moe_sort_workspace_size(desc) bytes."""
    import torch
    return torch.empty(max(moe_sort_workspace_size(desc), 256), dtype=torch.uint8, device=device)


class _DispatchView:
    """A dispatch descriptor's fields as the checks below want them."""

    def __init__(self, d):
        T = _torch()
        self.i32, self.f32, self.u8, self.dtype = T.i32, T.f32, T.u8, _torch_dtype(d.dtype)
        self.slots, self.hidden, self.num_local = d.num_tokens * d.topk, d.hidden, d.num_local
        self.logits = d.num_tokens * d.num_experts
        self.tokens, self.rows = (d.num_tokens, d.hidden), (d.max_rows or self.slots, d.hidden)
        self.token_stride, self.row_stride = (d.token_stride or d.hidden, 1), (d.row_stride or d.hidden, 1)

    def token_tensor(self, name, t, dev):
        # the usual case in one line, every other one (a single row or column, a fault) by the book
        if t.dtype is not self.dtype or t.get_device() != dev or t.shape != self.tokens or t.stride() != self.token_stride:
            _rows_tensor(name, t, self.dtype, *self.tokens, self.token_stride[0], dev)

    def expert_tensor(self, name, t, dev):
        if t.dtype is not self.dtype or t.get_device() != dev or t.shape != self.rows or t.stride() != self.row_stride:
            _rows_tensor(name, t, self.dtype, *self.rows, self.row_stride[0], dev, at_least=True)


_views = {}  # (view's class, descriptor bytes) -> view: a descriptor may change between calls, its bytes say whether it did


def _view(cls, desc):
    key = (cls, bytes(desc))
    v = _views.get(key)
    if v is None:
        if len(_views) >= 1024:
            _views.clear()
        v = _views[key] = cls(desc)
    return v


def moe_sort_tokens(desc, topk_ids, counts, offsets, row_to_slot, slot_to_row, workspace, stream=None):
    """Expert ids int32 [T, k] -> counts, offsets, row_to_slot, slot_to_row (int32), as moe_route_permute writes them."""
    v, dev = _view(_DispatchView, desc), _device_of(topk_ids)
    n, i32 = v.slots, v.i32
    _array("topk_ids", topk_ids, i32, n, dev)
    _array("counts", counts, i32, v.num_local, dev)
    _array("offsets", offsets, i32, v.num_local + 1, dev)
    _array("row_to_slot", row_to_slot, i32, n, dev)
    _array("slot_to_row", slot_to_row, i32, n, dev)
    _array("workspace", workspace, v.u8, 0, dev)
    _launch(lib().moe_sort_tokens, dev, stream, ctypes.byref(desc), topk_ids.data_ptr(), counts.data_ptr(),
            offsets.data_ptr(), row_to_slot.data_ptr(), slot_to_row.data_ptr(), workspace.data_ptr(), workspace.numel())


def moe_dispatch(desc, x, slot_to_row, xs, stream=None):
    """Token rows x [T, H] -> expert-ordered rows xs [max_rows, H] (rows that no slot owns are left as they were)."""
    v, dev = _view(_DispatchView, desc), _device_of(x)
    v.token_tensor("x", x, dev)
    _array("slot_to_row", slot_to_row, v.i32, v.slots, dev)
    v.expert_tensor("xs", xs, dev)
    _launch(lib().moe_dispatch, dev, stream, ctypes.byref(desc), x.data_ptr(), slot_to_row.data_ptr(), xs.data_ptr())


def moe_dispatch_backward(desc, dxs, slot_to_row, dx, stream=None):
    """Gradient of moe_dispatch: dx[t] = the sum of the rows of dxs that token t went to."""
    v, dev = _view(_DispatchView, desc), _device_of(dxs)
    v.expert_tensor("dxs", dxs, dev)
    _array("slot_to_row", slot_to_row, v.i32, v.slots, dev)
    v.token_tensor("dx", dx, dev)
    _launch(lib().moe_dispatch_backward, dev, stream, ctypes.byref(desc), dxs.data_ptr(), slot_to_row.data_ptr(),
            dx.data_ptr())


def moe_combine(desc, ys, slot_to_row, topk_w, y, stream=None):
    """Expert-ordered rows ys -> y[t] = sum_j topk_w[t, j] * ys[slot_to_row[t, j]], in token order."""
    v, dev = _view(_DispatchView, desc), _device_of(ys)
    v.expert_tensor("ys", ys, dev)
    _array("slot_to_row", slot_to_row, v.i32, v.slots, dev)
    _array("topk_w", topk_w, v.f32, v.slots, dev)
    v.token_tensor("y", y, dev)
    _launch(lib().moe_combine, dev, stream, ctypes.byref(desc), ys.data_ptr(), slot_to_row.data_ptr(),
            topk_w.data_ptr(), y.data_ptr())


def moe_combine_backward(desc, dy, ys, slot_to_row, topk_w, dys, dw, topk_ids=None, dlogits=None, stream=None):
    """Gradients of moe_combine: dys (rows), dw [T, k] float32 and, where dlogits [T, E_tot] float32 is given
    (with topk_ids), the gradient of the routing logits under the softmax over the chosen ones."""
    v, dev = _view(_DispatchView, desc), _device_of(dy)
    v.token_tensor("dy", dy, dev)
    v.expert_tensor("ys", ys, dev)
    _array("slot_to_row", slot_to_row, v.i32, v.slots, dev)
    _array("topk_w", topk_w, v.f32, v.slots, dev)
    v.expert_tensor("dys", dys, dev)
    _array("dw", dw, v.f32, v.slots, dev)
    if topk_ids is not None:
        _array("topk_ids", topk_ids, v.i32, v.slots, dev)
    if dlogits is not None:
        _array("dlogits", dlogits, v.f32, v.logits, dev)
    _launch(lib().moe_combine_backward, dev, stream, ctypes.byref(desc), dy.data_ptr(), ys.data_ptr(),
            slot_to_row.data_ptr(), topk_w.data_ptr(), dys.data_ptr(), dw.data_ptr(), _ptr(topk_ids), _ptr(dlogits))


def make_mxfp4_desc(rows: int, k: int, dtype: str = "bf16", scale_layout: str = "rows", stride: int = 0) -> MoeMxfp4Desc:
    """Descriptor of MXFP4 rows and the values they come from.  dtype: "bf16", "f16" or "f32"; scale_layout: "rows"
    (UE8M0 bytes [rows, k / 32], what moe_layer's MXFP4 weights have) or "packed" (int32 words
    [ceil(k / 128), rows rounded up to 4]); stride: elements between rows of the values (0 = k)."""
    return MoeMxfp4Desc(rows, k, DTYPES[dtype], SCALE_LAYOUTS[scale_layout], stride)


def make_mxfp4_gemm_desc(rows: int, n: int, k: int, groups: int = 1, out_dtype: str = "bf16",
                         a_scale_layout: str = "packed", b_scale_layout: str = "packed", variant: int = -1,
                         out_stride: int = 0) -> MoeMxfp4GemmDesc:
    """Descriptor of a grouped MXFP4 product [rows, k] x [groups, n, k] -> [rows, n]."""
    return MoeMxfp4GemmDesc(rows, n, k, groups, DTYPES[out_dtype], SCALE_LAYOUTS[a_scale_layout],
                            SCALE_LAYOUTS[b_scale_layout], variant, out_stride)


class _Stored:
    """How many codes and scales rows of k MXFP4 values have, and in which type."""

    def __init__(self, rows, k, layout):
        packed = layout == MOE_SF_PACKED_MN
        self.n, self.u8 = rows * (k // 2), _torch().u8
        self.sf_type = _torch().i32 if packed else self.u8
        self.sf_n = (k // 32 + 3) // 4 * ((rows + 3) // 4 * 4) if packed else rows * (k // 32)

    def check(self, name, codes, sf, dev):
        _array(name, codes, self.u8, self.n, dev)
        _array(name + "_sf", sf, self.sf_type, self.sf_n, dev)


class _Mxfp4View:
    def __init__(self, d):
        self.stored, self.dtype = _Stored(d.rows, d.k, d.scale_layout), _torch_dtype(d.dtype)
        self.rows, self.k, self.stride = d.rows, d.k, d.stride or d.k


class _Mxfp4GemmView:
    def __init__(self, d):
        self.a = _Stored(d.rows, d.k, d.a_scale_layout)
        self.b = _Stored(d.groups * d.n, d.k, d.b_scale_layout)
        self.i32, self.offsets = _torch().i32, d.groups + 1
        self.dtype, self.rows, self.n, self.stride = _torch_dtype(d.out_dtype), d.rows, d.n, d.out_stride or d.n


def moe_quantize_mxfp4(desc, values, codes, sf, stream=None):
    """values [rows, k] -> E2M1 codes uint8 [rows, k / 2] and UE8M0 scales (uint8, or int32 words when packed)."""
    v, dev = _view(_Mxfp4View, desc), _device_of(values)
    _rows_tensor("values", values, v.dtype, v.rows, v.k, v.stride, dev)
    v.stored.check("codes", codes, sf, dev)
    _launch(lib().moe_quantize_mxfp4, dev, stream, ctypes.byref(desc), values.data_ptr(), codes.data_ptr(), sf.data_ptr())


def moe_dequantize_mxfp4(desc, codes, sf, values, dtype: Optional[str] = None, stream=None):
    """The values [rows, k] of codes and scales, in the descriptor's dtype (or the one named)."""
    if dtype is not None and DTYPES[dtype] != desc.dtype:
        desc = MoeMxfp4Desc(desc.rows, desc.k, DTYPES[dtype], desc.scale_layout, desc.stride)
    v, dev = _view(_Mxfp4View, desc), _device_of(codes)
    v.stored.check("codes", codes, sf, dev)
    _rows_tensor("values", values, v.dtype, v.rows, v.k, v.stride, dev)
    _launch(lib().moe_dequantize_mxfp4, dev, stream, ctypes.byref(desc), codes.data_ptr(), sf.data_ptr(),
            values.data_ptr())


def moe_mxfp4_gemm(desc, a, a_sf, b, b_sf, offsets, c, stream=None):
    """c[r] = a[r] @ b[e].T for the rows of each group e (offsets int32 [groups + 1]; None: one group of all rows);
    a, b: E2M1 codes with their scales, c [rows, n].  Rows past the last group are left as they were."""
    v, dev = _view(_Mxfp4GemmView, desc), _device_of(a)
    v.a.check("a", a, a_sf, dev)
    v.b.check("b", b, b_sf, dev)
    if offsets is not None:
        _array("offsets", offsets, v.i32, v.offsets, dev)
    _rows_tensor("c", c, v.dtype, v.rows, v.n, v.stride, dev)
    _launch(lib().moe_mxfp4_gemm, dev, stream, ctypes.byref(desc), a.data_ptr(), a_sf.data_ptr(), b.data_ptr(),
            b_sf.data_ptr(), _ptr(offsets), c.data_ptr())


def make_balance_desc(num_tokens: int, num_experts: int, topk: int, num_seqs: int = 1, dtype: str = "f32",
                      score: str = "softmax", logit_stride: int = 0, grad_stride: int = 0) -> MoeBalanceDesc:
    """Descriptor of the router's balance loss.  dtype of the logits: "bf16", "f16" or "f32"; score: "softmax" or
    "sigmoid" (of each logit, over the token's sum); strides in elements (0 = num_experts)."""
    return MoeBalanceDesc(num_tokens, num_experts, topk, num_seqs, DTYPES[dtype], SCORES[score], logit_stride, grad_stride)


def moe_balance_workspace_size(desc: MoeBalanceDesc) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_balance_workspace_size(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def alloc_balance_workspace(desc: MoeBalanceDesc, device="cuda"):
    """A uint8 device tensor of moe_balance_workspace_size(desc) bytes."""
    import torch
    return torch.empty(max(moe_balance_workspace_size(desc), 256), dtype=torch.uint8, device=device)


class _BalanceView:
    def __init__(self, d):
        T = _torch()
        self.i32, self.f32, self.u8, self.bool, self.dtype = T.i32, T.f32, T.u8, T.bool, _torch_dtype(d.dtype)
        self.rows, self.cols, self.slots, self.seqs = d.num_tokens, d.num_experts, d.num_tokens * d.topk, d.num_seqs
        self.logit_stride, self.grad_stride = d.logit_stride or d.num_experts, d.grad_stride or d.num_experts

    def inputs(self, logits, mask, seq_offsets, dev):
        _rows_tensor("logits", logits, self.dtype, self.rows, self.cols, self.logit_stride, dev)
        if mask is not None:
            _array("mask", mask, self.bool if mask.dtype is self.bool else self.u8, self.rows, dev)
        if seq_offsets is not None:
            _array("seq_offsets", seq_offsets, self.i32, self.seqs + 1, dev)


def moe_balance_loss(desc, logits, topk_ids, counts, tokens, prob_sums, balance, workspace, z=None, mask=None,
                     seq_offsets=None, stream=None):
    """Counts int32 [S, E_tot], tokens int32 [S], prob_sums [S, E_tot], the balance loss [S] and, where given, the z loss
    [S] of the routing logits [T, E_tot] and the experts chosen, topk_ids int32 [T, k].  mask (bool or uint8 [T]): the
    tokens that count; seq_offsets int32 [S + 1]: the sequences' tokens (None: one sequence of all tokens).  With no tokens
    at all (num_tokens 0) nothing is written: clear counts and tokens first where they are summed over GPUs."""
    v, dev = _view(_BalanceView, desc), _device_of(logits)
    v.inputs(logits, mask, seq_offsets, dev)
    _array("topk_ids", topk_ids, v.i32, v.slots, dev)
    _array("counts", counts, v.i32, v.seqs * v.cols, dev)
    _array("tokens", tokens, v.i32, v.seqs, dev)
    _array("prob_sums", prob_sums, v.f32, v.seqs * v.cols, dev)
    _array("balance", balance, v.f32, v.seqs, dev)
    if z is not None:
        _array("z", z, v.f32, v.seqs, dev)
    _array("workspace", workspace, v.u8, 0, dev)
    _launch(lib().moe_balance_loss, dev, stream, ctypes.byref(desc), logits.data_ptr(), topk_ids.data_ptr(), _ptr(mask),
            _ptr(seq_offsets), counts.data_ptr(), tokens.data_ptr(), prob_sums.data_ptr(), balance.data_ptr(), _ptr(z),
            workspace.data_ptr(), workspace.numel())


def moe_balance_loss_backward(desc, logits, counts, tokens, dbalance, dlogits, dz=None, mask=None, seq_offsets=None,
                              add=None, stream=None):
    """Gradient of the routing logits: dlogits [T, E_tot] float32 = add (dlogits itself, say, or None) + the gradient of
    sum_s dbalance[s] * balance[s] + dz[s] * z[s], from the counts and tokens of moe_balance_loss."""
    v, dev = _view(_BalanceView, desc), _device_of(logits)
    v.inputs(logits, mask, seq_offsets, dev)
    _array("counts", counts, v.i32, v.seqs * v.cols, dev)
    _array("tokens", tokens, v.i32, v.seqs, dev)
    _array("dbalance", dbalance, v.f32, v.seqs, dev)
    if dz is not None:
        _array("dz", dz, v.f32, v.seqs, dev)
    for name, t in (("add", add), ("dlogits", dlogits)):
        if t is not None:
            _rows_tensor(name, t, v.f32, v.rows, v.cols, v.grad_stride, dev)
    _launch(lib().moe_balance_loss_backward, dev, stream, ctypes.byref(desc), logits.data_ptr(), _ptr(mask),
            _ptr(seq_offsets), counts.data_ptr(), tokens.data_ptr(), dbalance.data_ptr(), _ptr(dz), _ptr(add),
            dlogits.data_ptr())


def make_int4_desc(rows: int, k: int, group: int = 128, dtype: str = "bf16", scale_dtype: str = "bf16",
                   zeros: bool = False, stride: int = 0) -> MoeInt4Desc:
    """Descriptor of 4-bit rows with a scale (and a zero point) per group, and the values they come from.  dtype,
    scale_dtype: "bf16", "f16" or "f32"; group: 32, 64 or a multiple of 128; stride: elements between rows of the values
    (0 = k)."""
    return MoeInt4Desc(rows, k, group, DTYPES[dtype], DTYPES[scale_dtype], int(zeros), stride)


def make_w4_gemm_desc(rows: int, n: int, k: int, groups: int = 1, weight_format: str = "int4", group_size: int = 128,
                      scale_dtype: str = "bf16", zeros: bool = False, dtype: str = "bf16", out_dtype: str = "bf16",
                      activation: Optional[str] = None, activation_clamp: Optional[float] = None,
                      activation_alpha: float = 1.0, activation_up_bias: float = 0.0, a_stride: int = 0,
                      out_stride: int = 0) -> MoeW4GemmDesc:
    """Descriptor of a grouped product of 16-bit rows [rows, k] with 4-bit weights [groups, n, k] -> [rows, n]; with an
    activation ("swiglu", "swigluoai") the weights are [groups, 2n, k], gate rows before up rows.  weight_format: "int4",
    or "mxfp4" (group_size 32, scale_dtype "ue8m0")."""
    return MoeW4GemmDesc(rows, n, k, groups, W4_FORMATS[weight_format], group_size,
                         MOE_DT_U8 if scale_dtype == "ue8m0" else DTYPES[scale_dtype], int(zeros), DTYPES[dtype],
                         DTYPES[out_dtype], -1 if activation is None else ACTIVATIONS[activation],
                         math.inf if activation_clamp is None else activation_clamp, activation_alpha,
                         activation_up_bias, a_stride, out_stride)


class _Int4View:
    def __init__(self, d):
        self.rows, self.k, self.stride, self.codes = d.rows, d.k, d.stride or d.k, d.rows * (d.k // 2)
        self.n = d.rows * (d.k // d.group) if d.group > 0 else 0
        self.dtype, self.scale, self.u8, self.zeros = _torch_dtype(d.dtype), _torch_dtype(d.scale_dtype), _torch().u8, d.zeros

    def check(self, values, codes, scales, zeros, dev):
        _rows_tensor("values", values, self.dtype, self.rows, self.k, self.stride, dev)
        _array("codes", codes, self.u8, self.codes, dev)
        _array("scales", scales, self.scale, self.n, dev)
        if zeros is not None:
            _array("zeros", zeros, self.u8, self.n, dev)


class _W4GemmView:
    def __init__(self, d):
        self.rows, self.n, self.k, self.offsets = d.rows, d.n, d.k, d.groups + 1
        self.a_stride, self.out_stride = d.a_stride or d.k, d.out_stride or d.n
        b_rows = d.groups * d.n * (1 if d.activation < 0 else 2)
        self.codes, self.scales_n = b_rows * (d.k // 2), b_rows * (d.k // d.group_size) if d.group_size > 0 else 0
        self.dtype, self.out, self.scale = _torch_dtype(d.dtype), _torch_dtype(d.out_dtype), _torch_dtype(d.scale_dtype)
        self.u8, self.i32 = _torch().u8, _torch().i32


def moe_quantize_int4(desc, values, codes, scales, zeros=None, stream=None):
    """values [rows, k] -> codes uint8 [rows, k / 2], scales [rows, k / group] and, where the descriptor has them, zero
    points uint8 [rows, k / group]."""
    v, dev = _view(_Int4View, desc), _device_of(values)
    v.check(values, codes, scales, zeros, dev)
    _launch(lib().moe_quantize_int4, dev, stream, ctypes.byref(desc), values.data_ptr(), codes.data_ptr(),
            scales.data_ptr(), _ptr(zeros))


def moe_dequantize_int4(desc, codes, scales, zeros, values, dtype: Optional[str] = None, stream=None):
    """The values [rows, k] of codes, scales and zero points (or None), in the descriptor's dtype (or the one named)."""
    if dtype is not None and DTYPES[dtype] != desc.dtype:
        desc = MoeInt4Desc(desc.rows, desc.k, desc.group, DTYPES[dtype], desc.scale_dtype, desc.zeros, desc.stride)
    v, dev = _view(_Int4View, desc), _device_of(codes)
    v.check(values, codes, scales, zeros, dev)
    _launch(lib().moe_dequantize_int4, dev, stream, ctypes.byref(desc), codes.data_ptr(), scales.data_ptr(), _ptr(zeros),
            values.data_ptr())


def moe_w4_gemm(desc, a, b, b_scales, b_zeros, offsets, c, stream=None):
    """c[r] = a[r] @ w[e].T (with an activation: act of the gate and up halves) for the rows of each group e (offsets
    int32 [groups + 1]; None: one group of all rows), w the values of b, b_scales and b_zeros (None without zero
    points).  Rows past the last group are left as they were."""
    v, dev = _view(_W4GemmView, desc), _device_of(a)
    _rows_tensor("a", a, v.dtype, v.rows, v.k, v.a_stride, dev)
    _array("b", b, v.u8, v.codes, dev)
    _array("b_scales", b_scales, v.scale, v.scales_n, dev)
    if b_zeros is not None:
        _array("b_zeros", b_zeros, v.u8, v.scales_n, dev)
    if offsets is not None:
        _array("offsets", offsets, v.i32, v.offsets, dev)
    _rows_tensor("c", c, v.out, v.rows, v.n, v.out_stride, dev)
    _launch(lib().moe_w4_gemm, dev, stream, ctypes.byref(desc), a.data_ptr(), b.data_ptr(), b_scales.data_ptr(),
            _ptr(b_zeros), _ptr(offsets), c.data_ptr())
