"""ctypes binding of libep.so: the same entry points as include/ep.h.

Argument marshalling only: tensors become device pointers, torch's current
stream becomes the HIP stream, and a non-zero status becomes an exception.
Every step of the path runs in the HIP kernels; there is no fallback -- if the
library is missing or the tensors are not on the GPU, calls raise.
"""
from __future__ import annotations

import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libep.so")

EP_OK = 0
EP_BF16 = 0
EP_FP8_E4M3 = 1
EP_FP8_E4M3_POW2 = 2
EP_MXFP8_E4M3 = 3
EP_F16 = 4
EP_INT8 = 6
EP_F32 = 7                   # the router's logits only
EP_SCALES_MN_MAJOR = 0x100   # OR-ed into an FP8 dtype: scales stored transposed
EP_READ_X_AHEAD = 0x200      # OR-ed into ep_layout_dispatch's dtype: x read into the MALL during the layout
EP_GRAD_F32 = 0x400          # OR-ed into a weights' gradient's dtype: fp32 gradients
EP_GRAD_ACCUMULATE = 0x800   # OR-ed into it: added to what the gradients hold
EP_ACT_NONE = 0
EP_ACT_RELU = 1
EP_ACT_GELU = 2
EP_ACT_SILU = 3
EP_ACT_SWIGLU = 4
EP_SCORE_SOFTMAX = 0
EP_SCORE_SIGMOID = 1
_FP8_DTYPES = (EP_FP8_E4M3, EP_FP8_E4M3_POW2, EP_MXFP8_E4M3)
EP_FLAG_BAD_EXPERT = 1
EP_FLAG_OVERFLOW = 2
EP_MAX_EXPERTS = 1024
EP_MAX_TOPK = 64
EP_MAX_HIDDEN = 65536
EP_NOALLOC_SCRATCH_BYTES = 4 << 20


class EpError(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__("%s failed with status %d: %s" % (fn, status, text))
        self.status = status


class ep_layout_t(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64),
        ("num_recv_rows", ctypes.c_int64),
        ("num_topk", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("num_groups", ctypes.c_int32),
        ("capacity", ctypes.c_int32),
        ("num_tokens_per_expert", ctypes.c_void_p),
        ("expert_offsets", ctypes.c_void_p),
        ("num_tokens_per_group", ctypes.c_void_p),
        ("slot_idx", ctypes.c_void_p),
        ("recv_src", ctypes.c_void_p),
        ("error_flags", ctypes.c_void_p),
    ]


class ep_router_t(ctypes.Structure):
    _fields_ = [
        ("num_experts", ctypes.c_int32),
        ("num_topk", ctypes.c_int32),
        ("score", ctypes.c_int32),
        ("num_groups", ctypes.c_int32),
        ("topk_groups", ctypes.c_int32),
        ("group_top", ctypes.c_int32),
        ("renormalize", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


# name -> (restype, argtypes), mirroring include/ep.h
_i64, _i32, _u32, _vp, _sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_size_t
_LP = ctypes.POINTER(ep_layout_t)
_RP = ctypes.POINTER(ep_router_t)
_f32 = ctypes.c_float
SIGNATURES = {
    "ep_layout_init": (ctypes.c_int, [_LP, _i64, _i32, _i32, _i32, _i32]),
    "ep_num_recv_rows": (_i64, [_i64, _i32, _i32, _i32]),
    "ep_layout_workspace_bytes": (_sz, [_i64, _i32, _i32]),
    "ep_get_layout": (ctypes.c_int, [_vp, _LP, _vp, _sz, _vp]),
    "ep_get_layout_noalloc": (ctypes.c_int, [_vp, _LP, _vp]),
    "ep_dispatch": (ctypes.c_int, [_vp, _LP, _i32, _i32, _vp, _vp, _vp]),
    "ep_layout_dispatch": (ctypes.c_int, [_vp, _LP, _vp, _sz, _vp, _i32, _i32, _vp, _vp, _vp]),
    "ep_scales_to_mn_major": (ctypes.c_int, [_vp, _i64, _i32, _i32, _vp, _vp]),
    "ep_combine": (ctypes.c_int, [_vp, _vp, _LP, _i32, _vp, _vp]),
    "ep_combine_fp8": (ctypes.c_int, [_vp, _vp, _vp, _LP, _i32, _vp, _vp]),
    "ep_combine_f16": (ctypes.c_int, [_vp, _vp, _LP, _i32, _vp, _vp]),
    "ep_combine_mxfp8": (ctypes.c_int, [_vp, _vp, _vp, _LP, _i32, _vp, _vp]),
    "ep_dequant_mxfp8": (ctypes.c_int, [_vp, _vp, _i64, _i32, _vp, _vp]),
    "ep_group_layout_init": (ctypes.c_int, [_LP, _i64, _i32, _i32]),
    "ep_group_layout_workspace_bytes": (_sz, [_i64, _i32, _i32]),
    "ep_get_group_layout": (ctypes.c_int, [_vp, _vp, _i32, _i32, _LP, _vp, _vp, _vp, _vp, _sz, _vp]),
    "ep_combine_groups": (ctypes.c_int, [_vp, _LP, _i32, _vp, _vp]),
    "ep_dequant_fp8": (ctypes.c_int, [_vp, _vp, _i64, _i32, _vp, _vp]),
    "ep_cast_e4m3_bits": (ctypes.c_int, [_u32, _i64, _i32, _vp, _vp]),
    "ep_copy": (ctypes.c_int, [_vp, _vp, _sz, _vp]),
    "ep_expert_gemm": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _LP, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
    "ep_expert_gemm_grad_x": (ctypes.c_int, [_vp, _vp, _LP, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
    "ep_expert_gemm_grad_w": (ctypes.c_int, [_vp, _vp, _LP, _i32, _i32, _i32, _vp, _vp, _vp]),
    "ep_linear": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
    "ep_linear_grad_x": (ctypes.c_int, [_vp, _vp, _i64, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
    "ep_linear_grad_w": (ctypes.c_int, [_vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp]),
    "ep_act_grad": (ctypes.c_int, [_vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp]),
    "ep_combine_grad": (ctypes.c_int, [_vp, _vp, _vp, _LP, _i32, _i32, _vp, _vp, _vp]),
    "ep_quantize_int8": (ctypes.c_int, [_vp, _LP, _i64, _i32, _i32, _vp, _vp, _vp]),
    "ep_linear_int8": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp]),
    "ep_route": (ctypes.c_int, [_vp, _vp, _i64, _RP, _i32, _vp, _vp, _vp]),
    "ep_route_grad": (ctypes.c_int, [_vp, _vp, _vp, _i64, _RP, _i32, _vp, _vp]),
    "ep_block_norm": (ctypes.c_int, [_vp, _vp, _vp, _vp, _f32, _vp, _i64, _i32, _i32, _f32, _vp, _vp, _vp]),
    "ep_block_norm_grad_workspace_bytes": (_sz, [_i64, _i32]),
    "ep_block_norm_grad": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _f32, _vp, _i64, _i32, _i32, _f32,
                                          _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "ep_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "ep_version": (ctypes.c_char_p, []),
}

_lib = None


def library_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded libep.so.  Raises if it has not been built."""
    global _lib, _devices
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError("libep.so is not built (%s); run `python -m "
                               "combine_moe_layout_amd.build`" % _LIB_PATH)
        L = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib, _devices = L, torch.cuda.device_count()
    return _lib


def _check(fn: str, status: int) -> None:
    if status != EP_OK:
        raise EpError(fn, status, lib().ep_status_string(status).decode())


# the current stream's handle of a device by number, without making a Stream object (2.7 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# the current device's number, without a check of whether the GPU has been initialised, and how many
# devices there are (set with the library: where there is one, it is the current one)
_devices = 0
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: torch.Tensor | None, name: str, dtype=None) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return t.data_ptr()


class EpLayout:
    """Device arrays of one routing layout plus the ep_layout_t that points at
    them (the handle passed from ep_get_layout to ep_dispatch / ep_combine)."""

    def __init__(self, num_tokens: int, num_topk: int, num_experts: int, num_groups: int = 1,
                 capacity: int = 0, with_recv_src: bool = False, device=None):
        self.struct = ep_layout_t()
        _check("ep_layout_init", lib().ep_layout_init(ctypes.byref(self.struct), num_tokens,
                                                      num_topk, num_experts, num_groups, capacity))
        self._alloc(with_recv_src, device,
                    lib().ep_layout_workspace_bytes(num_tokens, num_topk, num_experts))

    def _alloc(self, with_recv_src: bool, device, workspace_bytes: int) -> None:
        """Device arrays for the sizes in self.struct, and the struct's pointers to them."""
        s = self.struct
        dev = torch.device("cuda") if device is None else torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.num_tokens_per_expert = torch.empty(s.num_experts, **i32)
        self.expert_offsets = torch.empty(s.num_experts + 1, **i32)
        self.num_tokens_per_group = torch.empty(s.num_groups, **i32)
        self.slot_idx = torch.empty((s.num_tokens, s.num_topk), **i32)
        self.recv_src = torch.empty(s.num_recv_rows, **i32) if with_recv_src else None
        self.error_flags = torch.empty(1, **i32)
        s.num_tokens_per_expert = self.num_tokens_per_expert.data_ptr()
        s.expert_offsets = self.expert_offsets.data_ptr()
        s.num_tokens_per_group = self.num_tokens_per_group.data_ptr()
        s.slot_idx = self.slot_idx.data_ptr() if s.num_tokens > 0 else None
        s.recv_src = self.recv_src.data_ptr() if with_recv_src and self.recv_src.numel() else None
        s.error_flags = self.error_flags.data_ptr()
        self.workspace = torch.empty(workspace_bytes, dtype=torch.uint8, device=dev)

    @property
    def num_tokens(self) -> int:
        return self.struct.num_tokens

    @property
    def num_topk(self) -> int:
        return self.struct.num_topk

    @property
    def num_experts(self) -> int:
        return self.struct.num_experts

    @property
    def num_recv_rows(self) -> int:
        return self.struct.num_recv_rows


class EpGroupLayout(EpLayout):
    """The per-group dedup layout: an EpLayout whose "experts" are the G groups,
    with kg = min(k, G) entries per token (ep_group_layout_init).  It is
    accepted wherever an EpLayout is, so ep_dispatch sends to the groups."""

    def __init__(self, num_tokens: int, num_topk: int, num_experts: int, num_groups: int,
                 with_recv_src: bool = False, device=None):
        self.struct = ep_layout_t()
        _check("ep_group_layout_init", lib().ep_group_layout_init(
            ctypes.byref(self.struct), num_tokens, num_topk, num_groups))
        self.source_topk = num_topk
        self.source_experts = num_experts
        self._alloc(with_recv_src, device,
                    lib().ep_group_layout_workspace_bytes(num_tokens, num_topk, num_groups))


# ----------------------------------------------------------------------------- entry points
def ep_num_recv_rows(num_tokens: int, num_topk: int, num_experts: int, capacity: int = 0) -> int:
    return int(lib().ep_num_recv_rows(num_tokens, num_topk, num_experts, capacity))


def ep_layout_workspace_bytes(num_tokens: int, num_topk: int, num_experts: int) -> int:
    return int(lib().ep_layout_workspace_bytes(num_tokens, num_topk, num_experts))


def ep_get_layout(topk_idx: torch.Tensor, layout: EpLayout, stream=None) -> EpLayout:
    """topk_idx: int64 [T, k] on the GPU.  Fills layout's arrays."""
    if tuple(topk_idx.shape) != (layout.num_tokens, layout.num_topk):
        raise ValueError("topk_idx shape %s does not match the layout" % (tuple(topk_idx.shape),))
    _check("ep_get_layout", lib().ep_get_layout(
        _ptr(topk_idx, "topk_idx", torch.int64) if topk_idx.numel() else None,
        ctypes.byref(layout.struct), layout.workspace.data_ptr(), layout.workspace.numel(),
        _stream(stream)))
    return layout


def ep_get_layout_noalloc(topk_idx: torch.Tensor, layout: EpLayout, stream=None) -> EpLayout:
    """ep_get_layout with the library's own fixed per-GPU workspace instead of
    layout.workspace (for callers that cannot allocate at call time)."""
    if tuple(topk_idx.shape) != (layout.num_tokens, layout.num_topk):
        raise ValueError("topk_idx shape %s does not match the layout" % (tuple(topk_idx.shape),))
    _check("ep_get_layout_noalloc", lib().ep_get_layout_noalloc(
        _ptr(topk_idx, "topk_idx", torch.int64) if topk_idx.numel() else None,
        ctypes.byref(layout.struct), _stream(stream)))
    return layout


def _dispatch_types(recv_dtype: int):
    """(x dtype, recv_x dtype, recv_scales dtype) of a receive dtype (with or
    without EP_SCALES_MN_MAJOR)."""
    recv_dtype &= ~(EP_SCALES_MN_MAJOR | EP_READ_X_AHEAD)
    if recv_dtype == EP_INT8:
        return torch.bfloat16, torch.int8, torch.float32
    if recv_dtype == EP_F16:
        return torch.float16, torch.float16, None
    if recv_dtype == EP_MXFP8_E4M3:
        return torch.bfloat16, torch.uint8, torch.uint8
    if recv_dtype in _FP8_DTYPES:
        return torch.bfloat16, torch.uint8, torch.float32
    return torch.bfloat16, torch.bfloat16, None


def _check_scales(recv_dtype: int, recv_scales, R: int, H: int) -> None:
    """Every FP8 scale layout holds H/128 four-byte words per receive row; int8 rows have one scale."""
    if (recv_dtype & ~EP_READ_X_AHEAD) == EP_INT8 and recv_scales is not None:
        if tuple(recv_scales.shape) != (R,):
            raise ValueError("recv_scales must have shape %s" % ((R,),))
    if (recv_dtype & ~(EP_SCALES_MN_MAJOR | EP_READ_X_AHEAD)) in _FP8_DTYPES and recv_scales is not None:
        if recv_scales.numel() * recv_scales.element_size() != R * (H // 128) * 4:
            raise ValueError("recv_scales does not hold %d rows of %d channels' scales" % (R, H))


def ep_dispatch(x: torch.Tensor, layout: EpLayout, recv_dtype: int, recv_x: torch.Tensor,
                recv_scales: torch.Tensor | None = None, stream=None) -> None:
    """x bf16 [T, H] -> recv_x: bf16 [R, H]; uint8 [R, H] FP8 codes with
    recv_scales fp32 [R, H/128] (EP_FP8_E4M3, EP_FP8_E4M3_POW2) or uint8
    [R, H/32] E8M0 bytes (EP_MXFP8_E4M3), or their transposes [H/128, R] and
    [H/32, R] with EP_SCALES_MN_MAJOR.  EP_F16: x and recv_x fp16.  EP_INT8:
    recv_x int8 with recv_scales fp32 [R]."""
    T, H = layout.num_tokens, x.shape[-1]
    if tuple(x.shape) != (T, H) or tuple(recv_x.shape) != (layout.num_recv_rows, H):
        raise ValueError("dispatch buffers do not match the layout")
    _check_scales(recv_dtype, recv_scales, layout.num_recv_rows, H)
    xt, rt, st = _dispatch_types(recv_dtype)
    _check("ep_dispatch", lib().ep_dispatch(
        _ptr(x, "x", xt), ctypes.byref(layout.struct), H, recv_dtype,
        _ptr(recv_x, "recv_x", rt), _ptr(recv_scales, "recv_scales", st),
        _stream(stream)))


def ep_layout_dispatch(topk_idx: torch.Tensor, layout: EpLayout, x: torch.Tensor, recv_dtype: int,
                       recv_x: torch.Tensor, recv_scales: torch.Tensor | None = None,
                       stream=None) -> EpLayout:
    """ep_get_layout followed by ep_dispatch; one launch for decode-sized batches."""
    T, H = layout.num_tokens, x.shape[-1]
    if tuple(topk_idx.shape) != (T, layout.num_topk):
        raise ValueError("topk_idx shape %s does not match the layout" % (tuple(topk_idx.shape),))
    if tuple(x.shape) != (T, H) or tuple(recv_x.shape) != (layout.num_recv_rows, H):
        raise ValueError("dispatch buffers do not match the layout")
    _check_scales(recv_dtype, recv_scales, layout.num_recv_rows, H)
    xt, rt, st = _dispatch_types(recv_dtype)
    _check("ep_layout_dispatch", lib().ep_layout_dispatch(
        _ptr(topk_idx, "topk_idx", torch.int64) if topk_idx.numel() else None,
        ctypes.byref(layout.struct), layout.workspace.data_ptr(), layout.workspace.numel(),
        _ptr(x, "x", xt), H, recv_dtype, _ptr(recv_x, "recv_x", rt),
        _ptr(recv_scales, "recv_scales", st), _stream(stream)))
    return layout


def ep_combine(expert_out: torch.Tensor, topk_weights: torch.Tensor, layout: EpLayout,
               out: torch.Tensor, stream=None) -> None:
    """expert_out bf16 [R, H], topk_weights fp32 [T, k] -> out bf16 [T, H]."""
    H = expert_out.shape[-1]
    if (tuple(expert_out.shape) != (layout.num_recv_rows, H)
            or tuple(topk_weights.shape) != (layout.num_tokens, layout.num_topk)
            or tuple(out.shape) != (layout.num_tokens, H)):
        raise ValueError("combine buffers do not match the layout")
    _check("ep_combine", lib().ep_combine(
        _ptr(expert_out, "expert_out", torch.bfloat16), _ptr(topk_weights, "topk_weights", torch.float32),
        ctypes.byref(layout.struct), H, _ptr(out, "out", torch.bfloat16), _stream(stream)))


def ep_combine_f16(expert_out: torch.Tensor, topk_weights: torch.Tensor, layout: EpLayout,
                   out: torch.Tensor, stream=None) -> None:
    """expert_out fp16 [R, H], topk_weights fp32 [T, k] -> out fp16 [T, H]."""
    H = expert_out.shape[-1]
    if (tuple(expert_out.shape) != (layout.num_recv_rows, H)
            or tuple(topk_weights.shape) != (layout.num_tokens, layout.num_topk)
            or tuple(out.shape) != (layout.num_tokens, H)):
        raise ValueError("combine buffers do not match the layout")
    _check("ep_combine_f16", lib().ep_combine_f16(
        _ptr(expert_out, "expert_out", torch.float16), _ptr(topk_weights, "topk_weights", torch.float32),
        ctypes.byref(layout.struct), H, _ptr(out, "out", torch.float16), _stream(stream)))


def ep_combine_fp8(expert_q: torch.Tensor, expert_scales: torch.Tensor, topk_weights: torch.Tensor,
                   layout: EpLayout, out: torch.Tensor, stream=None) -> None:
    """expert_q uint8 [R, H] E4M3 codes, expert_scales fp32 [R, H/128],
    topk_weights fp32 [T, k] -> out bf16 [T, H]."""
    H = expert_q.shape[-1]
    if (tuple(expert_q.shape) != (layout.num_recv_rows, H)
            or tuple(expert_scales.shape) != (layout.num_recv_rows, H // 128)
            or tuple(topk_weights.shape) != (layout.num_tokens, layout.num_topk)
            or tuple(out.shape) != (layout.num_tokens, H)):
        raise ValueError("combine buffers do not match the layout")
    _check("ep_combine_fp8", lib().ep_combine_fp8(
        _ptr(expert_q, "expert_q", torch.uint8), _ptr(expert_scales, "expert_scales", torch.float32),
        _ptr(topk_weights, "topk_weights", torch.float32), ctypes.byref(layout.struct), H,
        _ptr(out, "out", torch.bfloat16), _stream(stream)))


def ep_combine_mxfp8(expert_q: torch.Tensor, expert_scales: torch.Tensor, topk_weights: torch.Tensor,
                     layout: EpLayout, out: torch.Tensor, stream=None) -> None:
    """expert_q uint8 [R, H] E4M3 codes, expert_scales uint8 [R, H/32] E8M0 bytes,
    topk_weights fp32 [T, k] -> out bf16 [T, H]."""
    H = expert_q.shape[-1]
    if (tuple(expert_q.shape) != (layout.num_recv_rows, H)
            or tuple(expert_scales.shape) != (layout.num_recv_rows, H // 32)
            or tuple(topk_weights.shape) != (layout.num_tokens, layout.num_topk)
            or tuple(out.shape) != (layout.num_tokens, H)):
        raise ValueError("combine buffers do not match the layout")
    _check("ep_combine_mxfp8", lib().ep_combine_mxfp8(
        _ptr(expert_q, "expert_q", torch.uint8), _ptr(expert_scales, "expert_scales", torch.uint8),
        _ptr(topk_weights, "topk_weights", torch.float32), ctypes.byref(layout.struct), H,
        _ptr(out, "out", torch.bfloat16), _stream(stream)))


def ep_get_group_layout(topk_idx: torch.Tensor, topk_weights: torch.Tensor | None,
                        layout: EpGroupLayout, recv_topk_idx: torch.Tensor | None = None,
                        recv_topk_weights: torch.Tensor | None = None, stream=None,
                        is_token_in_group: torch.Tensor | None = None) -> EpGroupLayout:
    """topk_idx int64 [T, k] (and topk_weights fp32 [T, k] when
    recv_topk_weights is wanted) -> the group layout's arrays, plus optional
    recv_topk_idx int64 [T*kg, k] / recv_topk_weights fp32 [T*kg, k] and
    is_token_in_group uint8 (or bool) [T, G]."""
    T, k = layout.num_tokens, layout.source_topk
    if tuple(topk_idx.shape) != (T, k):
        raise ValueError("topk_idx shape %s does not match the layout" % (tuple(topk_idx.shape),))
    rows = (layout.num_recv_rows, k)
    for name, t in (("topk_weights", topk_weights),):
        if t is not None and tuple(t.shape) != (T, k):
            raise ValueError("%s shape does not match the layout" % name)
    for name, t in (("recv_topk_idx", recv_topk_idx), ("recv_topk_weights", recv_topk_weights)):
        if t is not None and tuple(t.shape) != rows:
            raise ValueError("%s must have shape %s" % (name, rows))
    member = None
    if is_token_in_group is not None:
        if tuple(is_token_in_group.shape) != (T, layout.num_experts):
            raise ValueError("is_token_in_group must have shape %s" % ((T, layout.num_experts),))
        member = is_token_in_group.view(torch.uint8) if is_token_in_group.dtype == torch.bool else is_token_in_group
    _check("ep_get_group_layout", lib().ep_get_group_layout(
        _ptr(topk_idx, "topk_idx", torch.int64) if topk_idx.numel() else None,
        _ptr(topk_weights, "topk_weights", torch.float32) if topk_weights is not None and topk_weights.numel() else None,
        k, layout.source_experts, ctypes.byref(layout.struct),
        _ptr(recv_topk_idx, "recv_topk_idx", torch.int64) if recv_topk_idx is not None and recv_topk_idx.numel() else None,
        _ptr(recv_topk_weights, "recv_topk_weights", torch.float32) if recv_topk_weights is not None and recv_topk_weights.numel() else None,
        _ptr(member, "is_token_in_group", torch.uint8) if member is not None and member.numel() else None,
        layout.workspace.data_ptr(), layout.workspace.numel(), _stream(stream)))
    return layout


def ep_combine_groups(z: torch.Tensor, layout: EpGroupLayout, out: torch.Tensor,
                      stream=None) -> None:
    """z bf16 [T*kg, H] (one already-weighted row per (token, group)) -> out
    bf16 [T, H], the unit-weight sum of each token's group rows."""
    H = z.shape[-1]
    if tuple(z.shape) != (layout.num_recv_rows, H) or tuple(out.shape) != (layout.num_tokens, H):
        raise ValueError("group combine buffers do not match the layout")
    _check("ep_combine_groups", lib().ep_combine_groups(
        _ptr(z, "z", torch.bfloat16), ctypes.byref(layout.struct), H,
        _ptr(out, "out", torch.bfloat16), _stream(stream)))


# The matrix products and the gradients.  Their tensors may live on any one GPU: the call
# runs there, on the given stream or that GPU's current one.
def _elem(dtype: int) -> torch.dtype:
    return torch.float16 if dtype == EP_F16 else torch.bfloat16


def _width(n: int, act: int) -> int:
    return 2 * n if act == EP_ACT_SWIGLU else n


class _Call:
    """The tensors of one call: each is checked (type, shape, device, contiguous) as its pointer is
    taken, and outputs against every other tensor's memory."""
    __slots__ = ("device", "ranges")

    def __init__(self, first: torch.Tensor, name: str, dims: int, layout: EpLayout | None = None):
        if first.dim() != dims:
            raise ValueError("%s must have %d dimensions" % (name, dims))
        if not first.is_cuda:
            raise ValueError("%s must be a GPU tensor" % name)
        self.device = first.get_device()
        self.ranges = []
        if layout is not None and layout.expert_offsets.get_device() != self.device:
            raise ValueError("the layout and %s are on different devices" % name)

    def operand(self, t: torch.Tensor | None, name: str, dtype: torch.dtype, shape: tuple) -> int | None:
        """Device pointer (None stays None)."""
        if t is None:
            return None
        if t.dtype is not dtype or t.shape != shape or t.get_device() != self.device or not t.is_contiguous():
            self.refuse(t, name, dtype, shape)
        p = t.data_ptr()
        if p == 0:                  # no elements
            return None
        self.ranges.append((p, p + t.nbytes, name))
        return p

    def refuse(self, t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple) -> None:
        if t.dtype is not dtype:
            raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
        if t.shape != shape:
            raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))
        if t.get_device() != self.device:
            raise ValueError("%s must be a GPU tensor on the call's device %d" % (name, self.device))
        raise ValueError("%s must be contiguous" % name)

    def output(self, t: torch.Tensor | None, name: str, dtype: torch.dtype, shape: tuple,
               may_be: tuple = ()) -> int | None:
        """The same for an output, which must not share memory with a tensor taken before it
        (but may be one of those named in may_be, from its first element on)."""
        p = self.operand(t, name, dtype, shape)
        if p is not None:
            mine = self.ranges.pop()
            end = mine[1]
            for lo, hi, other in self.ranges:
                if lo < end and p < hi and not (lo == p and other in may_be):
                    raise ValueError("%s overlaps %s" % (name, other))
            self.ranges.append(mine)
        return p

    def run(self, fn: str, stream, *args) -> None:
        """The entry point on the tensors' device, with the stream as its last argument."""
        f = getattr(lib(), fn)
        if _devices == 1 or self.device == _device():
            if stream is None and _raw_stream is not None:
                status = f(*args, _raw_stream(self.device))
            else:
                status = f(*args, _stream(stream))
        else:
            with torch.cuda.device(self.device):
                status = f(*args, _stream(stream))
        if status != EP_OK:
            _check(fn, status)


def ep_expert_gemm(x: torch.Tensor, weights: torch.Tensor, layout: EpLayout, out: torch.Tensor,
                   dtype: int, act: int = EP_ACT_NONE, x_scales: torch.Tensor | None = None,
                   weight_scales: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                   preact: torch.Tensor | None = None, stream=None) -> None:
    """x [R, K] (what ep_dispatch wrote with this dtype), weights [E, W, K] -> out [R, N]:
    act(x W_e^T + bias_e) for the rows of each expert e; W = N, or 2N for EP_ACT_SWIGLU.
    bf16 / fp16: all of that type.  FP8: uint8 codes, x_scales fp32 [R, K/128] ([K/128, R] with
    EP_SCALES_MN_MAJOR), weight_scales fp32 [E, W/128, K/128].  MXFP8: x_scales uint8 [R, K/32],
    weight_scales uint8 [E, W, K/32].  INT8: int8 codes, x_scales fp32 [R], weight_scales fp32
    [E, W].  FP8 and INT8 results are bf16.  preact [R, W]: the product itself."""
    c = _Call(x, "x", 2, layout)
    R, E, K, N = layout.num_recv_rows, layout.num_experts, x.shape[1], out.shape[-1]
    W, base = _width(N, act), dtype & ~EP_SCALES_MN_MAJOR
    et = _elem(base)
    if base in _FP8_DTYPES:
        qt, mx = torch.uint8, base == EP_MXFP8_E4M3
        st = torch.uint8 if mx else torch.float32
        xs = (R, K // 32) if mx else (K // 128, R) if dtype & EP_SCALES_MN_MAJOR else (R, K // 128)
        ws = (E, W, K // 32) if mx else (E, W // 128, K // 128)
    elif dtype == EP_INT8:
        qt, st, xs, ws = torch.int8, torch.float32, (R,), (E, W)
    else:
        qt, st, xs, ws = et, torch.float32, (), ()
        if x_scales is not None or weight_scales is not None:
            raise ValueError("dtype %d has no scales" % dtype)
    c.run("ep_expert_gemm", stream, c.operand(x, "x", qt, (R, K)), c.operand(x_scales, "x_scales", st, xs),
          c.operand(weights, "weights", qt, (E, W, K)),
          c.operand(weight_scales, "weight_scales", st, ws), c.operand(bias, "bias", et, (E, W)),
          ctypes.byref(layout.struct), K, N, dtype, act, c.output(preact, "preact", et, (R, W)),
          c.output(out, "out", et, (R, N)))


def ep_expert_gemm_grad_x(dy: torch.Tensor, weights: torch.Tensor, layout: EpLayout,
                          dx: torch.Tensor, dtype: int, act: int = EP_ACT_NONE,
                          preact: torch.Tensor | None = None, stream=None) -> None:
    """dy [R, N], weights [E, N, K] -> dx = (dy W_e) act'(preact): [R, K], or with EP_ACT_SWIGLU
    [R, 2K]; preact has dx's shape (none for EP_ACT_NONE)."""
    c = _Call(dy, "dy", 2, layout)
    if weights.dim() != 3:
        raise ValueError("weights must have 3 dimensions")
    R, E, N, K, et = layout.num_recv_rows, layout.num_experts, dy.shape[1], weights.shape[2], _elem(dtype)
    shape = (R, _width(K, act))
    c.run("ep_expert_gemm_grad_x", stream, c.operand(dy, "dy", et, (R, N)),
          c.operand(weights, "weights", et, (E, N, K)), ctypes.byref(layout.struct), K, N, dtype, act,
          c.operand(preact, "preact", et, shape), c.output(dx, "dx", et, shape))


def ep_expert_gemm_grad_w(dy: torch.Tensor, x: torch.Tensor, layout: EpLayout,
                          dweights: torch.Tensor, dtype: int, dbias: torch.Tensor | None = None,
                          stream=None) -> None:
    """dy [R, N], x [R, K] -> dweights [E, N, K] (and dbias [E, N]): dy_e^T x_e over the rows of
    each expert, in dtype's type or, with EP_GRAD_F32, fp32; EP_GRAD_ACCUMULATE adds."""
    c = _Call(dy, "dy", 2, layout)
    R, E, N, K = layout.num_recv_rows, layout.num_experts, dy.shape[1], x.shape[-1]
    et = _elem(dtype & ~(EP_GRAD_F32 | EP_GRAD_ACCUMULATE))
    gt = torch.float32 if dtype & EP_GRAD_F32 else et
    c.run("ep_expert_gemm_grad_w", stream, c.operand(dy, "dy", et, (R, N)), c.operand(x, "x", et, (R, K)),
          ctypes.byref(layout.struct), K, N, dtype, c.output(dweights, "dweights", gt, (E, N, K)),
          c.output(dbias, "dbias", gt, (E, N)))


def ep_linear(x: torch.Tensor, weights: torch.Tensor, out: torch.Tensor, dtype: int,
              act: int = EP_ACT_NONE, bias: torch.Tensor | None = None,
              residual: torch.Tensor | None = None, preact: torch.Tensor | None = None,
              stream=None) -> None:
    """x [rows, K], weights [W, K] -> out [rows, N] = act(x W^T + bias) + residual; W = N, or 2N
    for EP_ACT_SWIGLU.  preact [rows, W]: the product itself.  out may be the residual."""
    c = _Call(x, "x", 2)
    T, K, N, et = x.shape[0], x.shape[1], out.shape[-1], _elem(dtype)
    W = _width(N, act)
    res = c.operand(residual, "residual", et, (T, N))
    c.run("ep_linear", stream, c.operand(x, "x", et, (T, K)), c.operand(weights, "weights", et, (W, K)),
          c.operand(bias, "bias", et, (W,)), res, T, K, N, dtype, act,
          c.output(preact, "preact", et, (T, W)), c.output(out, "out", et, (T, N), may_be=("residual",)))


def ep_linear_grad_x(dy: torch.Tensor, weights: torch.Tensor, dx: torch.Tensor, dtype: int,
                     act: int = EP_ACT_NONE, preact: torch.Tensor | None = None, stream=None) -> None:
    """dy [rows, N], weights [N, K] -> dx = (dy W) act'(preact), as ep_expert_gemm_grad_x."""
    c = _Call(dy, "dy", 2)
    if weights.dim() != 2:
        raise ValueError("weights must have 2 dimensions")
    T, N, K, et = dy.shape[0], dy.shape[1], weights.shape[1], _elem(dtype)
    shape = (T, _width(K, act))
    c.run("ep_linear_grad_x", stream, c.operand(dy, "dy", et, (T, N)), c.operand(weights, "weights", et, (N, K)),
          T, K, N, dtype, act, c.operand(preact, "preact", et, shape), c.output(dx, "dx", et, shape))


def ep_linear_grad_w(dy: torch.Tensor, x: torch.Tensor, dweights: torch.Tensor, dtype: int,
                     dbias: torch.Tensor | None = None, stream=None) -> None:
    """dy [rows, N], x [rows, K] -> dweights [N, K] = dy^T x, dbias [N], as ep_expert_gemm_grad_w."""
    c = _Call(dy, "dy", 2)
    T, N, K = dy.shape[0], dy.shape[1], x.shape[-1]
    et = _elem(dtype & ~(EP_GRAD_F32 | EP_GRAD_ACCUMULATE))
    gt = torch.float32 if dtype & EP_GRAD_F32 else et
    c.run("ep_linear_grad_w", stream, c.operand(dy, "dy", et, (T, N)), c.operand(x, "x", et, (T, K)), T, K, N,
          dtype, c.output(dweights, "dweights", gt, (N, K)), c.output(dbias, "dbias", gt, (N,)))


def ep_quantize_int8(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, dtype: int,
                     layout: EpLayout | None = None, stream=None) -> None:
    """x [rows, n] (bf16, or fp16 with EP_F16) -> q int8 [rows, n] and scales fp32 [rows], one for
    each row; with a layout, its used receive rows alone (rows = R)."""
    c = _Call(x, "x", 2, layout)
    rows, n, et = x.shape[0], x.shape[1], _elem(dtype)
    if layout is not None and rows != layout.num_recv_rows:
        raise ValueError("x must have the layout's %d receive rows" % layout.num_recv_rows)
    c.run("ep_quantize_int8", stream, c.operand(x, "x", et, (rows, n)),
          None if layout is None else ctypes.byref(layout.struct), rows, n, dtype,
          c.output(q, "q", torch.int8, (rows, n)), c.output(scales, "scales", torch.float32, (rows,)))


def ep_linear_int8(x: torch.Tensor, x_scales: torch.Tensor, weights: torch.Tensor,
                   weight_scales: torch.Tensor, out: torch.Tensor, act: int = EP_ACT_NONE,
                   bias: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                   preact: torch.Tensor | None = None, stream=None) -> None:
    """ep_linear on codes: x int8 [rows, K] and x_scales fp32 [rows], weights int8 [W, K] and
    weight_scales fp32 [W]; bias, residual, preact and out bf16."""
    c = _Call(x, "x", 2)
    T, K, N, et = x.shape[0], x.shape[1], out.shape[-1], torch.bfloat16
    W = _width(N, act)
    res = c.operand(residual, "residual", et, (T, N))
    c.run("ep_linear_int8", stream, c.operand(x, "x", torch.int8, (T, K)),
          c.operand(x_scales, "x_scales", torch.float32, (T,)),
          c.operand(weights, "weights", torch.int8, (W, K)),
          c.operand(weight_scales, "weight_scales", torch.float32, (W,)),
          c.operand(bias, "bias", et, (W,)), res, T, K, N, act, c.output(preact, "preact", et, (T, W)),
          c.output(out, "out", et, (T, N), may_be=("residual",)))


class EpRouter:
    """How a router chooses (ep_router_t): the handle of ep_route and ep_route_grad."""

    def __init__(self, num_experts: int, num_topk: int, score: int = EP_SCORE_SOFTMAX, num_groups: int = 1,
                 topk_groups: int = 1, group_top: int = 1, renormalize: bool = True, scale: float = 1.0):
        self.struct = ep_router_t(num_experts, num_topk, score, num_groups, topk_groups, group_top,
                                  int(renormalize), scale)
        # the library's own checks, on a call with nothing to do
        _check("ep_route", lib().ep_route(None, None, 0, ctypes.byref(self.struct), EP_F32, None, None, None))

    @property
    def num_experts(self) -> int:
        return self.struct.num_experts

    @property
    def num_topk(self) -> int:
        return self.struct.num_topk


def _logits_type(dtype: int) -> torch.dtype:
    return torch.float32 if dtype == EP_F32 else _elem(dtype)


def ep_route(logits: torch.Tensor, router: EpRouter, topk_idx: torch.Tensor, topk_weights: torch.Tensor,
             dtype: int, bias: torch.Tensor | None = None, stream=None) -> None:
    """logits [T, E] (fp32, bf16 or fp16, as dtype says) and bias fp32 [E] -> topk_idx int64 [T, k]
    (-1: none) and topk_weights fp32 [T, k], what ep_get_layout and ep_combine take."""
    c = _Call(logits, "logits", 2)
    T, E, k = logits.shape[0], router.num_experts, router.num_topk
    c.run("ep_route", stream, c.operand(logits, "logits", _logits_type(dtype), (T, E)),
          c.operand(bias, "bias", torch.float32, (E,)), T, ctypes.byref(router.struct), dtype,
          c.output(topk_idx, "topk_idx", torch.int64, (T, k)),
          c.output(topk_weights, "topk_weights", torch.float32, (T, k)))


def ep_route_grad(d_topk_weights: torch.Tensor, logits: torch.Tensor, topk_idx: torch.Tensor,
                  router: EpRouter, d_logits: torch.Tensor, dtype: int, stream=None) -> None:
    """d_topk_weights fp32 [T, k] (what ep_combine_grad gives), ep_route's logits and topk_idx ->
    d_logits [T, E] of logits' type."""
    c = _Call(logits, "logits", 2)
    T, E, k, lt = logits.shape[0], router.num_experts, router.num_topk, _logits_type(dtype)
    c.run("ep_route_grad", stream, c.operand(d_topk_weights, "d_topk_weights", torch.float32, (T, k)),
          c.operand(logits, "logits", lt, (T, E)), c.operand(topk_idx, "topk_idx", torch.int64, (T, k)), T,
          ctypes.byref(router.struct), dtype, c.output(d_logits, "d_logits", lt, (T, E)))


def ep_block_norm(y: torch.Tensor | None, residual: torch.Tensor | None, out: torch.Tensor | None,
                  dtype: int, eps: float = 1e-6, post_weight: torch.Tensor | None = None,
                  gate: torch.Tensor | None = None, residual_scale: float = 1.0,
                  pre_weight: torch.Tensor | None = None, normed: torch.Tensor | None = None,
                  stream=None) -> None:
    """x = residual_scale residual + gate norm(y) post_weight -> out; norm(x) pre_weight -> normed.
    y, residual, out, normed [rows, H], weights [H], gate fp32 [rows].  Without post_weight y is
    not normed; y or residual, and out or pre_weight with normed, may be left out.  out or normed
    may be y or residual."""
    first, name = (residual, "residual") if y is None else (y, "y")
    if first is None:
        raise ValueError("y or residual is needed")
    c = _Call(first, name, 2)
    shape, et = tuple(first.shape), _elem(dtype)
    H = shape[1]
    args = (c.operand(y, "y", et, shape), c.operand(post_weight, "post_weight", et, (H,)),
            c.operand(gate, "gate", torch.float32, (shape[0],)), c.operand(residual, "residual", et, shape),
            residual_scale, c.operand(pre_weight, "pre_weight", et, (H,)), shape[0], H, dtype, eps)
    rows = ("y", "residual")
    c.run("ep_block_norm", stream, *args, c.output(out, "out", et, shape, may_be=rows),
          c.output(normed, "normed", et, shape, may_be=rows))


def ep_block_norm_grad_workspace_bytes(rows: int, hidden: int) -> int:
    return int(lib().ep_block_norm_grad_workspace_bytes(rows, hidden))


def ep_block_norm_grad(d_out: torch.Tensor | None, d_normed: torch.Tensor | None, y: torch.Tensor | None,
                       residual: torch.Tensor | None, dtype: int, workspace: torch.Tensor | None = None,
                       eps: float = 1e-6, post_weight: torch.Tensor | None = None,
                       gate: torch.Tensor | None = None, residual_scale: float = 1.0,
                       pre_weight: torch.Tensor | None = None, d_y: torch.Tensor | None = None,
                       d_residual: torch.Tensor | None = None, d_gate: torch.Tensor | None = None,
                       d_post_weight: torch.Tensor | None = None, d_pre_weight: torch.Tensor | None = None,
                       stream=None) -> None:
    """Gradients of ep_block_norm from d_out and d_normed [rows, H] (either may be left out) and its
    inputs; every gradient may be left out.  Weights' gradients have dtype's type or, with
    EP_GRAD_F32, fp32 (EP_GRAD_ACCUMULATE adds), and need a uint8 workspace of
    ep_block_norm_grad_workspace_bytes.  d_y and d_residual may be d_out or d_normed."""
    first, name = (d_normed, "d_normed") if d_out is None else (d_out, "d_out")
    if first is None:
        raise ValueError("d_out or d_normed is needed")
    c = _Call(first, name, 2)
    shape, et = tuple(first.shape), _elem(dtype & ~(EP_GRAD_F32 | EP_GRAD_ACCUMULATE))
    T, H = shape
    gt = torch.float32 if dtype & EP_GRAD_F32 else et
    args = (c.operand(d_out, "d_out", et, shape), c.operand(d_normed, "d_normed", et, shape),
            c.operand(y, "y", et, shape), c.operand(post_weight, "post_weight", et, (H,)),
            c.operand(gate, "gate", torch.float32, (T,)), c.operand(residual, "residual", et, shape),
            residual_scale, c.operand(pre_weight, "pre_weight", et, (H,)), T, H, dtype, eps)
    size = 0 if workspace is None else workspace.numel()
    rows = ("d_out", "d_normed")
    c.run("ep_block_norm_grad", stream, *args, c.output(d_y, "d_y", et, shape, may_be=rows),
          c.output(d_residual, "d_residual", et, shape, may_be=rows), c.output(d_gate, "d_gate", torch.float32, (T,)),
          c.output(d_post_weight, "d_post_weight", gt, (H,)), c.output(d_pre_weight, "d_pre_weight", gt, (H,)),
          c.output(workspace, "workspace", torch.uint8, (size,)), size)


def ep_act_grad(dy: torch.Tensor, preact: torch.Tensor, dz: torch.Tensor, dtype: int, act: int,
                stream=None) -> None:
    """dz = dy act'(preact): dy [rows, n], preact and dz [rows, n] ([rows, 2n] for EP_ACT_SWIGLU)."""
    c = _Call(dy, "dy", 2)
    T, n, et = dy.shape[0], dy.shape[1], _elem(dtype)
    shape = (T, _width(n, act))
    d, z = c.operand(dy, "dy", et, (T, n)), c.operand(preact, "preact", et, shape)
    # element by element: dz may be an input of its own width
    c.run("ep_act_grad", stream, d, z, T, n, dtype, act,
          c.output(dz, "dz", et, shape, may_be=("preact",) if act == EP_ACT_SWIGLU else ("dy", "preact")))


def ep_combine_grad(dout: torch.Tensor, expert_out: torch.Tensor | None, topk_weights: torch.Tensor,
                    layout: EpLayout, d_expert_out: torch.Tensor,
                    d_topk_weights: torch.Tensor | None, dtype: int, stream=None) -> None:
    """Gradients of ep_combine (EP_BF16) or ep_combine_f16 (EP_F16): dout [T, H] -> d_expert_out
    [R, H] (used rows) and d_topk_weights fp32 [T, k] (None to skip; expert_out is then unused)."""
    c = _Call(dout, "dout", 2, layout)
    T, k, R, H, et = layout.num_tokens, layout.num_topk, layout.num_recv_rows, dout.shape[1], _elem(dtype)
    c.run("ep_combine_grad", stream, c.operand(dout, "dout", et, (T, H)),
          c.operand(expert_out, "expert_out", et, (R, H)),
          c.operand(topk_weights, "topk_weights", torch.float32, (T, k)), ctypes.byref(layout.struct), H, dtype,
          c.output(d_expert_out, "d_expert_out", et, (R, H)),
          c.output(d_topk_weights, "d_topk_weights", torch.float32, (T, k)))


def ep_dequant_fp8(q: torch.Tensor, scales: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    rows, H = q.shape
    if tuple(y.shape) != (rows, H) or tuple(scales.shape) != (rows, H // 128):
        raise ValueError("dequant buffers disagree")
    _check("ep_dequant_fp8", lib().ep_dequant_fp8(
        _ptr(q, "q", torch.uint8), _ptr(scales, "scales", torch.float32), rows, H,
        _ptr(y, "y", torch.bfloat16), _stream(stream)))


def ep_dequant_mxfp8(q: torch.Tensor, scales: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    rows, H = q.shape
    if tuple(y.shape) != (rows, H) or tuple(scales.shape) != (rows, H // 32):
        raise ValueError("dequant buffers disagree")
    _check("ep_dequant_mxfp8", lib().ep_dequant_mxfp8(
        _ptr(q, "q", torch.uint8), _ptr(scales, "scales", torch.uint8), rows, H,
        _ptr(y, "y", torch.bfloat16), _stream(stream)))


def ep_scales_to_mn_major(scales: torch.Tensor, hidden: int, recv_dtype: int, scales_mn: torch.Tensor,
                          stream=None) -> None:
    """Row-major scales of an FP8 dispatch (fp32 [R, H/128] or MXFP8 uint8
    [R, H/32]) -> their MN-major layout ([H/128, R] or [H/32, R])."""
    recv_dtype &= ~EP_SCALES_MN_MAJOR
    if recv_dtype not in _FP8_DTYPES:
        raise ValueError("recv_dtype %d has no scales" % recv_dtype)
    per_row = hidden // 32 if recv_dtype == EP_MXFP8_E4M3 else hidden // 128
    rows = scales.shape[0]
    if tuple(scales.shape) != (rows, per_row) or tuple(scales_mn.shape) != (per_row, rows):
        raise ValueError("scale buffers disagree: %s -> %s" % (tuple(scales.shape), tuple(scales_mn.shape)))
    st = torch.uint8 if recv_dtype == EP_MXFP8_E4M3 else torch.float32
    _check("ep_scales_to_mn_major", lib().ep_scales_to_mn_major(
        _ptr(scales, "scales", st), rows, hidden, recv_dtype, _ptr(scales_mn, "scales_mn", st),
        _stream(stream)))


def ep_cast_e4m3_bits(first: int, n: int, method: int, out: torch.Tensor, stream=None) -> None:
    if out.numel() < n:
        raise ValueError("out too small")
    _check("ep_cast_e4m3_bits", lib().ep_cast_e4m3_bits(
        first & 0xFFFFFFFF, n, method, _ptr(out, "out", torch.uint8), _stream(stream)))


def ep_copy(src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() < nbytes:
        raise ValueError("dst too small")
    _check("ep_copy", lib().ep_copy(_ptr(src, "src"), _ptr(dst, "dst"), nbytes, _stream(stream)))


def ep_version() -> str:
    return lib().ep_version().decode()
