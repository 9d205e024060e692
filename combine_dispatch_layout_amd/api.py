"""Python binding of libcdl (argument marshalling only).

Every step of the hot path runs in the HIP kernels of ``libcdl.so``; this
module checks tensor devices, dtypes and shapes, allocates outputs with torch
(device memory only) and passes raw pointers and the current HIP stream to
the C ABI declared in ``include/cdl.h``.  There is no CPU fallback: if the
library is not built, or a tensor is not on a GPU, the call raises.

The calls mirror the dispatcher pages' flow ([0.4.4 diff]
_DeepEPDispatcherImplNormal: preprocess -> permute -> post-reorder combine;
[deepep.py] _DeepEPDispatcherImplLowLatency: low-latency dispatch returning
masked_m, and combine with the top-k weights):

    lay = dispatch_layout(topk_ids, expert_begin, num_local_experts)
    rows = dispatch(x, lay)                      # [R, H] bf16, expert-major
    lay, rows = permute(x, topk_ids, expert_begin, num_local_experts)  # both
    q, scales = dispatch_fp8(x, lay)             # [R, H] e4m3fn + [R, H/128] f32
    buf, masked_m, ll_map = dispatch_ll(x, lay, cap)   # [L, cap, H]
    out = combine(expert_out, lay.src2dst, topk_weights)  # [T, H] bf16

and the local experts in MXFP4, or the whole layer for a few tokens:

    lay, q, s = permute_mxfp4(x, topk_ids, expert_begin, num_local_experts)
    h, hs = grouped_swiglu_mxfp4(q, s, w13_q, w13_s, lay.counts, lay.seg_indptr)
    y = grouped_mxfp4(h, hs, w2_q, w2_s, lay.counts, lay.seg_indptr)   # [rows, H] bf16
    out = combine(y, lay.src2dst, topk_weights)
    out = moe_layer(x, topk_ids, topk_weights, w13, w2, expert_begin)  # few tokens
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcdl.so")

CDL_OK = 0
CDL_STATUS_ROWS_OVERFLOW = 1
CDL_STATUS_LL_OVERFLOW = 2
CDL_STATUS_MAP_RANGE = 4
CDL_STATUS_REORDER_OVERFLOW = 8
CDL_ERR_SCRATCH = -7
NOALLOC_SCRATCH_BYTES = 1 << 20
FP8_GROUP = 128
FP8_SCALE_UE8M0 = 1
FP8_SCALE_COLMAJOR = 2
FP8_SCALE_PACKED = 4
MXFP4_GROUP = 32
MOE_LAYER_MAX_TOKENS = 128

_lib = None


class CdlError(RuntimeError):
    """A libcdl call returned a negative status code."""

    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__("%s: %s (code %d)" % (what, status_string(code), code))


def library():
    """Load libcdl.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                "libcdl.so is not built at %s; run __graft_entry__.build() or "
                "python -m combine_dispatch_layout_amd.build" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        L.cdl_dispatch_layout_workspace_size.argtypes = [i64, i32, i32]
        L.cdl_dispatch_layout_workspace_size.restype = sz
        L.cdl_dispatch_layout.argtypes = [vp, i64, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
        L.cdl_dispatch_layout.restype = ctypes.c_int
        L.cdl_dispatch_layout_aligned.argtypes = [vp, i64, i32, i32, i32, i32, vp, vp, vp, vp,
                                                  i64, vp, vp, sz, vp]
        L.cdl_dispatch_layout_aligned.restype = ctypes.c_int
        L.cdl_permute.argtypes = [vp, i64, i64, i32, vp, i32, i32, i32, vp, vp, vp, vp, i64, vp,
                                  i64, vp, vp, sz, vp]
        L.cdl_permute.restype = ctypes.c_int
        L.cdl_permute_noalloc.argtypes = [vp, i64, i64, i32, vp, i32, i32, i32, vp, vp, vp, vp,
                                          i64, vp, i64, vp, vp]
        L.cdl_permute_noalloc.restype = ctypes.c_int
        L.cdl_permute_fp8.argtypes = [vp, i64, i64, i32, vp, i32, i32, i32, vp, vp, vp, vp, i64,
                                      vp, vp, i32, i64, vp, vp, sz, vp]
        L.cdl_fp8_scale_bytes.argtypes = [i64, i64, i32, i64]
        L.cdl_fp8_scale_bytes.restype = sz
        L.cdl_dispatch_fp8_ex.argtypes = [vp, i64, i64, i32, vp, vp, vp, i32, i64, vp, vp]
        L.cdl_dispatch_fp8_ex.restype = ctypes.c_int
        L.cdl_dispatch_ll_fp8.argtypes = [vp, i64, i64, i32, vp, i32, i32, vp, vp, vp, i64, vp, vp,
                                          i32, vp, vp, vp, vp]
        L.cdl_dispatch_ll_fp8.restype = ctypes.c_int
        L.cdl_permute_fp8.restype = ctypes.c_int
        L.cdl_rank_layout_workspace_size.argtypes = [i64, i32, i32, i32, i32]
        L.cdl_rank_layout_workspace_size.restype = sz
        L.cdl_permute_fp8_tensor.argtypes = [vp, i64, i64, i32, vp, i32, i32, i32, vp, vp, vp,
                                             vp, i64, vp, vp, i64, vp, vp, sz, vp]
        L.cdl_permute_fp8_tensor.restype = ctypes.c_int
        L.cdl_permute_fp8_workspace_size.argtypes = [i64, i32, i32, i64, i32, i64]
        L.cdl_permute_fp8_workspace_size.restype = sz
        L.cdl_rank_layout.argtypes = [vp, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
        L.cdl_rank_layout.restype = ctypes.c_int
        L.cdl_dispatch.argtypes = [vp, i64, i64, i32, vp, vp, i64, vp, vp]
        L.cdl_dispatch.restype = ctypes.c_int
        L.cdl_dispatch_fp8.argtypes = [vp, i64, i64, i32, vp, vp, vp, i64, vp, vp]
        L.cdl_dispatch_fp8.restype = ctypes.c_int
        L.cdl_dispatch_ll.argtypes = [vp, i64, i64, i32, vp, i32, i32, vp, vp, vp, i64, vp, vp,
                                      vp, vp, vp]
        L.cdl_permute_ll.argtypes = [vp, i64, i64, i32, vp, i32, i32, vp, vp, vp, vp, i64, i64, vp,
                                     vp, vp, vp, vp, sz, vp]
        L.cdl_permute_ll.restype = ctypes.c_int
        L.cdl_permute_ll_fp8.argtypes = [vp, i64, i64, i32, vp, i32, i32, vp, vp, vp, vp, i64, i64,
                                         vp, vp, i32, vp, vp, vp, vp, sz, vp]
        L.cdl_permute_ll_fp8.restype = ctypes.c_int
        L.cdl_dispatch_ll.restype = ctypes.c_int
        L.cdl_combine.argtypes = [vp, i64, i64, vp, vp, i64, i32, vp, vp, vp]
        L.cdl_combine.restype = ctypes.c_int
        L.cdl_combine_timed.argtypes = [vp, i64, i64, vp, vp, i64, i32, vp, vp, vp, vp, vp]
        L.cdl_combine_timed.restype = ctypes.c_int
        L.cdl_quant_mxfp4.argtypes = [vp, i64, i64, vp, vp, vp]
        L.cdl_quant_mxfp4.restype = ctypes.c_int
        L.cdl_dequant_mxfp4.argtypes = [vp, vp, i64, i64, vp, vp]
        L.cdl_dequant_mxfp4.restype = ctypes.c_int
        L.cdl_dispatch_mxfp4.argtypes = [vp, i64, i64, i32, vp, vp, vp, i64, vp, vp]
        L.cdl_dispatch_mxfp4.restype = ctypes.c_int
        L.cdl_permute_mxfp4.argtypes = [vp, i64, i64, i32, vp, i32, i32, i32, vp, vp, vp, vp, i64,
                                        vp, vp, i64, vp, vp, sz, vp]
        L.cdl_permute_mxfp4.restype = ctypes.c_int
        L.cdl_permute_ll_mxfp4.argtypes = [vp, i64, i64, i32, vp, i32, i32, vp, vp, vp, vp, i64,
                                           i64, vp, vp, vp, vp, vp, vp, sz, vp]
        L.cdl_permute_ll_mxfp4.restype = ctypes.c_int
        grouped = [vp, vp, i64, i64, vp, vp, i32, i64, vp, vp, i64]
        L.cdl_grouped_mxfp4.argtypes = grouped + [vp, vp, vp]
        L.cdl_grouped_mxfp4.restype = ctypes.c_int
        L.cdl_grouped_swiglu_mxfp4.argtypes = grouped + [vp, vp, vp, vp]
        L.cdl_grouped_swiglu_mxfp4.restype = ctypes.c_int
        L.cdl_moe_layer_workspace_size.argtypes = [i64, i32, i64, i32]
        L.cdl_moe_layer_workspace_size.restype = sz
        layer = [vp, i64, i64, i32, vp, vp, i32, i32, i64]
        L.cdl_moe_layer.argtypes = layer + [vp, vp, vp, vp, sz, vp]
        L.cdl_moe_layer.restype = ctypes.c_int
        L.cdl_moe_layer_mxfp4.argtypes = layer + [vp, vp, vp, vp, vp, vp, sz, vp]
        L.cdl_moe_layer_mxfp4.restype = ctypes.c_int
        L.cdl_ll_expected_m.argtypes = [i64, i32, i32, i32]
        L.cdl_ll_expected_m.restype = i64
        L.cdl_status_string.argtypes = [ctypes.c_int]
        L.cdl_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return library().cdl_status_string(int(code)).decode()


def _check(rc: int, what: str) -> None:
    if rc != CDL_OK:
        raise CdlError(rc, what)


# Every entry point has its argtypes declared (library()), so pointers pass as
# plain ints: no ctypes object per argument.
def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# torch's raw current-stream query: the stream handle without building a
# torch.cuda.Stream object (a few microseconds per call otherwise)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device):
    if _raw_stream is not None:
        return _raw_stream(device.index if device.index is not None else torch.cuda.current_device())
    return torch.cuda.current_stream(device).cuda_stream


def _need_gpu(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor (libcdl has no CPU path)" % name)


def _need(t: torch.Tensor, name: str, dtype, shape=None) -> None:
    _need_gpu(t, name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _same_device(dev: torch.device, **tensors) -> None:
    """Every given tensor (None skipped) lives on `dev`: the kernels of one
    call run on one device and take every pointer as that device's memory."""
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError("%s is on %s, the call's inputs on %s" % (name, t.device, dev))


def _need_q_rows(t: torch.Tensor, H: int) -> None:
    """out_q of the normal-mode fp8 calls: [rows, H] bytes.  The kernels
    write H bytes per destination row at row * H, up to rows rows, so a
    narrower buffer would be written past its end."""
    _need(t, "out_q", torch.uint8)
    if t.dim() != 2 or t.shape[1] != H:
        raise ValueError("out_q must be [rows, H] with H = %d, got %s" % (H, tuple(t.shape)))


_ROW_DTYPES_2 = (torch.bfloat16, torch.float16, torch.int16)
_ROW_DTYPES_1 = (torch.uint8, torch.int8, torch.float8_e4m3fn, torch.float8_e5m2)


def _rows16(t: torch.Tensor, name: str) -> torch.Tensor:
    """[n, H] rows of 1- or 2-byte elements viewed as 16-bit words.  The
    scatter moves bits, so any such dtype is dispatched exactly: bf16 hidden
    states, or rows already quantised to fp8 per tensor, whose permuted
    buffer stays fp8."""
    _need_gpu(t, name)
    if t.dim() != 2:
        raise ValueError("%s must be [rows, H]" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.dtype in _ROW_DTYPES_2:
        return t.view(torch.int16)
    if t.dtype in _ROW_DTYPES_1:
        if t.shape[1] % 2:
            raise ValueError("%s: rows of 1-byte elements need an even width" % name)
        return t.view(torch.int16)
    raise TypeError("%s must have 1- or 2-byte elements (bf16, fp16, fp8, int8), got %s"
                    % (name, t.dtype))


@dataclasses.dataclass
class Layout:
    """Caller-owned routing layout: the explicit form of the pages' dispatch
    ``handle``.  Device tensors; nothing here is synchronised."""
    T: int
    k: int
    expert_begin: int
    num_local_experts: int
    topk_ids: torch.Tensor          # [T, k] int32 (global ids)
    counts: torch.Tensor            # [L] int32 (true counts)
    seg_indptr: torch.Tensor        # [L+1] int64 (segments padded to `alignment`)
    src2dst: torch.Tensor           # [T*k] int32
    reorder_buf: torch.Tensor       # [T*k + L*(alignment-1)] int32 (first R entries valid)
    alignment: int = 1

    def num_rows(self) -> int:
        """R, the number of dispatched rows (synchronises with the device)."""
        return int(self.seg_indptr[self.num_local_experts].item())

    @property
    def reorder_topk_ids(self) -> torch.Tensor:
        """Local expert of every dispatched row (synchronises for R)."""
        return self.reorder_buf[: self.num_rows()]


def layout_workspace_size(T: int, k: int, L: int) -> int:
    n = library().cdl_dispatch_layout_workspace_size(T, k, L)
    if n == 0:
        raise CdlError(-2, "cdl_dispatch_layout_workspace_size")
    return int(n)


def dispatch_layout(topk_ids: torch.Tensor, expert_begin: int, num_local_experts: int,
                    workspace: Optional[torch.Tensor] = None, alignment: int = 1) -> Layout:
    """Per-expert counts, seg_indptr, src2dst and reorder_topk_ids of the
    rank's slots (global ids outside [expert_begin, expert_begin+L) are
    invalid).  With alignment > 1 every expert segment is padded to a
    multiple of `alignment` rows (padding rows have reorder id -1).  int64
    ids are narrowed to int32 here."""
    lay, ws = _new_layout(topk_ids, expert_begin, num_local_experts, workspace, alignment)
    rc = library().cdl_dispatch_layout_aligned(
        _ptr(lay.topk_ids), lay.T, lay.k, lay.expert_begin, lay.num_local_experts,
        lay.alignment, _ptr(lay.counts), _ptr(lay.seg_indptr), _ptr(lay.src2dst),
        _ptr(lay.reorder_buf), lay.reorder_buf.numel(), None, _ptr(ws),
        ws.numel() * ws.element_size(), _stream(lay.topk_ids.device))
    _check(rc, "cdl_dispatch_layout_aligned")
    return lay


def _new_layout(topk_ids: torch.Tensor, expert_begin: int, num_local_experts: int,
                workspace: Optional[torch.Tensor], alignment: int = 1):
    _need_gpu(topk_ids, "topk_ids")
    if topk_ids.dim() != 2:
        raise ValueError("topk_ids must be [T, k]")
    if topk_ids.dtype != torch.int32:
        topk_ids = topk_ids.to(torch.int32)
    topk_ids = topk_ids.contiguous()
    T, k = topk_ids.shape
    L = int(num_local_experts)
    dev = topk_ids.device
    ws_bytes = layout_workspace_size(T, k, L)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    elif workspace.numel() * workspace.element_size() < ws_bytes:
        raise ValueError("workspace too small: need %d bytes" % ws_bytes)
    A = int(alignment)
    if A < 1:
        raise ValueError("alignment must be >= 1")
    lay = Layout(T, k, int(expert_begin), L, topk_ids,
                 torch.empty(L, dtype=torch.int32, device=dev),
                 torch.empty(L + 1, dtype=torch.int64, device=dev),
                 torch.empty(T * k, dtype=torch.int32, device=dev),
                 torch.empty(max(T * k + L * (A - 1), 1), dtype=torch.int32, device=dev), A)
    return lay, workspace


def permute(x: torch.Tensor, topk_ids: torch.Tensor, expert_begin: int, num_local_experts: int,
            out: Optional[torch.Tensor] = None, rows: Optional[int] = None,
            status: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None,
            alignment: int = 1) -> Tuple[Layout, torch.Tensor]:
    """Layout + normal-mode scatter in one call (two kernels, one for T*k <= 4096).  `out` holds
    `rows` rows (default T*k + L*(alignment-1), an upper bound on R); the
    first R rows receive the dispatched rows (padding rows are not written).
    Returns (layout, out).  x holds bf16 rows, or any 1- or 2-byte element
    type (rows are copied bit for bit; `out` has x's dtype)."""
    xw = _rows16(x, "x")
    lay, ws = _new_layout(topk_ids, expert_begin, num_local_experts, workspace, alignment)
    T, k, L = lay.T, lay.k, lay.num_local_experts
    if x.shape[0] != T:
        raise ValueError("x must be [T, H] with T = %d" % T)
    if out is None:
        out = torch.empty(lay.reorder_buf.numel() if rows is None else int(rows), x.shape[1],
                          dtype=x.dtype, device=x.device)
    if out.dtype != x.dtype or out.dim() != 2 or out.shape[1] != x.shape[1]:
        raise ValueError("out must be [rows, H] of x's dtype")
    ow = _rows16(out, "out")
    H = xw.shape[1]
    if status is not None:
        _need(status, "status", torch.int32)
    _same_device(x.device, topk_ids=lay.topk_ids, out=out, status=status, workspace=ws)
    rc = library().cdl_permute(_ptr(xw), T, H, k, _ptr(lay.topk_ids), lay.expert_begin, L,
                               lay.alignment, _ptr(lay.counts), _ptr(lay.seg_indptr),
                               _ptr(lay.src2dst), _ptr(lay.reorder_buf), lay.reorder_buf.numel(),
                               _ptr(ow), ow.shape[0], _ptr(status), _ptr(ws),
                               ws.numel() * ws.element_size(), _stream(x.device))
    _check(rc, "cdl_permute")
    return lay, out


def permute_fp8(x: torch.Tensor, topk_ids: torch.Tensor, expert_begin: int,
                num_local_experts: int, rows: Optional[int] = None,
                out_q: Optional[torch.Tensor] = None, out_scales: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                alignment: int = 1, scale_flags: int = 0):
    """Layout + fp8 (e4m3fn, groups of 128) scatter in one call.  Returns
    (layout, q [rows, H] uint8, scales [rows, H/128] fp32)."""
    _need(x, "x", torch.bfloat16)
    lay, ws = _new_layout(topk_ids, expert_begin, num_local_experts, workspace, alignment)
    T, k, L = lay.T, lay.k, lay.num_local_experts
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError("x must be [T, H] with T = %d" % T)
    H = x.shape[1]
    if H % FP8_GROUP:
        raise CdlError(-3, "permute_fp8 (H must be a multiple of 128)")
    n = lay.reorder_buf.numel() if rows is None else int(rows)
    if out_q is None:
        out_q = torch.empty(n, H, dtype=torch.uint8, device=x.device)
    if out_scales is None:
        out_scales = new_scale_tensor(out_q.shape[0], H, scale_flags, x.device)
    _need_q_rows(out_q, H)
    _check_scale_buffer(out_scales, out_q.shape[0], H, scale_flags, out_q.shape[0])
    if status is not None:
        _need(status, "status", torch.int32)
    _same_device(x.device, topk_ids=lay.topk_ids, out_q=out_q, out_scales=out_scales,
                 status=status, workspace=ws)
    rc = library().cdl_permute_fp8(_ptr(x), T, H, k, _ptr(lay.topk_ids), lay.expert_begin, L,
                                   lay.alignment, _ptr(lay.counts), _ptr(lay.seg_indptr),
                                   _ptr(lay.src2dst), _ptr(lay.reorder_buf),
                                   lay.reorder_buf.numel(), _ptr(out_q), _ptr(out_scales),
                                   int(scale_flags), out_q.shape[0], _ptr(status), _ptr(ws),
                                   ws.numel() * ws.element_size(), _stream(x.device))
    _check(rc, "cdl_permute_fp8")
    return lay, out_q, out_scales


def permute_fp8_tensor(x: torch.Tensor, topk_ids: torch.Tensor, expert_begin: int,
                       num_local_experts: int, scale: Optional[torch.Tensor] = None,
                       rows: Optional[int] = None, out_q: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, alignment: int = 1):
    """Layout + scatter with every row cast to fp8 per tensor:
    e4m3fn(clamp(x / scale, +-448)), scale a device fp32 scalar or None for 1
    (the w8a8 per-tensor permuted buffer).  Returns (layout, q [rows, H] uint8
    holding e4m3fn bytes)."""
    _need(x, "x", torch.bfloat16)
    lay, ws = _new_layout(topk_ids, expert_begin, num_local_experts, workspace, alignment)
    T, k, L = lay.T, lay.k, lay.num_local_experts
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError("x must be [T, H] with T = %d" % T)
    H = x.shape[1]
    n = lay.reorder_buf.numel() if rows is None else int(rows)
    if out_q is None:
        out_q = torch.empty(n, H, dtype=torch.uint8, device=x.device)
    _need_q_rows(out_q, H)
    if scale is not None:
        _need(scale, "scale", torch.float32)
        if scale.numel() != 1:
            raise ValueError("scale must hold one value")
    if status is not None:
        _need(status, "status", torch.int32)
    _same_device(x.device, topk_ids=lay.topk_ids, out_q=out_q, scale=scale, status=status,
                 workspace=ws)
    rc = library().cdl_permute_fp8_tensor(_ptr(x), T, H, k, _ptr(lay.topk_ids), lay.expert_begin,
                                          L, lay.alignment, _ptr(lay.counts),
                                          _ptr(lay.seg_indptr), _ptr(lay.src2dst),
                                          _ptr(lay.reorder_buf), lay.reorder_buf.numel(),
                                          _ptr(out_q), _ptr(scale), out_q.shape[0],
                                          _ptr(status), _ptr(ws),
                                          ws.numel() * ws.element_size(), _stream(x.device))
    _check(rc, "cdl_permute_fp8_tensor")
    return lay, out_q


@dataclasses.dataclass
class RankLayout:
    """Where a token batch goes before the exchange (device tensors)."""
    num_tokens_per_rank: torch.Tensor       # [R] int32
    num_tokens_per_rdma_rank: torch.Tensor  # [R / ranks_per_node] int32
    num_tokens_per_expert: torch.Tensor     # [E] int32 (global experts)
    is_token_in_rank: torch.Tensor          # [T, R] bool


def rank_layout(topk_ids: torch.Tensor, num_experts: int, num_ranks: int,
                ranks_per_node: int = 1) -> RankLayout:
    """Per-rank / per-node token counts, per-expert slot counts and the
    token-in-rank table of global top-k ids (ids outside [0, E) are
    unrouted)."""
    _need_gpu(topk_ids, "topk_ids")
    if topk_ids.dim() != 2:
        raise ValueError("topk_ids must be [T, k]")
    ids = topk_ids.to(torch.int32).contiguous()
    T, k = ids.shape
    E, R, rpn = int(num_experts), int(num_ranks), int(ranks_per_node)
    wsb = library().cdl_rank_layout_workspace_size(T, k, E, R, rpn)
    if wsb == 0:
        raise CdlError(-3, "cdl_rank_layout_workspace_size (sizes)")
    dev = ids.device
    ws = torch.empty(wsb, dtype=torch.uint8, device=dev)
    out = RankLayout(torch.empty(R, dtype=torch.int32, device=dev),
                     torch.empty(R // rpn, dtype=torch.int32, device=dev),
                     torch.empty(E, dtype=torch.int32, device=dev),
                     torch.empty(T, R, dtype=torch.bool, device=dev))
    rc = library().cdl_rank_layout(_ptr(ids), T, k, E, R, rpn, _ptr(out.num_tokens_per_rank),
                                   _ptr(out.num_tokens_per_rdma_rank),
                                   _ptr(out.num_tokens_per_expert), _ptr(out.is_token_in_rank),
                                   _ptr(ws), wsb, _stream(dev))
    _check(rc, "cdl_rank_layout")
    return out


def permute_fp8_workspace_size(T: int, k: int, L: int, H: int, scale_flags: int,
                               rows: int) -> int:
    """Workspace bytes for permute_fp8 (rows = output rows) and
    permute_ll_fp8 (rows = L * cap) in a scale format: the layout workspace
    size for every valid format."""
    n = library().cdl_permute_fp8_workspace_size(T, k, L, H, scale_flags, rows)
    if n == 0:
        raise CdlError(-3, "cdl_permute_fp8_workspace_size")
    return int(n)


def fp8_scale_bytes(rows: int, H: int, scale_flags: int = 0, rows_per_mat: int = 0) -> int:
    n = library().cdl_fp8_scale_bytes(rows, H, scale_flags, rows_per_mat or max(rows, 1))
    if n == 0 and rows > 0:
        raise CdlError(-3, "cdl_fp8_scale_bytes (format)")
    return int(n)


def new_scale_tensor(rows: int, H: int, scale_flags: int, device, rows_per_mat: int = 0):
    """A scale buffer of the right size, typed and shaped for its format:
    fp32 [rows, G] (row-major), fp32 [mats, G, ld] (column-major), int32
    [rows, ceil(G/4)] or [mats, ceil(G/4), ld] (packed exponent bytes)."""
    G = H // FP8_GROUP
    rpm = rows_per_mat or max(rows, 1)
    packed = bool(scale_flags & FP8_SCALE_PACKED)
    dtype = torch.int32 if packed else torch.float32
    words = -(-G // 4) if packed else G
    if scale_flags & FP8_SCALE_COLMAJOR:
        mats = -(-rows // rpm) if rows else 0
        ld = -(-rpm // 4) * 4
        t = torch.empty(mats, words, ld, dtype=dtype, device=device)
    else:
        t = torch.empty(rows, words, dtype=dtype, device=device)
    assert t.numel() * 4 == fp8_scale_bytes(rows, H, scale_flags, rpm)
    return t


def dispatch(x: torch.Tensor, layout: Layout, out: Optional[torch.Tensor] = None,
             rows: Optional[int] = None, status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Normal-mode scatter: out[src2dst[t*k+j]] = x[t].  Allocates [R, H]
    (reading R from the device) unless `out` or `rows` is given.  x holds bf16
    rows, or any 1- or 2-byte element type (e.g. fp8 rows quantised per
    tensor): rows are copied bit for bit and `out` has x's dtype."""
    T, k = layout.T, layout.k
    xw = _rows16(x, "x")
    if x.shape[0] != T:
        raise ValueError("x must be [T, H] with T = %d" % T)
    if out is None:
        n = layout.num_rows() if rows is None else int(rows)
        out = torch.empty(n, x.shape[1], dtype=x.dtype, device=x.device)
    if out.dtype != x.dtype or out.dim() != 2 or out.shape[1] != x.shape[1]:
        raise ValueError("out must be [rows, H] of x's dtype")
    ow = _rows16(out, "out")
    H = xw.shape[1]
    if status is not None:
        _need(status, "status", torch.int32)
    _same_device(x.device, src2dst=layout.src2dst, out=out, status=status)
    rc = library().cdl_dispatch(_ptr(xw), T, H, k, _ptr(layout.src2dst), _ptr(ow), ow.shape[0],
                                _ptr(status), _stream(x.device))
    _check(rc, "cdl_dispatch")
    return out


def dispatch_fp8(x: torch.Tensor, layout: Layout, out_q: Optional[torch.Tensor] = None,
                 out_scales: Optional[torch.Tensor] = None, rows: Optional[int] = None,
                 status: Optional[torch.Tensor] = None,
                 scale_flags: int = 0) -> Tuple[torch.Tensor, torch.Tensor]:
    """Normal-mode scatter with per-token groups of 128 quantised to
    e4m3fn.  Returns (q [rows, H] uint8 holding e4m3fn bytes, scales in the
    `scale_flags` format -- fp32 [rows, H/128] by default);
    ``q.view(torch.float8_e4m3fn)`` reinterprets."""
    T, k = layout.T, layout.k
    _need(x, "x", torch.bfloat16)
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError("x must be [T, H] with T = %d" % T)
    H = x.shape[1]
    if H % FP8_GROUP:
        raise CdlError(-3, "dispatch_fp8 (H must be a multiple of 128)")
    if out_q is None:
        n = layout.num_rows() if rows is None else int(rows)
        out_q = torch.empty(n, H, dtype=torch.uint8, device=x.device)
    if out_scales is None:
        out_scales = new_scale_tensor(out_q.shape[0], H, scale_flags, x.device)
    _need_q_rows(out_q, H)
    _check_scale_buffer(out_scales, out_q.shape[0], H, scale_flags, out_q.shape[0])
    if status is not None:
        _need(status, "status", torch.int32)
    _same_device(x.device, src2dst=layout.src2dst, out_q=out_q, out_scales=out_scales,
                 status=status)
    rc = library().cdl_dispatch_fp8_ex(_ptr(x), T, H, k, _ptr(layout.src2dst), _ptr(out_q),
                                       _ptr(out_scales), int(scale_flags), out_q.shape[0],
                                       _ptr(status), _stream(x.device))
    _check(rc, "cdl_dispatch_fp8_ex")
    return out_q, out_scales


def _check_scale_buffer(t: torch.Tensor, rows: int, H: int, scale_flags: int, rpm: int) -> None:
    _need_gpu(t, "out_scales")
    if not t.is_contiguous():
        raise ValueError("out_scales must be contiguous")
    need = fp8_scale_bytes(rows, H, scale_flags, rpm)
    if t.numel() * t.element_size() < need:
        raise ValueError("out_scales holds %d bytes, the format needs %d"
                         % (t.numel() * t.element_size(), need))


def dispatch_ll(x: torch.Tensor, layout: Layout, cap: int, out: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None):
    """Low-latency dispatch into a padded [L, cap, H] buffer.  Returns (out,
    masked_m [L] int32, ll_src2dst [T*k] int32).  Rows at or beyond
    masked_m[e] are left as they were (never cleared)."""
    T, k, L = layout.T, layout.k, layout.num_local_experts
    _need(x, "x", torch.bfloat16)
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError("x must be [T, H] with T = %d" % T)
    H = x.shape[1]
    if out is None:
        out = torch.empty(L, cap, H, dtype=torch.bfloat16, device=x.device)
    _need(out, "out", torch.bfloat16, (L, cap, H))
    masked_m = torch.empty(L, dtype=torch.int32, device=x.device)
    ll_map = torch.empty(T * k, dtype=torch.int32, device=x.device)
    if status is not None:
        _need(status, "status", torch.int32)
    _same_device(x.device, topk_ids=layout.topk_ids, out=out, status=status)
    rc = library().cdl_dispatch_ll(_ptr(x), T, H, k, _ptr(layout.topk_ids), layout.expert_begin,
                                   L, _ptr(layout.src2dst), _ptr(layout.seg_indptr),
                                   _ptr(layout.counts), int(cap), _ptr(out), _ptr(masked_m),
                                   _ptr(ll_map), _ptr(status), _stream(x.device))
    _check(rc, "cdl_dispatch_ll")
    return out, masked_m, ll_map


def dispatch_ll_fp8(x: torch.Tensor, layout: Layout, cap: int, scale_flags: int = 0,
                    out_q: Optional[torch.Tensor] = None,
                    out_scales: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None):
    """Low-latency dispatch with fp8 rows.  Returns (q [L, cap, H] uint8,
    scales (every expert's cap rows are one matrix of the format), masked_m,
    ll_src2dst)."""
    T, k, L = layout.T, layout.k, layout.num_local_experts
    _need(x, "x", torch.bfloat16)
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError("x must be [T, H] with T = %d" % T)
    H = x.shape[1]
    if H % FP8_GROUP:
        raise CdlError(-3, "dispatch_ll_fp8 (H must be a multiple of 128)")
    if out_q is None:
        out_q = torch.empty(L, cap, H, dtype=torch.uint8, device=x.device)
    _need(out_q, "out_q", torch.uint8, (L, cap, H))
    if out_scales is None:
        out_scales = new_scale_tensor(L * cap, H, scale_flags, x.device, rows_per_mat=cap)
        if not scale_flags & FP8_SCALE_COLMAJOR:
            out_scales = out_scales.view(L, cap, -1)
    _check_scale_buffer(out_scales, L * cap, H, scale_flags, cap)
    masked_m = torch.empty(L, dtype=torch.int32, device=x.device)
    ll_map = torch.empty(T * k, dtype=torch.int32, device=x.device)
    if status is not None:
        _need(status, "status", torch.int32)
    _same_device(x.device, topk_ids=layout.topk_ids, out_q=out_q, out_scales=out_scales,
                 status=status)
    rc = library().cdl_dispatch_ll_fp8(_ptr(x), T, H, k, _ptr(layout.topk_ids),
                                       layout.expert_begin, L, _ptr(layout.src2dst),
                                       _ptr(layout.seg_indptr), _ptr(layout.counts), int(cap),
                                       _ptr(out_q), _ptr(out_scales), int(scale_flags),
                                       _ptr(masked_m), _ptr(ll_map), _ptr(status),
                                       _stream(x.device))
    _check(rc, "cdl_dispatch_ll_fp8")
    return out_q, out_scales, masked_m, ll_map


def permute_ll(x: torch.Tensor, topk_ids: torch.Tensor, expert_begin: int,
               num_local_experts: int, cap: int, out: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """The low-latency dispatch in one call: layout + padded [L, cap, H]
    scatter.  Returns (layout, out, masked_m, ll_src2dst)."""
    _need(x, "x", torch.bfloat16)
    lay, ws = _new_layout(topk_ids, expert_begin, num_local_experts, workspace, 1)
    T, k, L = lay.T, lay.k, lay.num_local_experts
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError("x must be [T, H] with T = %d" % T)
    H = x.shape[1]
    if out is None:
        out = torch.empty(L, cap, H, dtype=torch.bfloat16, device=x.device)
    _need(out, "out", torch.bfloat16, (L, cap, H))
    masked_m = torch.empty(L, dtype=torch.int32, device=x.device)
    ll_map = torch.empty(T * k, dtype=torch.int32, device=x.device)
    if status is not None:
        _need(status, "status", torch.int32)
    _same_device(x.device, topk_ids=lay.topk_ids, out=out, status=status, workspace=ws)
    rc = library().cdl_permute_ll(_ptr(x), T, H, k, _ptr(lay.topk_ids), lay.expert_begin, L,
                                  _ptr(lay.counts), _ptr(lay.seg_indptr), _ptr(lay.src2dst),
                                  _ptr(lay.reorder_buf), lay.reorder_buf.numel(), int(cap),
                                  _ptr(out), _ptr(masked_m), _ptr(ll_map), _ptr(status), _ptr(ws),
                                  ws.numel() * ws.element_size(), _stream(x.device))
    _check(rc, "cdl_permute_ll")
    return lay, out, masked_m, ll_map


def permute_ll_fp8(x: torch.Tensor, topk_ids: torch.Tensor, expert_begin: int,
                   num_local_experts: int, cap: int, scale_flags: int = 0,
                   out_q: Optional[torch.Tensor] = None,
                   out_scales: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """permute_ll with fp8 rows.  Returns (layout, q [L, cap, H] uint8,
    scales, masked_m, ll_src2dst)."""
    _need(x, "x", torch.bfloat16)
    lay, ws = _new_layout(topk_ids, expert_begin, num_local_experts, workspace, 1)
    T, k, L = lay.T, lay.k, lay.num_local_experts
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError("x must be [T, H] with T = %d" % T)
    H = x.shape[1]
    if H % FP8_GROUP:
        raise CdlError(-3, "permute_ll_fp8 (H must be a multiple of 128)")
    if out_q is None:
        out_q = torch.empty(L, cap, H, dtype=torch.uint8, device=x.device)
    _need(out_q, "out_q", torch.uint8, (L, cap, H))
    if out_scales is None:
        out_scales = new_scale_tensor(L * cap, H, scale_flags, x.device, rows_per_mat=cap)
        if not scale_flags & FP8_SCALE_COLMAJOR:
            out_scales = out_scales.view(L, cap, -1)
    _check_scale_buffer(out_scales, L * cap, H, scale_flags, cap)
    masked_m = torch.empty(L, dtype=torch.int32, device=x.device)
    ll_map = torch.empty(T * k, dtype=torch.int32, device=x.device)
    if status is not None:
        _need(status, "status", torch.int32)
    _same_device(x.device, topk_ids=lay.topk_ids, out_q=out_q, out_scales=out_scales,
                 status=status, workspace=ws)
    rc = library().cdl_permute_ll_fp8(_ptr(x), T, H, k, _ptr(lay.topk_ids), lay.expert_begin, L,
                                      _ptr(lay.counts), _ptr(lay.seg_indptr), _ptr(lay.src2dst),
                                      _ptr(lay.reorder_buf), lay.reorder_buf.numel(), int(cap),
                                      _ptr(out_q), _ptr(out_scales), int(scale_flags),
                                      _ptr(masked_m), _ptr(ll_map), _ptr(status), _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(x.device))
    _check(rc, "cdl_permute_ll_fp8")
    return lay, out_q, out_scales, masked_m, ll_map


def combine(y: torch.Tensor, map_: torch.Tensor, topk_weights: torch.Tensor,
            out: Optional[torch.Tensor] = None,
            status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t] = bf16(sum over valid j of w[t,j] * y[map[t*k+j]]) with fp32
    accumulation.  `y` is [rows, H] or the low-latency [L, cap, H] buffer;
    `map_` is src2dst or ll_src2dst."""
    _need_gpu(y, "y")
    if y.dtype != torch.bfloat16 or not y.is_contiguous():
        raise TypeError("y must be a contiguous bfloat16 tensor")
    H = y.shape[-1]
    y_rows = y.numel() // H if H else 0
    _need(topk_weights, "topk_weights", torch.float32)
    if topk_weights.dim() != 2:
        raise ValueError("topk_weights must be [T, k]")
    T, k = topk_weights.shape
    _need(map_, "map", torch.int32, (T * k,))
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=y.device)
    _need(out, "out", torch.bfloat16, (T, H))
    if status is not None:
        _need(status, "status", torch.int32)
    _same_device(y.device, map=map_, topk_weights=topk_weights, out=out, status=status)
    rc = library().cdl_combine(_ptr(y), y_rows, H, _ptr(map_), _ptr(topk_weights), T, k,
                               _ptr(out), _ptr(status), _stream(y.device))
    _check(rc, "cdl_combine")
    return out


def ll_expected_m(T: int, num_ranks: int, k: int, num_experts: int) -> int:
    return int(library().cdl_ll_expected_m(T, num_ranks, k, num_experts))


# ---------------------------------------------------------------------------
# MXFP4 rows, the grouped product, and the layer of a few tokens
# ---------------------------------------------------------------------------

def _launch(what: str, dev: torch.device, *args) -> None:
    """One call of the C ABI on the device's current stream, with that device
    current (the tensors' device need not be the caller's current one)."""
    fn = getattr(library(), what)
    if dev.index == torch.cuda.current_device():
        rc = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _stream(dev))
    _check(rc, what)


def _mx_width(H: int, what: str) -> None:
    if H < 1 or H % MXFP4_GROUP:
        raise CdlError(-3, "%s (row length must be a multiple of %d)" % (what, MXFP4_GROUP))


def _mx_out(out_q: Optional[torch.Tensor], out_scales: Optional[torch.Tensor], lead, H: int, device):
    """The two buffers of [*lead, H] MXFP4 rows: given ones checked, missing
    ones allocated."""
    if out_q is None:
        out_q = torch.empty(*lead, H // 2, dtype=torch.uint8, device=device)
    if out_scales is None:
        out_scales = torch.empty(*lead, H // MXFP4_GROUP, dtype=torch.uint8, device=device)
    _need(out_q, "out_q", torch.uint8, (*lead, H // 2))
    _need(out_scales, "out_scales", torch.uint8, (*lead, H // MXFP4_GROUP))
    return out_q, out_scales


def _mx_rows(q: torch.Tensor, scales: torch.Tensor, name: str) -> int:
    """Row length of MXFP4 rows q [..., H / 2] with scales [..., H / 32]."""
    _need(q, name, torch.uint8)
    if q.dim() < 1:
        raise ValueError("%s must have rows" % name)
    H = 2 * q.shape[-1]
    _mx_width(H, name)
    _need(scales, name + " scales", torch.uint8, (*q.shape[:-1], H // MXFP4_GROUP))
    return H


def quant_mxfp4(x: torch.Tensor, out_q: Optional[torch.Tensor] = None,
                out_scales: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Rows of x [..., H] bf16 to MXFP4: (q [..., H / 2], scales [..., H / 32]),
    uint8.  Groups of 32 share the smallest power-of-two scale that keeps
    their largest magnitude within 6."""
    _need(x, "x", torch.bfloat16)
    if x.dim() < 1:
        raise ValueError("x must be [..., H]")
    H = x.shape[-1]
    _mx_width(H, "quant_mxfp4")
    out_q, out_scales = _mx_out(out_q, out_scales, x.shape[:-1], H, x.device)
    _same_device(x.device, out_q=out_q, out_scales=out_scales)
    _launch("cdl_quant_mxfp4", x.device, _ptr(x), x.numel() // H, H, _ptr(out_q), _ptr(out_scales))
    return out_q, out_scales


def dequant_mxfp4(q: torch.Tensor, scales: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """MXFP4 rows q [..., H / 2], scales [..., H / 32] as bf16 [..., H] (exact)."""
    H = _mx_rows(q, scales, "q")
    if out is None:
        out = torch.empty(*q.shape[:-1], H, dtype=torch.bfloat16, device=q.device)
    _need(out, "out", torch.bfloat16, (*q.shape[:-1], H))
    _same_device(q.device, scales=scales, out=out)
    _launch("cdl_dequant_mxfp4", q.device, _ptr(q), _ptr(scales), out.numel() // H, H, _ptr(out))
    return out


def _mx_tokens(x: torch.Tensor, T: int) -> int:
    _need(x, "x", torch.bfloat16)
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError("x must be [T, H] with T = %d" % T)
    _mx_width(x.shape[1], "x")
    return x.shape[1]


def _mx_lead(out_q: Optional[torch.Tensor], out_scales: Optional[torch.Tensor], rows) -> int:
    """Destination rows of a normal-mode scatter: a given buffer's, else `rows`."""
    for name, t in (("out_q", out_q), ("out_scales", out_scales)):
        if t is not None:
            if t.dim() != 2:
                raise ValueError("%s must be [rows, bytes]" % name)
            return t.shape[0]
    return int(rows)


def dispatch_mxfp4(x: torch.Tensor, layout: Layout, out_q: Optional[torch.Tensor] = None,
                   out_scales: Optional[torch.Tensor] = None, rows: Optional[int] = None,
                   status: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Normal-mode scatter with the rows quantised to MXFP4.  Returns
    (q [rows, H / 2], scales [rows, H / 32])."""
    T, k = layout.T, layout.k
    H = _mx_tokens(x, T)
    if out_q is None and out_scales is None and rows is None:
        rows = layout.num_rows()
    out_q, out_scales = _mx_out(out_q, out_scales, (_mx_lead(out_q, out_scales, rows),), H, x.device)
    if status is not None:
        _need(status, "status", torch.int32)
    _same_device(x.device, src2dst=layout.src2dst, out_q=out_q, out_scales=out_scales, status=status)
    _launch("cdl_dispatch_mxfp4", x.device, _ptr(x), T, H, k, _ptr(layout.src2dst), _ptr(out_q),
            _ptr(out_scales), out_q.shape[0], _ptr(status))
    return out_q, out_scales


def permute_mxfp4(x: torch.Tensor, topk_ids: torch.Tensor, expert_begin: int, num_local_experts: int,
                  rows: Optional[int] = None, out_q: Optional[torch.Tensor] = None,
                  out_scales: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, alignment: int = 1):
    """Layout + MXFP4 scatter in one call.  Returns (layout, q [rows, H / 2],
    scales [rows, H / 32]); `rows` defaults to the upper bound of permute."""
    lay, ws = _new_layout(topk_ids, expert_begin, num_local_experts, workspace, alignment)
    T, k, L = lay.T, lay.k, lay.num_local_experts
    H = _mx_tokens(x, T)
    n = _mx_lead(out_q, out_scales, lay.reorder_buf.numel() if rows is None else rows)
    out_q, out_scales = _mx_out(out_q, out_scales, (n,), H, x.device)
    if status is not None:
        _need(status, "status", torch.int32)
    _same_device(x.device, topk_ids=lay.topk_ids, out_q=out_q, out_scales=out_scales, status=status,
                 workspace=ws)
    _launch("cdl_permute_mxfp4", x.device, _ptr(x), T, H, k, _ptr(lay.topk_ids), lay.expert_begin, L,
            lay.alignment, _ptr(lay.counts), _ptr(lay.seg_indptr), _ptr(lay.src2dst), _ptr(lay.reorder_buf),
            lay.reorder_buf.numel(), _ptr(out_q), _ptr(out_scales), out_q.shape[0], _ptr(status), _ptr(ws),
            ws.numel() * ws.element_size())
    return lay, out_q, out_scales


def permute_ll_mxfp4(x: torch.Tensor, topk_ids: torch.Tensor, expert_begin: int, num_local_experts: int,
                     cap: int, out_q: Optional[torch.Tensor] = None,
                     out_scales: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None):
    """permute_ll with MXFP4 rows.  Returns (layout, q [L, cap, H / 2], scales
    [L, cap, H / 32], masked_m, ll_src2dst)."""
    lay, ws = _new_layout(topk_ids, expert_begin, num_local_experts, workspace, 1)
    T, k, L = lay.T, lay.k, lay.num_local_experts
    H = _mx_tokens(x, T)
    out_q, out_scales = _mx_out(out_q, out_scales, (L, int(cap)), H, x.device)
    masked_m = torch.empty(L, dtype=torch.int32, device=x.device)
    ll_map = torch.empty(T * k, dtype=torch.int32, device=x.device)
    if status is not None:
        _need(status, "status", torch.int32)
    _same_device(x.device, topk_ids=lay.topk_ids, out_q=out_q, out_scales=out_scales, status=status,
                 workspace=ws)
    _launch("cdl_permute_ll_mxfp4", x.device, _ptr(x), T, H, k, _ptr(lay.topk_ids), lay.expert_begin, L,
            _ptr(lay.counts), _ptr(lay.seg_indptr), _ptr(lay.src2dst), _ptr(lay.reorder_buf),
            lay.reorder_buf.numel(), int(cap), _ptr(out_q), _ptr(out_scales), _ptr(masked_m), _ptr(ll_map),
            _ptr(status), _ptr(ws), ws.numel() * ws.element_size())
    return lay, out_q, out_scales, masked_m, ll_map


def _grouped_args(q, scales, w_q, w_scales, counts, seg_indptr, status):
    """Checked operands of the grouped products: (rows shape, K, L, weight
    rows, cap)."""
    K = _mx_rows(q, scales, "q")
    if _mx_rows(w_q, w_scales, "w_q") != K or w_q.dim() != 3:
        raise ValueError("w_q must be [L, N, K / 2] with K = %d, got %s" % (K, tuple(w_q.shape)))
    L, N = w_q.shape[:2]
    _need(counts, "counts", torch.int32, (L,))
    if seg_indptr is not None:
        _need(seg_indptr, "seg_indptr", torch.int64, (L + 1,))
        if q.dim() != 2:
            raise ValueError("q must be [rows, K / 2] with seg_indptr, got %s" % (tuple(q.shape),))
        cap = 0
    else:
        if q.dim() != 3 or q.shape[0] != L:
            raise ValueError("q must be [L, cap, K / 2] without seg_indptr, got %s" % (tuple(q.shape),))
        cap = q.shape[1]
    if status is not None:
        _need(status, "status", torch.int32)
    _same_device(q.device, scales=scales, w_q=w_q, w_scales=w_scales, counts=counts, seg_indptr=seg_indptr,
                 status=status)
    return q.shape[:-1], K, L, N, cap


def grouped_mxfp4(q: torch.Tensor, scales: torch.Tensor, w_q: torch.Tensor, w_scales: torch.Tensor,
                  counts: torch.Tensor, seg_indptr: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Each row times its expert's weights, both MXFP4, in bf16 with fp32
    accumulation.  w_q [L, N, K / 2].  With seg_indptr, q is [rows, K / 2] and
    expert e owns the counts[e] rows from seg_indptr[e]; without, q is the
    padded [L, cap, K / 2] buffer and counts its masked_m.  Rows of no expert
    are left as they were.  A quantised infinity is the number 6 * 2^127 here
    (the format has none), so it need not make its results infinite; a NaN
    does make them NaN.  Returns out [rows, N] or [L, cap, N]."""
    lead, K, L, N, cap = _grouped_args(q, scales, w_q, w_scales, counts, seg_indptr, status)
    if out is None:
        out = torch.empty(*lead, N, dtype=torch.bfloat16, device=q.device)
    _need(out, "out", torch.bfloat16, (*lead, N))
    _same_device(q.device, out=out)
    _launch("cdl_grouped_mxfp4", q.device, _ptr(q), _ptr(scales), lead.numel(), K, _ptr(w_q), _ptr(w_scales),
            L, N, _ptr(counts), _ptr(seg_indptr), cap, _ptr(out), _ptr(status))
    return out


def grouped_swiglu_mxfp4(q: torch.Tensor, scales: torch.Tensor, w_q: torch.Tensor, w_scales: torch.Tensor,
                         counts: torch.Tensor, seg_indptr: Optional[torch.Tensor] = None,
                         out_q: Optional[torch.Tensor] = None, out_scales: Optional[torch.Tensor] = None,
                         status: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The gate/up product with SwiGLU, quantised again in its epilogue: w_q
    [L, 2 I, K / 2] holds the I gate rows, then the I up rows.  Returns (q
    [rows, I / 2], scales [rows, I / 32]), the operand of the down product;
    rows and counts as for grouped_mxfp4."""
    lead, K, L, N, cap = _grouped_args(q, scales, w_q, w_scales, counts, seg_indptr, status)
    if N % 2:
        raise ValueError("w_q must hold as many gate as up rows, got %d rows" % N)
    I = N // 2
    _mx_width(I, "grouped_swiglu_mxfp4")
    out_q, out_scales = _mx_out(out_q, out_scales, lead, I, q.device)
    _same_device(q.device, out_q=out_q, out_scales=out_scales)
    _launch("cdl_grouped_swiglu_mxfp4", q.device, _ptr(q), _ptr(scales), lead.numel(), K, _ptr(w_q),
            _ptr(w_scales), L, I, _ptr(counts), _ptr(seg_indptr), cap, _ptr(out_q), _ptr(out_scales),
            _ptr(status))
    return out_q, out_scales


def moe_layer_workspace_size(T: int, k: int, I: int, L: int) -> int:
    n = library().cdl_moe_layer_workspace_size(T, k, I, L)
    if n == 0:
        raise CdlError(-3, "cdl_moe_layer_workspace_size (at most %d tokens)" % MOE_LAYER_MAX_TOKENS)
    return int(n)


def _layer_args(x, topk_ids, topk_weights, I, L, out, workspace):
    _need(x, "x", torch.bfloat16)
    if x.dim() != 2:
        raise ValueError("x must be [T, H]")
    T, H = x.shape
    _need_gpu(topk_ids, "topk_ids")
    if topk_ids.dim() != 2 or topk_ids.shape[0] != T:
        raise ValueError("topk_ids must be [T, k] with T = %d" % T)
    k = topk_ids.shape[1]
    ids = topk_ids.to(torch.int32).contiguous()
    _need(topk_weights, "topk_weights", torch.float32, (T, k))
    if out is None:
        out = torch.empty(T, H, dtype=torch.bfloat16, device=x.device)
    _need(out, "out", torch.bfloat16, (T, H))
    need = moe_layer_workspace_size(T, k, I, L)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    _need_gpu(workspace, "workspace")
    if not workspace.is_contiguous() or workspace.numel() * workspace.element_size() < need:
        raise ValueError("workspace too small: need %d bytes" % need)
    _same_device(x.device, topk_ids=ids, topk_weights=topk_weights, out=out, workspace=workspace)
    return T, H, k, ids, out, workspace


def moe_layer(x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor, w13: torch.Tensor,
              w2: torch.Tensor, expert_begin: int = 0, out: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The local experts of a few tokens (T <= 128, T * k <= 4096) in two
    kernels: out[t] = sum over local slots of w[t, j] * W2[e] h, h =
    silu(gate) * up from w13 [L, 2 I, H] bf16 (gate rows, then up rows), w2
    [L, H, I] bf16."""
    _need(w13, "w13", torch.bfloat16)
    _need(w2, "w2", torch.bfloat16)
    if w13.dim() != 3 or w13.shape[1] % 2:
        raise ValueError("w13 must be [L, 2 I, H], got %s" % (tuple(w13.shape),))
    L, I = w13.shape[0], w13.shape[1] // 2
    T, H, k, ids, out, ws = _layer_args(x, topk_ids, topk_weights, I, L, out, workspace)
    if tuple(w13.shape) != (L, 2 * I, H) or tuple(w2.shape) != (L, H, I):
        raise ValueError("w13 must be [L, 2 I, H] and w2 [L, H, I] with H = %d, got %s and %s"
                         % (H, tuple(w13.shape), tuple(w2.shape)))
    _same_device(x.device, w13=w13, w2=w2)
    _launch("cdl_moe_layer", x.device, _ptr(x), T, H, k, _ptr(ids), _ptr(topk_weights), int(expert_begin), L,
            I, _ptr(w13), _ptr(w2), _ptr(out), _ptr(ws), ws.numel() * ws.element_size())
    return out


def moe_layer_mxfp4(x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor, w13_q: torch.Tensor,
                    w13_scales: torch.Tensor, w2_q: torch.Tensor, w2_scales: torch.Tensor, expert_begin: int = 0,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_layer with MXFP4 weights (w13_q [L, 2 I, H / 2], w2_q [L, H, I / 2]
    and their scales); the activations stay bf16."""
    H13, I2 = _mx_rows(w13_q, w13_scales, "w13_q"), _mx_rows(w2_q, w2_scales, "w2_q")
    if w13_q.dim() != 3 or w13_q.shape[1] != 2 * I2:
        raise ValueError("w13_q must be [L, 2 I, H / 2] with I = %d, got %s" % (I2, tuple(w13_q.shape)))
    L, I = w13_q.shape[0], I2
    T, H, k, ids, out, ws = _layer_args(x, topk_ids, topk_weights, I, L, out, workspace)
    if H13 != H or tuple(w2_q.shape) != (L, H, I // 2):
        raise ValueError("w13_q and w2_q must be [L, 2 I, H / 2] and [L, H, I / 2] with H = %d, got %s and %s"
                         % (H, tuple(w13_q.shape), tuple(w2_q.shape)))
    _same_device(x.device, w13_q=w13_q, w13_scales=w13_scales, w2_q=w2_q, w2_scales=w2_scales)
    _launch("cdl_moe_layer_mxfp4", x.device, _ptr(x), T, H, k, _ptr(ids), _ptr(topk_weights),
            int(expert_begin), L, I, _ptr(w13_q), _ptr(w13_scales), _ptr(w2_q), _ptr(w2_scales), _ptr(out),
            _ptr(ws), ws.numel() * ws.element_size())
    return out
