"""MI355X-native MoE expert-parallel layout / dispatch / combine.

Thin PyTorch binding over libep.so (include/ep.h).  PyTorch only provides
device memory and the current HIP stream; every step of the path runs in the
library's gfx950 kernels.  The functions carry the C entry points' names:

  ep_get_layout(topk_idx, num_experts, ...)        -> Layout
  ep_get_layout_noalloc(topk_idx, layout, ...)     -> layout (the library's own scratch)
  ep_dispatch(x, layout, ...)                      -> (recv_x, recv_scales, recv_topk_weights)
  ep_dispatch_with_layout(x, topk_idx, num_experts, ...)
                                                   -> (layout, recv_x, recv_scales, recv_topk_weights)
  ep_combine(y, layout, ...)                       -> (combined_x, combined_topk_weights)
  ep_cast_fp8(x, group=128)                        -> (x_fp8, scales)
  ep_dispatch_partitioned(x, layout, topk_idx, ...) -> (recv_x, recv_scales, recv_topk_idx,
                                                        recv_topk_weights)
  ep_combine_partitioned(y, layout, ...)            -> combined_x
  ep_combine_reduced(y, layout, topk_idx, ...)      -> combined_x
  ep_expert_linear(x, w, layout, ...)               -> (out, checkpoint)
  ep_expert_wgrad(dy, x, layout, ...)               -> (dw, db)
  ep_expert_activation_backward(dh, pre, layout, ...) -> (dpre, h, dweights)
  ep_moe_decode(x, topk_idx, topk_weights, w1, w2, ...) -> out
  ep_cast_fp8_blocks(w, ...)                        -> ((codes, scales), transposed pair or None)
  ep_block_linear(x, w, layout=None, ...)           -> out
  ep_gated_ffn(x, w1, w2, ...)                      -> (out, z or None)
  ep_gated_ffn_backward(dout, x, z, w1, w2, ...)    -> (dx, dw1, dw2)

Semantics follow the DeepEP v2 test page ("DeepEP test target API
reference", sec. 2.1 dispatch, 2.2 combine, 3.1-3.2 the V1 layout tensors and
unweighted combine, 4.2 the per-token e4m3 cast); the layout object plays the
part of the page's handle.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple, Union

import torch

from . import _abi
from ._abi import (EP_DEV_BAD_EXPERT, EP_DEV_CAPACITY, EP_DEV_RECV_OVERFLOW, EpError,
                   LayoutParams, LayoutPtrs)

__all__ = ["load_library", "Layout", "ep_get_layout", "ep_get_layout_noalloc", "ep_dispatch",
           "ep_dispatch_with_layout",
           "ep_combine", "ep_cast_fp8", "logfmt_row_bytes", "ep_logfmt_encode",
           "ep_logfmt_decode", "ep_combine_logfmt",
           "ep_dispatch_partitioned", "ep_combine_partitioned", "ep_combine_reduced",
           "ep_expert_linear",
           "ep_expert_wgrad", "ep_expert_activation_backward", "ep_moe_decode",
           "ep_cast_fp8_blocks", "ep_block_linear", "ep_gated_ffn", "ep_gated_ffn_backward",
           "worst_case_recv_rows", "ep_probe_dispatch_stores", "EpError", "EP_DEV_BAD_EXPERT", "EP_DEV_CAPACITY",
           "EP_DEV_RECV_OVERFLOW"]


def load_library() -> ctypes.CDLL:
    return _abi.load()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    """The raw handle of the current stream of `device` (torch's current
    stream, which HIP graph capture also records into)."""
    idx = device.index if device.index is not None else torch._C._cuda_getDevice()
    return torch._C._cuda_getCurrentRawStream(idx)


def _launch(name: str, device, fn, *tensors_then_args):
    """Call entry point `fn` with `device` current (the library launches on the
    calling thread's current device), after checking that every tensor given
    before the plain arguments lives on it.  Usage:
    _launch(name, dev, fn, [tensors...], arg0, arg1, ...)."""
    tensors, args = tensors_then_args[0], tensors_then_args[1:]
    cur = torch._C._cuda_getDevice()
    idx = cur if device.index is None else device.index
    for t in tensors:
        if t is not None and t.get_device() != idx:
            raise ValueError(f"{name}: all tensors must be on cuda:{idx}, found {t.device}")
    if idx == cur:
        rc = fn(*args)
    else:
        with torch.cuda.device(idx):
            rc = fn(*args)
    _abi.check(name, rc)


def _need_cuda(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check(t: Optional[torch.Tensor], name: str, dtypes, cols=None, min_rows=None, rows=None):
    """A GPU buffer the kernels will read or write: contiguous, of one of
    `dtypes`, 2-D with `cols` columns (1-D when cols is None) and `rows` rows
    exactly or at least `min_rows`.  Catches a buffer the kernels would
    overrun before anything is launched."""
    if t is None:
        return
    _need_cuda(t, name)
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if cols is None:
        n = t.numel()
        if (rows is not None and n != rows) or (min_rows is not None and n < min_rows):
            raise ValueError(f"{name} has {n} elements, needs {rows if rows is not None else min_rows}")
        return
    if t.dim() != 2 or t.shape[1] != cols:
        raise ValueError(f"{name} must be [rows, {cols}], not {list(t.shape)}")
    if (rows is not None and t.shape[0] != rows) or (min_rows is not None and t.shape[0] < min_rows):
        raise ValueError(f"{name} has {t.shape[0]} rows, needs "
                         f"{rows if rows is not None else f'at least {min_rows}'}")


_F8 = (torch.float8_e4m3fn, torch.uint8)
_BF16 = (torch.bfloat16,)
_F32 = (torch.float32,)
_I64 = (torch.int64,)


def worst_case_recv_rows(num_tokens, num_topk, num_experts, expert_alignment=1, capacity=0,
                         num_partitions=1, partition_major=False) -> int:
    p = LayoutParams(num_tokens=num_tokens, num_topk=num_topk, num_experts=num_experts,
                     expert_alignment=expert_alignment, num_partitions=num_partitions,
                     capacity=capacity, partition_major=1 if partition_major else 0)
    return int(load_library().ep_worst_case_recv_rows(ctypes.byref(p)))


class Layout:
    """Device-resident receive layout (the dispatch "handle").

    Tensors: num_tokens_per_expert [S], expert_offset [S+1] (R at [S]), S the
    receive segments (E, or P for a partition-major layout),
    num_tokens_per_partition [P], is_token_in_partition [T, P] uint8,
    dst_slot [T, K], src_of_slot [max_recv_rows], status [1]; with the
    partition layout also partition_offset [P+1], num_tokens_per_group [P/G]
    and, for P <= 64, token_slot [T, P] and partition_src [T*P] (the token of
    each partition row) (else None).  A buffer may be replaced or dropped by
    assigning the attribute; resizing one in place is not supported (the
    calls pass each buffer's address as it was when last assigned)."""

    def __init__(self, params: LayoutParams, device, partition_layout: bool = False):
        T, K, P = params.num_tokens, params.num_topk, params.num_partitions
        S = P if params.partition_major else params.num_experts
        i32 = dict(dtype=torch.int32, device=device)
        self.params = params
        self.device = device
        self.num_tokens_per_expert = torch.empty(S, **i32)
        self.expert_offset = torch.empty(S + 1, **i32)
        self.num_tokens_per_partition = torch.empty(P, **i32)
        self.is_token_in_partition = torch.empty((T, P), dtype=torch.uint8, device=device)
        self.dst_slot = torch.empty((T, K), **i32)
        self.src_of_slot = torch.empty(max(params.max_recv_rows, 1), **i32)
        self.status = torch.zeros(1, **i32)
        self.partition_offset = self.token_slot = self.num_tokens_per_group = None
        self.partition_src = None
        if partition_layout:
            G = params.partitions_per_group or P
            self.partition_offset = torch.empty(P + 1, **i32)
            self.num_tokens_per_group = torch.empty(P // G, **i32)
            if P <= _abi.EP_MAX_SLOT_PARTITIONS:      # token_slot only up to 64 partitions
                self.token_slot = torch.empty((T, P), **i32)
                self.partition_src = torch.empty(max(T * P, 1), **i32)
        nbytes = load_library().ep_get_layout_workspace_bytes(ctypes.byref(params))
        self.workspace = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
        self._ptrs = None

    @property
    def num_tokens(self):
        return self.params.num_tokens

    @property
    def num_topk(self):
        return self.params.num_topk

    @property
    def num_experts(self):
        return self.params.num_experts

    @property
    def partition_major(self) -> bool:
        return bool(self.params.partition_major)

    @property
    def num_segments(self) -> int:
        """Receive segments: experts, or partitions when partition-major."""
        return self.params.num_partitions if self.params.partition_major else self.params.num_experts

    @property
    def max_recv_rows(self) -> int:
        return int(self.params.max_recv_rows)

    @property
    def num_partitions(self):
        return self.params.num_partitions

    _BUFFERS = frozenset(("num_tokens_per_expert", "expert_offset", "num_tokens_per_partition",
                          "is_token_in_partition", "dst_slot", "src_of_slot", "status",
                          "partition_offset", "token_slot", "num_tokens_per_group",
                          "partition_src"))

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name in Layout._BUFFERS:
            # a replaced (or dropped) buffer: the pointer struct must not keep
            # the old address, whose memory torch may hand out again
            object.__setattr__(self, "_ptrs", None)

    def ptrs(self) -> LayoutPtrs:
        """The buffers' device pointers as the C struct, built on first use
        after any buffer attribute was (re)assigned."""
        if self._ptrs is None:
            opt = [None if t is None else t.data_ptr()
                   for t in (self.partition_offset, self.token_slot, self.num_tokens_per_group,
                             self.partition_src)]
            self._ptrs = LayoutPtrs(self.num_tokens_per_expert.data_ptr(),
                                    self.expert_offset.data_ptr(),
                                    self.num_tokens_per_partition.data_ptr(),
                                    self.is_token_in_partition.data_ptr(), self.dst_slot.data_ptr(),
                                    self.src_of_slot.data_ptr(), self.status.data_ptr(), *opt)
        return self._ptrs

    def num_partition_rows(self) -> int:
        """Rp, rows of the non-expanded partition layout (synchronises)."""
        if self.partition_offset is None:
            raise ValueError("layout was built without the partition layout")
        return int(self.partition_offset[-1].item())

    def num_recv_rows(self) -> int:
        """R, the receive rows in use (synchronises: the page's do_cpu_sync)."""
        return int(self.expert_offset[-1].item())

    def check(self) -> int:
        """Synchronise and raise on device status bits; returns the bits."""
        st = int(self.status.item())
        if st & EP_DEV_BAD_EXPERT:
            raise ValueError("topk_idx holds an expert id outside [-1, num_experts)")
        if st & EP_DEV_CAPACITY:
            raise RuntimeError("an expert received more pairs than the fixed capacity")
        if st & EP_DEV_RECV_OVERFLOW:
            raise RuntimeError("receive rows exceed the allocated buffer")
        return st


def ep_get_layout(topk_idx: torch.Tensor, num_experts: int, expert_alignment: int = 1,
                  num_partitions: int = 1, capacity: int = 0,
                  max_recv_rows: Optional[int] = None,
                  cumulative_expert_stats: Optional[torch.Tensor] = None,
                  layout: Optional[Layout] = None, partition_layout: bool = False,
                  partitions_per_group: int = 0, partition_major: bool = False) -> Layout:
    """Derive the receive layout from topk_idx (int64 [T, K], -1 = none).
    capacity > 0 selects the fixed-capacity ("expand") layout.
    partition_layout=True also derives the non-expanded per-partition layout
    (token_slot etc., P <= 64); partitions_per_group sets G for
    num_tokens_per_group (0: one group).  partition_major=True groups the
    receive rows by partition instead of expert (pairs in (t, k) order inside
    each partition's segment; the per-expert tables then hold one entry per
    partition).  A `layout` of the same shape may be passed in to be
    rewritten in place."""
    lib = load_library()
    layout, params = _prepare_layout(topk_idx, num_experts, expert_alignment, num_partitions,
                                     capacity, max_recv_rows, cumulative_expert_stats, layout,
                                     partition_layout, partitions_per_group, partition_major)
    ptrs = layout.ptrs()
    _launch("ep_get_layout", topk_idx.device, lib.ep_get_layout,
            [cumulative_expert_stats, layout.workspace, layout.status],
            _ptr(topk_idx), ctypes.byref(params), ctypes.byref(ptrs),
            _ptr(cumulative_expert_stats), _ptr(layout.workspace),
            layout.workspace.numel(), _stream(topk_idx.device))
    return layout


def ep_get_layout_noalloc(topk_idx: torch.Tensor, layout: Layout,
                          cumulative_expert_stats: Optional[torch.Tensor] = None) -> Layout:
    """ep_get_layout into an existing `layout` (same shapes) with no
    workspace: the library's static per-GPU scratch is used instead (calls
    that overlap on one GPU race).  Allocates nothing."""
    lib = load_library()
    p = layout.params
    layout, params = _prepare_layout(topk_idx, p.num_experts, p.expert_alignment,
                                     p.num_partitions, p.capacity, p.max_recv_rows,
                                     cumulative_expert_stats, layout,
                                     layout.partition_offset is not None,
                                     p.partitions_per_group, bool(p.partition_major))
    ptrs = layout.ptrs()
    _launch("ep_get_layout_noalloc", topk_idx.device, lib.ep_get_layout_noalloc,
            [cumulative_expert_stats, layout.status],
            _ptr(topk_idx), ctypes.byref(params), ctypes.byref(ptrs),
            _ptr(cumulative_expert_stats), _stream(topk_idx.device))
    return layout


def _prepare_layout(topk_idx, num_experts, expert_alignment, num_partitions, capacity,
                    max_recv_rows, cumulative_expert_stats, layout, partition_layout,
                    partitions_per_group, partition_major=False):
    """(layout, params) for a layout call: a new Layout, or `layout` checked
    against these shapes."""
    _need_cuda(topk_idx, "topk_idx")
    if topk_idx.dtype != torch.int64 or topk_idx.dim() != 2:
        raise ValueError("topk_idx must be int64 [T, K]")
    T, K = topk_idx.shape
    pm = 1 if partition_major else 0
    if max_recv_rows is None:
        max_recv_rows = worst_case_recv_rows(T, K, num_experts, expert_alignment, capacity,
                                             num_partitions, partition_major)
    params = LayoutParams(num_tokens=T, num_topk=K, num_experts=num_experts,
                          expert_alignment=expert_alignment, num_partitions=num_partitions,
                          capacity=capacity, partitions_per_group=partitions_per_group,
                          partition_major=pm, max_recv_rows=int(max_recv_rows))
    if layout is None:
        layout = Layout(params, topk_idx.device, partition_layout)
    elif ((layout.params.num_tokens, layout.params.num_topk, layout.params.num_experts,
           layout.params.num_partitions, layout.params.max_recv_rows,
           layout.params.partitions_per_group or num_partitions, layout.params.partition_major)
          != (T, K, num_experts, num_partitions, int(max_recv_rows),
              partitions_per_group or num_partitions, pm)
          or (layout.partition_offset is not None) != partition_layout):
        raise ValueError("layout buffers do not match these shapes")
    else:
        layout.params = params
    if cumulative_expert_stats is not None:
        _need_cuda(cumulative_expert_stats, "cumulative_expert_stats")
        S = num_partitions if partition_major else num_experts
        if cumulative_expert_stats.dtype != torch.int32 or cumulative_expert_stats.numel() != S:
            raise ValueError("cumulative_expert_stats must be int32 [receive segments]")
    return layout, params


def _is_fp8(t: torch.Tensor) -> bool:
    return t.dtype in (torch.float8_e4m3fn, torch.uint8)


# Scale formats of the fp8 rows: fp32 amax/448, fp32 rounded up to a power of
# two, or that power of two as one UE8M0 byte (biased exponent).
_FP8_DTYPES = {"fp32": _abi.EP_DTYPE_FP8_E4M3, "pow2": _abi.EP_DTYPE_FP8_E4M3_POW2,
               "ue8m0": _abi.EP_DTYPE_FP8_E4M3_UE8M0}


def _fp8_dtype(scale_fmt: str) -> int:
    if scale_fmt not in _FP8_DTYPES:
        raise ValueError(f"scale_fmt must be one of {sorted(_FP8_DTYPES)}")
    return _FP8_DTYPES[scale_fmt]


def _scale_dtype(scale_fmt: str):
    return torch.uint8 if scale_fmt == "ue8m0" else torch.float32


def ep_dispatch(x: Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]], layout: Layout,
                topk_weights: Optional[torch.Tensor] = None, recv_fp8: bool = False,
                scale_group: int = 128, zero_padding: bool = False,
                num_recv_rows: Optional[int] = None,
                out: Optional[Sequence[Optional[torch.Tensor]]] = None,
                scale_fmt: str = "fp32"):
    """Permute token rows into the receive buffer.

    x: bf16 [T, H], or (fp8 codes [T, H], scales [T, H/G]: float32, or uint8
    UE8M0 bytes).  With bf16 x and recv_fp8=True the rows are cast to e4m3 on
    the fly with scales in `scale_fmt` ("fp32", "pow2" or "ue8m0").  Returns
    (recv_x, recv_scales or None, recv_topk_weights or None); recv buffers
    have num_recv_rows rows (default: the layout's max_recv_rows)."""
    lib = load_library()
    x, x_scales, scale_group, x_dtype, recv_dtype, scale_fmt = _x_and_dtypes(
        x, recv_fp8, scale_group, scale_fmt)
    bufs = _dispatch_buffers(x, layout, topk_weights, recv_dtype, scale_group, scale_fmt,
                             num_recv_rows, out)
    recv_x, recv_s, recv_w, rows = bufs
    params = layout.params
    ptrs = layout.ptrs()
    _launch("ep_dispatch", x.device, lib.ep_dispatch,
            [x_scales, topk_weights, recv_x, recv_s, recv_w, layout.status],
            _ptr(x), x_dtype, _ptr(x_scales), recv_dtype, x.shape[1], scale_group,
            _ptr(topk_weights), ctypes.byref(params), ctypes.byref(ptrs),
            _ptr(recv_x), _ptr(recv_s), _ptr(recv_w), rows,
            1 if zero_padding else 0, _stream(x.device))
    return recv_x, recv_s, recv_w


def ep_dispatch_with_layout(x: Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]],
                            topk_idx: torch.Tensor, num_experts: int, expert_alignment: int = 1,
                            topk_weights: Optional[torch.Tensor] = None, num_partitions: int = 1,
                            capacity: int = 0, max_recv_rows: Optional[int] = None,
                            cumulative_expert_stats: Optional[torch.Tensor] = None,
                            layout: Optional[Layout] = None, recv_fp8: bool = False,
                            scale_group: int = 128, zero_padding: bool = False,
                            num_recv_rows: Optional[int] = None,
                            out: Optional[Sequence[Optional[torch.Tensor]]] = None,
                            scale_fmt: str = "fp32", partition_major: bool = False):
    """ep_get_layout followed by ep_dispatch in one call (the layout's slots
    are derived by the dispatch kernels).  Arguments as the two calls; returns
    (layout, recv_x, recv_scales or None, recv_topk_weights or None), bit for
    bit what the two calls return."""
    lib = load_library()
    layout, params = _prepare_layout(topk_idx, num_experts, expert_alignment, num_partitions,
                                     capacity, max_recv_rows, cumulative_expert_stats, layout,
                                     False, 0, partition_major)
    x, x_scales, scale_group, x_dtype, recv_dtype, scale_fmt = _x_and_dtypes(
        x, recv_fp8, scale_group, scale_fmt)
    recv_x, recv_s, recv_w, rows = _dispatch_buffers(x, layout, topk_weights, recv_dtype,
                                                     scale_group, scale_fmt, num_recv_rows, out)
    ptrs = layout.ptrs()
    _launch("ep_dispatch_with_layout", x.device, lib.ep_dispatch_with_layout,
            [topk_idx, cumulative_expert_stats, layout.workspace, layout.status, x_scales,
             topk_weights, recv_x, recv_s, recv_w],
            _ptr(topk_idx), ctypes.byref(params), ctypes.byref(ptrs),
            _ptr(cumulative_expert_stats), _ptr(layout.workspace), layout.workspace.numel(),
            _ptr(x), x_dtype, _ptr(x_scales), recv_dtype, x.shape[1], scale_group,
            _ptr(topk_weights), _ptr(recv_x), _ptr(recv_s), _ptr(recv_w), rows,
            1 if zero_padding else 0, _stream(x.device))
    return layout, recv_x, recv_s, recv_w


def _dispatch_buffers(x, layout, topk_weights, recv_dtype, scale_group, scale_fmt,
                      num_recv_rows, out):
    """(recv_x, recv_scales, recv_topk_weights, rows) of a dispatch: the
    buffers given in `out`, checked, or new ones."""
    T, H = x.shape
    if T != layout.num_tokens:
        raise ValueError("x rows != layout tokens")
    rows = layout.max_recv_rows if num_recv_rows is None else int(num_recv_rows)
    dev = x.device
    recv_x = recv_s = recv_w = None
    if out is not None:
        recv_x, recv_s, recv_w = (list(out) + [None, None, None])[:3]
    fp8_out = recv_dtype != _abi.EP_DTYPE_BF16
    if recv_x is None:
        recv_x = torch.empty((rows, H), dtype=torch.float8_e4m3fn if fp8_out else torch.bfloat16,
                             device=dev)
    if fp8_out and recv_s is None:
        recv_s = torch.empty((rows, H // scale_group), dtype=_scale_dtype(scale_fmt), device=dev)
    if topk_weights is not None:
        _check(topk_weights, "topk_weights", _F32, layout.num_topk, rows=T)
        if recv_w is None:
            recv_w = torch.empty(rows, dtype=torch.float32, device=dev)
    _check(recv_x, "recv_x", _F8 if fp8_out else _BF16, H, min_rows=rows)
    if fp8_out:
        _check(recv_s, "recv_scales", (_scale_dtype(scale_fmt),), H // scale_group, min_rows=rows)
    _check(recv_w, "recv_topk_weights", _F32, min_rows=rows)
    return recv_x, recv_s, recv_w, rows


def ep_combine(y: torch.Tensor, layout: Layout, topk_weights: Optional[torch.Tensor] = None,
               bias: Union[None, torch.Tensor, Tuple[torch.Tensor, torch.Tensor]] = None,
               recv_topk_weights: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None):
    """Reduce expert outputs y (bf16 [rows, H], the receive layout) back to the
    tokens: out[t] = bias0 + bias1 + sum_k w[t,k] * y[dst_slot[t,k]] (fp32,
    k ascending, bf16 round to nearest even).  Returns (combined_x,
    combined_topk_weights or None)."""
    lib = load_library()
    _need_cuda(y, "y")
    if y.dtype != torch.bfloat16:
        raise ValueError("y must be bf16")
    rows, H = y.shape
    T, K = layout.num_tokens, layout.num_topk
    b0 = b1 = None
    if isinstance(bias, (tuple, list)):
        b0, b1 = (list(bias) + [None, None])[:2]
    elif bias is not None:
        b0 = bias
    for name, b in (("bias0", b0), ("bias1", b1)):
        if b is not None:
            _need_cuda(b, name)
            if b.dtype != torch.bfloat16 or tuple(b.shape) != (T, H):
                raise ValueError(f"{name} must be bf16 [T, H]")
    _check(topk_weights, "topk_weights", _F32, K, rows=T)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=y.device)
    _check(out, "out", _BF16, H, rows=T)
    cw = None
    if recv_topk_weights is not None:
        _check(recv_topk_weights, "recv_topk_weights", _F32, min_rows=rows)
        cw = torch.empty((T, K), dtype=torch.float32, device=y.device)
    params = layout.params
    ptrs = layout.ptrs()
    _launch("ep_combine", y.device, lib.ep_combine,
            [topk_weights, b0, b1, recv_topk_weights, out, layout.status],
            _ptr(y), H, rows, _ptr(topk_weights), _ptr(b0), _ptr(b1),
            ctypes.byref(params), ctypes.byref(ptrs), _ptr(recv_topk_weights),
            _ptr(cw), _ptr(out), _stream(y.device))
    return out, cw


def ep_probe_dispatch_stores(recv_x: torch.Tensor, layout: Layout, pattern: int = 0x3F803F80):
    """A measurement aid, not a step of the method: the bf16 dispatch's row
    stores (same kernel, grid and order) with every token row replaced by the
    32-bit `pattern`, so that no token row is read.  Writes
    recv_x[dst_slot[t, k]] for every kept pair; returns recv_x."""
    lib = load_library()
    _need_cuda(recv_x, "recv_x")
    if recv_x.dtype != torch.bfloat16 or recv_x.dim() != 2:
        raise ValueError("recv_x must be bf16 [rows, H]")
    _check(recv_x, "recv_x", _BF16, recv_x.shape[1])
    params = layout.params
    ptrs = layout.ptrs()
    _launch("ep_probe_dispatch_stores", recv_x.device, lib.ep_probe_dispatch_stores,
            [recv_x, layout.status], recv_x.shape[1], int(pattern) & 0xFFFFFFFF,
            ctypes.byref(params), ctypes.byref(ptrs), _ptr(recv_x), recv_x.shape[0],
            _stream(recv_x.device))
    return recv_x


def logfmt_row_bytes(hidden: int) -> int:
    """Bytes of one row of the 10-bit logarithmic payload (hidden a positive
    multiple of 128)."""
    n = int(load_library().ep_logfmt_row_bytes(int(hidden)))
    if n < 0:
        raise ValueError("hidden must be a positive multiple of 128")
    return n


_U8 = (torch.uint8,)


def ep_logfmt_encode(y: torch.Tensor, out: Optional[torch.Tensor] = None,
                     layout: Optional[Layout] = None) -> torch.Tensor:
    """bf16 rows [rows, H] -> 10-bit logarithmic payload, uint8
    [rows, logfmt_row_bytes(H)] (the use_logfmt format of the low-latency
    combine; layout and rounding in include/ep.h).  With `layout` (the
    receive layout the rows belong to) only rows that hold a pair are
    encoded; the others are left as they are (a combine never reads them)."""
    lib = load_library()
    _need_cuda(y, "y")
    if y.dtype != torch.bfloat16 or y.dim() != 2:
        raise ValueError("y must be bf16 [rows, H]")
    rows, H = y.shape
    rb = logfmt_row_bytes(H)
    if out is None:
        out = torch.empty((rows, rb), dtype=torch.uint8, device=y.device)
    _check(out, "out", _U8, rb, rows=rows)
    if layout is None:
        _launch("ep_logfmt_encode", y.device, lib.ep_logfmt_encode, [out],
                _ptr(y), rows, H, None, None, _ptr(out), _stream(y.device))
        return out
    if rows > layout.max_recv_rows:
        raise ValueError("y has more rows than the layout's max_recv_rows")
    params = layout.params
    ptrs = layout.ptrs()
    _launch("ep_logfmt_encode", y.device, lib.ep_logfmt_encode, [out, layout.src_of_slot],
            _ptr(y), rows, H, ctypes.byref(params), ctypes.byref(ptrs), _ptr(out),
            _stream(y.device))
    return out


def ep_logfmt_decode(payload: torch.Tensor, hidden: int,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """10-bit logarithmic payload -> bf16 rows [rows, hidden] (exact)."""
    lib = load_library()
    rb = logfmt_row_bytes(hidden)
    _check(payload, "payload", _U8, rb)
    rows = payload.shape[0]
    if out is None:
        out = torch.empty((rows, hidden), dtype=torch.bfloat16, device=payload.device)
    _check(out, "out", _BF16, hidden, rows=rows)
    _launch("ep_logfmt_decode", payload.device, lib.ep_logfmt_decode, [out],
            _ptr(payload), rows, hidden, _ptr(out), _stream(payload.device))
    return out


def ep_combine_logfmt(payload: torch.Tensor, hidden: int, layout: Layout,
                      topk_weights: Optional[torch.Tensor] = None,
                      bias: Union[None, torch.Tensor, Tuple[torch.Tensor, torch.Tensor]] = None,
                      recv_topk_weights: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None):
    """ep_combine over payload rows from ep_logfmt_encode (uint8
    [rows, logfmt_row_bytes(hidden)]): bit for bit the combine of the decoded
    rows.  Returns (combined_x, combined_topk_weights or None)."""
    lib = load_library()
    rb = logfmt_row_bytes(hidden)
    _check(payload, "payload", _U8, rb)
    rows, H = payload.shape[0], hidden
    T, K = layout.num_tokens, layout.num_topk
    b0 = b1 = None
    if isinstance(bias, (tuple, list)):
        b0, b1 = (list(bias) + [None, None])[:2]
    elif bias is not None:
        b0 = bias
    for name, b in (("bias0", b0), ("bias1", b1)):
        if b is not None:
            _need_cuda(b, name)
            if b.dtype != torch.bfloat16 or tuple(b.shape) != (T, H):
                raise ValueError(f"{name} must be bf16 [T, H]")
    _check(topk_weights, "topk_weights", _F32, K, rows=T)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=payload.device)
    _check(out, "out", _BF16, H, rows=T)
    cw = None
    if recv_topk_weights is not None:
        _check(recv_topk_weights, "recv_topk_weights", _F32, min_rows=rows)
        cw = torch.empty((T, K), dtype=torch.float32, device=payload.device)
    params = layout.params
    ptrs = layout.ptrs()
    _launch("ep_combine_logfmt", payload.device, lib.ep_combine_logfmt,
            [topk_weights, b0, b1, recv_topk_weights, out, layout.status],
            _ptr(payload), H, rows, _ptr(topk_weights), _ptr(b0), _ptr(b1),
            ctypes.byref(params), ctypes.byref(ptrs), _ptr(recv_topk_weights),
            _ptr(cw), _ptr(out), _stream(payload.device))
    return out, cw


def ep_cast_fp8(x: torch.Tensor, group: int = 128,
                out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, scale_fmt: str = "fp32"):
    """Per (token, group of `group` channels) cast of bf16 rows to e4m3.
    Returns (codes float8_e4m3fn [T, H], scales [T, H/group]): float32 for
    scale_fmt "fp32" (amax/448) and "pow2" (rounded up to a power of two),
    uint8 biased exponents for "ue8m0"."""
    lib = load_library()
    _need_cuda(x, "x")
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bf16")
    out_dtype = _fp8_dtype(scale_fmt)
    T, H = x.shape
    if out is None:
        q = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=x.device)
        s = torch.empty((T, H // group), dtype=_scale_dtype(scale_fmt), device=x.device)
    else:
        q, s = out
    _check(q, "x_fp8", _F8, H, rows=T)
    _check(s, "scales", (_scale_dtype(scale_fmt),), H // group, rows=T)
    _launch("ep_cast_fp8", x.device, lib.ep_cast_fp8, [q, s],
            _ptr(x), T, H, group, out_dtype, _ptr(q), _ptr(s), _stream(x.device))
    return q, s


def _x_and_dtypes(x, recv_fp8, scale_group, scale_fmt="fp32"):
    """(x, x_scales, G, x_dtype, recv_dtype, scale_fmt) for a dispatch call;
    fp8 input with uint8 scales is UE8M0."""
    x_scales = None
    if isinstance(x, (tuple, list)):
        x, x_scales = x
    _need_cuda(x, "x")
    H = x.shape[1]
    if _is_fp8(x):
        if x_scales is None:
            raise ValueError("fp8 x needs its scales")
        _need_cuda(x_scales, "x_scales")
        if x_scales.dtype == torch.uint8:
            scale_fmt = "ue8m0"
        elif x_scales.dtype != torch.float32:
            raise ValueError("fp8 scales must be float32 or uint8 (UE8M0)")
        elif scale_fmt == "ue8m0":
            scale_fmt = "fp32"
        d = _fp8_dtype(scale_fmt)
        if x_scales.dim() != 2 or x_scales.shape[0] != x.shape[0] or x_scales.shape[1] < 1 \
                or H % x_scales.shape[1] != 0:
            raise ValueError("x_scales must be [T, H / group]")
        return x, x_scales, H // x_scales.shape[1], d, d, scale_fmt
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bf16 or fp8")
    recv = _fp8_dtype(scale_fmt) if recv_fp8 else _abi.EP_DTYPE_BF16
    return x, None, scale_group, _abi.EP_DTYPE_BF16, recv, scale_fmt


def ep_dispatch_partitioned(x: Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]],
                            layout: Layout, topk_idx: torch.Tensor,
                            topk_weights: Optional[torch.Tensor] = None, recv_fp8: bool = False,
                            scale_group: int = 128, num_recv_rows: Optional[int] = None,
                            out: Optional[Sequence[Optional[torch.Tensor]]] = None,
                            scale_fmt: str = "fp32"):
    """Non-expanded dispatch: token t's row goes once to every partition q
    that owns one of its experts, at layout.token_slot[t, q].  Returns
    (recv_x, recv_scales or None, recv_topk_idx int64 [rows, K] with the
    partition-local expert id or -1, recv_topk_weights float32 [rows, K] or
    None).  rows defaults to T*P, the worst case; `out` may supply the four
    buffers (None entries are allocated)."""
    lib = load_library()
    if layout.token_slot is None:
        raise ValueError("the partitioned dispatch needs token_slot: partition_layout=True, P <= 64")
    x, x_scales, scale_group, x_dtype, recv_dtype, scale_fmt = _x_and_dtypes(
        x, recv_fp8, scale_group, scale_fmt)
    T, H = x.shape
    K = layout.num_topk
    if T != layout.num_tokens:
        raise ValueError("x rows != layout tokens")
    _check(topk_idx, "topk_idx", _I64, K, rows=T)
    rows = T * layout.num_partitions if num_recv_rows is None else int(num_recv_rows)
    dev = x.device
    fp8_out = recv_dtype != _abi.EP_DTYPE_BF16
    recv_x = recv_s = recv_i = recv_w = None
    if out is not None:
        recv_x, recv_s, recv_i, recv_w = (list(out) + [None] * 4)[:4]
    if recv_x is None:
        recv_x = torch.empty((rows, H), dtype=torch.float8_e4m3fn if fp8_out else torch.bfloat16,
                             device=dev)
    if fp8_out and recv_s is None:
        recv_s = torch.empty((rows, H // scale_group), dtype=_scale_dtype(scale_fmt), device=dev)
    if recv_i is None:
        recv_i = torch.empty((rows, K), dtype=torch.int64, device=dev)
    if topk_weights is not None:
        _check(topk_weights, "topk_weights", _F32, K, rows=T)
        if recv_w is None:
            recv_w = torch.empty((rows, K), dtype=torch.float32, device=dev)
    else:
        recv_w = None
    _check(recv_x, "recv_x", _F8 if fp8_out else _BF16, H, min_rows=rows)
    if fp8_out:
        _check(recv_s, "recv_scales", (_scale_dtype(scale_fmt),), H // scale_group, min_rows=rows)
    _check(recv_i, "recv_topk_idx", _I64, K, min_rows=rows)
    _check(recv_w, "recv_topk_weights", _F32, K, min_rows=rows)
    params = layout.params
    ptrs = layout.ptrs()
    _launch("ep_dispatch_partitioned", dev, lib.ep_dispatch_partitioned,
            [x_scales, topk_idx, topk_weights, recv_x, recv_s, recv_i, recv_w, layout.status],
            _ptr(x), x_dtype, _ptr(x_scales), recv_dtype, H, scale_group,
            _ptr(topk_idx), _ptr(topk_weights), ctypes.byref(params),
            ctypes.byref(ptrs), _ptr(recv_x), _ptr(recv_s), _ptr(recv_i),
            _ptr(recv_w), rows, _stream(dev))
    return recv_x, recv_s, recv_i, recv_w


def _biases(bias, T, H):
    b0 = b1 = None
    if isinstance(bias, (tuple, list)):
        b0, b1 = (list(bias) + [None, None])[:2]
    elif bias is not None:
        b0 = bias
    for name, b in (("bias0", b0), ("bias1", b1)):
        if b is not None:
            _need_cuda(b, name)
            if b.dtype != torch.bfloat16 or tuple(b.shape) != (T, H):
                raise ValueError(f"{name} must be bf16 [T, H]")
    return b0, b1


def ep_combine_partitioned(y: torch.Tensor, layout: Layout,
                           bias: Union[None, torch.Tensor, Tuple[torch.Tensor, torch.Tensor]] = None,
                           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Plain sum of the partitions' rows back to the tokens (fp32, partition
    order, bias first, bf16 round to nearest even)."""
    lib = load_library()
    if layout.token_slot is None:
        raise ValueError("the partitioned combine needs token_slot: partition_layout=True, P <= 64")
    _need_cuda(y, "y")
    if y.dtype != torch.bfloat16:
        raise ValueError("y must be bf16")
    rows, H = y.shape
    T = layout.num_tokens
    b0, b1 = _biases(bias, T, H)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=y.device)
    _check(out, "out", _BF16, H, rows=T)
    params = layout.params
    ptrs = layout.ptrs()
    _launch("ep_combine_partitioned", y.device, lib.ep_combine_partitioned,
            [b0, b1, out, layout.status],
            _ptr(y), H, rows, _ptr(b0), _ptr(b1), ctypes.byref(params),
            ctypes.byref(ptrs), _ptr(out), _stream(y.device))
    return out


def ep_combine_reduced(y: torch.Tensor, layout: Layout, topk_idx: torch.Tensor,
                       topk_weights: Optional[torch.Tensor] = None,
                       bias: Union[None, torch.Tensor, Tuple[torch.Tensor, torch.Tensor]] = None,
                       out: Optional[torch.Tensor] = None,
                       bf16_partials: bool = False) -> torch.Tensor:
    """Two-level combine on the expanded layout: each partition's weighted
    pairs summed in fp32 (rounded to bf16 with bf16_partials), then the
    partials (and bias) summed in fp32 in partition order and rounded to bf16."""
    lib = load_library()
    _need_cuda(y, "y")
    if y.dtype != torch.bfloat16:
        raise ValueError("y must be bf16")
    rows, H = y.shape
    T, K = layout.num_tokens, layout.num_topk
    _check(topk_idx, "topk_idx", _I64, K, rows=T)
    b0, b1 = _biases(bias, T, H)
    _check(topk_weights, "topk_weights", _F32, K, rows=T)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=y.device)
    _check(out, "out", _BF16, H, rows=T)
    params = layout.params
    ptrs = layout.ptrs()
    _launch("ep_combine_reduced", y.device, lib.ep_combine_reduced,
            [topk_idx, topk_weights, b0, b1, out, layout.status],
            _ptr(y), H, rows, _ptr(topk_idx), _ptr(topk_weights), _ptr(b0),
            _ptr(b1), ctypes.byref(params), ctypes.byref(ptrs), _ptr(out),
            1 if bf16_partials else 0, _stream(y.device))
    return out


# Activations of the expert operators: the function, and whether it is gated
# (a row of pre-activations is then [gate | up] and the result half as wide).
_ACTS = {"none": _abi.EP_ACT_NONE, "silu": _abi.EP_ACT_SILU, "gelu": _abi.EP_ACT_GELU,
         "swiglu": _abi.EP_ACT_SWIGLU, "geglu": _abi.EP_ACT_GEGLU}
_FP8_ROW_GROUP = 128
_CHECKPOINT_GROUP = 32


def _activation(name: str):
    if name not in _ACTS:
        raise ValueError(f"activation must be one of {sorted(_ACTS)}")
    return _ACTS[name], name in ("swiglu", "geglu")


def _check3(t: torch.Tensor, name: str, dtypes, shape):
    _need_cuda(t, name)
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")


def _rows_and_scales(v, name):
    """(tensor, scales or None) of bf16 rows or of e4m3 codes with UE8M0
    scales per 128 channels, along the last dimension."""
    if not isinstance(v, (tuple, list)):
        _need_cuda(v, name)
        if v.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be bf16, or (fp8 codes, UE8M0 scales)")
        return v, None
    codes, scales = v
    _need_cuda(codes, name)
    if not _is_fp8(codes):
        raise ValueError(f"{name} must be bf16, or (fp8 codes, UE8M0 scales)")
    if codes.shape[-1] % _FP8_ROW_GROUP:
        raise ValueError(f"fp8 {name} needs a multiple of {_FP8_ROW_GROUP} channels")
    if scales is None or scales.dtype != torch.uint8:
        raise ValueError(f"{name}'s scales must be uint8 (scale_fmt='ue8m0')")
    _check3(scales, f"{name} scales", _U8, (*codes.shape[:-1], codes.shape[-1] // _FP8_ROW_GROUP))
    return codes, scales


def ep_expert_linear(x: Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]],
                     w: Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]], layout: Layout,
                     bias: Optional[torch.Tensor] = None, activation: str = "none",
                     residual: Optional[torch.Tensor] = None, transposed: bool = False,
                     checkpoint: Union[bool, Tuple[torch.Tensor, torch.Tensor], None] = None,
                     out: Optional[torch.Tensor] = None):
    """The experts' matrix product over the receive rows, with its epilogue:
    z[r] = w[e] x[r] + bias[e], out[r] = act(z[r]) + residual[r], e the expert
    of row r.

    x: bf16 [rows, K], or (e4m3 codes [rows, K], UE8M0 scales uint8
    [rows, K/128]) as ep_dispatch(recv_fp8=True, scale_fmt="ue8m0") gives them.
    w: the same type, [E, N, K] (scales [E, N, K/128]); with transposed=True
    (bf16) [E, K, N], which is the data gradient on the forward weights.
    bias: bf16 [E, N].  activation: "none", "silu", "gelu" (tanh form), or
    "swiglu" / "geglu" on z = [gate | up].  residual: bf16 like out.
    checkpoint=True (or the two buffers) also keeps z in 8 bits: (e4m3 codes
    [rows, N], UE8M0 scales uint8 [rows, N/32]) for
    ep_expert_activation_backward (fp8 rows are then multiplied exactly, at the
    bf16 products' rate).  Returns (out bf16 [rows, N or N/2],
    checkpoint or None).  Padding rows are left as they were."""
    lib = load_library()
    act, gated = _activation(activation)
    x, x_scales = _rows_and_scales(x, "x")
    w, w_scales = _rows_and_scales(w, "w")
    if (x_scales is None) != (w_scales is None):
        raise ValueError("x and w must both be bf16 or both be fp8")
    if x.dim() != 2 or w.dim() != 3:
        raise ValueError("x must be [rows, K] and w [E, N, K]")
    rows, K = x.shape
    E = layout.num_experts
    N = w.shape[2] if transposed else w.shape[1]
    _check3(w, "w", _F8 if w_scales is not None else _BF16, (E, K, N) if transposed else (E, N, K))
    M = N // 2 if gated else N
    dev = x.device
    if bias is not None:
        _check3(bias, "bias", _BF16, (E, N))
    if residual is not None:
        _check(residual, "residual", _BF16, M, min_rows=rows)
    if out is None:
        out = torch.empty((rows, M), dtype=torch.bfloat16, device=dev)
    _check(out, "out", _BF16, M, min_rows=rows)
    codes = scales = None
    if isinstance(checkpoint, (tuple, list)):
        codes, scales = checkpoint
    elif checkpoint:
        codes = torch.empty((rows, N), dtype=torch.float8_e4m3fn, device=dev)
        scales = torch.empty((rows, N // _CHECKPOINT_GROUP), dtype=torch.uint8, device=dev)
    if codes is not None:
        if N % _CHECKPOINT_GROUP:
            raise ValueError(f"a checkpoint needs a multiple of {_CHECKPOINT_GROUP} columns")
        _check(codes, "checkpoint codes", _F8, N, min_rows=rows)
        _check(scales, "checkpoint scales", _U8, N // _CHECKPOINT_GROUP, min_rows=rows)
    params = layout.params
    ptrs = layout.ptrs()
    _launch("ep_expert_linear", dev, lib.ep_expert_linear,
            [x_scales, w, w_scales, bias, residual, out, codes, scales, layout.status],
            _ptr(x), _abi.EP_DTYPE_BF16 if x_scales is None else _abi.EP_DTYPE_FP8_E4M3_UE8M0,
            _ptr(x_scales), _ptr(w), _ptr(w_scales), N, K, 1 if transposed else 0, _ptr(bias), act,
            _ptr(residual), ctypes.byref(params), ctypes.byref(ptrs), rows, _ptr(out),
            _ptr(codes), _ptr(scales), _stream(dev))
    return out, (None if codes is None else (codes, scales))


def ep_expert_wgrad(dy: torch.Tensor, x: Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]],
                    layout: Layout, bias_grad: bool = False, dtype: torch.dtype = torch.float32,
                    accumulate: Optional[Sequence[Optional[torch.Tensor]]] = None,
                    out: Optional[Sequence[Optional[torch.Tensor]]] = None):
    """The experts' weight gradient over the receive rows: dw[e] = sum of
    dy[r]^T x[r] over the rows of expert e, [E, N, K] in `dtype` (float32 or
    bfloat16), and with bias_grad db[e] = sum of dy[r], float32 [E, N].

    dy: bf16 [rows, N].  x: bf16 [rows, K], or (e4m3 codes, UE8M0 scales per
    128 channels), the rows of an fp8 dispatch kept for the backward pass.
    accumulate=(dw0, db0): gradients the new ones are added to (db0 None
    without bias_grad); `out` may name the result buffers, the same tensors
    included.  An expert without rows gets zeros (or its dw0).  Returns
    (dw, db or None)."""
    lib = load_library()
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("dtype must be float32 or bfloat16")
    x, x_scales = _rows_and_scales(x, "x")
    if x.dim() != 2 or dy.dim() != 2:
        raise ValueError("dy must be [rows, N] and x [rows, K]")
    rows, K = x.shape
    N = dy.shape[1]
    _check(dy, "dy", _BF16, N, rows=rows)
    E = layout.num_experts
    dev = dy.device
    dw, db = (list(out) + [None, None])[:2] if out is not None else (None, None)
    dw0, db0 = (list(accumulate) + [None, None])[:2] if accumulate is not None else (None, None)
    if accumulate is not None and dw0 is None:
        raise ValueError("accumulate needs the weight gradients to add to")
    if (db is not None or db0 is not None) and not bias_grad:
        raise ValueError("db is given without bias_grad")
    if accumulate is not None and bias_grad and db0 is None:
        raise ValueError("accumulate with bias_grad needs both gradients")
    if dw is None:
        dw = torch.empty((E, N, K), dtype=dtype, device=dev)
    if bias_grad and db is None:
        db = torch.empty((E, N), dtype=torch.float32, device=dev)
    for name, t in (("dw", dw), ("accumulate dw", dw0)):
        if t is not None:
            _check3(t, name, (dtype,), (E, N, K))
    for name, t in (("db", db), ("accumulate db", db0)):
        if t is not None:
            _check3(t, name, _F32, (E, N))
    params = layout.params
    ptrs = layout.ptrs()
    _launch("ep_expert_wgrad", dev, lib.ep_expert_wgrad,
            [x, x_scales, dw0, db0, dw, db, layout.status],
            _ptr(dy), _ptr(x),
            _abi.EP_DTYPE_BF16 if x_scales is None else _abi.EP_DTYPE_FP8_E4M3_UE8M0,
            _ptr(x_scales), N, K, ctypes.byref(params), ctypes.byref(ptrs), rows, _ptr(dw0),
            _ptr(db0), _ptr(dw), 1 if dtype == torch.bfloat16 else 0, _ptr(db), _stream(dev))
    return dw, db


def ep_expert_activation_backward(dh: torch.Tensor,
                                  pre: Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]],
                                  layout: Layout, activation: str = "swiglu",
                                  row_weights: Optional[torch.Tensor] = None,
                                  out: Optional[Sequence[Optional[torch.Tensor]]] = None):
    """The gradient through the experts' activation h = act(z).

    pre: z, as the checkpoint of ep_expert_linear (e4m3 codes [rows, N], UE8M0
    scales [rows, N/32]) or bf16 [rows, N].  dh: bf16 [rows, M] (M = N, N/2
    gated), the gradient of row_weights[r] * h[r] (float32 [rows], ep_dispatch's
    recv_topk_weights; 1 if None).  Returns (dpre bf16 [rows, N], row_weights *
    h bf16 [rows, M], dweights float32 [rows] = sum of dh * h).  Padding rows
    are left as they were; `out` may name the three buffers (None entries are
    allocated).

    With dh from the dispatched gradient dout of the layer, dweights is the
    gradient of the routing weights of y = w2 h.  Where y also has a bias b2,
    add (dout rows * b2[e]).sum(1); b2's own gradient is db of an
    ep_expert_wgrad over the dout rows times row_weights."""
    lib = load_library()
    act, gated = _activation(activation)
    scales = None
    if isinstance(pre, (tuple, list)):
        pre, scales = pre
    _need_cuda(pre, "pre")
    if pre.dim() != 2:
        raise ValueError("pre must be [rows, N]")
    rows, N = pre.shape
    M = N // 2 if gated else N
    if scales is None:
        _check(pre, "pre", _BF16, N)
    else:
        if N % _CHECKPOINT_GROUP:
            raise ValueError(f"a checkpoint needs a multiple of {_CHECKPOINT_GROUP} columns")
        _check(pre, "pre codes", _F8, N)
        _check(scales, "pre scales", _U8, N // _CHECKPOINT_GROUP, rows=rows)
    _check(dh, "dh", _BF16, M, rows=rows)
    _check(row_weights, "row_weights", _F32, min_rows=rows)
    dev = dh.device
    dpre, h, dw = (list(out) + [None] * 3)[:3] if out is not None else (None, None, None)
    if dpre is None:
        dpre = torch.empty((rows, N), dtype=torch.bfloat16, device=dev)
    if h is None:
        h = torch.empty((rows, M), dtype=torch.bfloat16, device=dev)
    if dw is None:
        dw = torch.empty(rows, dtype=torch.float32, device=dev)
    _check(dpre, "dpre", _BF16, N, min_rows=rows)
    _check(h, "h", _BF16, M, min_rows=rows)
    _check(dw, "dweights", _F32, min_rows=rows)
    params = layout.params
    ptrs = layout.ptrs()
    _launch("ep_expert_activation_backward", dev, lib.ep_expert_activation_backward,
            [pre, scales, row_weights, dpre, h, dw, layout.status],
            _ptr(dh), _ptr(pre), _ptr(scales), N, act, _ptr(row_weights), ctypes.byref(params),
            ctypes.byref(ptrs), rows, _ptr(dpre), _ptr(h), _ptr(dw), _stream(dev))
    return dpre, h, dw


def ep_moe_decode(x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: Optional[torch.Tensor],
                  w1: Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]],
                  w2: Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]],
                  activation: str = "swiglu", w1_bias: Optional[torch.Tensor] = None,
                  w2_bias: Optional[torch.Tensor] = None,
                  bias: Union[None, torch.Tensor, Tuple[torch.Tensor, torch.Tensor]] = None,
                  status: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A whole mixture-of-experts layer for a few tokens (at most 1024 (token,
    expert) pairs), without a layout: out[t] = bias0 + bias1 + sum_k w[t,k] *
    (w2[e] act(w1[e] x[t] + w1_bias[e]) + w2_bias[e]), e = topk_idx[t,k].

    x: bf16 [T, H].  topk_idx: int64 [T, K], -1 = none.  topk_weights: float32
    [T, K], or None for the plain sum.  w1: bf16 [E, N, H] (N = 2I for "swiglu"
    and "geglu", gate rows first) and w2: bf16 [E, H, I]; or both (e4m3 codes,
    UE8M0 scales uint8 per 128 channels).  w1_bias: bf16 [E, N], w2_bias: bf16
    [E, H].  bias: up to two bf16 [T, H] tensors, as ep_combine's (a residual,
    a shared expert's output).  status: int32 [1], gets EP_DEV_BAD_EXPERT when
    an id is outside [-1, E).  Returns bf16 [T, H]."""
    lib = load_library()
    act, gated = _activation(activation)
    w1, s1 = _rows_and_scales(w1, "w1")
    w2, s2 = _rows_and_scales(w2, "w2")
    if (s1 is None) != (s2 is None):
        raise ValueError("w1 and w2 must both be bf16 or both be fp8")
    if x.dim() != 2 or w1.dim() != 3 or w2.dim() != 3 or topk_idx.dim() != 2:
        raise ValueError("x must be [T, H], topk_idx [T, K], w1 [E, N, H] and w2 [E, H, I]")
    T, H = x.shape
    E, N = w1.shape[:2]
    inter = N // 2 if gated else N
    kinds = _BF16 if s1 is None else _F8
    _check(x, "x", _BF16, H)
    _check3(w1, "w1", kinds, (E, 2 * inter if gated else N, H))
    _check3(w2, "w2", kinds, (E, H, inter))
    K = topk_idx.shape[1]
    _check(topk_idx, "topk_idx", _I64, K, rows=T)
    _check(topk_weights, "topk_weights", _F32, K, rows=T)
    if w1_bias is not None:
        _check3(w1_bias, "w1_bias", _BF16, (E, N))
    if w2_bias is not None:
        _check3(w2_bias, "w2_bias", _BF16, (E, H))
    b0, b1 = _biases(bias, T, H)
    dev = x.device
    if status is not None:
        _check(status, "status", (torch.int32,), rows=1)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    _check(out, "out", _BF16, H, rows=T)
    nbytes = int(lib.ep_moe_decode_workspace_bytes(T, K, inter))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _launch("ep_moe_decode", dev, lib.ep_moe_decode,
            [topk_idx, topk_weights, w1, s1, w2, s2, w1_bias, w2_bias, b0, b1, status, out],
            _ptr(x), _ptr(topk_idx), _ptr(topk_weights), T, K, E, H, inter,
            _abi.EP_DTYPE_BF16 if s1 is None else _abi.EP_DTYPE_FP8_E4M3_UE8M0, _ptr(w1), _ptr(s1),
            _ptr(w1_bias), _ptr(w2), _ptr(s2), _ptr(w2_bias), act, _ptr(b0), _ptr(b1), _ptr(ws),
            nbytes, _ptr(status), _ptr(out), _stream(dev))
    return out


# The calls below are short against their checks, so each first asks all of them at
# once (_is), and goes through the ones that name the fault only when that fails.
def _is(t: Optional[torch.Tensor], dtype, shape, device: int) -> bool:
    """Whether a buffer (None: not given) is as its kernel takes it."""
    return t is None or (t.dtype is dtype and t.shape == shape and t.get_device() == device
                         and t.is_contiguous())


def _check_codes(v, name):
    """The shapes of 8-bit rows or weights are checked by the caller."""
    codes, scales = v
    _need_cuda(codes, name)
    _need_cuda(scales, f"{name} scales")
    if not _is_fp8(codes):
        raise ValueError(f"{name} must be (fp8 codes, float32 scales)")
    if codes.shape[-1] % _FP8_ROW_GROUP:
        raise ValueError(f"{name} needs a multiple of {_FP8_ROW_GROUP} channels")
    if scales.dtype != torch.float32:
        raise ValueError(f"{name}'s scales must be float32 (scale_fmt 'fp32' or 'pow2')")


def _pair(v, name):
    if not isinstance(v, (tuple, list)) or len(v) != 2:
        raise ValueError(f"{name} must be (fp8 codes, float32 scales)")
    return v


def _scale_blocks(n: int) -> int:
    return (n + _FP8_ROW_GROUP - 1) // _FP8_ROW_GROUP


def ep_cast_fp8_blocks(w: torch.Tensor, transposed: bool = False,
                       out: Optional[Sequence[torch.Tensor]] = None):
    """Weights to e4m3 with one fp32 scale per 128 x 128 block, for
    ep_block_linear: w bf16 [N, K] or [E, N, K] (N and K multiples of 8) to codes
    of its shape and scales [(E,) ceil(N/128), ceil(K/128)] = max(amax, 1e-4) /
    448.  With transposed=True also the same of the transposed matrices, codes
    [(E,) K, N] and scales [(E,) ceil(K/128), ceil(N/128)], the weights of the
    product's data gradient, from the same read.  `out` may name the buffers
    (codes, scales, and with transposed=True the other two).  Returns ((codes,
    scales), (codes_t, scales_t) or None)."""
    lib = load_library()
    _need_cuda(w, "w")
    if w.dtype != torch.bfloat16:
        raise ValueError("w must be bf16")
    if w.dim() not in (2, 3):
        raise ValueError("w must be [N, K] or [E, N, K]")
    lead, (N, K) = tuple(w.shape[:-2]), w.shape[-2:]
    dev = w.device
    shapes = [(*lead, N, K), (*lead, _scale_blocks(N), _scale_blocks(K))]
    if transposed:
        shapes += [(*lead, K, N), (*lead, _scale_blocks(K), _scale_blocks(N))]
    if out is None:
        bufs = [torch.empty(s, dtype=torch.float32 if i & 1 else torch.float8_e4m3fn, device=dev)
                for i, s in enumerate(shapes)]
    else:
        bufs = list(out)
        if len(bufs) != len(shapes):
            raise ValueError(f"out must be {len(shapes)} buffers")
        for i, (t, s) in enumerate(zip(bufs, shapes)):
            _check3(t, "scales" if i & 1 else "codes", _F32 if i & 1 else _F8, s)
    codes_t, scales_t = bufs[2:] if transposed else (None, None)
    _launch("ep_cast_fp8_blocks", dev, lib.ep_cast_fp8_blocks, bufs,
            _ptr(w), lead[0] if lead else 1, N, K, _ptr(bufs[0]), _ptr(bufs[1]), _ptr(codes_t),
            _ptr(scales_t), _stream(dev))
    return (bufs[0], bufs[1]), ((codes_t, scales_t) if transposed else None)


def ep_block_linear(x: Tuple[torch.Tensor, torch.Tensor], w: Tuple[torch.Tensor, torch.Tensor],
                    layout: Optional[Layout] = None, bias: Optional[torch.Tensor] = None,
                    activation: str = "none", residual: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The matrix product of 8-bit rows and weights with one fp32 scale for each
    block of 128, with its epilogue: out[r] = act(w x[r] + bias) + residual[r].

    x: (e4m3 codes [rows, K], float32 scales [rows, K/128]), as
    ep_dispatch(recv_fp8=True) and ep_cast_fp8(x, 128) give them.  w: (e4m3 codes
    [E, N, K], float32 scales [E, ceil(N/128), K/128]) of ep_cast_fp8_blocks.
    With a layout, row r takes the weights of its expert, and rows that hold no
    pair are left as they were; without one all rows take w [N, K], scales
    [ceil(N/128), K/128] (a shared expert; bias [N]).  bias: bf16 [E, N].
    activation: "none", "silu", "gelu" (tanh form), or "swiglu" / "geglu" on z =
    [gate | up] (N a multiple of 64, else of 8).  residual: bf16 like out.
    Returns out, bf16 [rows, N or N/2].

    The data gradient is the same call: the gradient rows through ep_cast_fp8 and
    the transposed pair of ep_cast_fp8_blocks."""
    lib = load_library()
    act, gated = _activation(activation)
    x, x_scales = _pair(x, "x")
    w, w_scales = _pair(w, "w")
    lead = () if layout is None else (layout.num_experts,)
    dev, on = x.device, x.get_device()
    if x.dim() != 2 or w.dim() != 2 + len(lead):
        _check_codes((x, x_scales), "x")
        _check_codes((w, w_scales), "w")
        raise ValueError("x must be [rows, K] and w [E, N, K], or [N, K] without a layout")
    rows, K = x.shape
    N = w.shape[-2]
    M = N // 2 if gated else N
    G, B = K // _FP8_ROW_GROUP, _scale_blocks(N)
    if not (on >= 0 and x.is_contiguous() and x.dtype in _F8 and K % _FP8_ROW_GROUP == 0
            and w.dtype in _F8 and _is(w, w.dtype, (*lead, N, K), on)
            and _is(x_scales, torch.float32, (rows, G), on)
            and _is(w_scales, torch.float32, (*lead, B, G), on)
            and _is(bias, torch.bfloat16, (*lead, N), on)
            and _is(residual, torch.bfloat16, (rows, M), on)
            and _is(out, torch.bfloat16, (rows, M), on)):
        _check_codes((x, x_scales), "x")
        _check_codes((w, w_scales), "w")
        _check3(w, "w", _F8, (*lead, N, K))
        _check3(x_scales, "x scales", _F32, (rows, G))
        _check3(w_scales, "w scales", _F32, (*lead, B, G))
        if bias is not None:
            _check3(bias, "bias", _BF16, (*lead, N))
        _check(residual, "residual", _BF16, M, min_rows=rows)
        _check(out, "out", _BF16, M, min_rows=rows)
    if out is None:
        out = torch.empty((rows, M), dtype=torch.bfloat16, device=dev)
    params = ptrs = ws = None
    nbytes = 0
    if layout is None:
        nbytes = lib.ep_block_linear_workspace_bytes(rows, N, K)
        if nbytes:
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    else:
        params, ptrs = ctypes.byref(layout.params), ctypes.byref(layout.ptrs())
    _launch("ep_block_linear", dev, lib.ep_block_linear,
            (x_scales, w, w_scales, bias, residual, out, None if layout is None else layout.status),
            x.data_ptr(), x_scales.data_ptr(), w.data_ptr(), w_scales.data_ptr(), N, K, _ptr(bias),
            act, _ptr(residual), params, ptrs, rows, _ptr(ws), nbytes, out.data_ptr(), _stream(dev))
    return out


def _ffn_sizes(x: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor, activation: str):
    act, gated = _activation(activation)
    if not gated:
        raise ValueError('the block\'s activation must be "swiglu" or "geglu"')
    if x.dim() != 2 or w2.dim() != 2:
        _need_cuda(x, "x")
        raise ValueError("x must be [T, H], w1 [2 I, H] and w2 [H, I]")
    T, H = x.shape
    inter = w2.shape[1]
    on = x.get_device()
    if not (on >= 0 and _is(x, torch.bfloat16, (T, H), on)
            and _is(w1, torch.bfloat16, (2 * inter, H), on)
            and _is(w2, torch.bfloat16, (H, inter), on)):
        _check(x, "x", _BF16, H)
        _check3(w1, "w1", _BF16, (2 * inter, H))
        _check3(w2, "w2", _BF16, (H, inter))
    return act, T, H, inter, on


def ep_gated_ffn(x: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor, activation: str = "swiglu",
                 residual: Optional[torch.Tensor] = None,
                 save: Union[bool, torch.Tensor] = False, out: Optional[torch.Tensor] = None):
    """The gated feed-forward block that every token passes (a shared expert):
    z = x w1^T = [gate | up], out = (f(gate) * up) w2^T + residual.

    x: bf16 [T, H].  w1: bf16 [2 I, H], gate rows first; w2: bf16 [H, I] (H and I
    multiples of 8).  activation: "swiglu" or "geglu".  residual: bf16 [T, H] (the
    stream, or ep_combine's output; it may be `out`).  save=True (or the buffer,
    bf16 [T, 2 I]) also keeps z for ep_gated_ffn_backward.  Returns (out bf16
    [T, H], z or None)."""
    lib = load_library()
    act, T, H, inter, on = _ffn_sizes(x, w1, w2, activation)
    dev = x.device
    z = save if isinstance(save, torch.Tensor) else None
    if not (_is(z, torch.bfloat16, (T, 2 * inter), on) and _is(residual, torch.bfloat16, (T, H), on)
            and _is(out, torch.bfloat16, (T, H), on)):
        _check(z, "z", _BF16, 2 * inter, rows=T)
        _check(residual, "residual", _BF16, H, rows=T)
        _check(out, "out", _BF16, H, rows=T)
    if z is None and save:
        z = torch.empty((T, 2 * inter), dtype=torch.bfloat16, device=dev)
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    nbytes = lib.ep_gated_ffn_workspace_bytes(T, H, inter, 0)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _launch("ep_gated_ffn", dev, lib.ep_gated_ffn, (w1, w2, residual, z, out),
            x.data_ptr(), T, H, inter, w1.data_ptr(), w2.data_ptr(), act, _ptr(residual), _ptr(z),
            ws.data_ptr(), nbytes, out.data_ptr(), _stream(dev))
    return out, z


def ep_gated_ffn_backward(dout: torch.Tensor, x: torch.Tensor, z: torch.Tensor, w1: torch.Tensor,
                          w2: torch.Tensor, activation: str = "swiglu",
                          dtype: torch.dtype = torch.float32,
                          accumulate: Optional[Sequence[Optional[torch.Tensor]]] = None,
                          out: Optional[Sequence[Optional[torch.Tensor]]] = None):
    """The gradients of ep_gated_ffn: (dx bf16 [T, H], dw1 [2 I, H], dw2 [H, I]),
    the weights' in `dtype` (float32 or bfloat16).

    dout: bf16 [T, H], the gradient of out (and of its residual).  z: what the
    forward pass kept.  accumulate=(dw1, dw2): gradients the new ones are added to;
    `out` may name the result buffers (dx, dw1, dw2; None entries are allocated),
    the same tensors included.  dz and h = f(gate) * up are rounded to bf16 on the
    way, sums are fp32."""
    lib = load_library()
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("dtype must be float32 or bfloat16")
    act, T, H, inter, on = _ffn_sizes(x, w1, w2, activation)
    dev = x.device
    dx, dw1, dw2 = (list(out) + [None] * 3)[:3] if out is not None else (None, None, None)
    in1, in2 = (list(accumulate) + [None, None])[:2] if accumulate is not None else (None, None)
    shape1, shape2 = (2 * inter, H), (H, inter)
    if not (dout is not None and _is(dout, torch.bfloat16, (T, H), on)
            and z is not None and _is(z, torch.bfloat16, (T, 2 * inter), on)
            and _is(dx, torch.bfloat16, (T, H), on)
            and _is(dw1, dtype, shape1, on) and _is(in1, dtype, shape1, on)
            and _is(dw2, dtype, shape2, on) and _is(in2, dtype, shape2, on)):
        if dout is None or z is None:
            raise ValueError("dout and z must be given")
        _check(dout, "dout", _BF16, H, rows=T)
        _check(z, "z", _BF16, 2 * inter, rows=T)
        _check(dx, "dx", _BF16, H, rows=T)
        for name, t, shape in (("dw1", dw1, shape1), ("accumulate dw1", in1, shape1),
                               ("dw2", dw2, shape2), ("accumulate dw2", in2, shape2)):
            if t is not None:
                _check3(t, name, (dtype,), shape)
    if dx is None:
        dx = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    if dw1 is None:
        dw1 = torch.empty(shape1, dtype=dtype, device=dev)
    if dw2 is None:
        dw2 = torch.empty(shape2, dtype=dtype, device=dev)
    nbytes = lib.ep_gated_ffn_workspace_bytes(T, H, inter, 1)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _launch("ep_gated_ffn_backward", dev, lib.ep_gated_ffn_backward,
            (dout, z, w1, w2, in1, in2, dx, dw1, dw2),
            dout.data_ptr(), x.data_ptr(), z.data_ptr(), T, H, inter, w1.data_ptr(), w2.data_ptr(),
            act, _ptr(in1), _ptr(in2), ws.data_ptr(), nbytes, dx.data_ptr(), dw1.data_ptr(),
            dw2.data_ptr(), 1 if dtype == torch.bfloat16 else 0, _stream(dev))
    return dx, dw1, dw2
