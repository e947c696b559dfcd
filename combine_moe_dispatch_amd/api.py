"""Thin ctypes binding over libmoe_dispatch.so.

Argument marshalling only: every step of routing, dispatch and combine runs in
the library's HIP kernels.  torch supplies device memory and the stream.  The
names and arguments follow the C ABI in include/moe_dispatch.h.  Importing this
module loads the library and raises ImportError when it has not been built
(``python -m combine_moe_dispatch_amd.build``); there is no fallback.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_dispatch.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python -m combine_moe_dispatch_amd.build` (hipcc, gfx950)")
_lib = ctypes.CDLL(LIB_PATH)

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_HIP = 0, 1, 2, 3
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_PAYLOAD_BF16, MOE_PAYLOAD_FP8_E4M3_B128 = 0, 1
MOE_DEV_CAPACITY, MOE_DEV_BAD_ID = 1, 2
MOE_MAX_EXPERTS, MOE_MAX_TOP_K = 1024, 32


class _Shape(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("num_ranks", ctypes.c_int32), ("rank_capacity", ctypes.c_int32),
                ("payload", ctypes.c_int32)]


class _Layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "expert_counts", "expert_offsets", "rank_counts", "rank_offsets",
        "token_row", "row_src", "status")]


_vp, _i32 = ctypes.c_void_p, ctypes.c_int32
_lib.moe_recv_rows.argtypes = [ctypes.POINTER(_Shape)]
_lib.moe_recv_rows.restype = ctypes.c_int64
_lib.moe_dispatch_workspace_size.argtypes = [ctypes.POINTER(_Shape)]
_lib.moe_dispatch_workspace_size.restype = ctypes.c_size_t
_lib.moe_route_topk.argtypes = [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp]
_lib.moe_route_topk.restype = _i32
_lib.moe_route_topk_grouped.argtypes = [_vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp]
_lib.moe_route_topk_grouped.restype = _i32
_lib.moe_dispatch.argtypes = [ctypes.POINTER(_Shape), _vp, _vp, _vp, _vp,
                              ctypes.POINTER(_Layout), _vp, ctypes.c_size_t, _vp]
_lib.moe_dispatch.restype = _i32
_lib.moe_expert_scale.argtypes = [ctypes.POINTER(_Shape), _vp, _vp, ctypes.POINTER(_Layout),
                                  _vp, _vp, _vp, _vp]
_lib.moe_expert_scale.restype = _i32
_lib.moe_combine.argtypes = [ctypes.POINTER(_Shape), _vp, _vp, ctypes.POINTER(_Layout),
                             _vp, _vp, _vp]
_lib.moe_combine.restype = _i32
_lib.moe_status_string.argtypes = [_i32]
_lib.moe_status_string.restype = ctypes.c_char_p


class MoeError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call}: {_lib.moe_status_string(status).decode()}")


def _check(status: int, call: str) -> None:
    if status != MOE_OK:
        raise MoeError(status, call)


@dataclasses.dataclass(frozen=True)
class Shape:
    """Sizes of one problem (mirrors moe_shape)."""
    num_tokens: int
    hidden: int
    num_experts: int
    top_k: int
    num_ranks: int
    rank_capacity: int   # 0 = packed regions
    payload: int = MOE_PAYLOAD_BF16

    def c(self) -> _Shape:
        return _Shape(self.num_tokens, self.hidden, self.num_experts, self.top_k,
                      self.num_ranks, self.rank_capacity, self.payload)

    @property
    def fp8(self) -> bool:
        return self.payload == MOE_PAYLOAD_FP8_E4M3_B128


@dataclasses.dataclass
class Layout:
    """Device metadata tensors (mirrors moe_layout); row_src may be None."""
    expert_counts: torch.Tensor
    expert_offsets: torch.Tensor
    rank_counts: torch.Tensor
    rank_offsets: torch.Tensor
    token_row: torch.Tensor
    row_src: Optional[torch.Tensor]
    status: torch.Tensor

    def c(self) -> _Layout:
        p = lambda t: None if t is None else t.data_ptr()
        return _Layout(p(self.expert_counts), p(self.expert_offsets), p(self.rank_counts),
                       p(self.rank_offsets), p(self.token_row), p(self.row_src), p(self.status))

    @staticmethod
    def empty(shape: Shape, device, with_row_src: bool = False) -> "Layout":
        i = dict(dtype=torch.int32, device=device)
        rows = moe_recv_rows(shape)
        return Layout(torch.empty(shape.num_experts, **i), torch.empty(shape.num_experts, **i),
                      torch.empty(shape.num_ranks, **i), torch.empty(shape.num_ranks, **i),
                      torch.empty(shape.num_tokens, shape.top_k, **i),
                      torch.full((rows,), -1, **i) if with_row_src else None,
                      torch.zeros(1, **i))


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _empty(stream, size, dtype, device, returned: bool = True) -> torch.Tensor:
    """Memory that a call on `stream` allocates for itself: from that stream's
    pool, whose blocks no other stream's queued work still uses.  If the caller
    gets it, the current stream is recorded, so that a dropped tensor is not
    reused while work queued there reads it."""
    if stream is None or device.type != "cuda":
        return torch.empty(size, dtype=dtype, device=device)
    own = stream if isinstance(stream, torch.cuda.Stream) else \
        torch.cuda.ExternalStream(_stream(stream), device=device)
    with torch.cuda.stream(own):
        t = torch.empty(size, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


# ---------------------------------------------------------------------------
# Argument checks made before each C call: every tensor must be a contiguous
# GPU tensor of the expected element type holding at least the elements the
# shape addresses (a wrong view or an undersized buffer would otherwise be
# read or written out of bounds by the kernels).  Shapes the library rejects
# are left to it, so its status code is what the caller sees.
# ---------------------------------------------------------------------------
def _gpu(t, name: str, call: str, *, dtype=None, itemsize: Optional[int] = None,
         numel: int = 0, optional: bool = False) -> None:
    if t is None:
        if optional or numel == 0:
            return
        raise ValueError(f"{call}: {name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{call}: {name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{call}: {name} must be a GPU tensor (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{call}: {name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{call}: {name} must be {dtype} (got {t.dtype})")
    if itemsize is not None and t.element_size() != itemsize:
        raise TypeError(f"{call}: {name} must have {itemsize}-byte elements (got {t.dtype})")
    if t.numel() < numel:
        raise ValueError(f"{call}: {name} holds {t.numel()} elements, the shape needs {numel}")


def _rows(shape: Shape) -> Optional[int]:
    """Receive rows of a valid shape, or None (the C call then reports it)."""
    n = _lib.moe_recv_rows(ctypes.byref(shape.c()))
    return None if n < 0 else int(n)


def _payload_rows(shape: Shape, rows: int, t, ts, name: str, call: str,
                  scales_optional: bool = False) -> None:
    """A buffer of `rows` payload rows (bf16, or e4m3 codes plus fp32 scales)."""
    if shape.fp8:
        _gpu(t, name, call, itemsize=1, numel=rows * shape.hidden)
        _gpu(ts, name + " scales", call, dtype=torch.float32,
             numel=rows * (shape.hidden // 128), optional=scales_optional)
    else:
        _gpu(t, name, call, itemsize=2, numel=rows * shape.hidden)


def _layout(lay: "Layout", shape: Shape, rows: int, call: str) -> None:
    if lay is None:
        raise ValueError(f"{call}: layout is required")
    E, N = shape.num_experts, shape.num_ranks
    for f, n in (("expert_counts", E), ("expert_offsets", E), ("rank_counts", N),
                 ("rank_offsets", N), ("status", 1)):
        _gpu(getattr(lay, f), "layout." + f, call, dtype=torch.int32, numel=n)
    _gpu(lay.token_row, "layout.token_row", call, dtype=torch.int32,
         numel=shape.num_tokens * shape.top_k)
    _gpu(lay.row_src, "layout.row_src", call, dtype=torch.int32, numel=rows, optional=True)


def _route_args(call, logits, bias, k, topk_ids, topk_weights):
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError(f"{call}: logits must be a 2-D tensor [T, E]")
    T, E = logits.shape
    _gpu(logits, "logits", call, dtype=torch.float32, numel=T * E)
    _gpu(bias, "bias", call, dtype=torch.float32, numel=E, optional=True)
    _gpu(topk_ids, "topk_ids", call, dtype=torch.int32, numel=T * k)
    _gpu(topk_weights, "topk_weights", call, dtype=torch.float32, numel=T * k)


def moe_recv_rows(shape: Shape) -> int:
    n = _lib.moe_recv_rows(ctypes.byref(shape.c()))
    if n < 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_recv_rows")
    return int(n)


def moe_dispatch_workspace_size(shape: Shape) -> int:
    return int(_lib.moe_dispatch_workspace_size(ctypes.byref(shape.c())))


def moe_route_topk(logits: torch.Tensor, bias: Optional[torch.Tensor], k: int, score: int,
                   topk_ids: Optional[torch.Tensor] = None,
                   topk_weights: Optional[torch.Tensor] = None, stream=None):
    """Top-k routing; returns (topk_ids int32 [T,k], topk_weights fp32 [T,k])."""
    T, E = logits.shape
    if topk_ids is None:
        topk_ids = _empty(stream, (T, k), torch.int32, logits.device)
    if topk_weights is None:
        topk_weights = _empty(stream, (T, k), torch.float32, logits.device)
    _route_args("moe_route_topk", logits, bias, k, topk_ids, topk_weights)
    _check(_lib.moe_route_topk(_ptr(logits), _ptr(bias), T, E, k, score, _ptr(topk_ids),
                               _ptr(topk_weights), _stream(stream)), "moe_route_topk")
    return topk_ids, topk_weights


def moe_route_topk_grouped(logits: torch.Tensor, bias: Optional[torch.Tensor], k: int, score: int,
                           n_groups: int, topk_groups: int,
                           topk_ids: Optional[torch.Tensor] = None,
                           topk_weights: Optional[torch.Tensor] = None, stream=None):
    """Group-limited top-k routing; returns (topk_ids, topk_weights)."""
    T, E = logits.shape
    if topk_ids is None:
        topk_ids = _empty(stream, (T, k), torch.int32, logits.device)
    if topk_weights is None:
        topk_weights = _empty(stream, (T, k), torch.float32, logits.device)
    _route_args("moe_route_topk_grouped", logits, bias, k, topk_ids, topk_weights)
    _check(_lib.moe_route_topk_grouped(_ptr(logits), _ptr(bias), T, E, k, score, n_groups,
                                       topk_groups, _ptr(topk_ids), _ptr(topk_weights),
                                       _stream(stream)), "moe_route_topk_grouped")
    return topk_ids, topk_weights


def moe_dispatch(shape: Shape, x: torch.Tensor, topk_ids: torch.Tensor, recv_x: torch.Tensor,
                 recv_scales: Optional[torch.Tensor], layout: Layout,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rows = _rows(shape)
    if rows is not None:
        c = "moe_dispatch"
        T, H, k = shape.num_tokens, shape.hidden, shape.top_k
        _gpu(x, "x", c, itemsize=2, numel=T * H)
        _gpu(topk_ids, "topk_ids", c, dtype=torch.int32, numel=T * k)
        _payload_rows(shape, rows, recv_x, recv_scales, "recv_x", c)
        _layout(layout, shape, rows, c)
        # the library compares the workspace's bytes with what the shape needs
        _gpu(workspace, "workspace", c, optional=True)
    _check(_lib.moe_dispatch(ctypes.byref(shape.c()), _ptr(x), _ptr(topk_ids), _ptr(recv_x),
                             _ptr(recv_scales), ctypes.byref(layout.c()), _ptr(workspace),
                             ws_bytes, _stream(stream)), "moe_dispatch")


_lib.moe_dispatch_static.argtypes = [ctypes.POINTER(_Shape), _vp, _vp, _vp, _vp,
                                     ctypes.POINTER(_Layout), _vp]
_lib.moe_dispatch_static.restype = _i32
MOE_STATIC_SCRATCH_BYTES = 4 << 20


def moe_dispatch_static(shape: Shape, x: torch.Tensor, topk_ids: torch.Tensor,
                        recv_x: torch.Tensor, recv_scales: Optional[torch.Tensor],
                        layout: Layout, stream=None) -> None:
    """moe_dispatch without a workspace: the library's per-GPU scratch array
    serves the multi-kernel layout path (calls on one GPU must not overlap)."""
    rows = _rows(shape)
    if rows is not None:
        c = "moe_dispatch_static"
        T, H, k = shape.num_tokens, shape.hidden, shape.top_k
        _gpu(x, "x", c, itemsize=2, numel=T * H)
        _gpu(topk_ids, "topk_ids", c, dtype=torch.int32, numel=T * k)
        _payload_rows(shape, rows, recv_x, recv_scales, "recv_x", c)
        _layout(layout, shape, rows, c)
    _check(_lib.moe_dispatch_static(ctypes.byref(shape.c()), _ptr(x), _ptr(topk_ids),
                                    _ptr(recv_x), _ptr(recv_scales), ctypes.byref(layout.c()),
                                    _stream(stream)), "moe_dispatch_static")


_lib.moe_dispatch_sources.argtypes = [ctypes.POINTER(_Shape), _i32, _vp, _vp, _vp, _vp,
                                      ctypes.POINTER(_Layout), _vp, _vp, _vp, ctypes.c_size_t,
                                      _vp]
_lib.moe_dispatch_sources.restype = _i32


def world_shape(shape: Shape, num_sources: int) -> Shape:
    """The shape of all sources together (num_tokens = S*T)."""
    return dataclasses.replace(shape, num_tokens=shape.num_tokens * num_sources)


def moe_dispatch_sources(shape: Shape, num_sources: int, x: torch.Tensor,
                         topk_ids: torch.Tensor, recv_x: torch.Tensor,
                         recv_scales: Optional[torch.Tensor], layout: Layout,
                         source_counts: torch.Tensor, source_offsets: torch.Tensor,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Every source rank dispatching at once; shape holds one source's sizes."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    world = world_shape(shape, num_sources) if num_sources >= 1 else shape
    rows = _rows(world)
    if rows is not None and num_sources >= 1:
        c = "moe_dispatch_sources"
        T, H, k = world.num_tokens, world.hidden, world.top_k
        _gpu(x, "x", c, itemsize=2, numel=T * H)
        _gpu(topk_ids, "topk_ids", c, dtype=torch.int32, numel=T * k)
        _payload_rows(world, rows, recv_x, recv_scales, "recv_x", c)
        _layout(layout, world, rows, c)
        _gpu(source_counts, "source_counts", c, dtype=torch.int32,
             numel=num_sources * shape.num_experts)
        _gpu(source_offsets, "source_offsets", c, dtype=torch.int32,
             numel=num_sources * shape.num_experts)
    _check(_lib.moe_dispatch_sources(ctypes.byref(shape.c()), num_sources, _ptr(x),
                                     _ptr(topk_ids), _ptr(recv_x), _ptr(recv_scales),
                                     ctypes.byref(layout.c()), _ptr(source_counts),
                                     _ptr(source_offsets), _ptr(workspace), ws_bytes,
                                     _stream(stream)), "moe_dispatch_sources")


def moe_expert_scale(shape: Shape, recv_x: torch.Tensor, recv_scales: Optional[torch.Tensor],
                     layout: Layout, alpha: torch.Tensor, y: torch.Tensor,
                     y_scales: Optional[torch.Tensor], stream=None) -> None:
    rows = _rows(shape)
    if rows is not None:
        c = "moe_expert_scale"
        _payload_rows(shape, rows, recv_x, recv_scales, "recv_x", c)
        _payload_rows(shape, rows, y, y_scales, "y", c)
        _gpu(alpha, "alpha", c, dtype=torch.float32, numel=shape.num_experts)
        _layout(layout, shape, rows, c)
    _check(_lib.moe_expert_scale(ctypes.byref(shape.c()), _ptr(recv_x), _ptr(recv_scales),
                                 ctypes.byref(layout.c()), _ptr(alpha), _ptr(y), _ptr(y_scales),
                                 _stream(stream)), "moe_expert_scale")


def moe_combine(shape: Shape, expert_y: torch.Tensor, expert_scales: Optional[torch.Tensor],
                layout: Layout, topk_weights: torch.Tensor, out: torch.Tensor,
                stream=None) -> None:
    rows = _rows(shape)
    if rows is not None:
        c = "moe_combine"
        T, H, k = shape.num_tokens, shape.hidden, shape.top_k
        _payload_rows(shape, rows, expert_y, expert_scales, "expert_y", c)
        _layout(layout, shape, rows, c)
        _gpu(topk_weights, "topk_weights", c, dtype=torch.float32, numel=T * k)
        _gpu(out, "out", c, itemsize=2, numel=T * H)
    _check(_lib.moe_combine(ctypes.byref(shape.c()), _ptr(expert_y), _ptr(expert_scales),
                            ctypes.byref(layout.c()), _ptr(topk_weights), _ptr(out),
                            _stream(stream)), "moe_combine")


_lib.moe_combine_partial_send.argtypes = [ctypes.POINTER(_Shape), _vp, _vp, ctypes.POINTER(_Layout),
                                  _vp, _vp, _vp, _vp, _vp]
_lib.moe_combine_partial_send.restype = _i32
_lib.moe_combine_partial_recv.argtypes = [ctypes.POINTER(_Shape), _vp, _vp, _vp, _vp]
_lib.moe_combine_partial_recv.restype = _i32


def partial_slots(shape: Shape) -> int:
    """M = min(k, N): partial rows per token of the two-stage combine."""
    return min(shape.top_k, shape.num_ranks)


def moe_combine_partial_send(shape: Shape, expert_y: torch.Tensor, expert_scales: Optional[torch.Tensor],
                     layout: Layout, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                     partial: torch.Tensor, partial_rank: torch.Tensor, stream=None) -> None:
    """Stage 1 of the two-stage combine: one bf16 row per (token, rank)."""
    rows = _rows(shape)
    if rows is not None:
        c = "moe_combine_partial_send"
        T, H, k, M = shape.num_tokens, shape.hidden, shape.top_k, partial_slots(shape)
        _payload_rows(shape, rows, expert_y, expert_scales, "expert_y", c)
        _layout(layout, shape, rows, c)
        _gpu(topk_ids, "topk_ids", c, dtype=torch.int32, numel=T * k)
        _gpu(topk_weights, "topk_weights", c, dtype=torch.float32, numel=T * k)
        _gpu(partial, "partial", c, itemsize=2, numel=T * M * H)
        _gpu(partial_rank, "partial_rank", c, dtype=torch.int32, numel=T * M)
    _check(_lib.moe_combine_partial_send(ctypes.byref(shape.c()), _ptr(expert_y), _ptr(expert_scales),
                                 ctypes.byref(layout.c()), _ptr(topk_ids), _ptr(topk_weights),
                                 _ptr(partial), _ptr(partial_rank), _stream(stream)),
           "moe_combine_partial_send")


def moe_combine_partial_recv(shape: Shape, partial: torch.Tensor, partial_rank: torch.Tensor,
                     out: torch.Tensor, stream=None) -> None:
    """Stage 2: sum of each token's partial rows."""
    if _rows(shape) is not None:
        c = "moe_combine_partial_recv"
        T, H, M = shape.num_tokens, shape.hidden, partial_slots(shape)
        _gpu(partial, "partial", c, itemsize=2, numel=T * M * H)
        _gpu(partial_rank, "partial_rank", c, dtype=torch.int32, numel=T * M)
        _gpu(out, "out", c, itemsize=2, numel=T * H)
    _check(_lib.moe_combine_partial_recv(ctypes.byref(shape.c()), _ptr(partial), _ptr(partial_rank),
                                 _ptr(out), _stream(stream)), "moe_combine_partial_recv")


_lib.moe_dispatch_recv.argtypes = [ctypes.POINTER(_Shape), _vp, _vp, ctypes.POINTER(_Layout),
                                   _vp, _vp, _vp, _vp]
_lib.moe_dispatch_recv.restype = _i32
_lib.moe_combine_send.argtypes = [ctypes.POINTER(_Shape), _vp, _vp, ctypes.POINTER(_Layout),
                                  _vp, _vp, _vp]
_lib.moe_combine_send.restype = _i32


def moe_dispatch_recv(shape: Shape, recv_x: torch.Tensor, recv_scales: Optional[torch.Tensor],
                      layout: Layout, gemm_x: torch.Tensor, gemm_scales: Optional[torch.Tensor],
                      gemm_offsets: torch.Tensor, stream=None) -> None:
    """Receive half of dispatch: receive regions -> dense grouped-GEMM input."""
    rows = _rows(shape)
    if rows is not None:
        c = "moe_dispatch_recv"
        _payload_rows(shape, rows, recv_x, recv_scales, "recv_x", c)
        _payload_rows(shape, shape.num_tokens * shape.top_k, gemm_x, gemm_scales, "gemm_x", c)
        _layout(layout, shape, rows, c)
        _gpu(gemm_offsets, "gemm_offsets", c, dtype=torch.int32, numel=shape.num_experts + 1)
    _check(_lib.moe_dispatch_recv(ctypes.byref(shape.c()), _ptr(recv_x), _ptr(recv_scales),
                                  ctypes.byref(layout.c()), _ptr(gemm_x), _ptr(gemm_scales),
                                  _ptr(gemm_offsets), _stream(stream)), "moe_dispatch_recv")


def moe_combine_send(shape: Shape, gemm_y: torch.Tensor, gemm_scales: Optional[torch.Tensor],
                     layout: Layout, expert_y: torch.Tensor,
                     expert_scales: Optional[torch.Tensor], stream=None) -> None:
    """Send half of the combine: dense expert outputs -> receive-region layout."""
    rows = _rows(shape)
    if rows is not None:
        c = "moe_combine_send"
        _payload_rows(shape, shape.num_tokens * shape.top_k, gemm_y, gemm_scales, "gemm_y", c)
        _payload_rows(shape, rows, expert_y, expert_scales, "expert_y", c)
        _layout(layout, shape, rows, c)
    _check(_lib.moe_combine_send(ctypes.byref(shape.c()), _ptr(gemm_y), _ptr(gemm_scales),
                                 ctypes.byref(layout.c()), _ptr(expert_y), _ptr(expert_scales),
                                 _stream(stream)), "moe_combine_send")


def moe_status_string(status: int) -> str:
    return _lib.moe_status_string(status).decode()


def alloc_recv(shape: Shape, device, fill: Optional[int] = None):
    """Receive buffer (bf16 rows or e4m3 codes) and, for fp8, its scales."""
    rows = moe_recv_rows(shape)
    if shape.fp8:
        buf = torch.empty(rows, shape.hidden, dtype=torch.uint8, device=device)
        sc = torch.empty(rows, shape.hidden // 128, dtype=torch.float32, device=device)
    else:
        buf = torch.empty(rows, shape.hidden, dtype=torch.int16, device=device)
        sc = None
    if fill is not None:
        buf.fill_(fill if shape.fp8 else (fill - 0x10000 if fill >= 0x8000 else fill))
        if sc is not None:
            sc.fill_(float("nan"))
    return buf, sc


def alloc_workspace(shape: Shape, device) -> Optional[torch.Tensor]:
    n = moe_dispatch_workspace_size(shape)
    return None if n == 0 else torch.empty(n, dtype=torch.uint8, device=device)


# ---------------------------------------------------------------------------
# include/moe_experts.h: the experts' matrix product, the balance loss and the
# gradients.  These calls run on the device of their tensors, which must all be
# on one; without a stream they use that device's current one.  What a call
# allocates (results not given, a workspace) comes from its stream's pool.
# ---------------------------------------------------------------------------
MOE_ACT_NONE, MOE_ACT_SILU, MOE_ACT_GELU, MOE_ACT_SWIGLU = 0, 1, 2, 3


class _Linear(ctypes.Structure):
    _fields_ = [("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32),
                ("activation", ctypes.c_int32)]


_f32, _size = ctypes.c_float, ctypes.c_size_t
_shape_p, _layout_p, _linear_p = (ctypes.POINTER(c) for c in (_Shape, _Layout, _Linear))
_lib.moe_expert_matmul.argtypes = [_shape_p, _linear_p, _vp, _vp, _layout_p, _vp, _vp, _vp, _vp,
                                   _vp, _vp, _vp]
_lib.moe_expert_matmul.restype = _i32
_lib.moe_expert_matmul_backward_workspace_size.argtypes = [_shape_p, _linear_p]
_lib.moe_expert_matmul_backward_workspace_size.restype = _size
_lib.moe_expert_matmul_backward.argtypes = [_shape_p, _linear_p, _vp, _vp, _layout_p, _vp, _vp,
                                            _vp, _vp, _vp, _vp, _size, _vp]
_lib.moe_expert_matmul_backward.restype = _i32
_lib.moe_combine_backward.argtypes = [_shape_p, _vp, _vp, _layout_p, _vp, _vp, _vp, _vp]
_lib.moe_combine_backward.restype = _i32
_lib.moe_balance_loss_workspace_size.argtypes = [_i32, _i32, _i32]
_lib.moe_balance_loss_workspace_size.restype = _size
_lib.moe_balance_loss.argtypes = [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _i32, _f32, _vp,
                                  _vp, _vp, _vp, _vp, _size, _vp]
_lib.moe_balance_loss.restype = _i32
_lib.moe_route_backward_workspace_size.argtypes = [_i32, _i32]
_lib.moe_route_backward_workspace_size.restype = _size
_lib.moe_route_backward.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _i32,
                                    _f32, _vp, _vp, _vp, _vp, _vp, _vp, _size, _vp]
_lib.moe_route_backward.restype = _i32

_F32, _I32 = (torch.float32,), (torch.int32,)
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)          # values, or their bits
_E4M3 = (torch.float8_e4m3fn, torch.uint8, torch.int8)
_BYTES = (torch.uint8, torch.int8)


@dataclasses.dataclass(frozen=True)
class Linear:
    """One linear layer of every expert (mirrors moe_linear)."""
    in_features: int
    out_features: int
    activation: int = MOE_ACT_NONE

    def c(self) -> _Linear:
        return _Linear(self.in_features, self.out_features, self.activation)

    @property
    def pre_features(self) -> int:
        """Columns before the activation (weight rows per expert)."""
        return self.out_features * (2 if self.activation == MOE_ACT_SWIGLU else 1)


def _all(call: str, specs) -> int:
    """Check (name, tensor, dtypes, elements, required) entries; returns the
    one device index all tensors are on."""
    dev = -1
    for name, t, dtypes, numel, required in specs:
        if t is None:
            if required and numel > 0:
                raise ValueError(f"{call}: {name} is required")
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{call}: {name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{call}: {name} must be a GPU tensor (got {t.device})")
        if t.dtype not in dtypes:
            raise TypeError(f"{call}: {name} must be {dtypes[0]} (got {t.dtype})")
        if not t.is_contiguous():
            raise ValueError(f"{call}: {name} must be contiguous")
        if t.numel() < numel:
            raise ValueError(f"{call}: {name} holds {t.numel()} elements, {numel} are needed")
        d = t.get_device()
        if dev < 0:
            dev = d
        elif d != dev:
            raise ValueError(f"{call}: {name} is on cuda:{d}, other tensors on cuda:{dev}")
    return dev


# the current stream's handle without a Stream object around it (0.1 against 2.9 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _run(call: str, dev: int, stream, fn, *args) -> None:
    if dev < 0:  # nothing to launch on: the library names what is wrong
        _check(fn(*args, None), call)
        return
    if getattr(stream, "device_index", dev) != dev:
        raise ValueError(f"{call}: stream is on cuda:{stream.device_index}, tensors on cuda:{dev}")
    handle = _raw_stream(dev) if stream is None else _stream(stream)
    if dev == torch.cuda.current_device():
        _check(fn(*args, handle), call)
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, handle), call)


def _workspace(nbytes: int, given, dev: int, stream):
    """The caller's workspace, or one of the call's own."""
    if given is not None or nbytes == 0:
        return given
    if dev < 0:
        return None
    return _empty(stream, nbytes, torch.uint8, torch.device("cuda", dev), returned=False)


def _nbytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _segments(shape: Shape, layout: Optional[Layout]):
    if layout is None:
        return ()
    return (("layout.expert_counts", layout.expert_counts, _I32, shape.num_experts, True),
            ("layout.expert_offsets", layout.expert_offsets, _I32, shape.num_experts, True))


def _maybe(c):
    return None if c is None else ctypes.byref(c)


def moe_expert_matmul(shape: Shape, linear: Linear, x: torch.Tensor,
                      x_scales: Optional[torch.Tensor], layout: Optional[Layout],
                      weight: torch.Tensor, weight_scales: Optional[torch.Tensor],
                      bias: Optional[torch.Tensor], residual: Optional[torch.Tensor],
                      y: torch.Tensor, pre: Optional[torch.Tensor] = None, stream=None) -> None:
    """y = act(x weight[e]^T + bias[e]) + residual on every expert's placed rows.

    layout None: a dense product over num_tokens rows (num_experts == top_k == 1)."""
    c, dev = "moe_expert_matmul", -1
    rows = _rows(shape)
    if rows is not None:
        E, K, F, P = shape.num_experts, linear.in_features, linear.out_features, linear.pre_features
        rows = rows if layout is not None else shape.num_tokens
        fp8 = shape.fp8
        rt = _E4M3 if fp8 else _BF16
        dev = _all(c, (("x", x, rt, rows * K, True),
                       ("x_scales", x_scales, _F32, rows * (K // 128) if fp8 else 0, fp8),
                       ("weight", weight, rt, E * P * K, True),
                       ("weight_scales", weight_scales, _F32,
                        E * (P // 128) * (K // 128) if fp8 else 0, fp8),
                       ("bias", bias, _F32, E * P, False),
                       ("residual", residual, _BF16, rows * F, False),
                       ("y", y, _BF16, rows * F, True), ("pre", pre, _BF16, rows * P, False),
                       *_segments(shape, layout)))
    lay = None if layout is None else layout.c()
    _run(c, dev, stream, _lib.moe_expert_matmul, ctypes.byref(shape.c()),
         ctypes.byref(linear.c()), _ptr(x), _ptr(x_scales), _maybe(lay), _ptr(weight),
         _ptr(weight_scales), _ptr(bias), _ptr(residual), _ptr(y), _ptr(pre))


def moe_expert_matmul_backward_workspace_size(shape: Shape, linear: Linear) -> int:
    return int(_lib.moe_expert_matmul_backward_workspace_size(ctypes.byref(shape.c()),
                                                              ctypes.byref(linear.c())))


def alloc_expert_workspace(shape: Shape, linear: Linear, device) -> Optional[torch.Tensor]:
    """Workspace of moe_expert_matmul_backward (None when none is needed)."""
    n = moe_expert_matmul_backward_workspace_size(shape, linear)
    return None if n == 0 else torch.empty(n, dtype=torch.uint8, device=device)


def moe_expert_matmul_backward(shape: Shape, linear: Linear, grad_y: torch.Tensor,
                               x: Optional[torch.Tensor], layout: Optional[Layout],
                               weight: Optional[torch.Tensor], pre: Optional[torch.Tensor],
                               grad_x: Optional[torch.Tensor],
                               grad_weight: Optional[torch.Tensor],
                               grad_bias: Optional[torch.Tensor],
                               workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of moe_expert_matmul (bf16); any of the three outputs may be None."""
    c, dev = "moe_expert_matmul_backward", -1
    rows = _rows(shape)
    if rows is not None:
        E, K, F, P = shape.num_experts, linear.in_features, linear.out_features, linear.pre_features
        rows = rows if layout is not None else shape.num_tokens
        dev = _all(c, (("grad_y", grad_y, _BF16, rows * F, True),
                       ("x", x, _BF16, rows * K, grad_weight is not None),
                       ("weight", weight, _BF16, E * P * K, grad_x is not None),
                       ("pre", pre, _BF16, rows * P, linear.activation != MOE_ACT_NONE),
                       ("grad_x", grad_x, _BF16, rows * K, False),
                       ("grad_weight", grad_weight, _BF16, E * P * K, False),
                       ("grad_bias", grad_bias, _F32, E * P, False),
                       ("workspace", workspace, _BYTES, 0, False), *_segments(shape, layout)))
    lay = None if layout is None else layout.c()
    _run(c, dev, stream, _lib.moe_expert_matmul_backward, ctypes.byref(shape.c()),
         ctypes.byref(linear.c()), _ptr(grad_y), _ptr(x), _maybe(lay), _ptr(weight), _ptr(pre),
         _ptr(grad_x), _ptr(grad_weight), _ptr(grad_bias), _ptr(workspace), _nbytes(workspace))


def moe_combine_backward(shape: Shape, grad_out: torch.Tensor, expert_y: Optional[torch.Tensor],
                         layout: Layout, topk_weights: Optional[torch.Tensor],
                         grad_y: Optional[torch.Tensor], grad_weights: Optional[torch.Tensor],
                         stream=None) -> None:
    """Gradients of moe_combine (bf16); either output may be None."""
    c, dev = "moe_combine_backward", -1
    rows = _rows(shape)
    if rows is not None:
        if layout is None:
            raise ValueError(f"{c}: layout is required")
        T, H, k = shape.num_tokens, shape.hidden, shape.top_k
        dev = _all(c, (("grad_out", grad_out, _BF16, T * H, True),
                       ("expert_y", expert_y, _BF16, rows * H, grad_weights is not None),
                       ("layout.token_row", layout.token_row, _I32, T * k, True),
                       ("topk_weights", topk_weights, _F32, T * k, grad_y is not None),
                       ("grad_y", grad_y, _BF16, rows * H, False),
                       ("grad_weights", grad_weights, _F32, T * k, False)))
    _run(c, dev, stream, _lib.moe_combine_backward, ctypes.byref(shape.c()), _ptr(grad_out),
         _ptr(expert_y), ctypes.byref(layout.c()), _ptr(topk_weights), _ptr(grad_y),
         _ptr(grad_weights))


def moe_balance_loss_workspace_size(T: int, E: int, num_seqs: int) -> int:
    return int(_lib.moe_balance_loss_workspace_size(T, E, num_seqs))


def moe_balance_loss(logits: torch.Tensor, bias: Optional[torch.Tensor], topk_ids: torch.Tensor,
                     score: int, coef: float, seq_offsets: Optional[torch.Tensor] = None,
                     expert_counts: Optional[torch.Tensor] = None,
                     expert_probs: Optional[torch.Tensor] = None,
                     seq_tokens: Optional[torch.Tensor] = None,
                     loss: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """Balance loss of a routed batch; returns (loss [1], expert_counts [S,E],
    expert_probs [S,E], seq_tokens [S])."""
    c = "moe_balance_loss"
    T, E, k = _router_sizes(c, logits, topk_ids)
    S = _num_seqs(c, seq_offsets)
    dev = logits.device
    if expert_counts is None:
        expert_counts = _empty(stream, (S, E), torch.int32, dev)
    if expert_probs is None:
        expert_probs = _empty(stream, (S, E), torch.float32, dev)
    if seq_tokens is None:
        seq_tokens = _empty(stream, S, torch.int32, dev)
    if loss is None:
        loss = _empty(stream, 1, torch.float32, dev)
    d = _all(c, (("logits", logits, _F32, T * E, True), ("bias", bias, _F32, E, False),
                 ("topk_ids", topk_ids, _I32, T * k, True),
                 ("seq_offsets", seq_offsets, _I32, S + 1, False),
                 ("expert_counts", expert_counts, _I32, S * E, True),
                 ("expert_probs", expert_probs, _F32, S * E, True),
                 ("seq_tokens", seq_tokens, _I32, S, True), ("loss", loss, _F32, 1, True),
                 ("workspace", workspace, _BYTES, 0, False)))
    ws = _workspace(_lib.moe_balance_loss_workspace_size(T, E, S), workspace, d, stream)
    _run(c, d, stream, _lib.moe_balance_loss, _ptr(logits), _ptr(bias), _ptr(topk_ids), T, E, k,
         score, _ptr(seq_offsets), S, coef, _ptr(expert_counts), _ptr(expert_probs),
         _ptr(seq_tokens), _ptr(loss), _ptr(ws), _nbytes(ws))
    return loss, expert_counts, expert_probs, seq_tokens


def moe_route_backward_workspace_size(T: int, E: int) -> int:
    return int(_lib.moe_route_backward_workspace_size(T, E))


def moe_route_backward(logits: torch.Tensor, bias: Optional[torch.Tensor], topk_ids: torch.Tensor,
                       topk_weights: Optional[torch.Tensor],
                       grad_weights: Optional[torch.Tensor], score: int, coef: float = 0.0,
                       seq_offsets: Optional[torch.Tensor] = None,
                       expert_counts: Optional[torch.Tensor] = None,
                       seq_tokens: Optional[torch.Tensor] = None,
                       grad_loss: Optional[torch.Tensor] = None,
                       grad_logits: Optional[torch.Tensor] = None,
                       grad_bias: Optional[torch.Tensor] = None, with_grad_bias: bool = False,
                       workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradient of the router's logits; returns (grad_logits [T,E], grad_bias [E]
    or None).  with_grad_bias: allocate grad_bias when none is given."""
    c = "moe_route_backward"
    T, E, k = _router_sizes(c, logits, topk_ids)
    S = _num_seqs(c, seq_offsets)
    dev = logits.device
    if grad_logits is None:
        grad_logits = _empty(stream, (T, E), torch.float32, dev)
    if grad_bias is None and with_grad_bias:
        grad_bias = _empty(stream, E, torch.float32, dev)
    d = _all(c, (("logits", logits, _F32, T * E, True), ("bias", bias, _F32, E, False),
                 ("topk_ids", topk_ids, _I32, T * k, True),
                 ("topk_weights", topk_weights, _F32, T * k, grad_weights is not None),
                 ("grad_weights", grad_weights, _F32, T * k, False),
                 ("seq_offsets", seq_offsets, _I32, S + 1, False),
                 ("expert_counts", expert_counts, _I32, S * E, False),
                 ("seq_tokens", seq_tokens, _I32, S, False),
                 ("grad_loss", grad_loss, _F32, 1, False),
                 ("grad_logits", grad_logits, _F32, T * E, True),
                 ("grad_bias", grad_bias, _F32, E, False),
                 ("workspace", workspace, _BYTES, 0, False)))
    need = 0 if grad_bias is None else _lib.moe_route_backward_workspace_size(T, E)
    ws = _workspace(need, workspace, d, stream)
    _run(c, d, stream, _lib.moe_route_backward, _ptr(logits), _ptr(bias), _ptr(topk_ids),
         _ptr(topk_weights), _ptr(grad_weights), T, E, k, score, _ptr(seq_offsets), S, coef,
         _ptr(expert_counts), _ptr(seq_tokens), _ptr(grad_loss), _ptr(grad_logits),
         _ptr(grad_bias), _ptr(ws), _nbytes(ws))
    return grad_logits, grad_bias


def _router_sizes(call, logits, topk_ids):
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError(f"{call}: logits must be a 2-D tensor [T, E]")
    if not isinstance(topk_ids, torch.Tensor) or topk_ids.dim() != 2 or \
            topk_ids.shape[0] != logits.shape[0]:
        raise ValueError(f"{call}: topk_ids must be a 2-D tensor [T, k]")
    return logits.shape[0], logits.shape[1], topk_ids.shape[1]


def _num_seqs(call, seq_offsets) -> int:
    if seq_offsets is None:
        return 1
    if not isinstance(seq_offsets, torch.Tensor) or seq_offsets.dim() != 1:
        raise ValueError(f"{call}: seq_offsets must be a 1-D tensor [S + 1]")
    if seq_offsets.numel() < 2:
        raise ValueError(f"{call}: seq_offsets must hold one sequence at least")
    return seq_offsets.numel() - 1
