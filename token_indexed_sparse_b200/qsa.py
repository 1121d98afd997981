"""Thin Python binding of libqsa_b200.so (argument marshalling only).

The paged-cache calls, which a decode step makes every few microseconds, go
through the compiled ``_qsa_torch`` where their arguments need nothing done to
them, and through this file otherwise.

Every step of the computation runs in the CUDA library; this module passes
device pointers of PyTorch tensors and the current CUDA stream through the C ABI
declared in ``include/qsa.h``.  There is no fallback: if the library is missing
or the tensors are not on a CUDA device, the call raises.
"""

from __future__ import annotations

import ctypes
import functools
import importlib.util
import math
import operator
import os
import warnings

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqsa_b200.so")
_lib = None
_short = None  # the compiled binding, bound to the library

QSA_OK = 0


class QSAError(RuntimeError):
    """A QSA C-ABI call returned a non-OK status."""

    def __init__(self, status: int, what: str):
        super().__init__(f"{what} failed: {status_string(status)} ({status})")
        self.status = status


def library() -> ctypes.CDLL:
    """Load the shared library (once); raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            f"QSA CUDA library not found at {_LIB_PATH}; build it with "
            "`python -m token_indexed_sparse_b200.build` (there is no CPU fallback)")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.qsa_status_string.restype = ctypes.c_char_p
    lib.qsa_status_string.argtypes = [i32]
    lib.qsa_version.restype = ctypes.c_char_p
    lib.qsa_version.argtypes = []
    for name in ("qsa_forward_workspace_size", "qsa_backward_workspace_size"):
        f = getattr(lib, name)
        f.restype = sz
        f.argtypes = [i64, i64, i32, i32, i32]
    lib.qsa_forward.restype = i32
    lib.qsa_forward.argtypes = [vp, vp, vp, vp, i64, i64, i32, i32, i32, f32, vp, vp, vp, sz, vp]
    lib.qsa_backward.restype = i32
    lib.qsa_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, i32, f32,
                                 vp, vp, vp, vp, sz, vp]
    lib.qsa_forward_ex.restype = i32
    lib.qsa_forward_ex.argtypes = lib.qsa_forward.argtypes + [vp, i32]
    lib.qsa_backward_ex.restype = i32
    lib.qsa_backward_ex.argtypes = lib.qsa_backward.argtypes + [vp, i32]
    lib.qsa_forward_kvwait.restype = i32
    lib.qsa_forward_kvwait.argtypes = lib.qsa_forward.argtypes + [vp, vp, i32]
    lib.qsa_backward_saved.restype = i32
    lib.qsa_backward_saved.argtypes = [vp, vp, vp, vp, vp, vp, vp, sz, i64, i64, i32, i32, i32, f32, vp, vp, vp, i32,
                                       vp, sz, vp, vp, vp, i32]
    lib.qsa_backward_kvwait.restype = i32
    lib.qsa_backward_kvwait.argtypes = lib.qsa_backward.argtypes[:16] + [i32] + lib.qsa_backward.argtypes[16:] + [
        vp, vp, i32]
    lib.qsa_launch_count.restype = i32
    lib.qsa_launch_count.argtypes = [i64, i64, i32, i32, i32, i32]
    lib.qsa_bitmap_routes.restype = i32
    lib.qsa_bitmap_routes.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, vp, vp, vp, vp]
    lib.qsa_selector_scores.restype = i32
    lib.qsa_selector_scores.argtypes = [vp, vp, i64, i64, i32, i32, f32, vp, vp, vp, vp, i64, vp, vp]
    lib.qsa_selector_topk.restype = i32
    lib.qsa_selector_topk.argtypes = [vp, i64, i64, i64, i32, vp, vp, vp, vp, vp, vp]
    lib.qsa_backward_fp32kv.restype = i32
    lib.qsa_backward_fp32kv.argtypes = lib.qsa_backward.argtypes
    lib.qsa_route_plan_scratch_size.restype = sz
    lib.qsa_route_plan_scratch_size.argtypes = [i64, i64]
    lib.qsa_route_plan.restype = i32
    lib.qsa_route_plan.argtypes = [vp, i64, i64, i32, vp, vp, vp, vp, vp, sz, vp]
    lib.qsa_tile_plan_scratch_size.restype = sz
    lib.qsa_tile_plan_scratch_size.argtypes = [i64, i64]
    lib.qsa_tile_plan.restype = i32
    lib.qsa_tile_plan.argtypes = [vp, i64, i64, i32, vp, vp, vp, vp, vp, sz, vp]
    lib.qsa_union_group.restype = i32
    lib.qsa_union_group.argtypes = [i32]
    lib.qsa_union_plan.restype = i32
    lib.qsa_union_plan.argtypes = [vp, i64, i64, i32, vp, vp, vp, vp, vp, vp]
    lib.qsa_cast_f32_to_bf16.restype = i32
    lib.qsa_cast_f32_to_bf16.argtypes = [vp, vp, i64, vp]
    rows = [vp, i64, i64]  # a [T, heads, 256] operand: pointer, token and head strides
    # block_table, kv_len, cu_q, T, B, n_pages, page_size, max_pages, H, G
    cache = [vp, vp, vp, i64, i32, i64, i32, i64, i32, i32]
    lib.qsa_rope.restype = i32
    lib.qsa_rope.argtypes = rows * 4 + [vp, vp, i64, i32, i32, i32, i32, f32, i32, vp]
    lib.qsa_cache_append.restype = i32
    lib.qsa_cache_append.argtypes = rows * 4 + [vp, i32, i32, f32, vp, vp] + cache + [vp]
    lib.qsa_paged_forward_workspace_size.restype = sz
    lib.qsa_paged_forward_workspace_size.argtypes = [i64, i32, i32, i32, i32, i64]
    lib.qsa_paged_forward.restype = i32
    lib.qsa_paged_forward.argtypes = [vp] * 4 + cache + [i32, f32, vp, vp, vp, sz, vp]
    lib.qsa_paged_causal_workspace_size.restype = sz
    lib.qsa_paged_causal_workspace_size.argtypes = [i64, i32, i32, i32, i64, i32, i32]
    lib.qsa_paged_causal.restype = i32
    lib.qsa_paged_causal.argtypes = [vp] * 3 + cache + [i32, i32, f32, vp, vp, vp, sz, vp]
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return library().qsa_status_string(int(status)).decode()


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(status: int, what: str):
    if status != QSA_OK:
        raise QSAError(status, what)


def _prep(x: torch.Tensor, dtype, name: str) -> torch.Tensor:
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    return x.contiguous()


def _out(t: torch.Tensor, shape, dtype, device, name: str) -> torch.Tensor:
    """A caller-provided output buffer.  The kernels write it in place through its
    pointer, so it must be exactly the dense tensor they expect: anything else
    is refused before the call (a strided or short buffer would be overrun)."""
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _sizes(q, k, routes):
    if q.dim() != 3 or k.dim() != 3 or routes.dim() != 2:
        raise ValueError("expected q [T,H,256], k/v [T_kv,G,256], routes [T,n_sel]")
    T, H, D = q.shape
    T_kv, G, Dk = k.shape
    if D != 256 or Dk != 256:
        raise ValueError("head dimension must be 256")
    if routes.shape[0] != T:
        raise ValueError("routes must have one row per query")
    return T, T_kv, H, G, routes.shape[1]


def forward_workspace_size(T, T_kv, H, G, n_sel) -> int:
    return int(library().qsa_forward_workspace_size(T, T_kv, H, G, n_sel))


def backward_workspace_size(T, T_kv, H, G, n_sel) -> int:
    return int(library().qsa_backward_workspace_size(T, T_kv, H, G, n_sel))


def launch_count(T, T_kv, H, G, n_sel, backward: bool) -> int:
    """Kernels one forward / backward call enqueues (0 for rejected sizes)."""
    return int(library().qsa_launch_count(T, T_kv, H, G, n_sel, 1 if backward else 0))


def _workspace(nbytes: int, device, given: torch.Tensor | None) -> torch.Tensor:
    if given is not None:  # a dense uint8 buffer: its element count is its size in bytes
        if given.device != device or given.dtype != torch.uint8 or not given.is_contiguous():
            raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
        return given
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _events(stage_events):
    """ctypes array of raw cudaEvent_t handles from torch.cuda.Event objects."""
    if not stage_events:
        return None, 0
    handles = []
    for e in stage_events:
        if e.cuda_event == 0:          # torch creates events lazily
            e.record()
        handles.append(e.cuda_event)
    return (ctypes.c_void_p * len(handles))(*handles), len(handles)


def _event_handle(e):
    """Raw cudaEvent_t of a recorded torch.cuda.Event, or None."""
    if e is None:
        return None
    if e.cuda_event == 0:
        raise ValueError("kv_ready must be a recorded torch.cuda.Event")
    return e.cuda_event


def forward(q, k, v, routes, scale: float = 1.0 / 16.0, *, out=None, lse=None, workspace=None,
            stage_events=None, kv_ready=None):
    """qsa_forward: returns ``(out [T,H,256] bf16, lse [T,H] float32)``.

    ``stage_events`` (optional list of torch.cuda.Event) are recorded after the
    route-sort and attention stages.  ``kv_ready`` (optional recorded
    torch.cuda.Event): k and v may still be being written until it fires; the
    route work runs first and the attention waits for it (qsa_forward_kvwait)."""
    lib = library()
    q = _prep(q, torch.bfloat16, "q")
    k = _prep(k, torch.bfloat16, "k")
    v = _prep(v, torch.bfloat16, "v")
    routes = _prep(routes, torch.int32, "routes")
    T, T_kv, H, G, n_sel = _sizes(q, k, routes)
    out = torch.empty_like(q) if out is None else _out(out, q.shape, torch.bfloat16, q.device, "out")
    lse = (torch.empty(T, H, dtype=torch.float32, device=q.device) if lse is None
           else _out(lse, (T, H), torch.float32, q.device, "lse"))
    ws_bytes = lib.qsa_forward_workspace_size(T, T_kv, H, G, n_sel)
    ws = _workspace(ws_bytes, q.device, workspace)
    ev, n_ev = _events(stage_events)
    st = lib.qsa_forward_kvwait(_ptr(q), _ptr(k), _ptr(v), _ptr(routes), T, T_kv, H, G, n_sel, float(scale),
                                _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(q.device),
                                _event_handle(kv_ready), ev, n_ev)
    _check(st, "qsa_forward")
    return out, lse


def backward(grad_out, q, k, v, out, lse, routes, scale: float = 1.0 / 16.0, *,
             dq=None, dk=None, dv=None, workspace=None, stage_events=None, kv_fp32: bool = False,
             kv_ready=None, saved_workspace=None):
    """qsa_backward: returns ``(dq, dk, dv)`` (bf16, shapes of q, k, v).

    ``stage_events`` (optional, up to 5 torch.cuda.Event) are recorded after
    each backward stage.  With ``kv_fp32`` dk and dv are FP32 (the sums before
    the BF16 rounding, for adding partials from several calls).  ``kv_ready``
    (optional recorded torch.cuda.Event): k and v may still be being written
    until it fires; the route work runs first and dQ waits for it
    (qsa_backward_kvwait).  ``saved_workspace``: the workspace tensor of the
    forward call on the same routes (still holding its route lists, which
    are then reused instead of sorting the routes again: qsa_backward_saved);
    ``routes`` then only gives n_sel."""
    lib = library()
    grad_out = _prep(grad_out, torch.bfloat16, "grad_out")
    q = _prep(q, torch.bfloat16, "q")
    k = _prep(k, torch.bfloat16, "k")
    v = _prep(v, torch.bfloat16, "v")
    out = _prep(out, torch.bfloat16, "out")
    lse = _prep(lse, torch.float32, "lse")
    routes = _prep(routes, torch.int32, "routes")
    T, T_kv, H, G, n_sel = _sizes(q, k, routes)
    kv_dtype = torch.float32 if kv_fp32 else torch.bfloat16
    dq = torch.empty_like(q) if dq is None else _out(dq, q.shape, torch.bfloat16, q.device, "dq")
    dk = (torch.empty(k.shape, dtype=kv_dtype, device=k.device) if dk is None
          else _out(dk, k.shape, kv_dtype, k.device, "dk"))
    dv = (torch.empty(v.shape, dtype=kv_dtype, device=v.device) if dv is None
          else _out(dv, v.shape, kv_dtype, v.device, "dv"))
    ws_bytes = lib.qsa_backward_workspace_size(T, T_kv, H, G, n_sel)
    ws = _workspace(ws_bytes, q.device, workspace)
    ev, n_ev = _events(stage_events)
    if saved_workspace is not None:
        fws = _workspace(0, q.device, saved_workspace)
        st = lib.qsa_backward_saved(_ptr(grad_out), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(fws),
                                    fws.numel(), T, T_kv, H, G, n_sel, float(scale), _ptr(dq), _ptr(dk), _ptr(dv),
                                    1 if kv_fp32 else 0, _ptr(ws), ws.numel(), _stream(q.device),
                                    _event_handle(kv_ready), ev, n_ev)
        _check(st, "qsa_backward_saved")
        return dq, dk, dv
    st = lib.qsa_backward_kvwait(_ptr(grad_out), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(routes),
                                 T, T_kv, H, G, n_sel, float(scale), _ptr(dq), _ptr(dk), _ptr(dv),
                                 1 if kv_fp32 else 0, _ptr(ws), ws.numel(), _stream(q.device),
                                 _event_handle(kv_ready), ev, n_ev)
    _check(st, "qsa_backward")
    return dq, dk, dv


def union_plan(routes, T_kv: int):
    """qsa_union_plan: ``(group, ucnt, ukey, uown)`` of the forward's query
    groups (route rows first, as qsa_route_plan); ``ukey`` / ``uown`` are
    ``[n_groups, group * n_sel]``, row i valid up to ``ucnt[i]``."""
    lib = library()
    routes = _prep(routes, torch.int32, "routes")
    T, n_sel = routes.shape
    group = lib.qsa_union_group(n_sel)
    if group < 1:
        raise ValueError("n_sel outside 1..16384")
    n_groups = (T + group - 1) // group
    dev = routes.device
    row_cnt = torch.empty(T, dtype=torch.int32, device=dev)
    row_cols = torch.empty(T, n_sel, dtype=torch.int32, device=dev)
    ucnt = torch.empty(n_groups, dtype=torch.int32, device=dev)
    ukey = torch.empty(n_groups, group * n_sel, dtype=torch.int32, device=dev)
    uown = torch.empty(n_groups, group * n_sel, dtype=torch.uint8, device=dev)
    _check(lib.qsa_union_plan(_ptr(routes), T, T_kv, n_sel, _ptr(row_cnt), _ptr(row_cols), _ptr(ucnt), _ptr(ukey),
                              _ptr(uown), _stream(dev)), "qsa_union_plan")
    return group, ucnt, ukey, uown


def cast_f32_to_bf16(x, out=None):
    """qsa_cast_f32_to_bf16: ``x`` (FP32, CUDA) rounded to BF16, to nearest even.

    The final rounding of FP32 dK/dV sums added up across calls (context
    parallelism), the same rounding the backward applies itself."""
    lib = library()
    x = _prep(x, torch.float32, "x")
    out = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device) if out is None else \
        _out(out, x.shape, torch.bfloat16, x.device, "out")
    if x.data_ptr() % 16 or out.data_ptr() % 16:
        raise ValueError("x and out must be 16-byte aligned")
    _check(lib.qsa_cast_f32_to_bf16(_ptr(x), _ptr(out), x.numel(), _stream(x.device)), "qsa_cast_f32_to_bf16")
    return out


def route_plan(routes, T_kv: int):
    """qsa_route_plan: ``(row_cnt, row_cols, quad_ptr, quad_ent)`` device tensors."""
    lib = library()
    routes = _prep(routes, torch.int32, "routes")
    T, n_sel = routes.shape
    dev = routes.device
    nq = (T_kv + 3) // 4
    row_cnt = torch.empty(T, dtype=torch.int32, device=dev)
    row_cols = torch.empty(T, n_sel, dtype=torch.int32, device=dev)
    quad_ptr = torch.empty(nq + 1, dtype=torch.int32, device=dev)
    quad_ent = torch.empty(T * n_sel, dtype=torch.int64, device=dev)
    scratch = torch.empty(max(256, lib.qsa_route_plan_scratch_size(T, T_kv)), dtype=torch.uint8, device=dev)
    st = lib.qsa_route_plan(_ptr(routes), T, T_kv, n_sel, _ptr(row_cnt), _ptr(row_cols), _ptr(quad_ptr),
                            _ptr(quad_ent), _ptr(scratch), scratch.numel(), _stream(dev))
    _check(st, "qsa_route_plan")
    return row_cnt, row_cols, quad_ptr, quad_ent


def tile_plan(routes, T_kv: int):
    """qsa_tile_plan: ``(row_cnt, row_cols, tile_ptr, tile_ent)`` device tensors."""
    lib = library()
    routes = _prep(routes, torch.int32, "routes")
    T, n_sel = routes.shape
    dev = routes.device
    nt = (T_kv + 127) // 128
    row_cnt = torch.empty(T, dtype=torch.int32, device=dev)
    row_cols = torch.empty(T, n_sel, dtype=torch.int32, device=dev)
    tile_ptr = torch.empty(nt + 1, dtype=torch.int32, device=dev)
    tile_ent = torch.empty(T * n_sel, dtype=torch.int64, device=dev)
    scratch = torch.empty(max(256, lib.qsa_tile_plan_scratch_size(T, T_kv)), dtype=torch.uint8, device=dev)
    st = lib.qsa_tile_plan(_ptr(routes), T, T_kv, n_sel, _ptr(row_cnt), _ptr(row_cols), _ptr(tile_ptr),
                           _ptr(tile_ent), _ptr(scratch), scratch.numel(), _stream(dev))
    _check(st, "qsa_tile_plan")
    return row_cnt, row_cols, tile_ptr, tile_ent


def bitmap_routes(sel_blocks, lo, hi, blk_base, tok_base, T_kv: int, n_sel: int, block_size: int = 4):
    """Bitmap selection -> route IDs on the GPU (``qsa_bitmap_routes``).

    Returns ``(routes [T, n_sel] int32, row_cnt [T] int32, max_cnt [1] int32)``,
    all on the device and produced asynchronously on the current stream.
    """
    lib = library()
    sel = _prep(sel_blocks, torch.uint8, "sel_blocks")
    dev = sel.device
    T, NB = sel.shape
    lo, hi, blk_base, tok_base = (_prep(x, torch.int32, n) for x, n in
                                  ((lo, "lo"), (hi, "hi"), (blk_base, "blk_base"), (tok_base, "tok_base")))
    routes = torch.empty((T, n_sel), dtype=torch.int32, device=dev)
    row_cnt = torch.empty((T,), dtype=torch.int32, device=dev)
    max_cnt = torch.empty((1,), dtype=torch.int32, device=dev)
    st = lib.qsa_bitmap_routes(_ptr(sel), _ptr(lo), _ptr(hi), _ptr(blk_base), _ptr(tok_base), T, NB, T_kv,
                               block_size, n_sel, _ptr(routes), _ptr(row_cnt), _ptr(max_cnt), _stream(dev))
    _check(st, "qsa_bitmap_routes")
    return routes, row_cnt, max_cnt


def _opt_i32(x, name):
    return None if x is None else _prep(x, torch.int32, name)


def selector_scores(qi, kbar, scale: float, pos=None, blk_base=None, tok_base=None, scores=None, status=None):
    """Candidate block scores on the tensor cores (``qsa_selector_scores``).

    ``qi`` [T, Hi, 128] and ``kbar`` [NB, 128] BF16 on the GPU.  Returns
    ``scores`` [T, NB] FP32 (entries that are not candidates are left as they
    were: NaN in a fresh tensor) and a one-element device status tensor.
    """
    lib = library()
    qi = _prep(qi, torch.bfloat16, "qi")
    kbar = _prep(kbar, torch.bfloat16, "kbar")
    T, Hi, Di = qi.shape
    NB = kbar.shape[0]
    dev = qi.device
    pos, blk_base, tok_base = (_opt_i32(x, n) for x, n in ((pos, "pos"), (blk_base, "blk_base"),
                                                           (tok_base, "tok_base")))
    if scores is None:
        scores = torch.full((T, NB), float("nan"), dtype=torch.float32, device=dev)
    elif (scores.device != dev or scores.dtype != torch.float32 or scores.dim() != 2 or scores.shape[0] != T
          or scores.shape[1] < NB or scores.stride(1) != 1):
        raise ValueError(f"scores must be a float32 [{T}, >= {NB}] tensor on {dev} with unit column stride")
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=dev)
    elif status.device != dev or status.dtype != torch.int32 or status.numel() < 1 or not status.is_contiguous():
        raise ValueError(f"status must be a contiguous int32 tensor on {dev}")
    st = lib.qsa_selector_scores(_ptr(qi), _ptr(kbar), T, NB, Hi, Di, scale, _ptr(pos), _ptr(blk_base),
                                 _ptr(tok_base), _ptr(scores), scores.stride(0), _ptr(status), _stream(dev))
    _check(st, "qsa_selector_scores")
    return scores, status


def selector_topk(scores, k: int, NB: int, pos=None, blk_base=None, tok_base=None):
    """Top-k local blocks and expanded token routes (``qsa_selector_topk``)."""
    lib = library()
    scores = _prep(scores, torch.float32, "scores")
    T = scores.shape[0]
    dev = scores.device
    pos, blk_base, tok_base = (_opt_i32(x, n) for x, n in ((pos, "pos"), (blk_base, "blk_base"),
                                                           (tok_base, "tok_base")))
    blocks = torch.empty((T, k), dtype=torch.int32, device=dev)
    routes = torch.empty((T, 4 * (k + 1)), dtype=torch.int32, device=dev)
    st = lib.qsa_selector_topk(_ptr(scores), scores.stride(0), T, NB, k, _ptr(pos), _ptr(blk_base), _ptr(tok_base),
                               _ptr(blocks), _ptr(routes), _stream(dev))
    _check(st, "qsa_selector_topk")
    return blocks, routes


def select(qi, kbar, scale: float, k: int, pos=None, blk_base=None, tok_base=None):
    """The whole selector: (scores, blocks, routes, status)."""
    scores, status = selector_scores(qi, kbar, scale, pos, blk_base, tok_base)
    blocks, routes = selector_topk(scores, k, kbar.shape[0], pos, blk_base, tok_base)
    return scores, blocks, routes, status


# ---------------------------------------------------------------------------
# serving from a paged K/V cache
# ---------------------------------------------------------------------------

def rope_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                     original_len: int = 4096, fast_turns: float = 32.0, slow_turns: float = 1.0, device="cuda"):
    """``(inv_freq [rotary_dim / 2] float64 on device, mscale)`` for ``rope`` and ``cache_append``.

    Pair i turns by ``base ** (-2 i / rotary_dim)`` per position.  ``scaling``
    for contexts ``factor`` times ``original_len``: ``"linear"`` divides every
    frequency by the factor; ``"yarn"`` (Peng et al., 2023) divides those of slow
    pairs, keeps those of fast ones, and grows q and k by ``0.1 ln(factor) + 1``.

    Between the two, the divided share grows linearly with the pair's index, as in
    the models published with this scaling; the paper's own ramp is linear in the
    turns that a pair makes over the original length, which gives other values.  It
    starts at the last whole index (0 at least) whose pair makes ``fast_turns`` turns
    or more and ends at the first whose pair makes ``slow_turns`` or fewer."""
    if rotary_dim < 16 or rotary_dim > 256 or rotary_dim % 16:
        raise ValueError("rotary_dim must be a multiple of 16, at most 256")
    if not base > 1.0 or not factor >= 1.0:
        raise ValueError("base must be above 1 and factor at least 1")
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    inv_freq, mscale = base ** (-2.0 * i / rotary_dim), 1.0
    if scaling == "linear":
        inv_freq = inv_freq / factor
    elif scaling == "yarn":
        if not fast_turns > slow_turns > 0.0 or original_len < 1:
            raise ValueError("yarn needs fast_turns > slow_turns > 0 and original_len >= 1")

        def index(turns):  # where base ** (-2 index / rotary_dim) * original_len is 2 pi turns
            return rotary_dim * math.log(original_len / (2.0 * math.pi * turns)) / (2.0 * math.log(base))

        kept, divided = max(math.floor(index(fast_turns)), 0), math.ceil(index(slow_turns))
        if divided > kept:
            share = ((i - kept) / (divided - kept)).clamp(0.0, 1.0)
        else:  # even pair 0 makes no more than slow_turns
            share = torch.ones_like(i)
        inv_freq = inv_freq * (1.0 - share) + inv_freq / factor * share
        mscale = 0.1 * math.log(factor) + 1.0
    elif scaling is not None:
        raise ValueError('scaling must be None, "linear" or "yarn"')
    return inv_freq.to(device), mscale


class _NoShortWay:
    """In place of the compiled binding where there is none for this PyTorch: takes nothing."""

    @staticmethod
    def rope(*args):
        return NotImplemented

    cache_append = paged_forward = paged_causal = rope


def _load_binding():
    from . import build

    path = build.binding_path()
    try:
        spec = importlib.util.spec_from_file_location("_qsa_torch", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        return module
    except ImportError as e:
        warnings.warn(f"{os.path.basename(path)} does not load ({e}): the paged-cache calls go through Python, some "
                      "10 us longer; build it with `python -m token_indexed_sparse_b200.build`", RuntimeWarning,
                      stacklevel=4)
        return None


def _short_way():
    """The compiled binding with the library's entry points (loads both once), or what takes nothing."""
    global _short
    if _short is None:
        lib = library()
        short = _load_binding()
        if short is None:
            short = _NoShortWay()
        else:
            short.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
                lib.qsa_rope, lib.qsa_cache_append, lib.qsa_paged_forward, lib.qsa_paged_forward_workspace_size,
                lib.qsa_paged_causal, lib.qsa_paged_causal_workspace_size)))
        _short = short
    return _short


# The long way: the same calls for arguments that have to be converted first, or refused.

def _enqueue(index: int, what: str, named, call, *args):
    """Runs a library call on CUDA device ``index`` (all tensors of ``named``,
    pairs of name and tensor or None, have to be on it), its current stream last
    in the arguments."""
    for name, t in named:
        if t is not None and t.get_device() != index or index < 0:
            raise ValueError(f"{what}: {name} must be on {f'cuda:{index}' if index >= 0 else 'a CUDA device'}, "
                             f"got {'nothing' if t is None else t.device}")
    if index == torch._C._cuda_getDevice():
        st = call(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            st = call(*args, torch._C._cuda_getCurrentRawStream(index))
    if st != QSA_OK:
        raise QSAError(st, what)


def _int32(x, name: str) -> int:
    """An int argument of the library (ctypes would keep the low 32 bits of a larger one)."""
    x = operator.index(x)
    if not -2**31 <= x < 2**31:
        raise ValueError(f"{name} must fit 32 bits, got {x}")
    return x


def _bad_rows(x: torch.Tensor, T: int | None, name: str):
    if x.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {x.dtype}")
    if x.dim() != 3 or x.shape[2] != 256 or (T is not None and x.shape[0] != T):
        raise ValueError(f"{name} must be [{'T' if T is None else T}, heads, 256], got {tuple(x.shape)}")
    raise ValueError(f"{name} must have contiguous dims")


def _rows(x: torch.Tensor, T: int | None, name: str):
    """Pointer and strides of a ``[T, heads, 256]`` BF16 operand (dims contiguous, the rest as it is)."""
    shape, stride = x.shape, x.stride()
    if (x.dtype != torch.bfloat16 or len(shape) != 3 or shape[2] != 256 or stride[2] != 1
            or (T is not None and shape[0] != T)):
        _bad_rows(x, T, name)
    _int32(shape[1], f"heads of {name}")
    # the stride of an axis of length one is free
    return x.data_ptr(), stride[0] if shape[0] > 1 else 0, stride[1] if shape[1] > 1 else 0


def _rows_out(x: torch.Tensor, out: torch.Tensor | None, name: str) -> torch.Tensor:
    if out is None:
        return torch.empty_like(x)
    if out.shape != x.shape:
        raise ValueError(f"{name} must have shape {tuple(x.shape)}, got {tuple(out.shape)}")
    return out


def _vector(x: torch.Tensor, n: int | None, dtype, name: str):
    """A contiguous vector (of ``n`` elements): its pointer."""
    if x.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if x.dim() != 1 or not x.is_contiguous() or (n is not None and x.shape[0] != n):
        raise ValueError(f"{name} must be a contiguous vector{'' if n is None else f' of {n}'}, got {tuple(x.shape)}")
    return x.data_ptr()


_NO_ROWS = (None, 0, 0)


def _rope(q, k, positions, inv_freq, interleaved, mscale, out_q, out_k, backward):
    q_rows = _rows(q, None, "q")
    T, H, _ = q.shape
    out_q = _rows_out(q, out_q, "out_q")
    k_rows = out_k_rows = _NO_ROWS
    G = 0
    if k is not None:
        k_rows = _rows(k, T, "k")
        G = k.shape[1]
        out_k = _rows_out(k, out_k, "out_k")
        out_k_rows = _rows(out_k, T, "out_k")
    elif out_k is not None:
        raise ValueError("out_k without k")
    _enqueue(q.get_device(), "qsa_rope",
             (("q", q), ("k", k), ("out_q", out_q), ("out_k", out_k), ("positions", positions),
              ("inv_freq", inv_freq)),
             library().qsa_rope, *q_rows, *k_rows, *_rows(out_q, T, "out_q"), *out_k_rows,
             _vector(positions, T, torch.int32, "positions"), _vector(inv_freq, None, torch.float64, "inv_freq"), T, H,
             G, 2 * inv_freq.shape[0], interleaved, mscale, backward)
    return out_q, out_k


def rope(q, k, positions, inv_freq, *, interleaved: bool = False, mscale: float = 1.0, out_q=None, out_k=None):
    """qsa_rope: ``(q', k')``, q ``[T, H, 256]`` and k ``[T, G, 256]`` (or None) turned to their positions.

    ``positions`` [T] int32, ``inv_freq`` [rotary_dim / 2] float64 and
    ``mscale`` as from ``rope_frequencies``; dims from rotary_dim up pass.  q and k
    may be slices of one projection (any strides between tokens and heads that
    are multiples of 8); ``out_q`` / ``out_k`` may be the inputs (in place)."""
    r = (_short or _short_way()).rope(q, k, positions, inv_freq, interleaved, mscale, out_q, out_k, False)
    if r is NotImplemented:
        return _rope(q, k, positions, inv_freq, interleaved, mscale, out_q, out_k, 0)
    return r if type(r) is tuple else _check(r, "qsa_rope")


def rope_backward(grad_q, grad_k, positions, inv_freq, *, interleaved: bool = False, mscale: float = 1.0,
                  out_q=None, out_k=None):
    """The gradient of ``rope``: ``(dq, dk)`` from the gradients of its outputs (the opposite turn)."""
    r = (_short or _short_way()).rope(grad_q, grad_k, positions, inv_freq, interleaved, mscale, out_q, out_k, True)
    if r is NotImplemented:
        return _rope(grad_q, grad_k, positions, inv_freq, interleaved, mscale, out_q, out_k, 1)
    return r if type(r) is tuple else _check(r, "qsa_rope")


def _bad_cache(k_pages, v_pages, block_table, kv_len, cu_q):
    for x, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        if x.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be {torch.bfloat16}, got {x.dtype}")
        if x.dim() != 4 or x.shape[3] != 256 or not x.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [n_pages, page_size, G, 256] tensor")
    if k_pages.shape != v_pages.shape:
        raise ValueError("k_pages and v_pages must have one shape")
    for x, name in ((block_table, "block_table"), (kv_len, "kv_len"), (cu_q, "cu_q")):
        if x.dtype != torch.int32:
            raise TypeError(f"{name} must be {torch.int32}, got {x.dtype}")
    raise ValueError(f"block_table must be a contiguous [B, max_pages], got {tuple(block_table.shape)}")


def _cache(k_pages, v_pages, block_table, kv_len, cu_q, T: int, H: int):
    """Checks a cache; returns the arguments (table, kv_len, cu_q, T, B, n_pages, page_size, max_pages, H, G)."""
    shape, table = k_pages.shape, block_table.shape
    if (k_pages.dtype != torch.bfloat16 or v_pages.dtype != torch.bfloat16 or len(shape) != 4 or shape[3] != 256
            or v_pages.shape != shape or not k_pages.is_contiguous() or not v_pages.is_contiguous()
            or block_table.dtype != torch.int32 or len(table) != 2 or not block_table.is_contiguous()):
        _bad_cache(k_pages, v_pages, block_table, kv_len, cu_q)
    B = _int32(table[0], "rows of block_table")
    _int32(shape[1], "the page size")
    _int32(shape[2], "KV heads")
    _int32(H, "query heads")
    return (block_table.data_ptr(), _vector(kv_len, B, torch.int32, "kv_len"),
            _vector(cu_q, B + 1, torch.int32, "cu_q (one longer than kv_len)"),
            T, B, shape[0], shape[1], table[1], H, shape[2])


def cache_append(k_new, v_new, k_pages, v_pages, block_table, kv_len, cu_q, *, q=None, inv_freq=None,
                 interleaved: bool = False, mscale: float = 1.0, out_q=None):
    """qsa_cache_append: writes the new tokens' K and V rows ``[T, G, 256]`` into the pages (in place).

    With ``inv_freq`` (see ``rope_frequencies``) k is turned to its position in
    the cache first, and ``q`` [T, H, 256] with it: returns the turned q (into
    ``out_q``, which may be q itself), else None."""
    r = (_short or _short_way()).cache_append(k_new, v_new, k_pages, v_pages, block_table, kv_len, cu_q, q, inv_freq,
                                              interleaved, mscale, out_q)
    if r is not NotImplemented:
        return r if type(r) is not int else _check(r, "qsa_cache_append")
    k_rows = _rows(k_new, None, "k_new")
    T, G, _ = k_new.shape
    v_rows = _rows(v_new, T, "v_new")
    if v_new.shape[1] != G:
        raise ValueError("k_new and v_new must have one shape")
    H = 12 * G
    q_rows = out_rows = _NO_ROWS
    if q is not None:
        if inv_freq is None:
            raise ValueError("q is only taken to be rotated: it needs inv_freq")
        q_rows = _rows(q, T, "q")
        H = q.shape[1]
        out_q = _rows_out(q, out_q, "out_q")
        out_rows = _rows(out_q, T, "out_q")
    elif out_q is not None:
        raise ValueError("out_q without q")
    cache = _cache(k_pages, v_pages, block_table, kv_len, cu_q, T, H)
    if cache[9] != G:
        raise ValueError(f"the pages hold {cache[9]} KV heads, k_new {G}")
    freq, rot = None, 0
    if inv_freq is not None:
        freq, rot = _vector(inv_freq, None, torch.float64, "inv_freq"), 2 * inv_freq.shape[0]
    _enqueue(k_new.get_device(), "qsa_cache_append",
             (("k_new", k_new), ("v_new", v_new), ("k_pages", k_pages), ("v_pages", v_pages),
              ("block_table", block_table), ("kv_len", kv_len), ("cu_q", cu_q), ("q", q), ("inv_freq", inv_freq),
              ("out_q", out_q)),
             library().qsa_cache_append, *k_rows, *v_rows, *q_rows, *out_rows, freq, rot, interleaved, mscale,
             k_pages.data_ptr(), v_pages.data_ptr(), *cache)
    return out_q


def _paged_io(q, out, lse):
    q = _prep(q, torch.bfloat16, "q")
    shape = q.shape
    if len(shape) != 3 or shape[2] != 256:
        raise ValueError(f"q must be [T, H, 256], got {tuple(shape)}")
    out = torch.empty_like(q) if out is None else _out(out, shape, torch.bfloat16, q.device, "out")
    lse = (torch.empty(shape[0], shape[1], dtype=torch.float32, device=q.device) if lse is None
           else _out(lse, shape[:2], torch.float32, q.device, "lse"))
    return q, out, lse, shape[0], shape[1]


@functools.lru_cache(maxsize=1024)
def paged_forward_workspace_size(T, H, G, n_sel, page_size, max_pages) -> int:
    for x, name in ((H, "H"), (G, "G"), (n_sel, "n_sel"), (page_size, "page_size")):
        _int32(x, name)
    return int(library().qsa_paged_forward_workspace_size(T, H, G, n_sel, page_size, max_pages))


@functools.lru_cache(maxsize=1024)
def paged_causal_workspace_size(T, H, G, page_size, max_pages, window: int = 0, sinks: int = 0) -> int:
    for x, name in ((H, "H"), (G, "G"), (page_size, "page_size"), (window, "window"), (sinks, "sinks")):
        _int32(x, name)
    return int(library().qsa_paged_causal_workspace_size(T, H, G, page_size, max_pages, window, sinks))


def status_word(workspace: torch.Tensor) -> torch.Tensor:
    """The status word of a call that was given ``workspace``: a one-element int32 view of it on the device.

    Once the call's work has completed it is 0, or nonzero if a kernel gave up on a bounded wait
    (the call's outputs are then invalid).  Nothing is read or waited for here: a program looks when
    it synchronises anyway, before the workspace goes into another call."""
    if workspace.dtype != torch.uint8 or workspace.dim() != 1 or not workspace.is_contiguous() or workspace.numel() < 4:
        raise ValueError("workspace must be a contiguous uint8 vector")
    return workspace[:4].view(torch.int32)


def paged_forward(q, k_pages, v_pages, routes, block_table, kv_len, cu_q, scale: float = 1.0 / 16.0, *, out=None,
                  lse=None, workspace=None):
    """qsa_paged_forward: ``(out [T, H, 256] bf16, lse [T, H] float32)`` of new tokens over a paged cache.

    ``routes`` [T, n_sel] int32 name positions of the row's own sequence (a set,
    as in ``forward``).  Pools ``[n_pages, page_size, G, 256]``, ``block_table``
    [B, max_pages], ``kv_len`` [B] and ``cu_q`` [B + 1] int32.  Rows of no
    sequence are left as they were in ``out`` and ``lse``."""
    r = (_short or _short_way()).paged_forward(q, k_pages, v_pages, routes, block_table, kv_len, cu_q, scale, out, lse,
                                               workspace)
    if r is not NotImplemented:
        return r if type(r) is tuple else _check(r, "qsa_paged_forward")
    q, out, lse, T, H = _paged_io(q, out, lse)
    routes = _prep(routes, torch.int32, "routes")
    cache = _cache(k_pages, v_pages, block_table, kv_len, cu_q, T, H)
    if routes.dim() != 2 or routes.shape[0] != T:
        raise ValueError("routes must have one row per query")
    n_sel = _int32(routes.shape[1], "the length of a row of routes")
    ws = _workspace(paged_forward_workspace_size(T, H, cache[9], n_sel, cache[6], cache[7]), q.device, workspace)
    _enqueue(q.get_device(), "qsa_paged_forward",
             (("k_pages", k_pages), ("v_pages", v_pages), ("routes", routes), ("block_table", block_table),
              ("kv_len", kv_len), ("cu_q", cu_q)),
             library().qsa_paged_forward, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), routes.data_ptr(),
             *cache, n_sel, scale, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel())
    return out, lse


def paged_causal(q, k_pages, v_pages, block_table, kv_len, cu_q, scale: float = 1.0 / 16.0, *, window: int = 0,
                 sinks: int = 0, out=None, lse=None, workspace=None):
    """qsa_paged_causal: ``(out [T, H, 256] bf16, lse [T, H] float32)`` of new tokens over a paged cache.

    A token at position p sees the positions ``j <= p`` of its sequence, with
    ``window`` above 0 only those with ``j > p - window`` or ``j < sinks``.  The
    cache as in ``paged_forward``.  The kernel's waits are bounded; a caller who wants to
    see that none gave up brings a ``workspace`` (``paged_causal_workspace_size``) and
    looks at its ``status_word``."""
    r = (_short or _short_way()).paged_causal(q, k_pages, v_pages, block_table, kv_len, cu_q, scale, window, sinks, out,
                                              lse, workspace)
    if r is not NotImplemented:
        return r if type(r) is tuple else _check(r, "qsa_paged_causal")
    window, sinks = _int32(window, "window"), _int32(sinks, "sinks")
    q, out, lse, T, H = _paged_io(q, out, lse)
    cache = _cache(k_pages, v_pages, block_table, kv_len, cu_q, T, H)
    ws = _workspace(paged_causal_workspace_size(T, H, cache[9], cache[6], cache[7], window, sinks), q.device,
                    workspace)
    _enqueue(q.get_device(), "qsa_paged_causal",
             (("k_pages", k_pages), ("v_pages", v_pages), ("block_table", block_table), ("kv_len", kv_len),
              ("cu_q", cu_q)),
             library().qsa_paged_causal, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), *cache, window, sinks,
             scale, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel())
    return out, lse
