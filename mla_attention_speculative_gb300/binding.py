"""Thin ctypes binding of libmla.so (argument marshalling only).

Every function here has the C entry point's name and forwards to it.  The
tensors are PyTorch CUDA tensors: PyTorch provides device memory and the
current stream, nothing else.  Every step of the attention runs in the
library's kernels; if the library is missing this module raises instead of
falling back to anything.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from typing import NamedTuple, Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmla.so")

MLA_OK = 0
MLA_ERR_INVALID_ARG = -1
MLA_ERR_UNSUPPORTED = -2
MLA_ERR_WORKSPACE = -3
MLA_ERR_CUDA = -4
MLA_ERR_TIMEOUT = -5

MODES = {"auto": 0, "absorbed": 1, "materialised": 2}
BRANCH_ABSORBED = 1
BRANCH_MATERIALISED = 2
BRANCH_NAMES = {1: "absorbed", 2: "materialised"}
DTYPES = {torch.bfloat16: 0, torch.float32: 1}
# element types of a paged key/value cache
CACHE_DTYPES = {**DTYPES, torch.float8_e4m3fn: 2}


class MlaError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({detail})")


class Geometry(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("kv_lora_rank", ctypes.c_int32),
                ("qk_nope_dim", ctypes.c_int32), ("v_dim", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
                ("dtype", ctypes.c_int32)]


class KVGeometry(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
                ("dtype", ctypes.c_int32), ("cache_dtype", ctypes.c_int32)]


class PageView(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("width", ctypes.c_int32)]


class KVCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


_lib = None

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SIGS = {
    "mla_max_absorbed_queries": (_I64, [_I32, _I32, _I32, _I64]),
    "mla_max_absorbed_queries_batch": (_I64, [_I32, _I32, _I32, _P, _I32]),
    "mla_select_branch": (_I32, [_P, _I32, _P, _I32, _I32, _P]),
    "mla_workspace_bytes": (_I32, [_P, _I32, _I32, _P, _I32, _P]),
    "mla_verify_attention": (_I32, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P,
                                    _I32, _I32, _P, _I32, _I32, _I32, _I32, _P, _P,
                                    ctypes.c_size_t, _P, _P]),
    "mla_verify_attention_noalloc": (_I32, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _P,
                                            _P, _P, _I32, _I32, _P, _I32, _I32, _I32, _P,
                                            _P, _P]),
    "mla_check_page_table": (_I32, [_P, _I32, _I32, _P, _I32, _I32]),
    "mla_sparse_workspace_bytes": (_I32, [_P, _I32, _I32, _P, _I32, _P]),
    "mla_indexer_pool_update": (_I32, [_P, _I32, _I64, _I64, _I32, _I32, _I64, _I32, _I32, _P,
                                       _I64, _P, _P, _P]),
    "mla_indexer_select_workspace_bytes": (_I32, [_I32, _I32, _I64, _P]),
    "mla_indexer_select": (_I32, [_P, _P, _I64, _I32, _I32, _I64, _I32, _I32, _P, _P, _P,
                                  ctypes.c_size_t, _P]),
    "mla_verify_attention_sparse": (_I32, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P,
                                           _I32, _I32, _P, _I32, _P, _I32, _I32, _I32, _P, _P,
                                           ctypes.c_size_t, _P]),
    "mla_select_draft_cap": (_I32, [ctypes.c_double, _P, _I32, _P, _I32, _I32, _P]),
    "mla_concat_snapshots": (_I32, [_P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _P, _I64, _P,
                                    _I32, _P, _P]),
    "mla_rollback_valid_prefix": (_I32, [_P, _I32, _I32, _P, _P, _I32, _I32, _I32, _I32, _I32,
                                         _P, _P]),
    "mla_page_step": (_I32, [_P, _P, _P, _I32, _P, _I32, _I32, _I32, _P, _I32, _P, _P, _P, _P, _P,
                             _P, _I32, _P, _P, _P]),
    "mla_append_latent": (_I32, [_P, _P, _I64, _P, _I64, _P, ctypes.c_float, _P, _I32, _I32, _P,
                                 _P, _I32, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "mla_append_kv": (_I32, [_P, _P, _I64, _P, _I64, _P, _I64, _P, _I32, _I32, _I32, _P, _P, _I32,
                             _P, _P, _P]),
    "mla_decode_workspace_bytes": (_I32, [_P, _I32, _I32, _I32, _P]),
    "mla_decode_attention": (_I32, [_P, _P, _I64, _P, _P, _I32, _P, _I32, _I32, _P, _P, _P,
                                    ctypes.c_size_t, _P]),
    "mla_chunk_workspace_bytes": (_I32, [_P, _I32, _I32, _I32, _I32, _P]),
    "mla_chunk_attention": (_I32, [_P, _P, _I64, _I32, _P, _P, _P, _P, _I32, _P, _I32, _I32, _P,
                                   _P, _P, ctypes.c_size_t, _P]),
    "mla_page_fork": (_I32, [_P, _P, _P, _I32, _P, _I32, _I32, _I32, _P, _P, _I32, _P, _P, _P, _P,
                             _P, _P, _P, _P, _P, _P, _P]),
    "mla_page_release": (_I32, [_P, _P, _I32, _P, _I32, _I32, _I32, _P, _P, _I32, _P, _P, _P, _P,
                                _P, _P]),
    "mla_page_compact_workspace_bytes": (_I32, [_I32, _P]),
    "mla_page_compact": (_I32, [_P, _I32, _P, _I32, _I32, _P, _P, _P, _P, _I32, _P, _P, _P, _P,
                                _P, ctypes.c_size_t, _P]),
    "mla_page_copy": (_I32, [_P, _I32, _I32, _I32, _P, _P, _P, _P, _I32, _P]),
    "mla_kernel_timing_enable": (_I32, [_I32]),
    "mla_kernel_timing_read": (_I32, [ctypes.c_char_p, ctypes.c_size_t, _P, _P, _I32, _P,
                                      _I32]),
    "mla_device_status": (_I32, [_P, _I32]),
    "mla_selftest_bounded_wait": (_I32, [_P]),
    "mla_status_string": (ctypes.c_char_p, [_I32]),
    "mla_last_error": (ctypes.c_char_p, []),
    "mla_version": (_I32, []),
}


def lib() -> ctypes.CDLL:
    """Load libmla.so (built in-tree by build_lib); raise if it is absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run "
                               "`python -m mla_attention_speculative_gb300.build_lib`")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


def status_string(status: int) -> str:
    return lib().mla_status_string(int(status)).decode()


def mla_last_error() -> str:
    return lib().mla_last_error().decode()


def _check(status: int, where: str):
    if status != MLA_OK:
        raise MlaError(status, where, mla_last_error())


def _lens_array(cache_lens: Sequence[int]):
    arr = (ctypes.c_int32 * len(cache_lens))(*[int(t) for t in cache_lens])
    return arr


def make_geometry(H, r, n, v, rope, dtype=torch.bfloat16, scale: Optional[float] = None):
    return Geometry(int(H), int(r), int(n), int(v), int(rope),
                    float(scale) if scale is not None else 0.0, DTYPES[dtype])


_GEOMS = {}


def _geometry(H, r, n, v, rope, dtype, scale):
    """A Geometry per distinct shape, built once (the call only reads it)."""
    key = (H, r, n, v, rope, dtype, scale)
    g = _GEOMS.get(key)
    if g is None:
        g = _GEOMS[key] = make_geometry(H, r, n, v, rope, dtype, scale)
    return g


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current_stream(dev: torch.device) -> int:
    """The raw handle of the current CUDA stream of `dev` (PyTorch's fast accessor
    when present, else the public one)."""
    if _raw_stream is not None:
        return _raw_stream(dev.index if dev.index is not None else torch.cuda.current_device())
    return torch.cuda.current_stream(dev).cuda_stream


def mla_max_absorbed_queries(r: int, n: int, v: int, cache_len: int = 0) -> int:
    return int(lib().mla_max_absorbed_queries(r, n, v, cache_len))


def mla_max_absorbed_queries_batch(r: int, n: int, v: int, cache_lens: Sequence[int]) -> int:
    arr = _lens_array(cache_lens)
    return int(lib().mla_max_absorbed_queries_batch(r, n, v, arr, len(cache_lens)))


def mla_select_branch(geom: Geometry, L: int, cache_lens: Sequence[int], mode="auto") -> int:
    arr = _lens_array(cache_lens)
    out = ctypes.c_int32(0)
    _check(lib().mla_select_branch(ctypes.byref(geom), L, arr, len(cache_lens),
                                   MODES.get(mode, mode), ctypes.byref(out)),
           "mla_select_branch")
    return out.value


def mla_workspace_bytes(geom: Geometry, L: int, cache_lens: Sequence[int], mode="auto") -> int:
    arr = _lens_array(cache_lens)
    out = ctypes.c_size_t(0)
    _check(lib().mla_workspace_bytes(ctypes.byref(geom), len(cache_lens), L, arr,
                                     MODES.get(mode, mode), ctypes.byref(out)),
           "mla_workspace_bytes")
    return out.value


def mla_sparse_workspace_bytes(geom: Geometry, L: int, cache_lens: Sequence[int],
                               topk_len: int) -> int:
    arr = _lens_array(cache_lens)
    out = ctypes.c_size_t(0)
    _check(lib().mla_sparse_workspace_bytes(ctypes.byref(geom), len(cache_lens), L, arr,
                                            int(topk_len), ctypes.byref(out)),
           "mla_sparse_workspace_bytes")
    return out.value


def mla_check_page_table(page_table, cache_lens: Sequence[int], page_size: int,
                         num_pages: int) -> None:
    """Host-side range check of a page table (any int array-like [B, max_pages]);
    raises MlaError (MLA_ERR_INVALID_ARG) naming the first bad entry."""
    t = torch.as_tensor(page_table, dtype=torch.int32).cpu().contiguous()
    if t.dim() != 2:
        raise ValueError("page_table must be [batch, max_pages]")
    lens = _lens_array(cache_lens)
    _check(lib().mla_check_page_table(t.data_ptr(), t.shape[0], t.shape[1], lens, int(page_size),
                                      int(num_pages)), "mla_check_page_table")


def mla_select_draft_cap(p: float, verify_cost: Sequence[float], drafter_cost,
                         max_cap: int):
    """(best cap, [speedup(0), ..., speedup(limit)]) from a measured verify-cost
    curve (verify_cost[w-1] = cost of a pass over w rows) and the drafter's
    cost (one number, or one per cap)."""
    dr = [float(drafter_cost)] if isinstance(drafter_cost, (int, float)) else \
        [float(x) for x in drafter_cost]
    vc = (ctypes.c_double * len(verify_cost))(*[float(x) for x in verify_cost])
    dc = (ctypes.c_double * len(dr))(*dr)
    n_out = max(1, min(int(max_cap), len(verify_cost) - 1) + 1)
    sp = (ctypes.c_double * n_out)()
    cap = lib().mla_select_draft_cap(float(p), vc, len(verify_cost), dc, len(dr), int(max_cap), sp)
    if cap < 0:
        raise MlaError(MLA_ERR_INVALID_ARG, "mla_select_draft_cap", mla_last_error())
    limit = min(int(max_cap), len(verify_cost) - 1, len(dr) - 1 if len(dr) > 1 else 1 << 30)
    return int(cap), [sp[i] for i in range(limit + 1)]


def new_workspace(nbytes: int, device) -> torch.Tensor:
    """An (uninitialised) workspace of at least `nbytes` bytes."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


class SnapshotWindow(ctypes.Structure):
    _fields_ = [("window_start", ctypes.c_int32), ("cache_offset", ctypes.c_int64),
                ("sequence_stride", ctypes.c_int64)]


def _words(t: torch.Tensor) -> torch.Tensor:
    """A 32-bit tensor seen as uint32 words (no copy)."""
    if t.element_size() != 4:
        raise ValueError("snapshot buffers hold 32-bit words")
    return t


def mla_concat_snapshots(S, s_strides, T, t_strides, X, x_strides, s: int, n: int, H: int,
                         Q: int, cache, windows, stream=None) -> bool:
    """Concatenate S || T into X and write the snapshot windows into `cache`
    (flat 32-bit device tensors; strides in words).  windows: list of
    (window_start, cache_offset, sequence_stride).  Returns True when the
    fused single-load kernel ran, False for the ordinary path."""
    for t in (S, T, X, cache):
        _words(t)
    arr = (SnapshotWindow * max(1, len(windows)))(*[SnapshotWindow(*w) for w in windows])
    st = lambda v: (ctypes.c_int64 * 3)(*[int(x) for x in v])
    if stream is None:
        stream = _current_stream(X.device)
    fused = ctypes.c_int32(0)
    _check(lib().mla_concat_snapshots(_ptr(S), st(s_strides), _ptr(T), st(t_strides), _ptr(X),
                                      st(x_strides), s, n, H, Q, _ptr(cache), cache.numel(),
                                      arr, len(windows), stream, ctypes.byref(fused)),
           "mla_concat_snapshots")
    return bool(fused.value)


def mla_rollback_valid_prefix(blocks, r: int, cell_pos, cell_seq, p0: int, p1: int = -1,
                              seq: int = 0, n_streams: int = 1, stream=None) -> torch.Tensor:
    """Leading valid pooled blocks after a rollback from p0 (device int32
    tensor of one element).  blocks: int32 [n_blocks, 8 + r]; cell_pos: int32
    [n_cells]; cell_seq: int64 [n_cells] owner bit masks."""
    dev = cell_pos.device
    out = torch.empty(1, dtype=torch.int32, device=dev)
    _dense(blocks=blocks, cell_pos=cell_pos, cell_seq=cell_seq)
    if stream is None:
        stream = _current_stream(dev)
    _check(lib().mla_rollback_valid_prefix(_ptr(blocks), blocks.shape[0], r, _ptr(cell_pos),
                                           _ptr(cell_seq), cell_pos.numel(), p0, p1, seq,
                                           n_streams, _ptr(out), stream),
           "mla_rollback_valid_prefix")
    return out


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _dense(**tensors):
    for name, t in tensors.items():
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous (row-major)")


def mla_device_status(clear: bool = True) -> int:
    """Wait for the device, then raise MlaError if a kernel's bounded wait ran out."""
    code = ctypes.c_int32(0)
    _check(lib().mla_device_status(ctypes.byref(code), 1 if clear else 0), "mla_device_status")
    return code.value


def mla_selftest_bounded_wait(stream=None) -> None:
    """Launch the library's failure-path self-test (a bounded wait that runs out
    after about a second); mla_device_status then raises MLA_ERR_TIMEOUT."""
    if stream is None:
        stream = _current_stream(torch.device("cuda", torch.cuda.current_device()))
    _check(lib().mla_selftest_bounded_wait(stream), "mla_selftest_bounded_wait")


def cache_strides(c_kv: torch.Tensor, k_rope: torch.Tensor, paged: bool):
    """(c_kv row stride, k_rope row stride, rows between sequences) in elements."""
    if c_kv.stride(-1) != 1 or k_rope.stride(-1) != 1:
        raise ValueError("cache rows must be contiguous in their last dimension")
    cs, ks = c_kv.stride(1), k_rope.stride(1)
    if paged:
        if c_kv.stride(0) != c_kv.shape[1] * cs or k_rope.stride(0) != k_rope.shape[1] * ks:
            raise ValueError("paged cache pages must be contiguous runs of rows")
        return cs, ks, 0
    if c_kv.stride(0) % cs or k_rope.stride(0) % ks or \
            c_kv.stride(0) // cs != k_rope.stride(0) // ks:
        raise ValueError("c_kv and k_rope must have the same rows per sequence")
    return cs, ks, c_kv.stride(0) // cs


def _verify_args(q_nope, q_rope, c_kv, k_rope, W_UK, W_UV, cache_lens, mode, out, workspace,
                 page_table, cache_lens_dev, scale, noalloc=False):
    """Checks, defaults and the C arguments of mla_verify_attention up to (not
    including) the stream and the branch pointer.  Returns (args, out, dev,
    keep), keep holding every tensor the arguments point into.  With
    ``noalloc`` the arguments are those of mla_verify_attention_noalloc (no
    mode, no workspace)."""
    B, L, H, n = q_nope.shape
    rope = q_rope.shape[-1]
    r = W_UK.shape[-1]
    v = W_UV.shape[-1]
    dev = q_nope.device
    _dense(q_nope=q_nope, q_rope=q_rope, W_UK=W_UK, W_UV=W_UV, out=out, page_table=page_table)
    geom = _geometry(H, r, n, v, rope, q_nope.dtype, scale)
    lens = [int(t) for t in cache_lens]
    arr = _lens_array(lens)
    paged = page_table is not None
    cs, ks, seq = cache_strides(c_kv, k_rope, paged)
    if cache_lens_dev is None:
        cache_lens_dev = torch.tensor(lens, dtype=torch.int32, device=dev)
    if out is None:
        out = torch.empty((B, L, H, v), dtype=q_nope.dtype, device=dev)
    page_size = c_kv.shape[1] if paged else 0
    max_pages = page_table.shape[1] if paged else 0
    num_pages = c_kv.shape[0] if paged else 0
    args = [ctypes.byref(geom), _ptr(q_nope), _ptr(q_rope), _ptr(c_kv), _ptr(k_rope), cs, ks, seq,
            _ptr(W_UK), _ptr(W_UV), _ptr(cache_lens_dev), arr, B, L, _ptr(page_table), page_size,
            max_pages, num_pages]
    if noalloc:
        args += [_ptr(out)]
    else:
        m = MODES.get(mode, mode)
        if workspace is None:  # (a given workspace that is too small is rejected by the call)
            workspace = new_workspace(mla_workspace_bytes(geom, L, lens, m), dev)
        args += [m, _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size()]
    keep = (q_nope, q_rope, c_kv, k_rope, W_UK, W_UV, page_table, cache_lens_dev, out, workspace)
    return args, out, dev, keep


def mla_verify_attention(q_nope: torch.Tensor, q_rope: torch.Tensor, c_kv: torch.Tensor,
                         k_rope: torch.Tensor, W_UK: torch.Tensor, W_UV: torch.Tensor,
                         cache_lens: Sequence[int], mode="auto",
                         out: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None,
                         page_table: Optional[torch.Tensor] = None,
                         cache_lens_dev: Optional[torch.Tensor] = None,
                         scale: Optional[float] = None, stream=None):
    """One verify call through the C ABI.  Returns (out, branch).

    q_nope [B,L,H,n], q_rope [B,L,H,rope], W_UK [H,n,r], W_UV [H,r,v]; the
    cache is c_kv [B,Tmax,r] / k_rope [B,Tmax,rope] (contiguous) or
    [num_pages,page,r] / [num_pages,page,rope] with ``page_table`` [B,max_pages].
    ``out`` and ``workspace`` are allocated with torch when not given.
    """
    args, out, dev, _ = _verify_args(q_nope, q_rope, c_kv, k_rope, W_UK, W_UV, cache_lens, mode,
                                     out, workspace, page_table, cache_lens_dev, scale)
    if stream is None:
        stream = _current_stream(dev)
    branch = ctypes.c_int32(0)
    st = lib().mla_verify_attention(*args, stream, ctypes.byref(branch))
    _check(st, "mla_verify_attention")
    return out, branch.value


class PreparedVerifyAttention:
    """mla_verify_attention with its arguments marshalled once.

    For a caller that repeats a call on the same device buffers, as a serving
    loop does when it writes each step's queries and new cache rows into fixed
    tensors: the tensors, shapes, cache lengths and mode are fixed when the
    object is made (with the same checks and defaults as
    mla_verify_attention); ``run()`` issues the call on the current stream
    (or ``stream``) with whatever the buffers hold then, and returns the
    branch taken.  The tensors must outlive the object.  The library entry
    point and its results are the same as for mla_verify_attention.
    """

    def __init__(self, q_nope, q_rope, c_kv, k_rope, W_UK, W_UV, cache_lens, mode="auto",
                 out=None, workspace=None, page_table=None, cache_lens_dev=None, scale=None):
        args, self.out, dev, self._keep = _verify_args(q_nope, q_rope, c_kv, k_rope, W_UK, W_UV,
                                                       cache_lens, mode, out, workspace,
                                                       page_table, cache_lens_dev, scale)
        self._fn = lib().mla_verify_attention
        types = _SIGS["mla_verify_attention"][1]
        # plain ints become ctypes values now, so a run converts nothing
        self._args = [types[i](a) if isinstance(a, int) else a for i, a in enumerate(args)]
        self._dev = dev.index if dev.index is not None else torch.cuda.current_device()
        self._branch = ctypes.c_int32(0)
        self._branch_ref = ctypes.byref(self._branch)

    def run(self, stream=None) -> int:
        if stream is None:
            stream = (_raw_stream(self._dev) if _raw_stream is not None else
                      torch.cuda.current_stream(self._dev).cuda_stream)
        st = self._fn(*self._args, stream, self._branch_ref)
        if st != MLA_OK:
            _check(st, "mla_verify_attention")
        return self._branch.value


def mla_kernel_timing_enable(on: bool = True) -> None:
    """Bracket every library kernel launch with CUDA events (benchmark instrumentation)."""
    _check(lib().mla_kernel_timing_enable(1 if on else 0), "mla_kernel_timing_enable")


def mla_kernel_timing_read(reset: bool = True) -> dict:
    """{kernel name: (launches, total device ms)} of the kernels launched since
    the last reset (waits for their events)."""
    cap = 64
    names = ctypes.create_string_buffer(4096)
    launches = (ctypes.c_int32 * cap)()
    ms = (ctypes.c_double * cap)()
    n = ctypes.c_int32(0)
    _check(lib().mla_kernel_timing_read(names, 4096, launches, ms, cap, ctypes.byref(n),
                                        1 if reset else 0), "mla_kernel_timing_read")
    keys = names.value.decode().split(";") if n.value else []
    return {k: (int(launches[i]), float(ms[i])) for i, k in enumerate(keys[:cap])
            if launches[i] > 0}


def mla_verify_attention_noalloc(q_nope: torch.Tensor, q_rope: torch.Tensor,
                                 c_kv: torch.Tensor, k_rope: torch.Tensor,
                                 W_UK: torch.Tensor, W_UV: torch.Tensor,
                                 cache_lens: Sequence[int], out: Optional[torch.Tensor] = None,
                                 page_table: Optional[torch.Tensor] = None,
                                 cache_lens_dev: Optional[torch.Tensor] = None,
                                 scale: Optional[float] = None, stream=None):
    """Absorbed-branch verify call that uses the library's static scratch
    instead of a workspace (for callers that cannot allocate device memory).
    Same tensors and checks as :func:`mla_verify_attention`; returns (out, branch)."""
    args, out, dev, _ = _verify_args(q_nope, q_rope, c_kv, k_rope, W_UK, W_UV, cache_lens,
                                     None, out, None, page_table, cache_lens_dev, scale,
                                     noalloc=True)
    if stream is None:
        stream = _current_stream(dev)
    branch = ctypes.c_int32(0)
    st = lib().mla_verify_attention_noalloc(*args, stream, ctypes.byref(branch))
    _check(st, "mla_verify_attention_noalloc")
    return out, branch.value


def mla_verify_attention_sparse(q_nope: torch.Tensor, q_rope: torch.Tensor, c_kv: torch.Tensor,
                                k_rope: torch.Tensor, W_UK: torch.Tensor, W_UV: torch.Tensor,
                                cache_lens: Sequence[int], topk: torch.Tensor,
                                out: Optional[torch.Tensor] = None,
                                workspace: Optional[torch.Tensor] = None,
                                page_table: Optional[torch.Tensor] = None,
                                cache_lens_dev: Optional[torch.Tensor] = None,
                                scale: Optional[float] = None, stream=None) -> torch.Tensor:
    """Absorbed verify call over selected cached positions (the sparse model's
    top-k attention).  ``topk`` is an int32 device tensor [B, L, k]: verify row
    l of sequence b attends to the positions topk[b, l, :] that lie in
    [0, T_b - L + l] (others, e.g. -1 padding, are skipped).  The other
    tensors are those of :func:`mla_verify_attention`.  Returns out."""
    _dense(topk=topk)
    if topk.dtype != torch.int32 or topk.dim() != 3 or tuple(topk.shape[:2]) != \
            tuple(q_nope.shape[:2]):
        raise ValueError("topk must be int32 [B, L, k] matching q_nope's B and L")
    k = topk.shape[2]
    args, out, dev, _ = _verify_args(q_nope, q_rope, c_kv, k_rope, W_UK, W_UV, cache_lens, None,
                                     out, None, page_table, cache_lens_dev, scale, noalloc=True)
    geom_ref, L, arr = args[0], args[13], args[11]
    if workspace is None:
        nbytes = ctypes.c_size_t(0)
        _check(lib().mla_sparse_workspace_bytes(geom_ref, len(cache_lens), L, arr, int(k),
                                                ctypes.byref(nbytes)),
               "mla_sparse_workspace_bytes")
        workspace = new_workspace(nbytes.value, dev)
    if stream is None:
        stream = _current_stream(dev)
    # (geometry .. B, L) + (topk, k) + (page table .. num_pages) + (out, workspace, bytes)
    cargs = args[:14] + [_ptr(topk), int(k)] + args[14:18] + \
        [_ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(), stream]
    _check(lib().mla_verify_attention_sparse(*cargs), "mla_verify_attention_sparse")
    return out


class IndexerPoolState(ctypes.Structure):
    """What a pool of indexer keys describes (mla_indexer_pool_state_t)."""
    _fields_ = [("length", ctypes.c_int64), ("batch", ctypes.c_int32), ("dim", ctypes.c_int32)]

    def __init__(self):
        super().__init__(-1, 0, 0)


def mla_indexer_pool_update(keys: torch.Tensor, cache_len: int, new_tokens: int,
                            pooled: torch.Tensor, state: IndexerPoolState, padded: bool = False,
                            stream=None) -> bool:
    """Pool the indexer keys of one step.  keys [batch, Tmax, dim] (bf16 or
    fp32, rows contiguous), pooled fp32 [batch, cap, dim]; ``state`` is
    updated.  Returns True when the incremental (tail-only) path ran."""
    if keys.dim() != 3 or keys.stride(-1) != 1 or not pooled.is_contiguous() or \
            pooled.dtype != torch.float32:
        raise ValueError("keys must be [batch, T, dim] with contiguous rows, pooled fp32 "
                         "[batch, cap, dim] contiguous")
    Bn, _, d = keys.shape
    inc = ctypes.c_int32(0)
    if stream is None:
        stream = _current_stream(keys.device)
    _check(lib().mla_indexer_pool_update(
        _ptr(keys), DTYPES[keys.dtype], keys.stride(1), keys.stride(0) // keys.stride(1), Bn, d,
        int(cache_len), int(new_tokens), 1 if padded else 0, _ptr(pooled), pooled.shape[1],
        ctypes.byref(state), ctypes.byref(inc), stream), "mla_indexer_pool_update")
    return bool(inc.value)


def mla_indexer_select(q: torch.Tensor, pooled: torch.Tensor, cache_len: int, k_windows: int,
                       stream=None):
    """(windows [batch, S, k], positions [batch, S, 4k]) int32: each new
    token's k best visible windows, ascending, and their positions."""
    _dense(q=q, pooled=pooled)
    Bn, S, d = q.shape
    dev = q.device
    wins = torch.empty((Bn, S, k_windows), dtype=torch.int32, device=dev)
    pos = torch.empty((Bn, S, 4 * k_windows), dtype=torch.int32, device=dev)
    nbytes = ctypes.c_size_t(0)
    _check(lib().mla_indexer_select_workspace_bytes(Bn, S, int(cache_len), ctypes.byref(nbytes)),
           "mla_indexer_select_workspace_bytes")
    ws = new_workspace(nbytes.value, dev)
    if stream is None:
        stream = _current_stream(dev)
    _check(lib().mla_indexer_select(_ptr(q), _ptr(pooled), pooled.shape[1], Bn, d, int(cache_len),
                                    S, int(k_windows), _ptr(wins), _ptr(pos), _ptr(ws),
                                    ws.numel(), stream), "mla_indexer_select")
    return wins, pos


# ---------------------------------------------------------------------------
# Paged serving steps: page tables, appends, the drafter's decode attention
# (inference only: no gradients are recorded)
#
# Every tensor starts on a 16-byte boundary (lengths and tables too: a slice of a
# larger array may not).  The functions check, marshal and allocate at each call,
# about 40 us of host time; a Prepared* object does so once, for fixed buffers,
# and its run() takes 3 to 4 us.
# ---------------------------------------------------------------------------

def _tensor(name: str, t: torch.Tensor, shape=None, dtype=None, dense: bool = True):
    """Check one tensor argument (a None in `shape` matches any size)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if shape is not None and (t.dim() != len(shape) or
                              any(w is not None and int(w) != g
                                  for w, g in zip(shape, t.shape))):
        want = "[" + ", ".join("*" if w is None else str(w) for w in shape) + "]"
        raise ValueError(f"{name} must be {want}, got {list(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    return t


def _one_device(**tensors) -> torch.device:
    """The CUDA device that every given tensor is on."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be on a CUDA device, got {t.device}")
        if dev is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, other tensors on {dev}")
        dev = t.device
    return dev


def _stream_object(handle: int, dev: torch.device):
    """The PyTorch stream of a raw handle.  (ExternalStream would take 0 for no handle
    and give some other stream.)"""
    return torch.cuda.ExternalStream(handle, device=dev) if handle else \
        torch.cuda.default_stream(dev)


def _allocating_on(stream, dev: torch.device):
    """Allocate for kernels of `stream` (a raw handle; None: the current one), so
    that freed memory is only reused behind them."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(_stream_object(int(stream), dev))


class _PreparedCall:
    """A C call whose arguments are marshalled once and issued by run().

    Runs share the object's buffers (outputs, and the workspace of the decode
    attention): on several streams each must wait for the one before."""

    def _prepare(self, name: str, args, dev: torch.device, keep, made=()):
        self._name = name
        self._fn = getattr(lib(), name)
        types = _SIGS[name][1]
        for t, a in zip(types, args):   # (ctypes would keep the low 32 bits)
            if t is _I32 and not -2 ** 31 <= a < 2 ** 31:
                raise ValueError(f"{name}: {a} does not fit a 32-bit integer")
        # plain numbers become ctypes values now, so a run converts nothing
        self._args = [types[i](a) if isinstance(a, (int, float)) else a
                      for i, a in enumerate(args)]
        self._dev = dev.index if dev.index is not None else torch.cuda.current_device()
        self._one_device = torch.cuda.device_count() == 1   # then it is the current one
        self._keep = keep
        self._made = [t for t in made if t is not None]
        self._home = _current_stream(torch.device("cuda", self._dev))
        self._streams = {self._home}

    def run(self, stream=None) -> None:
        """Issue the call on the current stream of the tensors' device (or on
        ``stream``, a raw handle) with what the buffers hold then."""
        if stream is None:
            stream = (_raw_stream(self._dev) if _raw_stream is not None else
                      torch.cuda.current_stream(self._dev).cuda_stream)
        if stream not in self._streams:
            self._made_for(int(stream))
            self._streams.add(stream)
        if self._one_device or torch.cuda.current_device() == self._dev:
            st = self._fn(*self._args, stream)
        else:
            with torch.cuda.device(self._dev):
                st = self._fn(*self._args, stream)
        if st != MLA_OK:
            _check(st, self._name)


    def _made_for(self, stream: int) -> None:
        """Before the first run on another stream than the one the buffers made here
        belong to: what that one still does with them (zeros, or earlier work on the
        same memory) comes first, and they are not reused before this stream is done
        with them.  (A capture cannot wait for work outside it; it begins behind a
        synchronisation.)"""
        if not self._made:
            return
        dev = torch.device("cuda", self._dev)
        s = _stream_object(stream, dev)
        with torch.cuda.stream(s):
            if not torch.cuda.is_current_stream_capturing():
                s.wait_stream(_stream_object(self._home, dev))
        for t in self._made:
            t.record_stream(s)


class PageStep(NamedTuple):
    """The outputs of mla_page_step (device tensors)."""
    cache_lens: torch.Tensor   # int32 [batch]
    held_pages: torch.Tensor   # int32 [batch]
    row_start: torch.Tensor    # int32 [batch + 1]
    positions: torch.Tensor    # int32 [max_rows]
    slots: torch.Tensor        # int64 [max_rows]
    free_span: torch.Tensor    # int32 [2]
    missing: torch.Tensor      # int32 [1]


class PreparedPageStep(_PreparedCall):
    """mla_page_step with its arguments marshalled once (fixed buffers, as in a
    serving loop or a captured graph); ``run()`` issues it and ``out`` holds
    its outputs.  The tensors must outlive the object."""

    def __init__(self, kept_lens, new_tokens, held_pages, page_table, free_pages, free_span,
                 page_size: int, num_pages: int, max_rows: int,
                 out: Optional[PageStep] = None):
        i32 = torch.int32
        _tensor("page_table", page_table, (None, None), i32)
        B, W = page_table.shape
        for name, t in (("kept_lens", kept_lens), ("new_tokens", new_tokens),
                        ("held_pages", held_pages)):
            _tensor(name, t, (B,), i32)
        _tensor("free_pages", free_pages, (None,), i32)
        _tensor("free_span", free_span, (2,), i32)
        max_rows = int(max_rows)
        if max_rows < 0:
            raise ValueError("max_rows must not be negative")
        shapes = (("cache_lens", (B,), i32), ("held_pages", (B,), i32),
                  ("row_start", (B + 1,), i32), ("positions", (max_rows,), i32),
                  ("slots", (max_rows,), torch.int64), ("free_span", (2,), i32),
                  ("missing", (1,), i32))
        if out is not None:
            for (name, shape, dtype), t in zip(shapes, out):
                _tensor("out." + name, t, shape, dtype)
        dev = _one_device(kept_lens=kept_lens, new_tokens=new_tokens, held_pages=held_pages,
                          page_table=page_table, free_pages=free_pages, free_span=free_span,
                          **({} if out is None else {"out_" + n[0]: t
                                                     for n, t in zip(shapes, out)}))
        made = ()
        if out is None:
            out = made = PageStep(*[torch.empty(shape, dtype=dtype, device=dev)
                                    for _, shape, dtype in shapes])
        self.out = out
        args = [_ptr(kept_lens), _ptr(new_tokens), _ptr(held_pages), B, _ptr(page_table), W,
                int(page_size), int(num_pages), _ptr(free_pages), free_pages.numel(),
                _ptr(free_span), _ptr(out.cache_lens), _ptr(out.held_pages), _ptr(out.row_start),
                _ptr(out.positions), _ptr(out.slots), max_rows, _ptr(out.free_span),
                _ptr(out.missing)]
        keep = (kept_lens, new_tokens, held_pages, page_table, free_pages, free_span, out)
        self._prepare("mla_page_step", args, dev, keep, made)


def mla_page_step(kept_lens, new_tokens, held_pages, page_table, free_pages, free_span,
                  page_size: int, num_pages: int, max_rows: int, out: Optional[PageStep] = None,
                  stream=None) -> PageStep:
    """Page table, cache lengths, positions and slots of one step, on the GPU.

    ``kept_lens``, ``new_tokens``, ``held_pages`` int32 [B]; ``page_table``
    int32 [B, max_pages] (its new entries are written); ``free_pages`` int32
    ids of which entries ``free_span[0] .. free_span[1] - 1`` are free.  The
    step's rows are the sequences' new tokens in order, at most ``max_rows``;
    rows behind them get slot and position -1.  ``missing`` counts the pages
    that the free list did not have.  Returns a :class:`PageStep`; its
    ``cache_lens``, ``held_pages`` and ``free_span`` are the next step's
    inputs."""
    with _allocating_on(stream, page_table.device):
        call = PreparedPageStep(kept_lens, new_tokens, held_pages, page_table, free_pages,
                                free_span, page_size, num_pages, max_rows, out)
        call.run(stream)
    return call.out


def _head_rows(name: str, t: torch.Tensor, dtype=None):
    """(rows, heads, width, elements between rows) of [rows, heads, width] with dense heads."""
    _tensor(name, t, (None, None, None), dtype, dense=False)
    N, H, D = t.shape
    if (D > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != D):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return N, H, D, (t.stride(0) if N > 1 else H * D)


def _row_cache(name: str, t: torch.Tensor, width: int, dtype):
    """(rows, elements between rows) of a cache [pages, page, width] or [rows, width]."""
    if t.dim() == 2:
        t = t.unsqueeze(0)
    _tensor(name, t, (None, None, width), dtype, dense=False)
    P, S, _ = t.shape
    stride = t.stride(1) if S > 1 else (t.stride(0) if P > 1 else width)
    if (width > 1 and t.stride(2) != 1) or (P > 1 and t.stride(0) != S * stride):
        raise ValueError(f"{name}: pages must be contiguous runs of rows")
    return P * S, stride


def _step_rows(positions, slots, rows: int):
    _tensor("positions", positions, (rows,), torch.int32)
    _tensor("slots", slots, (rows,), torch.int64)


class PreparedAppendLatent(_PreparedCall):
    """mla_append_latent with its arguments marshalled once; ``run()`` issues it,
    ``q_nope`` and ``q_rope`` are its outputs.  The tensors must outlive the
    object."""

    def __init__(self, q, kv, cos_sin, positions, slots, c_kv, k_rope, norm_weight=None,
                 eps: float = 1e-6, interleaved: bool = True, q_nope=None, q_rope=None):
        _tensor("kv", kv, (None, None), dense=False)
        if kv.dtype not in DTYPES:
            raise ValueError(f"kv must be bf16 or fp32, got {kv.dtype}")
        dt = kv.dtype
        _tensor("cos_sin", cos_sin, (None, None), torch.float32)
        rope, N = cos_sin.shape[1], kv.shape[0]
        r = kv.shape[1] - rope
        if r < 1 or (kv.shape[1] > 1 and kv.stride(1) != 1):
            raise ValueError("kv rows must be contiguous and hold the latent and the RoPE key")
        kvs = kv.stride(0) if N > 1 else kv.shape[1]
        _step_rows(positions, slots, N)
        rows, cs = _row_cache("c_kv", c_kv, r, dt)
        rows2, ks = _row_cache("k_rope", k_rope, rope, dt)
        if rows != rows2:
            raise ValueError("c_kv and k_rope must have the same rows")
        if norm_weight is not None:
            _tensor("norm_weight", norm_weight, (r,), dt)
        H, n, qs = 1, 16, 0
        if q is not None:
            _, H, width, qs = _head_rows("q", q, dt)
            n = width - rope
            if q.shape[0] != N or n < 1:
                raise ValueError("q must be [rows, H, n + rope] with kv's rows")
            if q_nope is not None:
                _tensor("q_nope", q_nope, (N, H, n), dt)
            if q_rope is not None:
                _tensor("q_rope", q_rope, (N, H, rope), dt)
        elif q_nope is not None or q_rope is not None:
            raise ValueError("q_nope and q_rope need q")
        dev = _one_device(kv=kv, q=q, cos_sin=cos_sin, positions=positions, slots=slots,
                          c_kv=c_kv, k_rope=k_rope, norm_weight=norm_weight, q_nope=q_nope,
                          q_rope=q_rope)
        made = []
        if q is not None:
            # (a skipped row is not written: it starts as zeros, not as whatever was there)
            if q_nope is None:
                q_nope = torch.zeros((N, H, n), dtype=dt, device=dev)
                made.append(q_nope)
            if q_rope is None:
                q_rope = torch.zeros((N, H, rope), dtype=dt, device=dev)
                made.append(q_rope)
        self.q_nope, self.q_rope = q_nope, q_rope
        geom = _geometry(H, r, n, n, rope, dt, None)
        args = [ctypes.byref(geom), _ptr(q), qs, _ptr(kv), kvs, _ptr(norm_weight), float(eps),
                _ptr(cos_sin), cos_sin.shape[0], 1 if interleaved else 0, _ptr(positions),
                _ptr(slots), N, _ptr(q_nope), _ptr(q_rope), _ptr(c_kv), _ptr(k_rope), cs, ks,
                rows]
        keep = (q, kv, cos_sin, positions, slots, c_kv, k_rope, norm_weight, q_nope, q_rope)
        self._prepare("mla_append_latent", args, dev, keep, made)


def mla_append_latent(q, kv, cos_sin, positions, slots, c_kv, k_rope, norm_weight=None,
                      eps: float = 1e-6, interleaved: bool = True, q_nope=None, q_rope=None,
                      stream=None):
    """The rows of a step into the paged latent cache.  Returns (q_nope, q_rope).

    ``q`` [N, H, n + rope] (or None), ``kv`` [N, r + rope] as the projections
    leave them; ``cos_sin`` fp32 [table, rope] (cosines, then sines);
    ``positions`` int32 [N], ``slots`` int64 [N] as mla_page_step gives them.
    c_kv gets the RMS-normalised latent (``norm_weight`` None: as it is),
    k_rope the rotated key; q is split into q_nope and the rotated q_rope, which
    mla_verify_attention takes as [B, L, H, *] views.  Rows with position -1
    are skipped."""
    with _allocating_on(stream, kv.device):
        call = PreparedAppendLatent(q, kv, cos_sin, positions, slots, c_kv, k_rope, norm_weight,
                                    eps, interleaved, q_nope, q_rope)
        call.run(stream)
    return call.q_nope, call.q_rope


def _kv_cache(k_cache, v_cache, dtype, kv_heads: int, dim: int, k_scale, v_scale):
    """The C description of a paged key/value cache, and its element type."""
    if dtype not in DTYPES:
        raise ValueError(f"q, k and v must be bf16 or fp32, got {dtype}")
    _tensor("k_cache", k_cache, (None, None, kv_heads, dim), dense=False)
    _tensor("v_cache", v_cache, k_cache.shape, k_cache.dtype, dense=False)
    if k_cache.dtype not in CACHE_DTYPES:
        raise ValueError(f"a cache must be bf16, fp32 or float8_e4m3fn, got {k_cache.dtype}")
    strides = [k_cache.stride(i) if k_cache.shape[i] > 1 else 0 for i in range(3)]
    if strides != [v_cache.stride(i) if v_cache.shape[i] > 1 else 0 for i in range(3)]:
        raise ValueError("k_cache and v_cache must have the same strides")
    if dim > 1 and (k_cache.stride(3) != 1 or v_cache.stride(3) != 1):
        raise ValueError("cache rows must be contiguous in their last dimension")
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t is not None:
            _tensor(name, t, (kv_heads,), torch.float32)
    return KVCache(_ptr(k_cache), _ptr(v_cache), strides[0], strides[1], strides[2],
                   k_cache.shape[1], k_cache.shape[0], _ptr(k_scale), _ptr(v_scale))


class PreparedAppendKV(_PreparedCall):
    """mla_append_kv with its arguments marshalled once; ``run()`` issues it and
    ``q_out`` is its output.  The tensors must outlive the object."""

    def __init__(self, q, k, v, cos_sin, positions, slots, k_cache, v_cache,
                 interleaved: bool = False, k_scale=None, v_scale=None, q_out=None):
        N, Hk, D, ks = _head_rows("k", k)
        dt = k.dtype
        _tensor("v", v, (N, Hk, D), dt, dense=False)
        vs = _head_rows("v", v)[3]
        cache = _kv_cache(k_cache, v_cache, dt, Hk, D, k_scale, v_scale)
        _step_rows(positions, slots, N)
        rope = table = 0
        if cos_sin is not None:
            _tensor("cos_sin", cos_sin, (None, None), torch.float32)
            table, rope = cos_sin.shape
            if rope < 1:
                raise ValueError("cos_sin must not be empty (None: no rotation)")
        H, qs = Hk, 0
        if q is not None:
            _tensor("q", q, (N, None, D), dt, dense=False)
            _, H, _, qs = _head_rows("q", q)
            if q_out is not None:
                _tensor("q_out", q_out, (N, H, D), dt)
        elif q_out is not None:
            raise ValueError("q_out needs q")
        dev = _one_device(k=k, q=q, v=v, cos_sin=cos_sin, positions=positions, slots=slots,
                          k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale,
                          q_out=q_out)
        made = []
        if q is not None and q_out is None:
            q_out = torch.zeros((N, H, D), dtype=dt, device=dev)
            made.append(q_out)
        self.q_out = q_out
        geom = KVGeometry(H, Hk, D, 0.0, DTYPES[dt], CACHE_DTYPES[k_cache.dtype])
        args = [ctypes.byref(geom), _ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(cos_sin), table,
                rope, 1 if interleaved else 0, _ptr(positions), _ptr(slots), N, _ptr(q_out),
                ctypes.byref(cache)]
        keep = (geom, cache, q, k, v, cos_sin, positions, slots, k_cache, v_cache, k_scale,
                v_scale, q_out)
        self._prepare("mla_append_kv", args, dev, keep, made)


def mla_append_kv(q, k, v, cos_sin, positions, slots, k_cache, v_cache, interleaved: bool = False,
                  k_scale=None, v_scale=None, q_out=None, stream=None):
    """The rows of a step into a paged key/value cache.  Returns the rotated q.

    ``q`` [N, H, D] (or None), ``k`` and ``v`` [N, Hkv, D] (views of one
    projection's rows will do); ``cos_sin`` fp32 [table, rope_dim] or None;
    caches [num_pages, page_size, Hkv, D] in any stride order (a cache laid
    out [pages, Hkv, page, D] is passed as ``cache.transpose(1, 2)``), of q's
    type or float8_e4m3fn with fp32 ``k_scale`` / ``v_scale`` [Hkv].  Rows
    with position -1 are skipped.  ``q_out`` may be ``q``; otherwise no output
    may overlap an input.

    The rows are a step's, packed: with an idle slot among the sequences the
    query that mla_decode_attention wants for sequence b is row
    ``row_start[b]`` (of mla_page_step), not b."""
    with _allocating_on(stream, k.device):
        call = PreparedAppendKV(q, k, v, cos_sin, positions, slots, k_cache, v_cache, interleaved,
                                k_scale, v_scale, q_out)
        call.run(stream)
    return call.q_out


def mla_decode_workspace_bytes(num_heads: int, num_kv_heads: int, head_dim: int, batch: int,
                               page_size: int, max_pages: int, dtype=torch.bfloat16,
                               cache_dtype=None) -> int:
    geom = KVGeometry(num_heads, num_kv_heads, head_dim, 0.0, DTYPES[dtype],
                      CACHE_DTYPES[cache_dtype if cache_dtype is not None else dtype])
    out = ctypes.c_size_t(0)
    _check(lib().mla_decode_workspace_bytes(ctypes.byref(geom), batch, page_size, max_pages,
                                            ctypes.byref(out)), "mla_decode_workspace_bytes")
    return out.value


def _softmax_scale(scale: Optional[float]) -> float:
    """The scale as the library takes it, in fp32, where 0 stands for 1/sqrt(head_dim)."""
    if scale is None:
        return 0.0
    fp32 = ctypes.c_float(float(scale)).value
    if not 0.0 < fp32 < float("inf"):
        raise ValueError(f"scale must be positive and finite in fp32 (None: 1/sqrt(head_dim)), "
                         f"got {scale}")
    return fp32


class PreparedDecodeAttention(_PreparedCall):
    """mla_decode_attention with its arguments marshalled once, for a decode loop
    over fixed buffers (lengths and tables are read on the device, so they may
    change between runs and under a captured graph); ``run()`` issues it,
    ``out`` and ``lse`` are its outputs.  The tensors must outlive the
    object.  It has one workspace: runs on several streams, and graphs that
    hold them, must not overlap (an object, or a ``workspace``, for each
    otherwise)."""

    def __init__(self, q, k_cache, v_cache, cache_lens, page_table, window: int = 0,
                 scale: Optional[float] = None, k_scale=None, v_scale=None, out=None, lse=None,
                 return_lse: bool = False, workspace=None):
        B, H, D, qs = _head_rows("q", q)
        _tensor("k_cache", k_cache, (None, None, None, D), dense=False)
        Hk = k_cache.shape[2]
        cache = _kv_cache(k_cache, v_cache, q.dtype, Hk, D, k_scale, v_scale)
        geom = KVGeometry(H, Hk, D, _softmax_scale(scale), DTYPES[q.dtype],
                          CACHE_DTYPES[k_cache.dtype])
        _tensor("cache_lens", cache_lens, (B,), torch.int32)
        _tensor("page_table", page_table, (B, None), torch.int32)
        if out is not None:
            _tensor("out", out, (B, H, D), q.dtype)
        if lse is not None:
            _tensor("lse", lse, (B, H), torch.float32)
        if workspace is not None:
            _tensor("workspace", workspace)
        dev = _one_device(q=q, k_cache=k_cache, v_cache=v_cache, cache_lens=cache_lens,
                          page_table=page_table, k_scale=k_scale, v_scale=v_scale, out=out,
                          lse=lse, workspace=workspace)
        made = []
        if out is None:
            out = torch.empty((B, H, D), dtype=q.dtype, device=dev)
            made.append(out)
        if lse is None and return_lse:
            lse = torch.empty((B, H), dtype=torch.float32, device=dev)
            made.append(lse)
        if workspace is None:
            nbytes = ctypes.c_size_t(0)
            with torch.cuda.device(dev):
                _check(lib().mla_decode_workspace_bytes(
                    ctypes.byref(geom), B, k_cache.shape[1], page_table.shape[1],
                    ctypes.byref(nbytes)), "mla_decode_workspace_bytes")
            workspace = new_workspace(nbytes.value, dev)
            made.append(workspace)
        self.out, self.lse = out, lse
        args = [ctypes.byref(geom), _ptr(q), qs, ctypes.byref(cache), _ptr(cache_lens), B,
                _ptr(page_table), page_table.shape[1], int(window), _ptr(out), _ptr(lse),
                _ptr(workspace), workspace.numel() * workspace.element_size()]
        keep = (geom, cache, q, k_cache, v_cache, cache_lens, page_table, k_scale, v_scale, out,
                lse, workspace)
        self._prepare("mla_decode_attention", args, dev, keep, made)


def mla_decode_attention(q, k_cache, v_cache, cache_lens, page_table, window: int = 0,
                         scale: Optional[float] = None, k_scale=None, v_scale=None, out=None,
                         lse=None, return_lse: bool = False, workspace=None, stream=None):
    """Attention of one new token per sequence over a paged key/value cache.
    Returns out, or (out, lse) with ``return_lse`` or ``lse``.

    ``q`` [B, H, D]; caches [num_pages, page_size, Hkv, D] in any stride order
    (see mla_append_kv), of q's type or float8_e4m3fn; ``cache_lens`` int32 [B]
    on the device, the new token included (0: an idle slot, zeros come back);
    ``page_table`` int32 [B, max_pages]; ``window`` > 0 keeps the last
    ``window`` positions."""
    with _allocating_on(stream, q.device):
        call = PreparedDecodeAttention(q, k_cache, v_cache, cache_lens, page_table, window, scale,
                                       k_scale, v_scale, out, lse, return_lse, workspace)
        call.run(stream)
    return (call.out, call.lse) if call.lse is not None else call.out


def mla_chunk_workspace_bytes(num_heads: int, num_kv_heads: int, head_dim: int, batch: int,
                              rows: int, page_size: int, max_pages: int, dtype=torch.bfloat16,
                              cache_dtype=None) -> int:
    geom = KVGeometry(num_heads, num_kv_heads, head_dim, 0.0, DTYPES[dtype],
                      CACHE_DTYPES[cache_dtype if cache_dtype is not None else dtype])
    out = ctypes.c_size_t(0)
    _check(lib().mla_chunk_workspace_bytes(ctypes.byref(geom), batch, rows, page_size, max_pages,
                                           ctypes.byref(out)), "mla_chunk_workspace_bytes")
    return out.value


class PreparedChunkAttention(_PreparedCall):
    """mla_chunk_attention with its arguments marshalled once, for steps over fixed
    buffers (lengths, row starts and tables are read on the device, so they may
    change between runs and under a captured graph); ``run()`` issues it,
    ``out`` and ``lse`` are its outputs.  The tensors must outlive the
    object.  It has one workspace: runs on several streams, and graphs that
    hold them, must not overlap (an object, or a ``workspace``, for each
    otherwise)."""

    def __init__(self, q, k_cache, v_cache, kept_lens, cache_lens, row_start, page_table,
                 window: int = 0, scale: Optional[float] = None, k_scale=None, v_scale=None,
                 out=None, lse=None, return_lse: bool = False, workspace=None):
        N, H, D, qs = _head_rows("q", q)
        _tensor("k_cache", k_cache, (None, None, None, D), dense=False)
        Hk = k_cache.shape[2]
        cache = _kv_cache(k_cache, v_cache, q.dtype, Hk, D, k_scale, v_scale)
        geom = KVGeometry(H, Hk, D, _softmax_scale(scale), DTYPES[q.dtype],
                          CACHE_DTYPES[k_cache.dtype])
        _tensor("page_table", page_table, (None, None), torch.int32)
        B = page_table.shape[0]
        _tensor("kept_lens", kept_lens, (B,), torch.int32)
        _tensor("cache_lens", cache_lens, (B,), torch.int32)
        _tensor("row_start", row_start, (B + 1,), torch.int32)
        if out is not None:
            _tensor("out", out, (N, H, D), q.dtype)
        if lse is not None:
            _tensor("lse", lse, (N, H), torch.float32)
        if workspace is not None:
            _tensor("workspace", workspace)
        dev = _one_device(q=q, k_cache=k_cache, v_cache=v_cache, kept_lens=kept_lens,
                          cache_lens=cache_lens, row_start=row_start, page_table=page_table,
                          k_scale=k_scale, v_scale=v_scale, out=out, lse=lse,
                          workspace=workspace)
        made = []
        # (a row outside every sequence is not written: it starts as zeros, not as whatever was
        # there)
        if out is None:
            out = torch.zeros((N, H, D), dtype=q.dtype, device=dev)
            made.append(out)
        if lse is None and return_lse:
            lse = torch.zeros((N, H), dtype=torch.float32, device=dev)
            made.append(lse)
        if workspace is None:
            nbytes = ctypes.c_size_t(0)
            with torch.cuda.device(dev):
                _check(lib().mla_chunk_workspace_bytes(
                    ctypes.byref(geom), B, N, k_cache.shape[1], page_table.shape[1],
                    ctypes.byref(nbytes)), "mla_chunk_workspace_bytes")
            workspace = new_workspace(nbytes.value, dev)
            made.append(workspace)
        self.out, self.lse = out, lse
        args = [ctypes.byref(geom), _ptr(q), qs, N, ctypes.byref(cache), _ptr(kept_lens),
                _ptr(cache_lens), _ptr(row_start), B, _ptr(page_table), page_table.shape[1],
                int(window), _ptr(out), _ptr(lse), _ptr(workspace),
                workspace.numel() * workspace.element_size()]
        keep = (geom, cache, q, k_cache, v_cache, kept_lens, cache_lens, row_start, page_table,
                k_scale, v_scale, out, lse, workspace)
        self._prepare("mla_chunk_attention", args, dev, keep, made)


def mla_chunk_attention(q, k_cache, v_cache, kept_lens, cache_lens, row_start, page_table,
                        window: int = 0, scale: Optional[float] = None, k_scale=None,
                        v_scale=None, out=None, lse=None, return_lse: bool = False,
                        workspace=None, stream=None):
    """Attention of a step's new rows over a paged key/value cache.  Returns out, or
    (out, lse) with ``return_lse`` or ``lse``.

    ``q`` [N, H, D], the step's rows as mla_append_kv returns them; caches as
    for mla_decode_attention, holding those rows; ``kept_lens`` int32 [B] (the
    one given to mla_page_step), ``cache_lens`` [B] and ``row_start`` [B + 1] as
    mla_page_step returns them: row i of a sequence sits at position kept + i and
    sees itself and what is before it, the last ``window`` positions where that
    is positive.  Rows behind the last sequence are left as they are."""
    with _allocating_on(stream, q.device):
        call = PreparedChunkAttention(q, k_cache, v_cache, kept_lens, cache_lens, row_start,
                                      page_table, window, scale, k_scale, v_scale, out, lse,
                                      return_lse, workspace)
        call.run(stream)
    return (call.out, call.lse) if call.lse is not None else call.out


# ---------------------------------------------------------------------------
# The pages of a cache as a pool.  ``shares`` int32 [num_pages] counts a page's
# holders beyond the first; it starts as zeros.
# ---------------------------------------------------------------------------

class PageFork(NamedTuple):
    """The outputs of mla_page_fork (device tensors, int32)."""
    cache_lens: torch.Tensor   # [batch]
    held_pages: torch.Tensor   # [batch]
    shares: torch.Tensor       # [num_pages]
    free_span: torch.Tensor    # [2]
    missing: torch.Tensor      # [1]
    move_src: torch.Tensor     # [batch], the first moves[0] of them
    move_dst: torch.Tensor     # [batch]
    move_rows: torch.Tensor    # [batch]
    moves: torch.Tensor        # [1]


class PageRelease(NamedTuple):
    """The outputs of mla_page_release (device tensors, int32)."""
    held_pages: torch.Tensor   # [batch]
    shares: torch.Tensor       # [num_pages]
    free_span: torch.Tensor    # [2]
    released: torch.Tensor     # [1]


class PageCompact(NamedTuple):
    """The outputs of mla_page_compact (device tensors, int32)."""
    page_table: torch.Tensor   # [batch, max_pages]
    shares: torch.Tensor       # [num_pages]
    free_span: torch.Tensor    # [2]
    move_src: torch.Tensor     # [num_pages / 2, at least 1], the first moves[0] of them
    move_dst: torch.Tensor     # [the same]
    moves: torch.Tensor        # [1]


class _PreparedPoolCall(_PreparedCall):
    """What the page calls share: int32 tensors checked, outputs checked or made."""

    def _pool(self, kind, inputs, shapes, out):
        for name, (t, shape) in inputs.items():
            _tensor(name, t, shape, torch.int32)
        if out is not None:
            if len(out) != len(shapes):
                raise ValueError(f"out must be a {kind.__name__}")
            for name, t in zip(kind._fields, out):
                _tensor("out." + name, t, shapes[name], torch.int32)
        given = {} if out is None else {"out_" + n: t for n, t in zip(kind._fields, out)}
        dev = _one_device(**{n: t for n, (t, _) in inputs.items()}, **given)
        made = ()
        if out is None:
            # (move lists are written as far as there are moves: the rest starts as zeros)
            out = made = kind(*[torch.zeros(shapes[n], dtype=torch.int32, device=dev)
                                if n.startswith("move_") else
                                torch.empty(shapes[n], dtype=torch.int32, device=dev)
                                for n in kind._fields])
        self.out = kind(*out)
        return dev, made


class PreparedPageFork(_PreparedPoolCall):
    """mla_page_fork with its arguments marshalled once; ``run()`` issues it and
    ``out`` holds its outputs.  The tensors must outlive the object."""

    def __init__(self, src_of, cache_lens, held_pages, page_table, shares, free_pages, free_span,
                 page_size: int, out: Optional[PageFork] = None):
        _tensor("page_table", page_table, (None, None), torch.int32)
        _tensor("shares", shares, (None,), torch.int32)
        B, W = page_table.shape
        P = shares.numel()
        inputs = dict(src_of=(src_of, (B,)), cache_lens=(cache_lens, (B,)),
                      held_pages=(held_pages, (B,)), page_table=(page_table, (B, W)),
                      shares=(shares, (P,)), free_pages=(free_pages, (None,)),
                      free_span=(free_span, (2,)))
        shapes = dict(cache_lens=(B,), held_pages=(B,), shares=(P,), free_span=(2,), missing=(1,),
                      move_src=(B,), move_dst=(B,), move_rows=(B,), moves=(1,))
        dev, made = self._pool(PageFork, inputs, shapes, out)
        o = self.out
        args = [_ptr(src_of), _ptr(cache_lens), _ptr(held_pages), B, _ptr(page_table), W,
                int(page_size), P, _ptr(shares), _ptr(free_pages), free_pages.numel(),
                _ptr(free_span), *[_ptr(t) for t in o]]
        self._prepare("mla_page_fork", args, dev, (inputs, o), made)


def mla_page_fork(src_of, cache_lens, held_pages, page_table, shares, free_pages, free_span,
                  page_size: int, out: Optional[PageFork] = None, stream=None) -> PageFork:
    """Fork sequences to idle slots: slot b takes the rows of sequence ``src_of[b]``
    where that is in [0, B) and slot b holds no pages.

    ``src_of``, ``cache_lens``, ``held_pages`` int32 [B]; ``page_table`` int32
    [B, max_pages] (the forked slots' entries are written); ``shares`` int32
    [num_pages]; ``free_pages`` and ``free_span`` as for mla_page_step.  Whole
    pages are shared; a last one that is not full is replaced by a free page, and
    the rows to copy are listed: ``mla_page_copy(caches, out.move_src,
    out.move_dst, out.moves, out.move_rows)``, for the caches of all layers, has
    to follow.  ``missing`` counts the slots that the free list had no page for.
    ``out.shares`` may be ``shares``."""
    with _allocating_on(stream, page_table.device):
        call = PreparedPageFork(src_of, cache_lens, held_pages, page_table, shares, free_pages,
                                free_span, page_size, out)
        call.run(stream)
    return call.out


class PreparedPageRelease(_PreparedPoolCall):
    """mla_page_release with its arguments marshalled once; ``run()`` issues it and
    ``out`` holds its outputs.  The tensors must outlive the object."""

    def __init__(self, kept_lens, held_pages, page_table, shares, free_pages, free_span,
                 page_size: int, out: Optional[PageRelease] = None):
        _tensor("page_table", page_table, (None, None), torch.int32)
        _tensor("shares", shares, (None,), torch.int32)
        B, W = page_table.shape
        P = shares.numel()
        inputs = dict(kept_lens=(kept_lens, (B,)), held_pages=(held_pages, (B,)),
                      page_table=(page_table, (B, W)), shares=(shares, (P,)),
                      free_pages=(free_pages, (None,)), free_span=(free_span, (2,)))
        shapes = dict(held_pages=(B,), shares=(P,), free_span=(2,), released=(1,))
        dev, made = self._pool(PageRelease, inputs, shapes, out)
        args = [_ptr(kept_lens), _ptr(held_pages), B, _ptr(page_table), W, int(page_size), P,
                _ptr(shares), _ptr(free_pages), free_pages.numel(), _ptr(free_span),
                *[_ptr(t) for t in self.out]]
        self._prepare("mla_page_release", args, dev, (inputs, self.out), made)


def mla_page_release(kept_lens, held_pages, page_table, shares, free_pages, free_span,
                     page_size: int, out: Optional[PageRelease] = None,
                     stream=None) -> PageRelease:
    """Give back the pages behind each sequence's ``kept_lens[b]`` rows (0: the
    sequence ends), those that no other sequence holds to the free list.

    ``free_pages`` has room for every page (as many entries as ``shares``) and is
    written outside ``free_span``; ``page_table`` is only read.  ``out.held_pages``,
    ``out.shares`` and ``out.free_span`` are the next call's inputs;
    ``out.shares`` may be ``shares``.  A sequence cut back into a page that others
    hold must be forked and released before rows are appended to it: they would
    overwrite the others' rows, and no call notices."""
    with _allocating_on(stream, page_table.device):
        call = PreparedPageRelease(kept_lens, held_pages, page_table, shares, free_pages,
                                   free_span, page_size, out)
        call.run(stream)
    return call.out


class PreparedPageCompact(_PreparedPoolCall):
    """mla_page_compact with its arguments marshalled once; ``run()`` issues it and
    ``out`` holds its outputs.  The tensors must outlive the object.  It has one
    workspace, as PreparedDecodeAttention has."""

    def __init__(self, held_pages, page_table, shares, free_pages,
                 out: Optional[PageCompact] = None, workspace=None):
        _tensor("page_table", page_table, (None, None), torch.int32)
        _tensor("shares", shares, (None,), torch.int32)
        B, W = page_table.shape
        P = shares.numel()
        M = max(1, P // 2)
        inputs = dict(held_pages=(held_pages, (B,)), page_table=(page_table, (B, W)),
                      shares=(shares, (P,)), free_pages=(free_pages, (None,)))
        shapes = dict(page_table=(B, W), shares=(P,), free_span=(2,), move_src=(M,),
                      move_dst=(M,), moves=(1,))
        if workspace is not None:
            _tensor("workspace", workspace)
        dev, made = self._pool(PageCompact, inputs, shapes, out)
        _one_device(page_table=page_table, workspace=workspace)
        if workspace is None:
            nbytes = ctypes.c_size_t(0)
            _check(lib().mla_page_compact_workspace_bytes(P, ctypes.byref(nbytes)),
                   "mla_page_compact_workspace_bytes")
            workspace = new_workspace(nbytes.value, dev)
            made = tuple(made) + (workspace,)
        o = self.out
        args = [_ptr(held_pages), B, _ptr(page_table), W, P, _ptr(shares), _ptr(o.page_table),
                _ptr(o.shares), _ptr(free_pages), free_pages.numel(), _ptr(o.free_span),
                _ptr(o.move_src), _ptr(o.move_dst), _ptr(o.moves), _ptr(workspace),
                workspace.numel() * workspace.element_size()]
        self._prepare("mla_page_compact", args, dev, (inputs, o, workspace), made)


def mla_page_compact(held_pages, page_table, shares, free_pages,
                     out: Optional[PageCompact] = None, workspace=None,
                     stream=None) -> PageCompact:
    """Bring all held pages to the front of the pool: with L of them, those at or
    beyond L go to the free places below, and L .. num_pages - 1 are free.

    Every page in use must be in a table row.  ``mla_page_copy(caches,
    out.move_src, out.move_dst, out.moves)``, for the caches of all layers, has
    to follow; ``free_pages`` (as many entries as ``shares``) is rewritten.
    ``out.page_table`` may be ``page_table`` and ``out.shares`` ``shares``."""
    with _allocating_on(stream, page_table.device):
        call = PreparedPageCompact(held_pages, page_table, shares, free_pages, out, workspace)
        call.run(stream)
    return call.out


def _page_view(name: str, t: torch.Tensor) -> PageView:
    """A cache [pages, page, width] or [pages, page, heads, width] in any stride order."""
    if not isinstance(t, torch.Tensor) or t.dim() not in (3, 4):
        raise ValueError(f"{name} must be [pages, page, width] or [pages, page, heads, width]")
    if t.numel() == 0 or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must not be empty and its rows contiguous in their last "
                         "dimension")
    eb = t.element_size()
    strides = [t.stride(i) * eb if t.shape[i] > 1 else 0 for i in range(t.dim() - 1)]
    heads = t.shape[2] if t.dim() == 4 else 1
    return PageView(_ptr(t), strides[0], strides[1], strides[2] if t.dim() == 4 else 0, heads,
                    t.shape[-1] * eb)


class PreparedPageCopy(_PreparedCall):
    """mla_page_copy with its arguments marshalled once; ``run()`` issues it.  The
    tensors must outlive the object."""

    def __init__(self, caches, move_src, move_dst, moves=None, move_rows=None):
        caches = list(caches)
        if not caches:
            raise ValueError("caches must not be empty")
        views = (PageView * len(caches))(*[_page_view(f"caches[{i}]", t)
                                           for i, t in enumerate(caches)])
        pages, page = caches[0].shape[:2]
        for i, t in enumerate(caches):
            if tuple(t.shape[:2]) != (pages, page):
                raise ValueError(f"caches[{i}] must have caches[0]'s pages of as many rows")
        _tensor("move_src", move_src, (None,), torch.int32)
        n = move_src.numel()
        _tensor("move_dst", move_dst, (n,), torch.int32)
        if moves is not None:
            _tensor("moves", moves, (1,), torch.int32)
        if move_rows is not None:
            _tensor("move_rows", move_rows, (n,), torch.int32)
        dev = _one_device(move_src=move_src, move_dst=move_dst, moves=moves, move_rows=move_rows,
                          **{f"caches[{i}]": t for i, t in enumerate(caches)})
        args = [views, len(caches), page, pages, _ptr(move_src), _ptr(move_dst), _ptr(move_rows),
                _ptr(moves), n]
        keep = (views, caches, move_src, move_dst, moves, move_rows)
        self._prepare("mla_page_copy", args, dev, keep)


def mla_page_copy(caches, move_src, move_dst, moves=None, move_rows=None, stream=None) -> None:
    """Copy pages in every cache tensor of a list at once (keys and values, or
    latents and RoPE keys, of all layers; at most 128): the first
    ``move_rows[i]`` rows (None: all) of page ``move_src[i]`` to page
    ``move_dst[i]``, for i < ``moves[0]`` (None: all entries).

    Caches are [num_pages, page_size, width] or [num_pages, page_size, heads,
    width], of any type and stride order with contiguous last dimension.
    Destinations must be distinct, and none a source."""
    PreparedPageCopy(caches, move_src, move_dst, moves, move_rows).run(stream)
