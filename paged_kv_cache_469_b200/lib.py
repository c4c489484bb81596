"""Python binding of libpa.so: argument marshalling only (ctypes; the module
``_binding`` for the calls that a decode step makes many times).

Every call forwards torch tensors' device pointers and the current CUDA
stream to the C ABI declared in ``include/pa.h``; every step of the
computation runs in the library's CUDA kernels.  There is no fallback: if
the library is missing or a call fails, an exception says so.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpa.so")

PA_OK, PA_ERR_INVALID, PA_ERR_UNSUPPORTED, PA_ERR_CUDA = 0, -1, -2, -3
PA_DTYPE_F32, PA_DTYPE_BF16 = 0, 1

# every symbol include/pa.h declares
EXPORTS = ("pa_status_string", "pa_reshape_and_cache", "pa_attention_workspace_size",
           "pa_workspace_init", "pa_workspace_status", "pa_attention_varlen",
           "pa_attention_varlen_write_cache", "pa_attention_varlen_static_scratch",
           "pa_plan_step", "pa_rope_append", "pa_rope_append_fp4", "pa_gather_fp4",
           "pa_attention_fp4_workspace_size", "pa_attention_varlen_fp4")

_lib = None


class PAError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {library().pa_status_string(status).decode()} ({status})")
        self.status = status


def library() -> ctypes.CDLL:
    """Load libpa.so (built in-tree by ``paged_kv_cache_469_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m paged_kv_cache_469_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        c_int, c_p, c_sz, c_f = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
        lib.pa_status_string.restype = ctypes.c_char_p
        lib.pa_status_string.argtypes = [c_int]
        lib.pa_reshape_and_cache.restype = c_int
        lib.pa_reshape_and_cache.argtypes = [c_p, c_p, c_p, c_p, c_p, c_int, c_int, c_int, c_int,
                                             c_int, c_int, c_p]
        lib.pa_attention_workspace_size.restype = c_sz
        lib.pa_attention_workspace_size.argtypes = [c_int, c_int, c_int, c_int, c_int]
        lib.pa_workspace_status.restype = c_int
        lib.pa_workspace_status.argtypes = [c_p, c_sz, c_p, c_p]
        lib.pa_workspace_init.restype = c_int
        lib.pa_workspace_init.argtypes = [c_p, c_sz, c_p]
        lib.pa_attention_varlen.restype = c_int
        lib.pa_attention_varlen.argtypes = [c_p, c_p, c_p, c_p, c_p, c_int, c_p, c_p, c_int,
                                            c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                            c_int, c_f, c_int, c_p, c_sz, c_p, c_p, c_p]
        lib.pa_attention_varlen_write_cache.restype = c_int
        lib.pa_attention_varlen_write_cache.argtypes = [
            c_p, c_p, c_p, c_p, c_p, c_p, c_p, c_p, c_int, c_p, c_p, c_int, c_int, c_int, c_int,
            c_int, c_int, c_int, c_int, c_int, c_f, c_int, c_p, c_sz, c_p, c_p, c_p]
        lib.pa_plan_step.restype = c_int
        lib.pa_plan_step.argtypes = [c_p, c_int, c_p, c_p, c_p, c_int, c_p, c_int, c_int, c_p,
                                     c_p, c_p, c_int, c_p]
        c_i64 = ctypes.c_int64
        lib.pa_rope_append.restype = c_int
        lib.pa_rope_append.argtypes = [c_p, c_p, c_i64, c_p, c_i64, c_p, c_i64, c_p, c_p, c_p,
                                       c_p, c_p, c_i64, c_int, c_int, c_int, c_int, c_int, c_int,
                                       c_int, c_int, c_int, c_p]
        lib.pa_rope_append_fp4.restype = c_int
        lib.pa_rope_append_fp4.argtypes = [c_p, c_p, c_i64, c_p, c_i64, c_p, c_i64, c_p, c_f, c_f,
                                           c_p, c_p, c_p, c_i64, c_int, c_int, c_int, c_int,
                                           c_int, c_int, c_int, c_int, c_int, c_p]
        lib.pa_gather_fp4.restype = c_int
        lib.pa_gather_fp4.argtypes = [c_p, c_p, c_p, c_f, c_f, c_p, c_int, c_int, c_int, c_int,
                                      c_int, c_int, c_p]
        lib.pa_attention_fp4_workspace_size.restype = c_sz
        lib.pa_attention_fp4_workspace_size.argtypes = [c_int, c_int, c_int, c_int, c_int]
        lib.pa_attention_varlen_fp4.restype = c_int
        lib.pa_attention_varlen_fp4.argtypes = [c_p, c_p, c_p, c_f, c_f, c_p, c_int, c_p, c_p,
                                                c_int, c_int, c_int, c_int, c_int, c_int, c_int,
                                                c_int, c_int, c_f, c_int, c_p, c_sz, c_p, c_p,
                                                c_p]
        _lib = lib
    return _lib


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return PA_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return PA_DTYPE_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _dev(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return t.data_ptr()


def _stream(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _host_i32(a):
    """(pointer, keep-alive) of an optional host int32 array."""
    if a is None:
        return None, None
    if isinstance(a, torch.Tensor):
        a = a.cpu().numpy()
    import numpy as np
    arr = np.ascontiguousarray(a, dtype=np.int32)
    return arr.ctypes.data, arr


def reshape_and_cache(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, slot_mapping: torch.Tensor, stream=None) -> None:
    """k, v: [T, Hkv, D]; caches: [num_blocks, Hkv, 16, D]; slot_mapping: int64 [T]."""
    num_blocks, hkv, bs, d = k_cache.shape
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    rc = library().pa_reshape_and_cache(
        _dev(k, "k"), _dev(v, "v"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        _dev(slot_mapping, "slot_mapping"), k.shape[0], hkv, d, bs, num_blocks, _dtype_code(k),
        _stream(stream))
    if rc != PA_OK:
        raise PAError(rc, "pa_reshape_and_cache")


def attention_workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                             max_seq_len: int) -> int:
    return int(library().pa_attention_workspace_size(num_seqs, num_q_heads, num_kv_heads,
                                                     head_dim, max_seq_len))


def new_workspace(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                  max_seq_len: int, device="cuda", stream=None) -> torch.Tensor:
    """A zeroed workspace (uint8 CUDA tensor) sized for steps up to these bounds."""
    n = attention_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_seq_len)
    if n == 0:
        raise ValueError("invalid workspace bounds")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    rc = library().pa_workspace_init(ws.data_ptr(), n, _stream(stream))
    if rc != PA_OK:
        raise PAError(rc, "pa_workspace_init")
    return ws


def workspace_status(workspace: torch.Tensor, stream=None) -> int:
    """Status word of a workspace (0 = every kernel so far ran to completion)."""
    out = ctypes.c_int(0)
    rc = library().pa_workspace_status(_dev(workspace, "workspace"), workspace.numel(),
                                       ctypes.addressof(out), _stream(stream))
    if rc != PA_OK:
        raise PAError(rc, "pa_workspace_status")
    return int(out.value)


def attention_varlen(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                     query_start_loc: torch.Tensor, *, max_query_len: int, max_seq_len: int,
                     scale: float, workspace: torch.Tensor | None, seq_lens_host=None,
                     query_start_loc_host=None, stream=None) -> torch.Tensor:
    """Paged attention over one flattened step (see pa_attention_varlen in pa.h)."""
    num_blocks, hkv, bs, d = k_cache.shape
    t, hq, _ = q.shape
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32 or \
            query_start_loc.dtype != torch.int32:
        raise TypeError("block_tables, seq_lens and query_start_loc must be int32")
    sl_ptr, sl_keep = _host_i32(seq_lens_host)
    qs_ptr, qs_keep = _host_i32(query_start_loc_host)
    ws_ptr, ws_n = (0, 0) if workspace is None else (_dev(workspace, "workspace"),
                                                     workspace.numel() * workspace.element_size())
    rc = library().pa_attention_varlen(
        _dev(out, "out"), _dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        _dev(block_tables, "block_tables"), block_tables.shape[1], _dev(seq_lens, "seq_lens"),
        _dev(query_start_loc, "query_start_loc"), seq_lens.shape[0], t, max_query_len,
        max_seq_len, hq, hkv, d, bs, num_blocks, float(scale), _dtype_code(q), ws_ptr, ws_n,
        sl_ptr, qs_ptr, _stream(stream))
    del sl_keep, qs_keep
    if rc != PA_OK:
        raise PAError(rc, "pa_attention_varlen")
    return out


def attention_varlen_write_cache(out: torch.Tensor, q: torch.Tensor, k_new: torch.Tensor,
                                 v_new: torch.Tensor, k_cache: torch.Tensor,
                                 v_cache: torch.Tensor, slot_mapping: torch.Tensor,
                                 block_tables: torch.Tensor, seq_lens: torch.Tensor,
                                 query_start_loc: torch.Tensor, *, max_query_len: int,
                                 max_seq_len: int, scale: float, workspace: torch.Tensor | None,
                                 seq_lens_host=None, query_start_loc_host=None,
                                 stream=None) -> torch.Tensor:
    """The step's cache write and attention in one call (see
    pa_attention_varlen_write_cache in pa.h)."""
    num_blocks, hkv, bs, d = k_cache.shape
    t, hq, _ = q.shape
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32 or \
            query_start_loc.dtype != torch.int32:
        raise TypeError("block_tables, seq_lens and query_start_loc must be int32")
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    sl_ptr, sl_keep = _host_i32(seq_lens_host)
    qs_ptr, qs_keep = _host_i32(query_start_loc_host)
    ws_ptr, ws_n = (0, 0) if workspace is None else (_dev(workspace, "workspace"),
                                                     workspace.numel() * workspace.element_size())
    rc = library().pa_attention_varlen_write_cache(
        _dev(out, "out"), _dev(q, "q"), _dev(k_new, "k_new"), _dev(v_new, "v_new"),
        _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"), _dev(slot_mapping, "slot_mapping"),
        _dev(block_tables, "block_tables"), block_tables.shape[1], _dev(seq_lens, "seq_lens"),
        _dev(query_start_loc, "query_start_loc"), seq_lens.shape[0], t, max_query_len,
        max_seq_len, hq, hkv, d, bs, num_blocks, float(scale), _dtype_code(q), ws_ptr, ws_n,
        sl_ptr, qs_ptr, _stream(stream))
    del sl_keep, qs_keep
    if rc != PA_OK:
        raise PAError(rc, "pa_attention_varlen_write_cache")
    return out


# bits of planner_state[1] (see pa_plan_step in pa.h)
PLAN_POOL_EMPTY, PLAN_ROW_FULL, PLAN_SLOTS_FULL, PLAN_BAD_LENGTH, PLAN_BAD_HEAD = 1, 2, 4, 8, 16


def new_planner_state(queue_head: int = 0, device="cuda") -> torch.Tensor:
    """int32[4] planner state: queue head, status bits, two words the call uses."""
    st = torch.zeros(4, dtype=torch.int32, device=device)
    st[0] = queue_head
    return st


def plan_step(free_queue: torch.Tensor, planner_state: torch.Tensor,
              num_computed: torch.Tensor, query_lens: torch.Tensor, block_tables: torch.Tensor,
              seq_lens: torch.Tensor, query_start_loc: torch.Tensor,
              slot_mapping: torch.Tensor, block_size: int = 16, stream=None) -> None:
    """Block allocation, seq_lens, query_start_loc and slot mapping of one step on
    the GPU (see pa_plan_step in pa.h); errors land in planner_state[1]."""
    for name, t in (("free_queue", free_queue), ("planner_state", planner_state),
                    ("num_computed", num_computed), ("query_lens", query_lens),
                    ("block_tables", block_tables), ("seq_lens", seq_lens),
                    ("query_start_loc", query_start_loc)):
        if t.dtype != torch.int32:
            raise TypeError(f"{name} must be int32")
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    num_seqs = query_lens.shape[0]
    if num_computed.shape[0] != num_seqs or seq_lens.shape[0] != num_seqs or \
            query_start_loc.shape[0] != num_seqs + 1 or block_tables.shape[0] != num_seqs or \
            planner_state.numel() != 4:
        raise ValueError("plan_step: inconsistent sizes")
    rc = library().pa_plan_step(
        _dev(free_queue, "free_queue"), free_queue.numel(), _dev(planner_state, "planner_state"),
        _dev(num_computed, "num_computed"), _dev(query_lens, "query_lens"), num_seqs,
        _dev(block_tables, "block_tables"), block_tables.shape[1], block_size,
        _dev(seq_lens, "seq_lens"), _dev(query_start_loc, "query_start_loc"),
        _dev(slot_mapping, "slot_mapping"), slot_mapping.numel(), _stream(stream))
    if rc != PA_OK:
        raise PAError(rc, "pa_plan_step")


_native = None


def _marshal():
    """The module ``_binding`` (built in-tree like the library), bound to the library."""
    global _native
    if _native is None:
        library()
        try:
            from . import _binding
        except ImportError as e:
            raise RuntimeError(f"the module _binding is missing ({e}): build it with "
                               "`python -m paged_kv_cache_469_b200.build`") from e
        _binding.load(LIB_PATH)
        _native = _binding
    return _native


def rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                v_cache: torch.Tensor, slot_mapping: torch.Tensor,
                positions: torch.Tensor | None, cos_sin: torch.Tensor | None, *,
                q_out: torch.Tensor | None = None, interleaved: bool = False,
                stream=None) -> torch.Tensor:
    """Queries and keys rotated to their positions, keys and values stored in their
    slots, in one launch (see pa_rope_append in pa.h).

    q: [T, Hq, D], k, v: [T, Hkv, D], each row contiguous (slices of a fused
    projection are fine); caches: [num_blocks, Hkv, 16, D]; slot_mapping,
    positions: int64 [T]; cos_sin: float32 [max_position, rotary_dim], the
    cosines and then the sines of a position's angles (None: nothing is
    rotated).  Returns q_out (a new tensor unless given, one of ``stream``: what
    is made by a call belongs to the stream that writes it)."""
    if q_out is None:
        with torch.cuda.stream(stream):
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    rc = _marshal().rope_append(q, k, v, k_cache, v_cache, slot_mapping, positions, cos_sin, q_out,
                                interleaved, None if stream is None else stream.cuda_stream)
    if rc != PA_OK:
        raise PAError(rc, "pa_rope_append")
    return q_out


def new_fp4_cache(num_blocks: int, num_kv_heads: int, head_dim: int,
                  device="cuda") -> torch.Tensor:
    """A zeroed 4-bit cache: uint8 [num_blocks, num_kv_heads, 18 * head_dim], K and
    V of 16 tokens of one kv-head per tile (the layout is in pa.h)."""
    return torch.zeros(num_blocks, num_kv_heads, 18 * head_dim, dtype=torch.uint8, device=device)


def rope_append_fp4(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kv_cache: torch.Tensor,
                    slot_mapping: torch.Tensor, positions: torch.Tensor | None,
                    cos_sin: torch.Tensor | None, *, k_scale: float = 1.0, v_scale: float = 1.0,
                    q_out: torch.Tensor | None = None, interleaved: bool = False,
                    stream=None) -> torch.Tensor:
    """``rope_append`` into a 4-bit cache (see pa_rope_append_fp4 in pa.h); k_scale and
    v_scale are the tensors' own scales."""
    if q_out is None:
        with torch.cuda.stream(stream):
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    rc = _marshal().rope_append_fp4(q, k, v, kv_cache, k_scale, v_scale, slot_mapping, positions,
                                    cos_sin, q_out, interleaved,
                                    None if stream is None else stream.cuda_stream)
    if rc != PA_OK:
        raise PAError(rc, "pa_rope_append_fp4")
    return q_out


def gather_fp4(kv_cache: torch.Tensor, slots: torch.Tensor, *, k_scale: float = 1.0,
               v_scale: float = 1.0, dtype=torch.bfloat16, k_out: torch.Tensor | None = None,
               v_out: torch.Tensor | None = None, stream=None):
    """K and V values ([n, Hkv, D] each, of ``dtype`` unless one is given) of the slots
    (int64 [n]) of a 4-bit cache; rows of slots outside the pool are left as they are
    (see pa_gather_fp4 in pa.h)."""
    if k_out is None or v_out is None:
        shape = (slots.shape[0], kv_cache.shape[1], kv_cache.shape[2] // 18)
        with torch.cuda.stream(stream):  # the fills come before the gather
            if k_out is None:
                k_out = torch.zeros(shape, dtype=dtype if v_out is None else v_out.dtype,
                                    device=kv_cache.device)
            if v_out is None:
                v_out = torch.zeros(shape, dtype=k_out.dtype, device=kv_cache.device)
    rc = _marshal().gather_fp4(kv_cache, slots, k_scale, v_scale, k_out, v_out,
                               None if stream is None else stream.cuda_stream)
    if rc != PA_OK:
        raise PAError(rc, "pa_gather_fp4")
    return k_out, v_out


def new_fp4_workspace(num_seqs: int, num_tokens: int, num_q_heads: int, num_kv_heads: int,
                      head_dim: int, device="cuda", stream=None) -> torch.Tensor:
    """A zeroed workspace of ``attention_varlen_fp4`` for steps up to these sizes."""
    n = int(library().pa_attention_fp4_workspace_size(num_seqs, num_tokens, num_q_heads,
                                                      num_kv_heads, head_dim))
    if n == 0:
        raise ValueError("invalid workspace bounds")
    with torch.cuda.stream(stream):
        ws = torch.empty(n, dtype=torch.uint8, device=device)
    if not ws.is_cuda:
        raise ValueError("the workspace must be on a CUDA device")
    with torch.cuda.device(ws.device):
        rc = library().pa_workspace_init(ws.data_ptr(), n, _stream(stream))
    if rc != PA_OK:
        raise PAError(rc, "pa_workspace_init")
    return ws


def _host_lengths(a, n: int):
    """(address, keep-alive) of n host lengths, or (0, None)."""
    if a is None:
        return 0, None
    if isinstance(a, torch.Tensor):
        a = a.cpu().numpy()
    if not (isinstance(a, np.ndarray) and a.dtype == np.int32 and a.flags.c_contiguous):
        a = np.ascontiguousarray(a, dtype=np.int32)
    if a.shape != (n,):
        raise ValueError("a host copy's size does not fit")
    return a.__array_interface__["data"][0], a


def attention_varlen_fp4(out: torch.Tensor, q: torch.Tensor, kv_cache: torch.Tensor,
                         block_tables: torch.Tensor, seq_lens: torch.Tensor,
                         query_start_loc: torch.Tensor, *, max_query_len: int, max_seq_len: int,
                         scale: float, workspace: torch.Tensor, k_scale: float = 1.0,
                         v_scale: float = 1.0, seq_lens_host=None, query_start_loc_host=None,
                         stream=None) -> torch.Tensor:
    """Paged attention of one flattened step over a 4-bit cache (see
    pa_attention_varlen_fp4 in pa.h)."""
    s = seq_lens.shape[0]
    sl_ptr, sl_keep = _host_lengths(seq_lens_host, s)
    qs_ptr, qs_keep = _host_lengths(query_start_loc_host, s + 1)
    rc = _marshal().attention_varlen_fp4(
        out, q, kv_cache, k_scale, v_scale, block_tables, seq_lens, query_start_loc,
        max_query_len, max_seq_len, scale, workspace, sl_ptr, qs_ptr,
        None if stream is None else stream.cuda_stream)
    del sl_keep, qs_keep
    if rc != PA_OK:
        raise PAError(rc, "pa_attention_varlen_fp4")
    return out
