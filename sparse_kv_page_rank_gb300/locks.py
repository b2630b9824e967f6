"""Thin ctypes binding of liblocks.so (argument marshalling only).

Every function here has the name of the C entry point it wraps and does
nothing but turn tensors into raw device pointers, fill the C structs and
check the returned status; all compute runs in the library's CUDA kernels.
Tensors are torch tensors (device memory, streams) or raw integer pointers.
The library must have been built (``sparse_kv_page_rank_gb300.build_lib``);
a missing library raises instead of falling back to anything else.
"""

from __future__ import annotations

import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_lib", "liblocks.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "locks.h")

LOCKS_OK = 0
LOCKS_ERR_INVALID_ARG = 1
LOCKS_ERR_UNSUPPORTED = 2
LOCKS_ERR_CUDA = 3
LOCKS_ERR_WORKSPACE = 4
LOCKS_ERR_DEVICE = 5
# bytes of the library-owned workspace behind locks_decode_step_static
LOCKS_STATIC_WS_BYTES = 8 << 20
LOCKS_DTYPE_BF16 = 0
LOCKS_DTYPE_F32 = 1
LOCKS_DTYPE_Q4 = 2
LOCKS_DTYPE_BF16_PACKED = 3
LOCKS_KV_BF16 = 0
LOCKS_KV_Q4 = 1
LOCKS_FLAG_UNFUSED = 0x1
LOCKS_FLAG_FUSED = 0x2


def q4_page_head_bytes(rank: int, page_size: int = 64) -> int:
    """Bytes of one page-head of a LOCKS_DTYPE_Q4 summary (LOCKS_Q4_BLOCK_BYTES)."""
    return (72 * rank + page_size * rank + 132 + 15) // 16 * 16


def kv_q4_block_bytes(page_size: int = 64) -> int:
    """Bytes of one page-head of a LOCKS_KV_Q4 cache (LOCKS_KV_Q4_BLOCK_BYTES)."""
    return 144 * page_size


LOCKS_DEVERR_BLOCK_TABLE = 0x1
LOCKS_DEVERR_SEL_PAGE = 0x2
LOCKS_DEVERR_LENGTHS = 0x4
LOCKS_DEVERR_PAGE_ID = 0x8
LOCKS_DEVERR_TIMEOUT = 0x10
LOCKS_DEVERR_POSITION = 0x20
LOCKSGEN_DEVERR_LOGITS = 0x40
LOCKSGEN_DEVERR_PARENT = 0x80
LOCKSGEN_MAX_BEAMS = 32
LOCKSGEN_MAX_KEEP = 64
LOCKSGEN_MAX_ROWS = 65535
LOCKSGEN_MAX_VOCAB = 1 << 22
LOCKSGEN_MAX_AXES = 4


class LocksError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


class locks_cache_t(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("n_summarized", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("pages_total", ctypes.c_int32),
                ("max_pages", ctypes.c_int32, 28), ("kv_format", ctypes.c_int32, 4)]


class locks_summary_t(ctypes.Structure):
    _fields_ = [("basis_t", ctypes.c_void_p), ("coeffs", ctypes.c_void_p),
                ("rank", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class locks_params_t(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("budget_tokens", ctypes.c_int32),
                ("scale", ctypes.c_float), ("flags", ctypes.c_int32)]


class lockskv_tokens_t(ctypes.Structure):
    _fields_ = [("cu_tokens", ctypes.c_void_p), ("total", ctypes.c_int32), ("max_tokens", ctypes.c_int32)]


class lockskv_append_t(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
                ("rope", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("q_stride", ctypes.c_int64), ("q_out_stride", ctypes.c_int64),
                ("num_q_heads", ctypes.c_int32), ("rope_rows", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class locksgen_axes_t(ctypes.Structure):
    _fields_ = [("positions", ctypes.c_void_p), ("axis_stride", ctypes.c_int64), ("num_axes", ctypes.c_int32),
                ("axis_of_pair", ctypes.c_uint8 * 64)]


class locksgen_choice_t(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("scores", ctypes.c_void_p), ("ended", ctypes.c_void_p),
                ("out_scores", ctypes.c_void_p), ("out_parents", ctypes.c_void_p), ("out_tokens", ctypes.c_void_p),
                ("out_ended", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("batch", ctypes.c_int32),
                ("beams", ctypes.c_int32), ("vocab", ctypes.c_int32), ("keep", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("end_token", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load liblocks.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"liblocks.so not built ({LIB_PATH}); run "
                               "python -m sparse_kv_page_rank_gb300.build_lib")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        C, S, R = P(locks_cache_t), P(locks_summary_t), P(locks_params_t)
        T, A, i64 = P(lockskv_tokens_t), P(lockskv_append_t), ctypes.c_int64
        sig = {
            "locks_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "locks_workspace_size": (ctypes.c_int, [C, S, R, P(sz)]),
            "locks_workspace_init": (ctypes.c_int, [vp, sz, vp]),
            "locks_build_summaries": (ctypes.c_int, [C, S, vp, i32, vp, sz, vp]),
            "locks_select": (ctypes.c_int, [C, S, R, vp, vp, vp, vp, vp, sz, vp]),
            "locks_page_scores": (ctypes.c_int, [C, S, R, vp, vp, vp, sz, vp]),
            "locks_sparse_attend": (ctypes.c_int, [C, R, vp, vp, vp, vp, vp, vp, sz, vp]),
            "locks_decode_step": (ctypes.c_int, [C, S, R, vp, vp, vp, vp, vp, vp, sz, vp]),
            "locks_decode_step_launches": (ctypes.c_int, [C, S, R, P(i32)]),
            "locks_dense_decode": (ctypes.c_int, [C, R, vp, vp, vp, vp, sz, vp]),
            "locks_exact_page_lse": (ctypes.c_int, [C, R, vp, vp, vp]),
            "locks_get_device_error": (ctypes.c_int, [vp, P(i32), vp]),
            "locks_decode_step_static": (ctypes.c_int, [C, S, R, vp, vp, vp, vp, vp, vp, vp]),
            "lockskv_append": (ctypes.c_int, [C, T, A, vp, sz, vp]),
            "lockskv_read": (ctypes.c_int, [C, T, vp, vp, vp, sz, vp]),
            "lockskv_prompt_workspace_size": (ctypes.c_int, [C, R, T, P(sz)]),
            "lockskv_prompt_attend": (ctypes.c_int, [C, R, T, vp, i64, vp, vp, vp, sz, vp]),
            "locksgen_append_axes": (ctypes.c_int, [C, T, A, P(locksgen_axes_t), vp, sz, vp]),
            "locksgen_select_workspace_size": (ctypes.c_int, [P(locksgen_choice_t), P(sz)]),
            "locksgen_select": (ctypes.c_int, [P(locksgen_choice_t), vp, sz, vp]),
            "locksgen_reorder_workspace_size": (ctypes.c_int, [C, i32, P(sz)]),
            "locksgen_reorder": (ctypes.c_int, [C, i32, i32, vp, vp, sz, vp]),
            "locksgen_attend_workspace_size": (ctypes.c_int, [C, R, i32, P(sz)]),
            "locksgen_attend": (ctypes.c_int, [C, R, i32, vp, vp, vp, vp, vp, sz, vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def declared_symbols() -> list[str]:
    """Entry points declared in include/locks.h."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"LOCKS_API\s+[\w\s\*]+?\b(locks_\w+)\s*\(", text)))


def status_string(status: int) -> str:
    return lib().locks_status_string(int(status)).decode()


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream, device: int | None = None) -> int | None:
    if stream is None:
        import torch
        # the current stream's handle without building a Stream object around it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if device is None else device)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, what: str):
    if status != LOCKS_OK:
        raise LocksError(status, what)


def make_cache(k_pool, v_pool, block_table, seq_lens, n_summarized=None, *, pages_total=None,
               num_kv_heads=None) -> locks_cache_t:
    """C struct for a paged cache given as tensors [pages_total][Hkv][P][d], or as
    4-bit blocks uint8 [pages_total][Hkv][kv_q4_block_bytes(P)] (v_pool None)."""
    fmt = LOCKS_KV_BF16
    if k_pool is not None and hasattr(k_pool, "shape"):
        if k_pool.dim() == 3:
            pt, hkv, nbytes = k_pool.shape
            P, d, fmt = nbytes // 144, 128, LOCKS_KV_Q4
            if nbytes != kv_q4_block_bytes(P):
                raise ValueError(f"{nbytes} bytes are no 4-bit block of whole tokens")
        else:
            pt, hkv, P, d = k_pool.shape
    else:
        pt, hkv, P, d = pages_total, num_kv_heads, 64, 128
    if block_table.shape[1] >= 1 << 27:  # beyond every limit, and more than the field holds
        raise LocksError(LOCKS_ERR_UNSUPPORTED, "make_cache")
    return locks_cache_t(_ptr(k_pool), _ptr(v_pool), _ptr(block_table), _ptr(seq_lens),
                         _ptr(n_summarized), int(block_table.shape[0]), int(hkv), int(d), int(P),
                         int(pt), int(block_table.shape[1]), fmt)


def make_tokens(cu_tokens, total: int, max_tokens: int) -> lockskv_tokens_t:
    """The newest tokens of a batch; cu_tokens None: one per sequence."""
    return lockskv_tokens_t(_ptr(cu_tokens), int(total), int(max_tokens))


_bf16 = None


def _row_stride(x, what: str) -> int:
    """Elements between the token rows of x [total][heads][128] (bf16, heads contiguous)."""
    global _bf16
    if _bf16 is None:
        import torch
        _bf16 = torch.bfloat16
    if x.dtype is not _bf16 or x.dim() != 3:
        raise ValueError(f"{what} must be bf16 [tokens][heads][128]")
    n, h, d = x.shape
    row, head, one = x.stride()
    if d != 128:
        raise ValueError(f"{what} must be bf16 [tokens][heads][128]")
    if one != 1 or (head != 128 and h > 1):
        raise ValueError(f"{what}: the heads of a token must be contiguous")
    return row if n > 1 else h * 128


def make_append(k, v, q=None, q_out=None, rope=None, rotary_dim: int = 0, positions=None,
                interleaved: bool = False) -> lockskv_append_t:
    """C struct of what lockskv_append writes, from tensors [total][heads][128]."""
    qs = qos = heads = rows = 0
    if q is not None:
        heads, qs, qos = q.shape[1], _row_stride(q, "q"), _row_stride(q_out, "q_out")
    if rope is not None:
        rows = rope.shape[0]
    return lockskv_append_t(k.data_ptr(), v.data_ptr(), _ptr(q), _ptr(q_out), _ptr(rope), _ptr(positions),
                            _row_stride(k, "k"), _row_stride(v, "v"), qs, qos, heads, rows, rotary_dim, interleaved)


def rope_axes(parts, cyclic: bool = False) -> list[int]:
    """The axis of each rotated pair when axis a has parts[a] of them.  The axes follow one
    another; or, ``cyclic``, they take turns: axis a > 0 has the pairs a, a + n, a + 2 n, ...
    (n axes) and axis 0 all others."""
    parts = [int(n) for n in parts]
    if not parts or min(parts) < 0:
        raise ValueError("an axis has a number of pairs")
    if not cyclic:
        return [a for a, n in enumerate(parts) for _ in range(n)]
    axes = [0] * sum(parts)
    for a in range(1, len(parts)):
        for i in range(parts[a]):
            if a + i * len(parts) >= len(axes):
                raise ValueError(f"axis {a} cannot take turns for {parts[a]} of {len(axes)} pairs")
            axes[a + i * len(parts)] = a
    return axes


def make_axes(axis_of_pair) -> locksgen_axes_t:
    """What ``LocksRuntime.append`` takes as ``axes``: the axis of each rotated pair
    (``rope_axes`` gives the usual ones).  The positions are set by the call."""
    axis_of_pair = [int(a) for a in axis_of_pair]
    if not 0 < len(axis_of_pair) <= 64 or min(axis_of_pair) < 0 or max(axis_of_pair) >= LOCKSGEN_MAX_AXES:
        raise ValueError(f"the axes of 1 to 64 pairs, each below {LOCKSGEN_MAX_AXES}")
    axes = locksgen_axes_t(None, 0, max(axis_of_pair) + 1, (ctypes.c_uint8 * 64)(*axis_of_pair))
    axes.pairs = len(axis_of_pair)
    return axes


def make_summary(basis_t, coeffs, rank: int, dtype: int = LOCKS_DTYPE_BF16) -> locks_summary_t:
    return locks_summary_t(_ptr(basis_t), _ptr(coeffs), int(rank), int(dtype))


def make_params(num_q_heads: int, budget_tokens: int, scale: float = 0.0, flags: int = 0) -> locks_params_t:
    return locks_params_t(int(num_q_heads), int(budget_tokens), float(scale), int(flags))


def locks_workspace_size(cache, summary, params) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().locks_workspace_size(ctypes.byref(cache), ctypes.byref(summary) if summary else None,
                                      ctypes.byref(params), ctypes.byref(n)), "locks_workspace_size")
    return int(n.value)


def locks_workspace_init(ws, nbytes: int, stream=None):
    _check(lib().locks_workspace_init(_ptr(ws), int(nbytes), _stream(stream)), "locks_workspace_init")


def locks_build_summaries(cache, summary, page_ids, n: int, ws=None, ws_bytes: int = 0, stream=None):
    _check(lib().locks_build_summaries(ctypes.byref(cache), ctypes.byref(summary), _ptr(page_ids), int(n),
                                       _ptr(ws), int(ws_bytes), _stream(stream)), "locks_build_summaries")


def locks_select(cache, summary, params, q, sel_pages, sel_count, page_lse, ws, ws_bytes: int, stream=None):
    _check(lib().locks_select(ctypes.byref(cache), ctypes.byref(summary), ctypes.byref(params), _ptr(q),
                              _ptr(sel_pages), _ptr(sel_count), _ptr(page_lse), _ptr(ws), int(ws_bytes),
                              _stream(stream)), "locks_select")


def locks_page_scores(cache, summary, params, q, page_lse, ws, ws_bytes: int, stream=None):
    _check(lib().locks_page_scores(ctypes.byref(cache), ctypes.byref(summary), ctypes.byref(params), _ptr(q),
                                   _ptr(page_lse), _ptr(ws), int(ws_bytes), _stream(stream)),
           "locks_page_scores")


def locks_sparse_attend(cache, params, q, sel_pages, sel_count, out, lse, ws, ws_bytes: int, stream=None):
    _check(lib().locks_sparse_attend(ctypes.byref(cache), ctypes.byref(params), _ptr(q), _ptr(sel_pages),
                                     _ptr(sel_count), _ptr(out), _ptr(lse), _ptr(ws), int(ws_bytes),
                                     _stream(stream)), "locks_sparse_attend")


def locks_decode_step(cache, summary, params, q, out, lse, sel_pages, sel_count, ws, ws_bytes: int,
                      stream=None):
    _check(lib().locks_decode_step(ctypes.byref(cache), ctypes.byref(summary), ctypes.byref(params), _ptr(q),
                                   _ptr(out), _ptr(lse), _ptr(sel_pages), _ptr(sel_count), _ptr(ws),
                                   int(ws_bytes), _stream(stream)), "locks_decode_step")


def locks_decode_step_static(cache, summary, params, q, out, lse, sel_pages=None, sel_count=None,
                             device_error=None, stream=None):
    """locks_decode_step in the library's own fixed device workspace (no
    workspace argument; for callers that cannot allocate device memory)."""
    _check(lib().locks_decode_step_static(ctypes.byref(cache), ctypes.byref(summary), ctypes.byref(params),
                                          _ptr(q), _ptr(out), _ptr(lse), _ptr(sel_pages), _ptr(sel_count),
                                          _ptr(device_error), _stream(stream)), "locks_decode_step_static")


def locks_decode_step_launches(cache, summary, params) -> int:
    n = ctypes.c_int32(0)
    _check(lib().locks_decode_step_launches(ctypes.byref(cache), ctypes.byref(summary), ctypes.byref(params),
                                            ctypes.byref(n)), "locks_decode_step_launches")
    return n.value


def locks_dense_decode(cache, params, q, out, lse, ws, ws_bytes: int, stream=None):
    _check(lib().locks_dense_decode(ctypes.byref(cache), ctypes.byref(params), _ptr(q), _ptr(out), _ptr(lse),
                                    _ptr(ws), int(ws_bytes), _stream(stream)), "locks_dense_decode")


def locks_exact_page_lse(cache, params, q, page_lse, stream=None):
    _check(lib().locks_exact_page_lse(ctypes.byref(cache), ctypes.byref(params), _ptr(q), _ptr(page_lse),
                                      _stream(stream)), "locks_exact_page_lse")


def locks_get_device_error(ws, stream=None) -> int:
    """Returns the device error bits (0 = none) and clears them."""
    code = ctypes.c_int32(0)
    st = lib().locks_get_device_error(_ptr(ws), ctypes.byref(code), _stream(stream))
    if st not in (LOCKS_OK, LOCKS_ERR_DEVICE):
        raise LocksError(st, "locks_get_device_error")
    return int(code.value)


def lockskv_append(cache, tokens, append, ws=None, ws_bytes: int = 0, stream=None):
    _check(lib().lockskv_append(ctypes.byref(cache), ctypes.byref(tokens), ctypes.byref(append), _ptr(ws),
                                int(ws_bytes), _stream(stream)), "lockskv_append")


def lockskv_read(cache, tokens, k_out, v_out, ws=None, ws_bytes: int = 0, stream=None):
    _check(lib().lockskv_read(ctypes.byref(cache), ctypes.byref(tokens), _ptr(k_out), _ptr(v_out), _ptr(ws),
                              int(ws_bytes), _stream(stream)), "lockskv_read")


def lockskv_prompt_workspace_size(cache, params, tokens) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().lockskv_prompt_workspace_size(ctypes.byref(cache), ctypes.byref(params), ctypes.byref(tokens),
                                               ctypes.byref(n)), "lockskv_prompt_workspace_size")
    return int(n.value)


def lockskv_prompt_attend(cache, params, tokens, q, q_stride: int, out, lse, ws, ws_bytes: int, stream=None):
    _check(lib().lockskv_prompt_attend(ctypes.byref(cache), ctypes.byref(params), ctypes.byref(tokens), _ptr(q),
                                       int(q_stride), _ptr(out), _ptr(lse), _ptr(ws), int(ws_bytes),
                                       _stream(stream)), "lockskv_prompt_attend")


def locksgen_append_axes(cache, tokens, append, axes, ws=None, ws_bytes: int = 0, stream=None):
    _check(lib().locksgen_append_axes(ctypes.byref(cache), ctypes.byref(tokens), ctypes.byref(append), ctypes.byref(axes),
                                      _ptr(ws), int(ws_bytes), _stream(stream)), "locksgen_append_axes")


def locksgen_select_workspace_size(choice) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().locksgen_select_workspace_size(ctypes.byref(choice), ctypes.byref(n)), "locksgen_select_workspace_size")
    return int(n.value)


def locksgen_select(choice, ws, ws_bytes: int, stream=None):
    _check(lib().locksgen_select(ctypes.byref(choice), _ptr(ws), int(ws_bytes), _stream(stream)), "locksgen_select")


def locksgen_reorder_workspace_size(cache, beams: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().locksgen_reorder_workspace_size(ctypes.byref(cache), int(beams), ctypes.byref(n)),
           "locksgen_reorder_workspace_size")
    return int(n.value)


def locksgen_reorder(caches, num_caches: int, beams: int, parents, ws, ws_bytes: int, stream=None):
    """caches: a ctypes array of num_caches locks_cache_t."""
    _check(lib().locksgen_reorder(caches, int(num_caches), int(beams), _ptr(parents), _ptr(ws), int(ws_bytes),
                                  _stream(stream)), "locksgen_reorder")


def locksgen_attend_workspace_size(cache, params, beams: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().locksgen_attend_workspace_size(ctypes.byref(cache), ctypes.byref(params), int(beams), ctypes.byref(n)),
           "locksgen_attend_workspace_size")
    return int(n.value)


def locksgen_attend(cache, params, beams: int, shared_pages, q, out, lse, ws, ws_bytes: int, stream=None):
    _check(lib().locksgen_attend(ctypes.byref(cache), ctypes.byref(params), int(beams), _ptr(shared_pages), _ptr(q),
                                 _ptr(out), _ptr(lse), _ptr(ws), int(ws_bytes), _stream(stream)), "locksgen_attend")
