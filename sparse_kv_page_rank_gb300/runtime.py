"""Device-side state of one paged cache for PyTorch callers.

``LocksRuntime`` owns the torch tensors the C ABI reads (pools, block table,
lengths, summaries, workspace), the C structs that point at them, and thin
methods that call the entry points of ``locks``.  It computes nothing itself.
"""

from __future__ import annotations

import torch

from . import locks as L


class LocksRuntime:
    """Holds a paged cache on ``device`` and calls liblocks.so on it.

    k_pool, v_pool: bf16 [pages_total][Hkv][P][128] with P = 64 or 16; or, for
    a cache held in 4 bits (LOCKS_KV_Q4), k_pool uint8 [pages_total][Hkv]
    [kv_q4_block_bytes(P)] and v_pool None.
    block_table int32 [B][max_pages]; seq_lens, n_summarized int32 [B].
    Summaries are allocated here.  bf16: one LOCKS_DTYPE_BF16_PACKED block per
    page-head (basis rows, then coefficients), with ``basis_t`` [pages_total]
    [Hkv][rank][128] and ``coeffs`` [..][P][rank] as views into it; with
    ``split`` two separate LOCKS_DTYPE_BF16 arrays of those shapes instead.
    With ``quantized``: one LOCKS_DTYPE_Q4 block per page-head (uint8
    [pages_total][Hkv][q4_page_head_bytes(rank, P)]).
    ``form``: "auto" (the library's choice: three kernels), or "unfused" /
    "fused" for LOCKS_FLAG_UNFUSED / LOCKS_FLAG_FUSED (the decode step as three
    kernels, or as two wherever the size limits allow).

    One workspace serves all decode calls and one all prompt attention: the
    caller orders calls of a kind that are on different streams, and replays of
    graphs that hold them (an event between them, or a LocksRuntime over the
    same tensors for each).
    """

    def __init__(self, k_pool: torch.Tensor, v_pool: torch.Tensor | None, block_table: torch.Tensor,
                 seq_lens: torch.Tensor, n_summarized: torch.Tensor, num_q_heads: int, rank: int,
                 budget_tokens: int, scale: float = 0.0, quantized: bool = False, form: str = "auto",
                 split: bool = False):
        if v_pool is None:
            assert k_pool.dtype == torch.uint8 and k_pool.dim() == 3 and k_pool.is_contiguous()
        else:
            assert k_pool.dtype == torch.bfloat16 and v_pool.dtype == torch.bfloat16
        assert block_table.dtype == torch.int32 and seq_lens.dtype == torch.int32
        self.device = k_pool.device
        self._index = k_pool.get_device()
        self.k_pool, self.v_pool = k_pool, v_pool
        self.block_table, self.seq_lens = block_table, seq_lens
        self.n_summarized = n_summarized.to(torch.int32)
        self.cache = L.make_cache(k_pool, v_pool, block_table, seq_lens, self.n_summarized)
        pt, hkv, P, d = self.cache.pages_total, self.cache.num_kv_heads, self.cache.page_size, self.cache.head_dim
        self.page_size = P
        self.batch = block_table.shape[0]
        self.num_kv_heads, self.num_q_heads = hkv, num_q_heads
        self.rank = rank
        self.quantized = quantized
        if quantized:
            self.basis_t = torch.zeros((pt, hkv, L.q4_page_head_bytes(rank, P)), dtype=torch.uint8,
                                       device=self.device)
            self.coeffs = None
            self.summary = L.make_summary(self.basis_t, None, rank, L.LOCKS_DTYPE_Q4)
        elif split:
            self.basis_t = torch.zeros((pt, hkv, rank, d), dtype=torch.bfloat16, device=self.device)
            self.coeffs = torch.zeros((pt, hkv, P, rank), dtype=torch.bfloat16, device=self.device)
            self.summary = L.make_summary(self.basis_t, self.coeffs, rank, L.LOCKS_DTYPE_BF16)
        else:
            self.blocks = torch.zeros((pt, hkv, rank * d + P * rank), dtype=torch.bfloat16, device=self.device)
            self.basis_t = self.blocks[:, :, :rank * d].unflatten(-1, (rank, d))
            self.coeffs = self.blocks[:, :, rank * d:].unflatten(-1, (P, rank))
            self.summary = L.make_summary(self.blocks, None, rank, L.LOCKS_DTYPE_BF16_PACKED)
        flags = {"auto": 0, "unfused": L.LOCKS_FLAG_UNFUSED, "fused": L.LOCKS_FLAG_FUSED}[form]
        self.params = L.make_params(num_q_heads, budget_tokens, scale, flags)
        self.k_max = min(budget_tokens // P, block_table.shape[1])
        self.ws_bytes = L.locks_workspace_size(self.cache, self.summary, self.params)
        self.ws = torch.empty(self.ws_bytes + 256, dtype=torch.uint8, device=self.device)
        off = (-self.ws.data_ptr()) % 256
        self.ws = self.ws[off:off + self.ws_bytes]
        L.locks_workspace_init(self.ws, self.ws_bytes)
        # the builder's own error word, so that builds may run on another
        # stream beside calls that use the main workspace
        self.build_ws = torch.zeros(512, dtype=torch.uint8, device=self.device)
        off = (-self.build_ws.data_ptr()) % 256
        self.build_ws = self.build_ws[off:off + 256]
        # the error word of the calls that write and read tokens, and the prompt
        # attention's workspace (grown to the largest call seen)
        self.kv_ws = torch.zeros(512, dtype=torch.uint8, device=self.device)
        off = (-self.kv_ws.data_ptr()) % 256
        self.kv_ws = self.kv_ws[off:off + 256]
        self.prompt_ws = None
        self._prompt_need = {}     # bytes by max_tokens
        self._prompt_captured = False
        self._prompt_held = []     # outgrown workspaces that a captured graph may still use
        B = self.batch
        self.sel_pages = torch.zeros((B, hkv, max(self.k_max, 1)), dtype=torch.int32, device=self.device)
        self.sel_count = torch.zeros((B, hkv), dtype=torch.int32, device=self.device)
        self.out = torch.zeros((B, num_q_heads, d), dtype=torch.bfloat16, device=self.device)
        self.lse = torch.zeros((B, num_q_heads), dtype=torch.float32, device=self.device)

    def set_summaries(self, basis_t: torch.Tensor, coeffs: torch.Tensor | None):
        """Install externally computed summaries (same layouts; coeffs is
        None for the quantised format)."""
        self.basis_t.copy_(basis_t)
        if self.coeffs is not None:
            self.coeffs.copy_(coeffs)

    def build_summaries(self, page_ids: torch.Tensor, stream=None):
        ids = page_ids.to(device=self.device, dtype=torch.int32).contiguous()
        L.locks_build_summaries(self.cache, self.summary, ids, ids.numel(), self.build_ws, 256, stream)

    def select(self, q: torch.Tensor, page_lse: torch.Tensor | None = None, stream=None):
        L.locks_select(self.cache, self.summary, self.params, q, self.sel_pages, self.sel_count, page_lse,
                       self.ws, self.ws_bytes, stream)
        return self.sel_pages, self.sel_count

    def page_scores(self, q: torch.Tensor, page_lse: torch.Tensor, stream=None):
        L.locks_page_scores(self.cache, self.summary, self.params, q, page_lse, self.ws, self.ws_bytes, stream)
        return page_lse

    def sparse_attend(self, q: torch.Tensor, stream=None):
        L.locks_sparse_attend(self.cache, self.params, q, self.sel_pages, self.sel_count, self.out, self.lse,
                              self.ws, self.ws_bytes, stream)
        return self.out, self.lse

    def decode_step(self, q: torch.Tensor, out=None, lse=None, keep_selection: bool = True, stream=None):
        out = self.out if out is None else out
        lse = self.lse if lse is None else lse
        sp, sc = (self.sel_pages, self.sel_count) if keep_selection else (None, None)
        L.locks_decode_step(self.cache, self.summary, self.params, q, out, lse, sp, sc, self.ws,
                            self.ws_bytes, stream)
        return out, lse

    def decode_step_launches(self) -> int:
        """Kernels one decode_step launches for this cache's shapes (2 or 3)."""
        return L.locks_decode_step_launches(self.cache, self.summary, self.params)

    def dense_decode(self, q: torch.Tensor, out=None, lse=None, stream=None):
        out = self.out if out is None else out
        lse = self.lse if lse is None else lse
        L.locks_dense_decode(self.cache, self.params, q, out, lse, self.ws, self.ws_bytes, stream)
        return out, lse

    def exact_page_lse(self, q: torch.Tensor, stream=None) -> torch.Tensor:
        pl = torch.full((self.batch, self.num_q_heads, self.block_table.shape[1]), float("nan"),
                        dtype=torch.float32, device=self.device)
        L.locks_exact_page_lse(self.cache, self.params, q, pl, stream)
        return pl

    def _new(self, shape, dtype, stream):
        """An output of a call on `stream`, whose memory belongs to that stream."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with self._on(stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def _on(self, stream):
        return torch.cuda.stream(torch.cuda.ExternalStream(stream, self.device) if isinstance(stream, int) else stream)

    def _capturing(self, stream) -> bool:
        """Whether the current stream, or the one that a call is given, is being captured."""
        if torch.cuda.is_current_stream_capturing():
            return True
        if stream is None:
            return False
        with self._on(stream):
            return torch.cuda.is_current_stream_capturing()

    def _launch_on(self, stream) -> int:
        """Handle of the stream of a call on tokens, which launches where the cache is or not at all."""
        if torch.cuda.current_device() != self._index:
            raise ValueError(f"the cache is on {self.device}, which is not the current device")
        return L._stream(stream, self._index)

    def _tokens(self, total: int, cu_tokens: torch.Tensor | None, max_tokens: int | None):
        if cu_tokens is None:
            return L.make_tokens(None, total, 1)
        if (cu_tokens.dtype is not torch.int32 or cu_tokens.numel() != self.batch + 1 or cu_tokens.get_device() != self._index
                or not cu_tokens.is_contiguous()):
            raise ValueError("cu_tokens must be contiguous int32 [batch + 1] on the device")
        return L.make_tokens(cu_tokens, total, total if max_tokens is None else max_tokens)

    def append(self, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor | None = None, *,
               rope: torch.Tensor | None = None, rotary_dim: int | None = None, interleaved: bool = False,
               positions: torch.Tensor | None = None, axes=None, cu_tokens: torch.Tensor | None = None,
               max_tokens: int | None = None, q_out: torch.Tensor | None = None, stream=None):
        """Writes the newest tokens of every sequence into the cache (seq_lens
        already counts them) and rotates their keys and queries.

        k, v: bf16 [total][Hkv][128], q: bf16 [total][Hq][128] (views into a
        fused projection are fine); rope: float32 [positions][rotary_dim], the
        cosines, then the sines; cu_tokens int32 [batch + 1] gives each
        sequence's rows and max_tokens the most that one has (default: total);
        without cu_tokens there is one token per sequence.  positions: int32
        [total], the table rows of the tokens (default: their positions in the
        sequences); or, with ``axes`` (``locks.make_axes``: the axis of each
        rotated pair), int32 [axes][total], a row per axis.  Returns the
        rotated queries (``q_out``, by default a new tensor; ``q`` itself
        rotates in place), or None without q."""
        shape = k.shape
        total = shape[0]
        index, handle = self._index, self._launch_on(stream)
        if (len(shape) != 3 or shape[1] != self.num_kv_heads or v.shape != shape or k.get_device() != index
                or v.get_device() != index):
            raise ValueError(f"k and v must be [tokens][{self.num_kv_heads}][128] on the device")
        if q is not None:
            shape = q.shape
            if len(shape) != 3 or shape[0] != total or shape[1] != self.num_q_heads or q.get_device() != index:
                raise ValueError(f"q must be [{total}][{self.num_q_heads}][128] on the device")
            if q_out is None:
                q_out = self._new(shape, torch.bfloat16, stream)
            elif q_out.shape != shape or q_out.get_device() != index:
                raise ValueError("q_out must have q's shape, on the device")
        elif q_out is not None:
            raise ValueError("q_out without q")
        if rope is None:
            rotary_dim = rotary_dim or 0
        else:
            if (rope.dtype is not torch.float32 or rope.dim() != 2 or rope.get_device() != index
                    or not rope.is_contiguous()):
                raise ValueError("rope must be contiguous float32 [positions][rotary_dim] on the device")
            cols = rope.shape[1]
            if rotary_dim is None:
                rotary_dim = cols
            elif rotary_dim != cols:
                raise ValueError("rope must have rotary_dim columns")
        if axes is not None:
            return self._append_axes(k, v, q, q_out, rope, rotary_dim, interleaved, positions, axes,
                                     self._tokens(total, cu_tokens, max_tokens), handle)
        if positions is not None and (positions.dtype is not torch.int32 or positions.numel() != total
                                      or positions.get_device() != index or not positions.is_contiguous()):
            raise ValueError("positions must be contiguous int32 [tokens] on the device")
        L.lockskv_append(self.cache, self._tokens(total, cu_tokens, max_tokens),
                         L.make_append(k, v, q, q_out, rope, rotary_dim, positions, interleaved),
                         self.kv_ws, 256, handle)
        return q_out

    def _append_axes(self, k, v, q, q_out, rope, rotary_dim, interleaved, positions, axes, tokens, handle):
        if rope is None or getattr(axes, "pairs", None) != rotary_dim // 2:
            raise ValueError("axes (locks.make_axes) need a rope, of whose pairs each has its axis")
        if (positions is None or positions.dtype is not torch.int32 or positions.dim() != 2
                or positions.shape[1] != tokens.total or positions.get_device() != self._index
                or (tokens.total > 1 and positions.stride(1) != 1)):
            raise ValueError("positions must be int32 [axes][tokens] on the device, an axis' tokens contiguous")
        n, total = positions.shape
        stride = positions.stride(0) if n > 1 else total
        if not axes.num_axes <= n <= L.LOCKSGEN_MAX_AXES or stride < total:
            raise ValueError(f"positions of {axes.num_axes} to {L.LOCKSGEN_MAX_AXES} axes are needed, that do not overlap")
        call = L.locksgen_axes_t(positions.data_ptr(), stride, n, axes.axis_of_pair)
        L.locksgen_append_axes(self.cache, tokens, L.make_append(k, v, q, q_out, rope, rotary_dim, None, interleaved),
                               call, self.kv_ws, 256, handle)
        return q_out

    def read_tokens(self, total: int, *, cu_tokens: torch.Tensor | None = None, max_tokens: int | None = None,
                    stream=None):
        """The newest tokens' keys and values as the cache holds them: two new
        bf16 tensors [total][Hkv][128] (rows of nobody are left unwritten)."""
        handle = self._launch_on(stream)
        k, v = (self._new((total, self.num_kv_heads, 128), torch.bfloat16, stream) for _ in range(2))
        L.lockskv_read(self.cache, self._tokens(total, cu_tokens, max_tokens), k, v, self.kv_ws, 256, handle)
        return k, v

    def prompt_attend(self, q: torch.Tensor, *, cu_tokens: torch.Tensor | None = None,
                      max_tokens: int | None = None, out=None, lse=None, stream=None):
        """Causal attention of the newest tokens, already in the cache, over it:
        q bf16 [total][Hq][128] -> out bf16 [total][Hq][128], lse float32
        [total][Hq] (new tensors by default).

        The workspace grows with the calls and is shared by all of them (see
        the class on calls that could overlap); a call is captured into a graph
        after one of the same max_tokens has run."""
        total = q.shape[0]
        index, handle = self._index, self._launch_on(stream)
        if q.dim() != 3 or q.shape[1] != self.num_q_heads or q.get_device() != index:
            raise ValueError(f"q must be [tokens][{self.num_q_heads}][128] on the device")
        stride = L._row_stride(q, "q")
        tokens = self._tokens(total, cu_tokens, max_tokens)
        if out is None:
            out = self._new(q.shape, torch.bfloat16, stream)
        elif (out.shape != q.shape or out.dtype is not torch.bfloat16 or out.get_device() != index
              or not out.is_contiguous()):
            raise ValueError("out must be contiguous bf16 of q's shape on the device")
        if lse is None:
            lse = self._new((total, self.num_q_heads), torch.float32, stream)
        elif (lse.shape != (total, self.num_q_heads) or lse.dtype is not torch.float32 or lse.get_device() != index
              or not lse.is_contiguous()):
            raise ValueError(f"lse must be contiguous float32 [{total}][{self.num_q_heads}] on the device")
        need = self._prompt_need.get(tokens.max_tokens)
        if need is None:
            need = L.lockskv_prompt_workspace_size(self.cache, self.params, tokens)
            self._prompt_need[tokens.max_tokens] = need
        capturing = self._capturing(stream)
        if self.prompt_ws is None or self.prompt_ws.numel() < need:
            self._grow_prompt_ws(need, capturing)
        self._prompt_captured |= capturing
        L.lockskv_prompt_attend(self.cache, self.params, tokens, q, stride, out, lse, self.prompt_ws,
                                self.prompt_ws.numel(), handle)
        return out, lse

    def _grow_prompt_ws(self, need: int, capturing: bool):
        if capturing:
            raise RuntimeError("prompt_attend needs a larger workspace: run a call of these sizes before the capture")
        # calls on any stream may still use the old one, and a captured graph keeps its address
        torch.cuda.synchronize(self.device)
        if self._prompt_captured:
            self._prompt_held.append(self.prompt_ws)
            self._prompt_captured = False
        err = 0 if self.prompt_ws is None else L.locks_get_device_error(self.prompt_ws)
        if self.prompt_ws is not None:  # in large steps, while they are cheap
            need = max(need, min(2 * self.prompt_ws.numel(), 256 << 20))
        ws = torch.empty(need + 256, dtype=torch.uint8, device=self.device)
        off = (-ws.data_ptr()) % 256
        self.prompt_ws = ws[off:off + need]
        L.locks_workspace_init(self.prompt_ws, need)
        if err:
            self.prompt_ws[:4].view(torch.int32).fill_(err)
        torch.cuda.synchronize(self.device)

    def device_error(self, stream=None) -> int:
        """LOCKS_DEVERR_* bits set since the last read, by the calls on the
        main workspace, by the builder and by the calls on tokens and prompts
        (all words are cleared)."""
        err = L.locks_get_device_error(self.ws, stream) | L.locks_get_device_error(self.build_ws, stream)
        err |= L.locks_get_device_error(self.kv_ws, stream)
        for ws in [self.prompt_ws, *self._prompt_held]:
            if ws is not None:
                err |= L.locks_get_device_error(ws, stream)
        return err
