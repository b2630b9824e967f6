"""Beam search over paged caches: choosing the beams, moving them in the
caches, attending with them.

``LocksBeams`` holds the workspaces of the calls and the C structs of the
layers' caches; it computes nothing itself.  A decode step of a model whose
layers have a ``LocksRuntime`` each, over one block table and one set of lengths:

    for rt, layer in zip(runtimes, layers):
        q = rt.append(k, v, q, rope=cos_sin)
        out, lse = beams.attend(q, shared_pages, layer=i)    # or rt.decode_step(q)
    scores, parents, tokens, ended = beams.select(logits, scores, ended)
    trail.append((parents.clone(), tokens.clone()))           # the next call overwrites them
    beams.reorder(parents)
    seq_lens += seq_lens > 0                                  # the chosen tokens come next

Rows r W .. r W + W - 1 of the caches are the W beams of request r.  Each row
has its own pages from its open page on; full pages may be shared
(``include/locksgen.h`` says how a request begins).
"""

from __future__ import annotations

import ctypes

import torch

from . import locks as L


_LOGITS = {torch.bfloat16: L.LOCKS_DTYPE_BF16, torch.float32: L.LOCKS_DTYPE_F32}


class LocksBeams:
    """Beam search with ``width`` beams per request.

    runtimes: the layers' ``LocksRuntime``, which share block_table, seq_lens and
    n_summarized (the same tensors) and have one page format; or none, with a
    ``device``, for ``select`` alone.  ``end_token`` ends a hypothesis (-1: none).

    One workspace serves all calls of a kind, and so do the outputs that are not given
    (as those of a ``LocksRuntime``'s decode calls): the next call of the same sizes
    overwrites them.  The caller orders calls that are on different streams, and
    replays of graphs that hold them (or has a LocksBeams for each).
    """

    def __init__(self, runtimes=None, width: int = 1, *, device=None, end_token: int = -1):
        self.runtimes = list(runtimes or [])
        if not 0 < width <= L.LOCKSGEN_MAX_BEAMS:
            raise ValueError(f"1 to {L.LOCKSGEN_MAX_BEAMS} beams")
        self.width, self.end_token = width, int(end_token)
        if self.runtimes:
            self.device, self._index = self.runtimes[0].device, self.runtimes[0]._index
        else:
            device = torch.device("cuda" if device is None else device)
            if device.type != "cuda":
                raise ValueError("beams need a CUDA device")
            self._index = torch.cuda.current_device() if device.index is None else device.index
            self.device = torch.device("cuda", self._index)
        self._select_ws = None
        self._select_need = {}  # bytes by sizes
        self._outs = {}         # outputs by sizes
        self._held = []         # all workspaces: a captured graph may still use an outgrown one
        if self.runtimes:
            rt = self.runtimes[0]
            if rt.batch % width:
                raise ValueError(f"{rt.batch} rows are no whole requests of {width} beams")
            for x in self.runtimes:
                if (x.block_table.data_ptr(), x.seq_lens.data_ptr(), x.n_summarized.data_ptr()) != (
                        rt.block_table.data_ptr(), rt.seq_lens.data_ptr(), rt.n_summarized.data_ptr()):
                    raise ValueError("the runtimes must share block_table, seq_lens and n_summarized")
            if not rt.block_table.is_contiguous():
                raise ValueError("block_table must be contiguous")
            self.requests = rt.batch // width
            self._caches = (L.locks_cache_t * len(self.runtimes))(*(x.cache for x in self.runtimes))
            self._reorder_ws = self._workspace(L.locksgen_reorder_workspace_size(rt.cache, width))
            self._attend_ws = self._workspace(max(L.locksgen_attend_workspace_size(x.cache, x.params, width)
                                                  for x in self.runtimes))

    def _workspace(self, need: int, stream=None) -> torch.Tensor:
        if torch.cuda.is_current_stream_capturing() or (stream is not None and self._on_stream(
                stream, torch.cuda.is_current_stream_capturing)):
            raise RuntimeError("a larger workspace is needed: run a call of these sizes before the capture")
        ws = torch.zeros(need + 256, dtype=torch.uint8, device=self.device)
        off = (-ws.data_ptr()) % 256
        torch.cuda.synchronize(self.device)  # before a call on any stream
        self._held.append(ws[off:off + need])
        return self._held[-1]

    def _launch_on(self, stream) -> int:
        if torch.cuda.current_device() != self._index:
            raise ValueError(f"the beams are on {self.device}, which is not the current device")
        return L._stream(stream, self._index)

    def _on_stream(self, stream, f):
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, self.device) if isinstance(stream, int) else stream):
            return f()

    def _here(self, x, dtype, shape, what):
        if x.dtype is not dtype or x.shape != shape or x.get_device() != self._index or not x.is_contiguous():
            raise ValueError(f"{what} must be contiguous {str(dtype)[6:]} {list(shape)} on the device")

    def select(self, logits: torch.Tensor, scores: torch.Tensor, ended: torch.Tensor | None = None, *,
               keep: int | None = None, out_scores=None, out_parents=None, out_tokens=None, out_ended=None, stream=None):
        """The ``keep`` (default: width) best continuations of every request.

        logits: bf16 or float32 [requests * width][vocab] (or [requests][width][vocab]), a
        row's elements contiguous; scores: float32 [requests][width], -inf for a row without a
        hypothesis; ended: int32 [requests][width], nonzero for a hypothesis that has
        ended, which continues as it is with the token ``end_token``.  Returns scores, parents, tokens
        and ended (None without an end_token), [requests][keep], best first; where there is no
        continuation the score is -inf and parent and token are -1.  The outputs are the object's
        own unless given, and the next call of these sizes overwrites them: copy the parents and
        tokens that are to be kept.  They may be given back as scores and ended where keep is width, or of one request
        the first width of them (``scores[:, :width]``)."""
        handle = self._launch_on(stream)
        W = self.width
        if logits.dim() == 3:
            n, w, vocab = logits.shape
            ok = w == W and (n == 1 or W == 1 or logits.stride(0) == W * logits.stride(1))
            row = logits.stride(0) if W == 1 else logits.stride(1)
        else:
            ok = logits.dim() == 2 and logits.shape[0] % W == 0
            n, vocab, row = (logits.shape[0] // W, logits.shape[1], logits.stride(0)) if ok else (0, 0, 0)
        dtype = _LOGITS.get(logits.dtype)
        if not ok or dtype is None or (vocab > 1 and logits.stride(-1) != 1) or logits.get_device() != self._index:
            raise ValueError(f"logits must be bf16 or float32 [requests * {W}][vocab] on the device, a row's elements contiguous")
        if self.runtimes and n != self.requests:
            raise ValueError(f"logits of {self.requests} requests are needed")
        keep = W if keep is None else int(keep)
        if not 0 < keep <= L.LOCKSGEN_MAX_KEEP:
            raise L.LocksError(L.LOCKS_ERR_INVALID_ARG if keep <= 0 else L.LOCKS_ERR_UNSUPPORTED, "locksgen_select")
        self._here(scores, torch.float32, (n, W), "scores")
        if ended is not None:
            self._here(ended, torch.int32, (n, W), "ended")
            if self.end_token < 0:
                raise ValueError("ended without an end_token")
        shape = (n, keep)
        own = self._outs.get(shape)
        if own is None:
            def make():
                return tuple(torch.empty(shape, dtype=t, device=self.device)
                             for t in (torch.float32, torch.int32, torch.int32, torch.int32))
            # memory that its first use follows on the same stream
            own = self._outs[shape] = make() if stream is None else self._on_stream(stream, make)
        if out_scores is None:
            out_scores = own[0]
        else:
            self._here(out_scores, torch.float32, shape, "out_scores")
        if out_parents is None:
            out_parents = own[1]
        else:
            self._here(out_parents, torch.int32, shape, "out_parents")
        if out_tokens is None:
            out_tokens = own[2]
        else:
            self._here(out_tokens, torch.int32, shape, "out_tokens")
        if out_ended is not None:
            self._here(out_ended, torch.int32, shape, "out_ended")
        elif self.end_token >= 0:
            out_ended = own[3]
        outs = out_scores, out_parents, out_tokens, out_ended
        if n == 0:
            return outs
        choice = L.locksgen_choice_t(logits.data_ptr(), scores.data_ptr(), L._ptr(ended), out_scores.data_ptr(),
                                     out_parents.data_ptr(), out_tokens.data_ptr(), L._ptr(out_ended),
                                     row if n * W > 1 else vocab, n, W, vocab, keep, dtype, self.end_token)
        key = (n, vocab, keep, dtype)
        need = self._select_need.get(key)
        if need is None:
            need = self._select_need[key] = L.locksgen_select_workspace_size(choice)
        ws = self._select_ws
        if ws is None or ws.numel() < need:  # in large steps, so that the outgrown ones are no more than the last
            ws = self._select_ws = self._workspace(need if ws is None else max(need, 2 * ws.numel()), stream)
        L.locksgen_select(choice, ws, ws.numel(), handle)
        return outs

    def reorder(self, parents: torch.Tensor, stream=None):
        """Every row becomes a copy of its parent (int32 [requests][width], as ``select`` gives them; -1:
        an idle row), in all layers: block_table, seq_lens, n_summarized and, where a beam is
        continued more than once, its open page.  In place."""
        handle = self._launch_on(stream)
        if not self.runtimes:
            raise ValueError("these beams have no caches")
        self._here(parents, torch.int32, (self.requests, self.width), "parents")
        L.locksgen_reorder(self._caches, len(self._caches), self.width, parents, self._reorder_ws,
                           self._reorder_ws.numel(), handle)

    def attend(self, q: torch.Tensor, shared_pages: torch.Tensor, layer: int = 0, out=None, lse=None, stream=None):
        """``LocksRuntime.dense_decode`` of layer ``layer`` for rows that share pages: the first
        shared_pages[r] (int32 [requests]) columns of the block table are the same in all rows of
        request r and are read once.  q bf16 [requests * width][Hq][128] -> out bf16 of the same
        shape, lse float32 [requests * width][Hq] (the runtime's own by default, as there)."""
        handle = self._launch_on(stream)
        if not self.runtimes:
            raise ValueError("these beams have no caches")
        rt = self.runtimes[layer]
        shape = (rt.batch, rt.num_q_heads, 128)
        self._here(q, torch.bfloat16, shape, "q")
        self._here(shared_pages, torch.int32, (self.requests,), "shared_pages")
        if out is None:
            out = rt.out
        else:
            self._here(out, torch.bfloat16, shape, "out")
        if lse is None:
            lse = rt.lse
        else:
            self._here(lse, torch.float32, shape[:2], "lse")
        L.locksgen_attend(rt.cache, rt.params, self.width, shared_pages, q, out, lse, self._attend_ws,
                          self._attend_ws.numel(), handle)
        return out, lse

    def device_error(self, stream=None) -> int:
        """LOCKS_DEVERR_* and LOCKSGEN_DEVERR_* bits that these calls have set since the last read
        (cleared)."""
        err = 0
        for ws in self._held:
            err |= L.locks_get_device_error(ws, stream)
        return err
