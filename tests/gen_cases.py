"""Cases and 64-bit references for beam search and positions with several axes,
written from include/locksgen.h alone."""

from __future__ import annotations

import math

import torch

from tests.kv_cases import Case


def shared_case(prompts, tails, hq, hkv, P, fmt, seed, nsum=None):
    """A cache of len(prompts) requests whose beams have lengths prompts[r] + tails[r][w] (None: an
    idle row) and share the prompt's full pages.  Returns (case, width, shared pages)."""
    W = len(tails[0])
    lens = [0 if t is None else n + t for n, row in zip(prompts, tails) for t in row]
    case = Case(lens, hq, hkv, P, fmt, seed, nsum=nsum)
    shared = [n // P for n in prompts]
    for r, s in enumerate(shared):
        rows = [r * W + w for w in range(W) if lens[r * W + w]]
        for row in rows[1:]:
            case.table[row, :s] = case.table[rows[0], :s]
    return case, W, torch.tensor(shared, dtype=torch.int32, device="cuda")


def reordered(table, lens, nsum, parents, P):
    """Lists: tables, lengths and counts of one request's rows after a reorder, and the copies
    (source page, destination page, tokens)."""
    W = len(parents)
    unused = [w for w in range(W) if w not in parents]
    first = {}
    for r, p in enumerate(parents):
        if p >= 0 and p not in first:
            first[p] = r
    owner = {r: p for p, r in first.items()}
    rest = [r for r in range(W) if parents[r] >= 0 and r not in owner] + [r for r in range(W) if parents[r] < 0]
    owner.update(zip(rest, unused))
    out, copies = [], []
    for r, p in enumerate(parents):
        o = owner[r]
        if p < 0 or (first[p] != r and lens[o] // P > lens[p] // P):
            out.append((list(table[o]), 0, 0))
            continue
        j, n = lens[p] // P, lens[p] % P
        out.append((list(table[p][:j]) + list(table[o][j:]), lens[p], nsum[p]))
        if first[p] != r and n:
            copies.append((table[p][j], table[o][j], -(-n // 16) * 16))
    return [list(x) for x in zip(*out)], copies


def candidates64(logits, scores, ended, end_token):
    """Scores [B][W][V] in 64 bits of all continuations (-inf: none), of logits [B][W][V]."""
    x = logits.double()
    s = scores.double()[..., None] + (x - x.logsumexp(dim=-1, keepdim=True))
    s = torch.where(x == -math.inf, -math.inf, s)
    s = torch.where(scores[..., None] == -math.inf, -math.inf, s)
    if ended is not None:
        over = (ended != 0)[..., None]
        own = torch.full_like(s, -math.inf)
        own[..., end_token] = scores.double()
        s = torch.where(over, own, s)
    return s
