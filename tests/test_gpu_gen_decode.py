"""A beam search whose steps use every way to attend: the page-selected decode, the dense one, the
prompt attention and the one that reads shared pages once, each directly after a reorder and again after
the next append, without a wait between the calls.

The truth is a cache in which every hypothesis has pages of its own, filled by appending its tokens
from the first to the last as the choices say they follow each other. Reordered beams give the same bits
as it does (the same pages' contents, lengths, summaries and counts), and the attention of shared pages
agrees with 64 bits within test_gpu_gen_attend's tolerances. The choices are held to test_gpu_gen_select's:
every (parent, token) against the 64-bit score of that continuation."""

import math

import pytest
import torch

from sparse_kv_page_rank_gb300.beams import LocksBeams
from sparse_kv_page_rank_gb300.runtime import LocksRuntime
from tests.kv_cases import D, dequant64
from tests.test_gpu_gen_attend import check as check_attend
from tests.test_gpu_gen_select import check as check_select

pytestmark = pytest.mark.gpu
HQ, HKV, V, RANK = 8, 2, 300, 4


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


def pool(pages, fmt, P):
    if fmt == "q4":
        return torch.full((pages, HKV, 144 * P), 255, dtype=torch.uint8, device="cuda"), None
    return tuple(torch.full((pages, HKV, P, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))


class Alone:
    """Every row's tokens (k, v [t][HKV][D], or None) in pages of its own."""

    def __init__(self, texts, nsum, cols, fmt, P, budget):
        self.fmt, self.P, self.hq, self.hkv, self.B = fmt, P, HQ, HKV, len(texts)
        self.lens = [0 if t is None else t[0].shape[0] for t in texts]
        self.table = torch.arange(self.B * cols, dtype=torch.int32, device="cuda").flip(0).view(self.B, cols).contiguous()
        seq = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.k, self.v = pool(self.B * cols, fmt, P)
        self.rt = LocksRuntime(self.k, self.v, self.table, seq, torch.tensor(nsum, dtype=torch.int32, device="cuda"), HQ, RANK, budget)
        k, v = (torch.cat([t[i] for t in texts if t is not None]) for i in range(2))
        cu = torch.tensor([0] + self.lens).cumsum(0).int().cuda()
        self.rt.append(k, v, cu_tokens=cu, max_tokens=max(self.lens))
        full = torch.cat([self.table[r, :n] for r, n in enumerate(nsum)])
        if full.numel():
            self.rt.build_summaries(full)

    def kv64(self, b):
        n = self.lens[b]
        pages = self.table[b, :-(-n // self.P)].long()
        k, v = dequant64(self.k[pages]) if self.fmt == "q4" else (self.k[pages].double(), self.v[pages].double())
        return [x.transpose(0, 1).reshape(HKV, -1, D)[:, :n] for x in (k, v)]


def attentions(rt, q):
    """What the calls on one token per row give, copied before the next one overwrites it."""
    live = rt.seq_lens > 0
    got = {}
    out, lse = rt.decode_step(q)
    got["decode_step"] = out.clone(), lse.clone()
    got["pages"] = rt.sel_pages.clone(), rt.sel_count.clone()
    got["dense_decode"] = [x.clone() for x in rt.dense_decode(q)]
    got["prompt_attend"] = [x[live] for x in rt.prompt_attend(q)]
    got["read_tokens"] = [x[live] for x in rt.read_tokens(rt.batch)]
    return got


def same(a, b, what):
    for name in a:
        for x, y in zip(a[name], b[name]):
            if name == "pages":
                continue
            assert torch.equal(x, y), (what, name)
    (pa, ca), (pb, cb) = a["pages"], b["pages"]
    assert torch.equal(ca, cb), what
    seen = torch.arange(pa.shape[-1], device="cuda") < ca[..., None]
    assert torch.equal(pa.masked_fill(~seen, -1), pb.masked_fill(~seen, -1)), what


@pytest.mark.parametrize("fmt,P,prompts,W,steps,budget", [
    ("bf16", 64, [900, 500], 4, 70, 256), ("q4", 64, [700], 3, 66, 128), ("bf16", 16, [200, 90, 40], 4, 36, 64),
    ("q4", 16, [250, 100], 5, 34, 64),
])
def test_search(fmt, P, prompts, W, steps, budget):
    g = torch.Generator().manual_seed(P + W)
    R, end = len(prompts), 3
    rows, cols = R * W, (max(prompts) + steps) // P + 2
    full = [n // P for n in prompts]
    pages = sum(f + W * (cols - f) for f in full)
    order, at = torch.randperm(pages, generator=g).int(), 0
    tab = torch.zeros(rows, cols, dtype=torch.int32)
    for r, f in enumerate(full):
        tab[r * W:r * W + W, :f] = order[at:at + f]
        at += f
        for w in range(W):
            tab[r * W + w, f:] = order[at:at + cols - f]
            at += cols - f
    tab = tab.cuda()
    lens = torch.tensor([n if w == 0 else 0 for n in prompts for w in range(W)], dtype=torch.int32).cuda()
    nsum = torch.tensor([n // P if w == 0 else 0 for n in prompts for w in range(W)], dtype=torch.int32).cuda()
    shared = torch.tensor(full, dtype=torch.int32).cuda()
    rt = LocksRuntime(*pool(pages, fmt, P), tab, lens, nsum, HQ, RANK, budget)
    beams = LocksBeams([rt], width=W, end_token=end)
    assert rt.n_summarized is nsum

    def draw(n):
        return [(torch.randn(n, HKV, D, generator=g) * s).bfloat16().cuda() for s in (2.0, 1.0)]

    texts = [None] * rows
    for r, n in enumerate(prompts):
        texts[r * W] = tuple(draw(n))
    k, v = (torch.cat([t[i] for t in texts if t is not None]) for i in range(2))
    cu = torch.tensor([0] + lens.tolist()).cumsum(0).int().cuda()
    rt.append(k, v, cu_tokens=cu, max_tokens=max(prompts))
    rt.build_summaries(torch.cat([tab[r * W, :f] for r, f in enumerate(full)]))
    scores = torch.full((R, W), -math.inf, device="cuda")
    scores[:, 0] = 0
    ended = torch.zeros(R, W, dtype=torch.int32, device="cuda")
    for step in range(steps):
        logits = (torch.randn(R, W, V, generator=g) * 1.5).cuda()
        was = scores.clone(), ended.clone()
        q = (torch.randn(2, rows, HQ, D, generator=g) * 2).bfloat16().cuda()
        new = draw(rows)
        look = step % 6 == 0 or step > steps - 3
        # one stretch of calls without a wait
        got = beams.select(logits, scores, ended)
        chosen = [x.clone() for x in got]
        scores, parents, tokens, ended = got
        beams.reorder(parents)
        after = attentions(rt, q[0]) if look else None
        counts = nsum.clone()
        lens += lens > 0
        rt.append(*new)
        then = attentions(rt, q[1]) if look else None
        out, lse = beams.attend(q[1], shared)
        torch.cuda.synchronize()
        assert beams.device_error() == 0 and rt.device_error() == 0
        check_select(chosen, logits, *was, end, W)
        p = chosen[1].tolist()
        texts = [None if p[i // W][i % W] < 0 else texts[i // W * W + p[i // W][i % W]] for i in range(rows)]
        if look:
            before = Alone(texts, counts.tolist(), cols, fmt, P, budget)
            same(after, attentions(before.rt, q[0]), (step, "reordered"))
            assert before.rt.device_error() == 0
        texts = [t if t is None else tuple(torch.cat([x, y[i:i + 1]]) for x, y in zip(t, new)) for i, t in enumerate(texts)]
        assert lens.tolist() == [0 if t is None else t[0].shape[0] for t in texts]
        if look:
            truth = Alone(texts, nsum.tolist(), cols, fmt, P, budget)
            same(then, attentions(truth.rt, q[1]), (step, "appended"))
            check_attend(truth, q[1], out, lse)
            assert truth.rt.device_error() == 0
        # pages that are full now get their summaries, but not in every step
        if step % 3 != 1:
            ids = []
            for i, n in enumerate(lens.tolist()):
                ids += tab[i, int(nsum[i]):n // P].tolist() if n else []
            if ids:
                rt.build_summaries(torch.tensor(sorted(set(ids)), dtype=torch.int32, device="cuda"))
            nsum.copy_(lens // P)
    assert int(nsum.max()) * P > budget  # pages were chosen among more than the budget's
