"""Beam search as a program runs it: a prompt whose tokens have positions with several axes, then
steps of append, attention of the beams, choice and reorder over two layers, in one captured graph, against a
search that holds every hypothesis' own keys and values.

The model is a toy: a step's logits and a token's keys, values and queries are fixed random tables' rows,
mixed with the attention's output, so that what a beam has seen decides what it says. The plain search
follows the library's own choices (a choice between nearly equal continuations is the library's to make, and
test_gpu_gen_select checks it) and compares the attention's output of every step with the definition."""

import pytest
import torch

from sparse_kv_page_rank_gb300 import locks as L
from sparse_kv_page_rank_gb300.beams import LocksBeams
from sparse_kv_page_rank_gb300.runtime import LocksRuntime
from tests.gen_cases import candidates64
from tests.kv_cases import D, attend64
from tests.test_gpu_gen_axes import rotated
from tests.test_gpu_kv_append import table

pytestmark = pytest.mark.gpu

HQ, HKV, V = 8, 2, 500


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


@pytest.mark.parametrize("fmt,P,prompts,W,steps", [
    ("bf16", 64, [130, 64, 7], 4, 70), ("q4", 16, [40, 33], 5, 40), ("bf16", 16, [31], 3, 50), ("q4", 64, [200, 1], 2, 20),
])
def test_search(fmt, P, prompts, W, steps):
    g = torch.Generator().manual_seed(P + W)
    R, end = len(prompts), 3
    rows, longest = R * W, max(prompts) + steps + 1
    cols = -(-longest // P)
    full = [n // P for n in prompts]
    # a request's rows: the prompt's full pages, shared, and pages of their own
    pages = sum(full) + sum(W * (cols - f) for f in full)
    order = torch.randperm(pages, generator=g).int()
    tab, at = torch.zeros(rows, cols, dtype=torch.int32), 0
    for r, f in enumerate(full):
        tab[r * W:r * W + W, :f] = order[at:at + f]
        at += f
        for w in range(W):
            tab[r * W + w, f:] = order[at:at + cols - f]
            at += cols - f
    tab = tab.cuda()
    lens = torch.tensor([n if w == 0 else 0 for n in prompts for w in range(W)], dtype=torch.int32).cuda()
    nsum = torch.zeros_like(lens)
    shared = torch.tensor(full, dtype=torch.int32).cuda()

    def pool():
        if fmt == "q4":
            return torch.full((pages, HKV, 144 * P), 255, dtype=torch.uint8, device="cuda"), None
        return tuple(torch.full((pages, HKV, P, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    rts = [LocksRuntime(*pool(), tab, lens, nsum, HQ, 2, 0) for _ in range(2)]
    beams = LocksBeams(rts, width=W, end_token=end)
    rope, axes = table(longest + 5, 128), L.make_axes(L.rope_axes([16, 24, 24]))
    word = (torch.randn(2, V, HQ + 2 * HKV, D, generator=g)).bfloat16().cuda()  # a token's q, k, v in each layer
    says = (torch.randn(HQ * D, V, generator=g) / 6).cuda()

    # the prompts
    text = [torch.randint(4, V, (n,), generator=g) for n in prompts]
    cu = torch.tensor([0] + [n if w == 0 else 0 for n in prompts for w in range(W)]).cumsum(0).int().cuda()
    tokens = torch.cat(text).cuda()
    pos = torch.stack([torch.cat([torch.arange(n) // (a + 1) for n in prompts]) for a in range(3)]).int().cuda()
    for layer, rt in enumerate(rts):
        q, k, v = word[layer][tokens].split([HQ, HKV, HKV], dim=1)
        rt.append(k, v, q, rope=rope, positions=pos, axes=axes, cu_tokens=cu, max_tokens=max(prompts))
    scores = torch.full((R, W), float("-inf")).cuda()
    scores[:, 0] = 0
    ended = torch.zeros(R, W, dtype=torch.int32).cuda()
    heard = torch.zeros(rows, HQ * D, device="cuda")  # the last layer's attention
    new = torch.zeros(rows, dtype=torch.long, device="cuda")
    where = torch.zeros(3, rows, dtype=torch.int32, device="cuda")
    trace = {n: torch.zeros(rows, HQ, D, dtype=torch.bfloat16, device="cuda") for n in ("q0", "q1", "o0", "o1")}
    parents, picked = (torch.zeros(R, W, dtype=torch.int32, device="cuda") for _ in range(2))
    logits = torch.zeros(rows, V, device="cuda")

    three = torch.tensor([[1], [2], [3]], device="cuda", dtype=torch.int32)

    def step():  # but for the toy model and the lengths, every kernel is the library's
        torch.matmul(heard, says, out=logits)
        beams.select(logits, scores, ended, out_scores=scores, out_parents=parents, out_tokens=picked, out_ended=ended)
        beams.reorder(parents)
        lens.add_(lens.clamp(max=1))
        new.copy_(picked.clamp(min=0).flatten())
        torch.div((lens - 1).clamp(min=0)[None], three, rounding_mode="floor", out=where)
        for layer, rt in enumerate(rts):
            q, k, v = word[layer].index_select(0, new).split([HQ, HKV, HKV], dim=1)
            q = rt.append(k, v, q, rope=rope, positions=where, axes=axes)
            o, _ = beams.attend(q, shared, layer=layer)
            trace[f"q{layer}"].copy_(q)
            trace[f"o{layer}"].copy_(o)
        heard.copy_(o.flatten(1))

    # each hypothesis' own keys and values (rotated, as the cache stores them), a list of rows' tensors per layer
    kv = [[None] * rows for _ in rts]
    first = 0
    for r, n in enumerate(prompts):
        for layer in range(2):
            _, k, v = word[layer][text[r].cuda()].split([HQ, HKV, HKV], dim=1)
            k = rotated(k, rope, pos[:, first:first + n], L.rope_axes([16, 24, 24]), False).bfloat16()
            kv[layer][r * W] = (k, v)
        first += n
    held = lambda x: x.double() if fmt == "bf16" else quantised64(x)
    graph = None
    for i in range(steps):
        was_s, was_e = scores.clone(), ended.clone()
        before = heard.clone()
        if i == 0:
            step()
        else:
            if graph is None:
                torch.cuda.synchronize()
                state = [x.clone() for x in (scores, ended, lens, tab, nsum, heard)]
                graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
                with torch.cuda.graph(graph, stream=stream):
                    step()
                torch.cuda.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(state, (scores, ended, lens, tab, nsum, heard)))  # nothing has run
            graph.replay()
        torch.cuda.synchronize()
        assert beams.device_error() == 0 and all(rt.device_error() == 0 for rt in rts)
        # the choice is among the best
        s = candidates64((before @ says).view(R, W, V), was_s, was_e, end).flatten(1)
        best = s.topk(W, dim=1).values
        assert ((scores.double() - best).abs()[torch.isfinite(best)] < 1e-3).all()
        assert (torch.isfinite(scores) == torch.isfinite(best)).all()
        # follow it
        p = (parents.long() + torch.arange(R, device="cuda")[:, None] * W).flatten().tolist()
        alive = (parents >= 0).flatten().tolist()
        for layer in range(2):
            old = kv[layer]
            kv[layer] = [old[p[r]] if alive[r] else None for r in range(rows)]
            _, k, v = word[layer][new].split([HQ, HKV, HKV], dim=1)
            k = rotated(k, rope, where, L.rope_axes([16, 24, 24]), False).bfloat16()
            for r in range(rows):
                if kv[layer][r] is not None:
                    kv[layer][r] = (torch.cat([kv[layer][r][0], k[r:r + 1]]), torch.cat([kv[layer][r][1], v[r:r + 1]]))
        for r in range(rows):
            assert int(lens[r]) == (0 if kv[0][r] is None else kv[0][r][0].shape[0])
        if i % 7 and i != steps - 1:
            continue
        for layer in range(2):
            for r in range(rows):
                if kv[layer][r] is None:
                    assert (trace[f"o{layer}"][r] == 0).all()
                    continue
                k, v = (held(x).transpose(0, 1) for x in kv[layer][r])
                for h in range(HKV):
                    sl = slice(h * 4, h * 4 + 4)
                    o, _, mean, _, mag = attend64(trace[f"q{layer}"][r, sl], k[h], v[h])
                    e = 2.0 ** -17 * mag[:, None] + 2.0 ** -21  # (as in test_gpu_gen_attend)
                    tol = (2.0 ** -8 + 2.0 ** -12 + 2 * e) * mean + 2.0 ** -8 * o.abs() + 2.0 ** -32 * v[h].abs().sum(dim=0)
                    assert ((trace[f"o{layer}"][r, sl].double() - o).abs() <= tol).all(), (i, layer, r, h)
    assert int(lens.max()) == max(prompts) + steps or bool(ended.any())


def quantised64(x):
    """What a 4-bit page holds for x bf16 [t][h][128], in 64 bits."""
    from tests.test_gpu_kv_append import quantised
    q, s = quantised(x)
    return q.double() * s.double().repeat_interleave(32, dim=-1)
