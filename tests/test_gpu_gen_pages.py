"""A caller that gives pages out one by one, as rows come to need them, and takes them back by the
rule of locksgen.h: no page that a row still needs is given out twice, none is lost, and every
hypothesis reads its own tokens."""

import random

import pytest
import torch

from sparse_kv_page_rank_gb300.beams import LocksBeams
from sparse_kv_page_rank_gb300.runtime import LocksRuntime

pytestmark = pytest.mark.gpu
P = 16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


def still_needed(table, lens, W, r):
    """Pages of request r that the rule keeps."""
    rows = range(r * W, r * W + W)
    live = [x for x in rows if lens[x]]
    if not live:
        return set()
    first = min(lens[x] // P for x in live)
    held = {p for x in live for p in table[x]}
    return (held | {p for x in rows if not lens[x] for p in table[x][first:]}) - {-1}


@pytest.mark.parametrize("W,requests,steps,left_behind", [(4, 1, 90, False), (5, 2, 70, False), (4, 2, 60, True)])
def test_pages_on_demand(W, requests, steps, left_behind):
    rng = random.Random(W + steps)
    rows, cols = W * requests, steps // P + 5
    pages = requests * (W * cols)  # more than rows ever hold, but far fewer than would be used up if some were lost
    k, v = (torch.zeros(pages, 1, P, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    free = list(range(pages))
    rng.shuffle(free)
    table = [[-1] * cols for _ in range(rows)]
    lens, text, given = [0] * rows, [None] * rows, [set() for _ in range(requests)]
    tab, seq = torch.zeros(rows, cols, dtype=torch.int32, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda")
    rt = LocksRuntime(k, v, tab, seq, torch.zeros_like(seq), 1, 2, 0)
    beams = LocksBeams([rt], width=W)

    def give(row, column):
        if table[row][column] < 0:
            table[row][column] = free.pop()
            given[row // W].add(table[row][column])

    def write(row, token):
        """The row's next token, into its own open page."""
        give(row, lens[row] // P)
        k[table[row][lens[row] // P], 0, lens[row] % P] = float(token)
        lens[row] += 1

    for r in range(requests):
        prompt = [rng.randrange(256) for _ in range(rng.randrange(1, 40))]
        row = r * W
        text[row] = prompt
        for t in prompt:
            write(row, t)
    most = 0
    for step in range(steps):
        parents = []
        for r in range(requests):
            live = [w for w in range(W) if lens[r * W + w]]
            longest = max(lens[r * W + w] for w in live)
            mine = [rng.choice(live) if rng.random() < 0.85 else -1 for _ in range(W)]
            # what is continued more than once is among the longest
            for i, p in enumerate(mine):
                if p >= 0 and p in mine[:i] and lens[r * W + p] != longest:
                    mine[i] = -1
            if all(p < 0 or lens[r * W + p] != longest for p in mine):
                mine[0] = max(live, key=lambda w: lens[r * W + w])
            parents.append(mine)
            for w in range(W):  # a page of its own where the live rows are
                for column in {lens[r * W + x] // P for x in live}:
                    if column >= lens[r * W + w] // P:
                        give(r * W + w, column)
        tab.copy_(torch.tensor(table, dtype=torch.int32))
        seq.copy_(torch.tensor(lens, dtype=torch.int32))
        beams.reorder(torch.tensor(parents, dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        assert beams.device_error() == 0, step
        old, table, lens = text, tab.tolist(), seq.tolist()
        text = [None if parents[i // W][i % W] < 0 else list(old[i // W * W + parents[i // W][i % W]]) for i in range(rows)]
        assert lens == [0 if t is None else len(t) for t in text]
        for r in range(requests):
            keep = still_needed(table, lens, W, r)
            assert keep <= given[r]
            back = given[r] - keep
            free.extend(back)
            given[r] = keep
            for row in range(r * W, r * W + W):  # the caller's own note that those are gone
                table[row] = [-1 if p in back else p for p in table[row]]
            most = max(most, len(keep))
        k[torch.tensor(free, device="cuda")] = -1.0  # as if another request wrote there
        # every live row but those left behind goes on
        for row in range(rows):
            if text[row] is not None and not (left_behind and row % W and rng.random() < 0.2):
                t = rng.randrange(256)
                text[row].append(t)
                write(row, t)
        for row in range(rows):
            if text[row] is not None:
                got = [int(k[table[row][i // P], 0, i % P, 0]) for i in range(0, len(text[row]), 5)]
                assert got == text[row][::5], (step, row)
        assert len(free) + sum(map(len, given)) == pages and len(set(free)) == len(free)
    assert most <= W * cols
