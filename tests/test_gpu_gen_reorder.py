"""Rows that follow their parents: block tables, lengths, counts and open pages, exactly."""

import pytest
import torch

from sparse_kv_page_rank_gb300 import locks as L
from sparse_kv_page_rank_gb300.beams import LocksBeams
from sparse_kv_page_rank_gb300.runtime import LocksRuntime
from tests.gen_cases import reordered
from tests.kv_cases import D, unpack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


class Rows:
    """Caches (layers) full of random tokens whose rows all have pages of their own."""

    def __init__(self, lens, W, hkv, P, fmt, cols, layers=1, seed=0, nsum=True):
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        pages = B * cols + 2
        self.lens, self.W, self.P, self.fmt, self.gen = list(lens), W, P, fmt, g
        self.table = torch.randperm(pages, generator=g)[:B * cols].view(B, cols).int().cuda()
        self.seq = torch.tensor(lens, dtype=torch.int32).cuda()
        self.nsum = torch.tensor([max(0, n) // P // 2 for n in lens], dtype=torch.int32).cuda()
        self.pools = []
        for _ in range(layers):
            if fmt == "q4":
                self.pools.append((torch.randint(0, 256, (pages, hkv, 144 * P), generator=g).to(torch.uint8).cuda(), None))
            else:
                self.pools.append(tuple(torch.randint(-30000, 30000, (pages, hkv, P, D), generator=g).short().cuda()
                                        .view(torch.bfloat16) for _ in range(2)))
        self.rts = [LocksRuntime(k, v, self.table, self.seq, self.nsum, hkv, 2, 0) for k, v in self.pools]
        self.beams = LocksBeams(self.rts, width=W)

    def flat(self):
        return [x.view(torch.uint8) if x.dtype is torch.uint8 else x.view(torch.int16) for kv in self.pools for x in kv if x is not None]

    def run(self, parents, call=None):
        """Reorders by parents [requests][W] and checks everything."""
        before = [x.clone() for x in self.flat()]
        table, lens, nsum = self.table.tolist(), self.seq.tolist(), self.nsum.tolist()
        p = torch.tensor(parents, dtype=torch.int32).cuda()
        (call or self.beams.reorder)(p)
        W, P = self.W, self.P
        want, copies = [[], [], []], []
        for r, mine in enumerate(parents):
            s = slice(r * W, r * W + W)
            out, c = reordered(table[s], lens[s], nsum[s], mine, P)
            copies += c
            for a, b in zip(want, out):
                a += b
        assert self.table.tolist() == want[0] and self.seq.tolist() == want[1] and self.nsum.tolist() == want[2]
        for x, old in zip(self.flat(), before):
            if self.fmt == "q4":
                # token by token: a token's codes and scales, as the format places them
                parts, was = unpack(x), unpack(old)
                for a, b in zip(parts, was):
                    a, b = (y.view(torch.int16) if y.dtype is torch.float16 else y for y in (a, b))
                    fresh = b.clone()
                    for src, dst, n in copies:
                        fresh[dst, :, :n] = b[src, :, :n]
                    assert torch.equal(a, fresh)
            else:
                fresh = old.clone()
                for src, dst, n in copies:
                    fresh[dst, :, :n] = old[src, :, :n]
                assert torch.equal(x, fresh)


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("P,W,hkv,lens,cols,parents", [
    (64, 4, 2, [130] * 4, 5, [[0, 0, 1, 3]]),
    (64, 4, 2, [130] * 4, 5, [[2, 2, 2, 2]]),
    (64, 4, 1, [130] * 4, 5, [[3, 2, 1, 0]]),
    (64, 4, 1, [128] * 4, 5, [[1, 1, 0, 1]]),               # open pages that are still empty
    (64, 4, 1, [320] * 4, 5, [[1, 1, 0, 1]]),               # tables that are full
    (64, 4, 1, [100, 0, 0, 0], 5, [[0, 0, 0, 0]]),          # the first step after a prompt
    (64, 4, 1, [0, 0, 0, 0], 3, [[0, 1, 2, 3]]),
    (16, 4, 3, [100] * 4, 9, [[0, -1, 0, -1]]),             # rows that become idle
    (16, 4, 3, [100] * 4, 9, [[-1, -1, -1, -1]]),
    (16, 1, 8, [33, 16, 1], 4, [[0], [0], [-1]]),
    (16, 3, 8, [33, 33, 33, 200, 200, 200, 7, 7, 7], 13, [[2, 2, 0], [1, 1, 1], [0, 2, 2]]),
    (64, 5, 2, [70, 70, 40, 70, 70], 3, [[4, 2, 0, 0, 4]]),  # row 2 has ended before the others
    (64, 32, 1, [65] * 32, 3, [[0] * 32]),
    (16, 32, 1, [65] * 64, 300, [[(7 * i * i) % 32 for i in range(32)], [i // 2 for i in range(32)]]),
])
def test_rows_follow_their_parents(fmt, P, W, hkv, lens, cols, parents):
    rows = Rows(lens, W, hkv, P, fmt, cols, seed=P + W)
    rows.run(parents)
    assert rows.beams.device_error() == 0


@pytest.mark.parametrize("fmt,layers", [("bf16", 3), ("q4", 2), ("bf16", 66)])
def test_layers_move_together(fmt, layers):
    rows = Rows([40] * 6, 3, 1, 16, fmt, 4, layers=layers)
    rows.run([[0, 0, 2], [1, 1, 1]])
    rows.run([[2, 0, 0], [2, 1, 0]])
    assert rows.beams.device_error() == 0


def test_many_steps_and_odd_tables():
    """Beams that grow and are moved many times never share a page that is still written."""
    W, P = 6, 16
    rows = Rows([5, 0, 0, 0, 0, 0] * 3, W, 2, P, "bf16", 9, seed=4)
    g = torch.Generator().manual_seed(1)
    rows.run([[0] * W] * 3)
    for step in range(120):
        rows.seq += rows.seq > 0
        rows.run([torch.randint(0, W, (W,), generator=g).tolist() for _ in range(3)])
        table, lens = rows.table.tolist(), rows.seq.tolist()
        for r in range(3):
            own = [p for w in range(W) for p in table[r * W + w][lens[r * W + w] // P:]]
            older = {p for w in range(W) for p in table[r * W + w][:lens[r * W + w] // P]}
            assert len(set(own)) == len(own) and not older & set(own)
    assert rows.beams.device_error() == 0


def test_without_counts_and_captured():
    rows = Rows([100] * 4, 4, 2, 64, "bf16", 4, seed=3)
    bare = [L.make_cache(k, v, rows.table, rows.seq) for k, v in rows.pools]
    array = (L.locks_cache_t * 1)(*bare)
    ws = torch.zeros(L.locksgen_reorder_workspace_size(bare[0], 4), dtype=torch.uint8, device="cuda")
    rows.nsum.zero_()
    rows.run([[1, 1, 3, 0]], lambda p: L.locksgen_reorder(array, 1, 4, p, ws, ws.numel()))
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    parents = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        rows.beams.reorder(parents)
    for mine in ([0, 1, 2, 3], [3, 3, 1, 3], [2, 0, 0, 1]):
        def call(p):
            parents.copy_(p)
            graph.replay()
            torch.cuda.synchronize()
        rows.run([mine], call)
    assert rows.beams.device_error() == 0


def test_what_only_the_device_can_see():
    rows = Rows([100] * 4, 4, 1, 64, "bf16", 3, seed=3)
    rows.beams.reorder(torch.tensor([[0, 4, -2, 0]], dtype=torch.int32).cuda())
    assert rows.beams.device_error() == L.LOCKSGEN_DEVERR_PARENT and rows.seq.tolist() == [100, 0, 0, 100]
    # the copy of a row shorter than the one whose pages it would take
    rows = Rows([100, 30, 100, 100], 4, 1, 64, "bf16", 3, seed=3)
    rows.run([[1, 1, 1, 0]])
    assert rows.beams.device_error() == L.LOCKS_DEVERR_LENGTHS and rows.seq.tolist() == [30, 0, 0, 100]
    # a row whose length no table holds has no copies, and its pages go to idle rows only
    for bad in (-5, 193):
        rows = Rows([100, bad, 100, 100], 4, 1, 64, "bf16", 3, seed=3)
        rows.beams.reorder(torch.tensor([[1, 0, 0, 3]], dtype=torch.int32).cuda())
        assert rows.beams.device_error() == L.LOCKS_DEVERR_LENGTHS
        # nobody's parents: 1 and 2; row 2, the other copy of row 0, comes first and gets row 1's
        assert rows.seq.tolist() == [0, 100, 0, 100]
    for bad in (-1, 1 << 20):
        rows = Rows([100] * 4, 4, 1, 64, "bf16", 3, seed=3)
        before = [x.clone() for x in rows.flat()]
        rows.table[2, 1] = bad
        rows.beams.reorder(torch.tensor([[2, 2, 2, 3]], dtype=torch.int32).cuda())
        assert rows.beams.device_error() == L.LOCKS_DEVERR_BLOCK_TABLE
        assert all(torch.equal(a, b) for a, b in zip(before, rows.flat()))


def test_refusals():
    rows = Rows([100] * 4, 4, 1, 64, "bf16", 3)
    good = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    for bad in (good.long(), good.view(4), good.cpu(), torch.zeros(1, 8, dtype=torch.int32, device="cuda")[:, ::2]):
        with pytest.raises(ValueError):
            rows.beams.reorder(bad)
    with pytest.raises(ValueError):
        LocksBeams(rows.rts, width=3)
    k, v = rows.pools[0]
    other = LocksRuntime(k, v, rows.table, rows.seq.clone(), rows.nsum, 1, 2, 0)
    with pytest.raises(ValueError):
        LocksBeams(rows.rts + [other], width=4)
    torch.cuda.synchronize()
    assert rows.seq.tolist() == [100] * 4 and rows.beams.device_error() == 0
