"""Attention of rows that share pages, against 64 bits and against the dense decode.

Tolerances, half a step per rounding.  Logits: 128 exact products added in float32, 2^-24 of
sum |q||k| each (4-bit pages: 32 at a time, then four scaled sums: no more), so a weight is off by
e = 2^-17 sum |q||k| scale + 2^-21 (the exponential and the exponent's rounding, of at most 2^6 in
base 2 for a weight that counts).  bf16 pages: the softmax weights are rounded to bf16, 2^-8.  4-bit
pages: weights and values s * code are rounded to half precision, 2^-11 each; a weight below
2^-14 is off by half of half precision's smallest step, 2^-25, where the row's largest is at
least 2^7, so by 2^-32 of that, which is no more than 1: 2^-32 sum |v| over all tokens.  The sums over
tokens and the joins are float32 (2^-12 for all, up to 2^12 additions in turn); the output is rounded
to bf16, 2^-8 of itself.  lse: the sum's share of the same."""

import math

import pytest
import torch

from sparse_kv_page_rank_gb300 import locks as L
from sparse_kv_page_rank_gb300.beams import LocksBeams
from tests.gen_cases import shared_case
from tests.kv_cases import D, attend64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


def check(case, q, out, lse, scale=None):
    g = case.hq // case.hkv
    for b, n in enumerate(case.lens):
        if n == 0:
            assert (out[b] == 0).all() and (lse[b] == -math.inf).all()
            continue
        k, v = case.kv64(b)
        for h in range(case.hkv):
            s = slice(h * g, h * g + g)
            o, l, mean, _, mag = attend64(q[b, s], k[h], v[h], scale=scale)
            e = 2.0 ** -17 * mag + 2.0 ** -21
            assert ((lse[b, s].double() - l).abs() <= e + 2.0 ** -12 + 2.0 ** -24 * l.abs()).all(), (b, h)
            weights = 2.0 ** -8 if case.fmt == "bf16" else 2.0 ** -10
            tol = (weights + 2.0 ** -12 + 2 * e[:, None]) * mean + 2.0 ** -8 * o.abs()
            if case.fmt == "q4":
                tol = tol + 2.0 ** -32 * v[h].abs().sum(dim=0)
            bad = (out[b, s].double() - o).abs() > tol
            assert not bad.any(), (b, h, (out[b, s].double() - o).abs().max())


CASES = [
    # prompts, tails by row (None: idle), hq, hkv, P
    ([130], [[3, 1, 3, 3]], 8, 2, 64),
    ([1000, 65, 700], [[90, 90], [64, 0], [200, 7]], 8, 8, 64),
    ([64], [[0, 0, 0]], 4, 1, 64),                                    # nothing but shared pages
    ([63, 1], [[1, 2], [5, 70]], 4, 4, 64),                           # no shared page
    ([333], [[10] * 8], 32, 8, 16),
    ([333, 50, 17], [[10] * 5, [0] * 5, [40, None, 40, 3, None]], 6, 2, 16),
    ([500], [[None, 20, None, 20]], 8, 2, 64),                        # the first row is idle
    ([500, 300], [[None, 20, None], [None, None, None]], 8, 2, 64),   # one row shares with nobody; an idle request
    ([2000], [[31]], 16, 1, 64),                                      # one beam, 16 heads
    ([1025], [[100] * 32], 4, 4, 16),                                 # 32 rows exactly
    ([1025], [[100] * 11], 9, 3, 64),                                 # 33 rows: two blocks, one of one row
    ([700], [[5, 9, 14, 100, 64, 63, 65]], 32, 2, 64),                # 16 heads x 7: four blocks
    ([15, 31, 16], [[0, 1, 2], [3, 0, 33], [1, 16, 17]], 3, 1, 16),
    ([1], [[0, 0]], 1, 1, 64),
    ([20011], [[77, 90, 100, 100]], 8, 2, 64),
    ([9000] * 12, [[13, 100]] * 12, 8, 4, 16),
]


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("prompts,tails,hq,hkv,P", CASES)
def test_cases(fmt, prompts, tails, hq, hkv, P):
    case, W, shared = shared_case(prompts, tails, hq, hkv, P, fmt, seed=hq + P + len(prompts))
    beams = LocksBeams([case.runtime()], width=W)
    q = case.query(case.B)
    out, lse = (x.clone() for x in beams.attend(q, shared))
    assert beams.device_error() == 0
    check(case, q, out, lse)
    # any smaller count of shared pages is right too, and a larger one is cut to the shortest row's
    fewer = (shared // 2).contiguous()
    other, lse2 = beams.attend(q, fewer)
    check(case, q, other, lse2)
    again, lse3 = beams.attend(q, shared)
    assert torch.equal(out, again) and torch.equal(lse, lse3)
    assert beams.device_error() == 0


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_counts_beyond_the_rows(fmt):
    case, W, shared = shared_case([300], [[0, 0]], 4, 2, 64, fmt, seed=5)
    beams = LocksBeams([case.runtime()], width=W)
    q = case.query(case.B)
    for n in (4, 5, 1 << 30, -3):
        out, lse = beams.attend(q, torch.full_like(shared, n))
        check(case, q, out, lse)
    assert beams.device_error() == 0


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_scale_and_large_values(fmt):
    case, W, shared = shared_case([700], [[33, 40, 1]], 8, 2, 64, fmt, seed=11)
    rt = case.runtime()
    rt.params.scale = 0.5
    beams = LocksBeams([rt], width=W)
    q = case.query(case.B, spread=6.0)
    out, lse = beams.attend(q, shared)
    check(case, q, out, lse, scale=0.5)


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_numbers_that_are_not_finite(fmt):
    """In a page that rows see they reach those rows' results only; past a row's end none."""
    case, W, shared = shared_case([100, 100], [[30, 40], [30, 40]], 4, 1, 64, fmt, seed=12)
    q = case.query(case.B)
    beams = LocksBeams([case.runtime()], width=W)
    clean = beams.attend(q, shared)[0].clone()
    page, slot = int(case.table[1, 2]), 3  # token 131 of row 1
    if fmt == "bf16":
        case.v[page, 0, slot, 7] = float("nan")
    else:
        block = case.k[page, 0]
        where = 136 * 64 + 32 * (slot % 8 // 2) + 2 * (slot % 2)  # its value scale of dimensions 0 .. 31
        block[where:where + 2] = torch.tensor([0, 0x7e], dtype=torch.uint8)
    out, _ = beams.attend(q, shared)
    assert torch.isnan(out[1]).any() and torch.equal(out[[0, 2, 3]], clean[[0, 2, 3]])


def test_differing_tables_are_told():
    case, W, shared = shared_case([300], [[10, 10, 10]], 4, 2, 64, "bf16", seed=5)
    beams = LocksBeams([case.runtime()], width=W)
    q = case.query(case.B)
    case.table[2, 1] = case.table[2, 4]
    beams.attend(q, shared)
    assert beams.device_error() == L.LOCKS_DEVERR_BLOCK_TABLE


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_bad_pages_and_lengths_are_skipped(fmt):
    case, W, shared = shared_case([300, 200], [[10, 10], [5, 6]], 4, 2, 64, fmt, seed=5)
    beams = LocksBeams([case.runtime()], width=W)
    q = case.query(case.B)
    good = beams.attend(q, shared)[0].clone()
    case.table[0, 4] = 1 << 24   # a page of row 0's own
    out, _ = beams.attend(q, shared)
    assert beams.device_error() == L.LOCKS_DEVERR_BLOCK_TABLE and torch.equal(out[1:], good[1:])
    case.table[2:4, 1] = -1      # a shared page of request 1
    out, _ = beams.attend(q, shared)
    assert beams.device_error() == L.LOCKS_DEVERR_BLOCK_TABLE and torch.equal(out[1], good[1])
    assert torch.isfinite(out).all()
    case.table[0, 4] = 0
    case.table[2:4, 1] = 0
    case.seq[0] = -4
    out, lse = beams.attend(q, shared)
    assert beams.device_error() == L.LOCKS_DEVERR_LENGTHS and (out[0] == 0).all() and (lse[0] == -math.inf).all()


def test_close_to_the_dense_decode_and_captured():
    case, W, shared = shared_case([3000, 900], [[64, 65, 66, 67], [64, 65, 66, 67]], 16, 4, 64, "bf16", seed=21)
    rt = case.runtime()
    beams, q = LocksBeams([rt], width=W), case.query(case.B)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    out, lse = torch.empty_like(q), torch.empty(case.B, 16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        beams.attend(q, shared, out=out, lse=lse)
    for n in (0, 1):
        case.seq -= n
        case.lens = [x - n for x in case.lens]
        q.copy_(case.query(case.B))
        graph.replay()
        torch.cuda.synchronize()
        check(case, q, out, lse)
        dense, dl = rt.dense_decode(q)
        assert (dl - lse).abs().max() < 1e-3 and (dense.float() - out.float()).abs().max() < 0.05
    # on a stream of its own, its outputs that stream's
    with torch.cuda.stream(stream):
        stream.wait_stream(torch.cuda.default_stream())
    o2, l2 = beams.attend(q, shared, stream=stream)
    stream.synchronize()
    assert torch.equal(o2, out) and torch.equal(l2, lse) and beams.device_error() == 0


def test_refusals():
    case, W, shared = shared_case([300], [[10, 10]], 4, 2, 64, "bf16", seed=5)
    beams, q = LocksBeams([case.runtime()], width=W), case.query(case.B)
    wide = torch.zeros(2, 8, D, dtype=torch.bfloat16, device="cuda")
    for args, kw in (((q.float(), shared), {}), ((q[:1], shared), {}), ((wide[:, ::2], shared), {}), ((q, shared.long()), {}),
                     ((q, shared.repeat(2)), {}), ((q, shared.cpu()), {}), ((q, shared), dict(out=q[:1])),
                     ((q, shared), dict(lse=torch.zeros(2, 4, device="cuda", dtype=torch.float64)))):
        with pytest.raises(ValueError):
            beams.attend(*args, **kw)
    with pytest.raises(IndexError):
        beams.attend(q, shared, layer=1)
    assert beams.device_error() == 0
