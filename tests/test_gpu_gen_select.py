"""Choosing beams, against all candidates in 64 bits.

Tolerance.  A score is s + x - lse, added in 64 bits and rounded once (2^-24 of it).  The
sum of exponentials is of float32: every term is off by 2^-22 (the exponential), 2^-24 of the
distance d to the maximum (the difference) and of its exponent (one rounding); the mean of d
under the weights of the largest-entropy row is below ln(vocab) < 13, and 64 additions
in turn or in trees add 2^-24 each at most: together 4 + 2 * 13 + 64 + 2 < 96 times 2^-24.
Candidates closer than twice that to each other, but not equal, may come in either order."""

import math

import pytest
import torch

from sparse_kv_page_rank_gb300 import locks as L
from sparse_kv_page_rank_gb300.beams import LocksBeams
from tests.gen_cases import candidates64

pytestmark = pytest.mark.gpu
TOL = 96 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


def check(got, logits, scores, ended, end_token, keep):
    B, W, V = logits.shape
    s = candidates64(logits, scores, ended, end_token).cpu()
    value, index = s.flatten(1).sort(dim=1, descending=True, stable=True)
    out_s, out_p, out_t, out_e = [None if x is None else x.cpu() for x in got]
    for b in range(B):
        n = min(keep, int((value[b] > -math.inf).sum()))
        assert (out_s[b, n:] == -math.inf).all() and (out_p[b, n:] == -1).all() and (out_t[b, n:] == -1).all()
        assert out_e is None or (out_e[b, n:] == 0).all()
        flat = out_p[b, :n].long() * V + out_t[b, :n].long()
        assert (out_p[b, :n] >= 0).all() and (out_p[b, :n] < W).all() and (out_t[b, :n] >= 0).all() and (out_t[b, :n] < V).all()
        assert flat.unique().numel() == n
        mine = s[b].flatten()[flat]
        assert ((out_s[b, :n].double() - mine).abs() <= TOL + 2.0 ** -24 * mine.abs()).all()
        for i in (flat != index[b, :n]).nonzero().flatten().tolist():
            # another order of what is not told apart, but never of what is equal
            assert 0 < abs(mine[i] - value[b, i]) <= 2 * TOL, (b, i, flat[i], index[b, i])
        if out_e is not None:
            old = torch.zeros(W, dtype=torch.int32) if ended is None else ended[b].cpu()
            assert torch.equal(out_e[b, :n] != 0, (old[out_p[b, :n].long()] != 0) | (out_t[b, :n] == end_token))


def make(B, W, V, dtype, seed, spread=3.0, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, W, V, generator=g) * spread
    if masked:
        x.masked_fill_(torch.rand(B, W, V, generator=g) < masked, -math.inf)
    scores = -(torch.randn(B, W, generator=g).abs() * 0.7 + 5)
    return x.to(dtype).cuda(), scores.cuda(), g


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,W,V,keep", [
    (1, 1, 1, 1), (1, 1, 5, 8), (2, 3, 7, 4), (1, 4, 32000, 4), (3, 8, 50257, 16), (2, 32, 8192, 64), (1, 32, 8185, 32),
    (5, 5, 8193, 5), (2, 2, 100003, 17), (1, 16, 128256, 33), (40, 4, 1000, 8), (1, 2, 300000, 16),
])
def test_sizes(dtype, B, W, V, keep):
    logits, scores, _ = make(B, W, V, dtype, seed=V + keep)
    beams = LocksBeams(width=W)
    got = beams.select(logits.view(B * W, V), scores, keep=keep)
    assert got[3] is None and beams.device_error() == 0
    check(got, logits, scores, None, -1, keep)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_at_any_alignment(dtype):
    V, W = 9001, 3
    wide = (torch.randn(2 * W, V + 40) * 3).to(dtype).cuda()
    for off in range(9):
        for logits in (wide[:, off:off + V], wide.flatten()[off:off + 2 * W * (V + 3)].view(2 * W, V + 3)[:, :V]):
            beams = LocksBeams(width=W)
            scores = torch.tensor([[-1.0, -2.0, -0.5]] * 2).cuda()
            got = beams.select(logits, scores)
            check(got, logits.reshape(2, W, V), scores, None, -1, W)
    # beams as an axis, and one row of a taller array
    x = (torch.randn(4, 2 * W, V) * 3).to(dtype).cuda()
    got = LocksBeams(width=W).select(x[:1, ::2], torch.zeros(1, W).cuda())
    check(got, x[:1, ::2], torch.zeros(1, W).cuda(), None, -1, W)
    got = LocksBeams(width=W).select(x[:, ::2], torch.zeros(4, W).cuda())
    check(got, x[:, ::2], torch.zeros(4, W).cuda(), None, -1, W)
    with pytest.raises(ValueError, match="logits"):  # rows that are not equally far apart
        LocksBeams(width=W).select(x[:2, :W], torch.zeros(2, W).cuda())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties_go_to_the_lowest(dtype):
    B, W, V = 2, 4, 20000
    for kind in ("equal", "few", "rising", "twins"):
        if kind == "equal":
            x = torch.zeros(B, W, V)
        elif kind == "few":
            x = torch.randint(0, 3, (B, W, V), generator=torch.Generator().manual_seed(1)).float()
        elif kind == "rising":  # the best of a part all in one place
            x = (torch.arange(V) // 64).float().expand(B, W, V).clone() / 32
        else:
            x = (torch.randn(B, 1, V, generator=torch.Generator().manual_seed(2)) * 3).expand(B, W, V).clone()
        x[1] = -x[1]  # negative zeros among them
        x, scores = x.to(dtype).cuda(), torch.full((B, W), -3.0).cuda()
        for keep in (1, 4, 16, 17, 64):
            got = LocksBeams(width=W).select(x, scores, keep=keep)
            s = candidates64(x, scores, None, -1).flatten(1)
            index = s.sort(dim=1, descending=True, stable=True).indices[:, :keep]
            assert torch.equal(got[1].long() * V + got[2].long(), index), (kind, keep)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masks(dtype):
    V, W, low = 12345, 4, torch.finfo(dtype).min
    logits, scores, g = make(6, W, V, dtype, seed=7, masked=0.9)
    logits[0, 1] = -math.inf                         # nothing left
    logits[1] = -math.inf                            # nothing at all
    logits[2, 0, 5:] = -math.inf                     # five candidates
    logits[2, 1:] = -math.inf
    logits[3] = low                                  # the type's lowest value everywhere
    logits[4] = torch.where(logits[4] == -math.inf, torch.tensor(low, dtype=dtype, device="cuda"), logits[4])
    scores[5, 1:] = -math.inf                        # the first step: one hypothesis
    logits[5, 1] = math.nan                          # whose others' logits are not read
    beams = LocksBeams(width=W)
    got = beams.select(logits, scores, keep=8)
    assert beams.device_error() == 0
    check(got, logits, scores, None, -1, 8)
    assert (got[1][1] == -1).all() and int((got[1][2] >= 0).sum()) <= 5 and (got[1][5] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ended_hypotheses(dtype):
    B, W, V, end = 3, 5, 3001, 77
    logits, scores, g = make(B, W, V, dtype, seed=8)
    ended = torch.tensor([[0, 1, 0, 0, 2], [1, 1, 1, 1, 1], [0, 0, 0, 0, 0]], dtype=torch.int32).cuda()
    scores[0, 1], scores[0, 4] = -1.0, -50.0
    logits[0, 1] = math.nan  # not read
    logits[2, 3, end] = 60   # ends now
    beams = LocksBeams(width=W, end_token=end)
    got = beams.select(logits, scores, ended)
    assert beams.device_error() == 0
    x = torch.nan_to_num(logits, nan=0.0)
    check(got, x, scores, ended, end, W)
    assert got[3][1].all() and int(got[3][2, 0]) == 1 and int(got[2][2, 0]) == end
    # in place
    s2, e2, want = scores.clone(), ended.clone(), [x.clone() for x in got]
    again = beams.select(logits, s2, e2, out_scores=s2, out_ended=e2)
    assert all(torch.equal(a, b) for a, b in zip(again, want)) and again[0] is s2 and again[3] is e2
    # and the object's own outputs handed back
    second = beams.select(logits, got[0], got[3])
    assert all(a is b for a, b in zip(second, got))
    check(second, x, want[0], want[3], end, W)


def test_bad_numbers_are_told_and_kept_out():
    V, W = 9000, 3
    for place, bad in ((8999, math.nan), (0, math.inf), (8200, -math.nan)):
        logits, scores, _ = make(2, W, V, torch.float32, seed=3)
        logits[0, 1, place] = bad
        beams = LocksBeams(width=W)
        got = beams.select(logits, scores)
        assert beams.device_error() == L.LOCKSGEN_DEVERR_LOGITS and beams.device_error() == 0
        clean = scores.clone()
        clean[0, 1] = -math.inf
        check(got, torch.nan_to_num(logits), clean, None, -1, W)
    for bad in (math.nan, math.inf):
        logits, scores, _ = make(2, W, V, torch.float32, seed=3)
        scores[1, 2] = bad
        beams = LocksBeams(width=W)
        got = beams.select(logits, scores)
        assert beams.device_error() == L.LOCKSGEN_DEVERR_LOGITS
        scores[1, 2] = -math.inf
        check(got, logits, scores, None, -1, W)
    # a row whose other entries are all masked
    logits = torch.full((1, 1, 10), -math.inf).cuda()
    logits[0, 0, 3] = math.nan
    beams = LocksBeams(width=1)
    assert int(beams.select(logits, torch.zeros(1, 1).cuda())[1][0, 0]) == -1
    assert beams.device_error() == L.LOCKSGEN_DEVERR_LOGITS


def test_the_same_bits_every_time_and_from_a_graph():
    logits, scores, _ = make(7, 6, 33333, torch.bfloat16, seed=5)
    beams = LocksBeams(width=6, end_token=2)
    ended = torch.zeros(7, 6, dtype=torch.int32).cuda()
    first = [x.clone() for x in beams.select(logits, scores, ended, keep=12)]
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(first, beams.select(logits, scores, ended, keep=12)))
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        out = beams.select(logits, scores, ended, keep=12)
    for seed in (5, 6):
        logits.copy_(make(7, 6, 33333, torch.bfloat16, seed=seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        check(out, logits, scores, ended, 2, 12)
    with pytest.raises(RuntimeError, match="before the capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=stream):
            beams.select(logits, scores, ended, keep=64)
    torch.cuda.synchronize()
    # a larger call beside it leaves the graph its workspace
    beams.select(logits, scores, ended, keep=64)
    graph.replay()
    torch.cuda.synchronize()
    check(out, logits, scores, ended, 2, 12)
    assert beams.device_error() == 0


def test_no_requests():
    got = LocksBeams(width=4).select(torch.empty(0, 100, device="cuda"), torch.empty(0, 4, device="cuda"))
    assert got[0].shape == (0, 4)


def test_refusals():
    logits, scores, _ = make(2, 3, 100, torch.float32, seed=1)
    beams, ended = LocksBeams(width=3), torch.zeros(2, 3, dtype=torch.int32).cuda()
    for args, kw in (((logits.half(), scores), {}), ((logits.transpose(1, 2), scores), {}), ((logits[:, :2], scores), {}),
                     ((logits, scores[:1]), {}), ((logits, scores.double()), {}), ((logits, scores, ended), {}),
                     ((logits, scores), dict(out_scores=scores.double())), ((logits, scores), dict(out_tokens=ended[:, :2])),
                     ((logits.cpu(), scores), {}), ((logits[0, :2], scores), {})):
        with pytest.raises(ValueError):
            beams.select(*args, **kw)
    for kw in (dict(keep=0), dict(keep=65)):
        with pytest.raises(L.LocksError):
            beams.select(logits, scores, **kw)
    with pytest.raises(L.LocksError):
        LocksBeams(width=3, end_token=100).select(logits, scores, ended)
    for width in (0, 33):
        with pytest.raises(ValueError):
            LocksBeams(width=width)
    with pytest.raises(ValueError):
        beams.reorder(ended)
    with pytest.raises(ValueError):
        beams.attend(logits, ended)
