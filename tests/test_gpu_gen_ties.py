"""Continuations that score the same in 64 bits although their logits differ: the lower beam, then the
larger logit, then the lower token, however many there are. Exact, no tolerance."""

import math

import pytest
import torch

from sparse_kv_page_rank_gb300.beams import LocksBeams

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


def by_logit(x):
    """Tokens of rows x [..., V], the larger logit first, then the lower token."""
    return (x.float() + 0.0).sort(dim=-1, descending=True, stable=True).indices


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("keep", [1, 4, 17, 64])
@pytest.mark.parametrize("score", [-3.0, -1e8, -1e15, -1e30, -3e38])
def test_one_beam_goes_by_its_logits(dtype, keep, score):
    g = torch.Generator().manual_seed(keep)
    for V in (40, 700, 9000, 60000):
        x = torch.randn(3, V, generator=g)
        x[1] *= 1e-20
        x[2].masked_fill_(torch.rand(V, generator=g) < 0.5, -math.inf)
        x = x.to(dtype)
        beams = LocksBeams(width=1)
        got = beams.select(x.cuda(), torch.full((3, 1), score).cuda(), keep=keep)
        assert beams.device_error() == 0
        n = min(keep, V)
        want = by_logit(x)[:, :n]
        live = torch.gather(x, 1, want) > -math.inf
        assert torch.equal(got[2][:, :n].cpu().long(), want.masked_fill(~live, -1)), V


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [30, 900, 20000])
@pytest.mark.parametrize("keep", [1, 3, 16, 40, 64])
def test_beams_that_tie(dtype, V, keep):
    """All logits are tiny and differ: all continuations of equal hypotheses score the same."""
    g = torch.Generator().manual_seed(V + keep)
    W = 4
    x = (torch.randn(2, W, V, generator=g) * 1e-20).to(dtype)
    scores = torch.tensor([[-4.0, -3.0, -5.0, -3.0], [-3.0, -math.inf, -3.0, -3.0]])
    beams = LocksBeams(width=W)
    _, parents, tokens, _ = (None if t is None else t.cpu() for t in beams.select(x.cuda(), scores.cuda(), keep=keep))
    assert beams.device_error() == 0
    for b, order in enumerate(([1, 3, 0, 2], [0, 2, 3])):
        want = [(w, t) for w in order for t in by_logit(x[b, w]).tolist()][:keep]
        assert list(zip(parents[b].tolist(), tokens[b].tolist()))[:len(want)] == want


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ended_beams_that_tie(dtype):
    """An ended hypothesis and continuations with its score."""
    V, end, W = 500, 77, 3
    x = (torch.randn(1, W, V, generator=torch.Generator().manual_seed(3)) * 1e-20).to(dtype)
    lse = torch.tensor(float(V), dtype=torch.float64).log()
    scores = torch.tensor([[-2.0, 0.0, -2.0]])
    scores[0, 1] = -2.0  # a live beam's continuations are ln V lower
    ended = torch.tensor([[1, 0, 1]], dtype=torch.int32)
    beams = LocksBeams(width=W, end_token=end)
    got = [t.cpu() for t in beams.select(x.cuda(), scores.cuda(), ended.cuda(), keep=5)]
    want = [(0, end), (2, end)] + [(1, t) for t in by_logit(x[0, 1]).tolist()[:3]]
    assert list(zip(got[1][0].tolist(), got[2][0].tolist())) == want
    assert got[3][0].tolist() == [1, 1] + [int(t == end) for _, t in want[2:]]
    assert (got[0][0, 2:].double() - (-2.0 - lse)).abs().max() < 1e-5
