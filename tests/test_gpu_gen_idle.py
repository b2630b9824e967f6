"""A live row's results are its own: what stands in the queries of idle rows of its request, which
append leaves as they were, has no part in a bit of them; nor have the queries of other live rows."""

import math

import pytest
import torch

from sparse_kv_page_rank_gb300.beams import LocksBeams
from tests.gen_cases import shared_case
from tests.test_gpu_gen_attend import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


def fills(g, shape):
    """What memory may hold: nothing, small and large numbers, and none."""
    yield torch.zeros(shape)
    for spread in (0.1, 3.0, 30.0, 1e4, 1e30):
        yield torch.randn(shape, generator=g) * spread
    for x in (math.nan, math.inf, -math.inf):
        yield torch.full(shape, x)
    mixed = torch.randn(shape, generator=g) * 20
    mixed[..., ::7] = math.nan
    yield mixed


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("P", [64, 16])
@pytest.mark.parametrize("prompts,tails,hq,hkv", [
    # long enough for several tiles in each CTA's piece
    ([16000], [[20, None, 20, None, 21, None, None, 9]], 32, 8),  # 32 rows of a pass, half of them idle
    ([9000, 7000], [[None, 5, 6, None], [40, None, None, 41]], 16, 8),
    ([16000], [[3, None, 3]], 16, 8),                             # up to 16 rows of a pass
    ([500, 70], [[3, None, 3], [None, 9, 9]], 4, 1),
])
def test_queries_of_idle_rows(fmt, P, prompts, tails, hq, hkv):
    case, W, shared = shared_case(prompts, tails, hq, hkv, P, fmt, seed=P + hq)
    beams = LocksBeams([case.runtime()], width=W)
    q = case.query(case.B)
    idle = [b for b, n in enumerate(case.lens) if n == 0]
    first = None
    for fill in fills(case.gen, (len(idle), hq, 128)):
        q[idle] = fill.bfloat16().cuda()
        out, lse = beams.attend(q, shared)
        if first is None:
            first = out.clone(), lse.clone()
            check(case, q, out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert beams.device_error() == 0


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("P", [64, 16])
def test_queries_of_other_live_rows(fmt, P):
    case, W, shared = shared_case([16000], [[20, 20, 20, 20]], 32, 8, P, fmt, seed=P)
    beams = LocksBeams([case.runtime()], width=W)
    q = case.query(case.B)
    first = [x.clone() for x in beams.attend(q, shared)]
    for fill in fills(case.gen, (2, 32, 128)):
        q[1::2] = fill.bfloat16().cuda()
        out, lse = beams.attend(q, shared)
        assert torch.equal(out[::2], first[0][::2]) and torch.equal(lse[::2], first[1][::2])
    assert beams.device_error() == 0
