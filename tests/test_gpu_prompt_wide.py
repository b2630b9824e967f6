"""Attention of new tokens where the block table is much wider than the sequences: the
same results in every form, among them the one that takes 4-bit pages' codes apart for
many row tiles, which only a table too wide for planes brings about.  Tolerances are
those of the file that is imported."""

import pytest
import torch

from tests.kv_cases import Case
from tests.test_gpu_prompt import check, cu_of

pytestmark = pytest.mark.gpu

PLANE_LIMIT = 4 << 30  # bytes of fp16 planes beyond which codes are converted in place


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


def beyond_planes(batch, hkv, P):
    """Columns of a table whose planes would exceed the limit."""
    return PLANE_LIMIT // (3 * batch * hkv * P * 256) + 1


@pytest.mark.parametrize("P,hq,hkv,lens,new", [
    (64, 32, 8, [3000], [600]),
    (16, 32, 8, [2500, 70, 0], [500, 70, 0]),
    (64, 8, 8, [1500, 900], [1500, 257]),
    (64, 48, 3, [2000], [700]),
])
def test_codes_for_many_tiles(P, hq, hkv, lens, new):
    case = Case(lens, hq, hkv, P, "q4", seed=sum(lens), extra_cols=beyond_planes(len(lens), hkv, P))
    rt, q = case.runtime(), case.query(sum(new), spread=1.5)
    first = None
    for _ in range(10):
        out, lse = rt.prompt_attend(q, cu_tokens=cu_of(new), max_tokens=max(new))
        assert first is None or (torch.equal(out, first[0]) and torch.equal(lse, first[1]))
        first = out, lse
    assert rt.device_error() == 0 and rt.prompt_ws.numel() < 1 << 30
    check(case, new, q, out, lse)


def test_codes_over_a_long_cache():
    """Some 300 blocks of codes per tile, again and again."""
    case = Case([40000], 4, 1, 64, "q4", seed=2)
    rt, q = case.runtime(), case.query(90)
    first = None
    for _ in range(50):
        out, lse = rt.prompt_attend(q, cu_tokens=cu_of([90]), max_tokens=90)
        assert first is None or (torch.equal(out, first[0]) and torch.equal(lse, first[1]))
        first = out, lse
    assert rt.device_error() == 0
    check(case, [90], q, out, lse)


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("P", [64, 16])
@pytest.mark.parametrize("new", [[2, 0, 3, 1], [60, 0, 33, 1], [300, 0, 299, 5]])
def test_short_sequences_in_a_wide_table(fmt, P, new):
    case = Case([700, 5, 300, 130], 8, 2, P, fmt, seed=P + sum(new), extra_cols=131072 // P)
    rt, q = case.runtime(), case.query(sum(new))
    out, lse = rt.prompt_attend(q, cu_tokens=cu_of(new), max_tokens=max(new))
    assert rt.device_error() == 0
    check(case, new, q, out, lse)
    q = case.query(4)
    out, lse = rt.dense_decode(q)
    assert rt.device_error() == 0
    check(case, [1] * 4, q, out, lse)
