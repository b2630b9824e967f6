"""max_tokens may be any number that is at least every sequence's new tokens."""

import pytest
import torch

from sparse_kv_page_rank_gb300 import locks as L
from sparse_kv_page_rank_gb300.build_lib import build
from tests.kv_cases import D, Case
from tests.test_gpu_prompt import check, cu_of

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("P,hq,hkv,batch,cols", [(64, 32, 8, 1, 128), (16, 4, 4, 3, 77), (64, 16, 1, 2, 2000), (16, 1, 1, 1, 1),
                                                 (64, 64, 64, 64, 2048)])
def test_the_plan_for_no_known_bound_is_that_of_the_whole_table(fmt, P, hq, hkv, batch, cols):
    build()
    c = L.locks_cache_t(k_pool=0x1000, v_pool=0x2000, block_table=0x3000, seq_lens=0x4000, batch=batch, num_kv_heads=hkv,
                        head_dim=128, page_size=P, pages_total=100, max_pages=cols, kv_format=fmt)
    p = L.make_params(hq, 0)
    want = L.lockskv_prompt_workspace_size(c, p, L.make_tokens(0xB000, 1000, cols * P))
    for most in (cols * P + 1, 1 << 30, MOST - 127, MOST):
        assert L.lockskv_prompt_workspace_size(c, p, L.make_tokens(0xB000, 1000, most)) == want


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("P,hq,hkv,lens,new", [(64, 4, 1, [700, 90], [400, 3]), (16, 8, 2, [40, 300, 5], [40, 200, 0]),
                                               (16, 1, 1, [16], [9])])
@pytest.mark.parametrize("most", [1 << 30, MOST])
def test_no_row_is_left_out_without_a_known_bound(fmt, P, hq, hkv, lens, new, most):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    case = Case(lens, hq, hkv, P, fmt, seed=sum(lens), extra_cols=0)
    rt, total = case.runtime(), sum(new)
    k, v = (torch.randn(total, hkv, D, generator=case.gen).bfloat16().cuda() for _ in range(2))
    rt.append(k, v, cu_tokens=cu_of(new), max_tokens=most)
    got = rt.read_tokens(total, cu_tokens=cu_of(new), max_tokens=most)
    known = rt.read_tokens(total, cu_tokens=cu_of(new), max_tokens=max(new))
    assert all(torch.equal(a, b) for a, b in zip(got, known))
    q = case.query(total)
    out, lse = rt.prompt_attend(q, cu_tokens=cu_of(new), max_tokens=most)
    assert rt.device_error() == 0
    check(case, new, q, out, lse)
