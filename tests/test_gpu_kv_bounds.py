"""4-bit pages at the largest scale that their format allows: every call that reads
them gives what 64 bits give.  Tolerances are those of the files that are imported."""

import re
from pathlib import Path

import pytest
import torch

from tests.kv_cases import D, Case, attend64, pack
from tests.test_gpu_kv_q4 import check as check_decode
from tests.test_gpu_prompt import check, cu_of

ROOT = Path(__file__).resolve().parents[1]


def max_scale():
    text = (ROOT / "include" / "locks.h").read_text()
    return float(re.search(r"#define LOCKS_KV_Q4_MAX_SCALE (\d+)", text).group(1))


def test_the_bound_is_the_largest_scale_with_a_finite_element():
    s = torch.tensor(max_scale())
    assert s.half().float() == s and torch.isfinite((s * 7).half())
    above = torch.nextafter(s.half().cpu(), torch.tensor(float("inf"), dtype=torch.float16)).float()
    assert torch.isinf((above * 7).half())


@pytest.mark.gpu
@pytest.mark.parametrize("where", ["k", "v", "both"])
@pytest.mark.parametrize("P,hq,hkv,n,new", [
    (64, 4, 1, 700, 5),     # few rows
    (64, 4, 1, 700, 60),    # codes
    (16, 4, 1, 700, 60),
    (64, 4, 1, 700, 300),   # planes
    (16, 16, 1, 700, 100),
])
def test_pages_at_the_bound(where, P, hq, hkv, n, new):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()
    case = Case([n], hq, hkv, P, "q4", seed=new)
    pages = case.k.shape[0]
    g = torch.Generator().manual_seed(new)
    kq, vq = (torch.randint(-7, 8, (pages, hkv, P, D), generator=g).float() for _ in range(2))
    small = torch.full((pages, hkv, P, 4), 0.1)
    bound = torch.full((pages, hkv, P, 4), max_scale())
    case.k.copy_(pack(kq, bound if where != "v" else small, vq, bound if where != "k" else small))
    rt = case.runtime()
    # logits of a few units either way
    q = case.query(new, spread=1.0 if where == "v" else 0.1 / max_scale())
    out, lse = rt.prompt_attend(q, cu_tokens=cu_of([new]), max_tokens=new)
    assert rt.device_error() == 0 and torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    check(case, [new], q, out, lse)
    last = q[-1:].contiguous()
    out, lse = rt.dense_decode(last)
    check_decode(case, last, out, lse)
    k, v = (x.transpose(0, 1).bfloat16() for x in case.kv64(0))
    got = rt.read_tokens(n, cu_tokens=cu_of([n]), max_tokens=n)
    assert rt.device_error() == 0
    for a, b in zip(got, (k, v)):
        assert torch.equal(a, b)
    # the page log-sum-exp of the first page
    lse = rt.exact_page_lse(last)[0, :, 0].double()
    for h in range(hq):
        _, rl, _, mag, _ = attend64(last[0, h:h + 1], case.kv64(0)[0][h * hkv // hq][:P], case.kv64(0)[1][h * hkv // hq][:P],
                                    ksc=case.scale64(0)[h * hkv // hq][:P])
        assert abs(float(lse[h] - rl)) <= float(2.0 ** -17 * mag + 2.0 ** -22 * (mag + 16) + P * 2.0 ** -24
                                                + 2.0 ** -22 * (rl.abs() + 17))
