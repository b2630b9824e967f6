"""Appending and reading of more rows than a CTA per token is used for, bit for bit as the
smaller calls are checked (see the file that is imported: no tolerance is needed)."""

import pytest
import torch

from tests.kv_cases import D, Case
from tests.test_gpu_kv_append import check_cache, quantised, rotated, rows_of, table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


MANY = [1, 0, 31, 64, 0, 17, 100] * 11  # 77 sequences, more than two rounds of the search for a row's


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("P,hq,hkv,lens,new,rot", [
    (64, 21, 3, [1500, 0, 90], [1490, 0, 77], 128),            # an odd number of rows, in several rounds of loads
    (16, 3, 1, [2000, 5], [1217, 5], 64),                      # fewer rows than one round
    (64, 32, 8, [n + 3 for n in MANY], MANY, 96),
    (16, 16, 1, [1300], [1300], 16),
    (64, 4, 4, [4000, 1], [3999, 1], 0),
])
def test_many_rows(fmt, interleaved, P, hq, hkv, lens, new, rot):
    case = Case(lens, hq, hkv, P, fmt, seed=rot + P + len(lens))
    rt = case.runtime()
    seq, at, cu = rows_of(lens, new)
    total, spare = sum(new), 5  # rows behind the last sequence
    assert total > 1216
    qkv = (torch.randn(total + spare, hq + 2 * hkv, D, generator=case.gen) * 3).bfloat16().cuda()
    qkv[:, :, 40] *= 20
    q, k, v = qkv.split([hq, hkv, hkv], dim=1)
    rope = table(max(lens) + 1, rot) if rot else None
    before = (case.k.clone(), None if case.v is None else case.v.clone())
    q_out = torch.full((total + spare, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    rt.append(k, v, q, rope=rope, interleaved=interleaved, cu_tokens=cu, max_tokens=max(new), q_out=q_out)
    assert rt.device_error() == 0
    assert torch.equal(q_out[:total], rotated(q[:total], rope, at, rot, interleaved).bfloat16())
    assert (q_out[total:] == 7).all()
    kr = rotated(k[:total], rope, at, rot, interleaved).bfloat16()
    check_cache(case, before, kr, v[:total], seq, at)
    ko, vo = rt.read_tokens(total + spare, cu_tokens=cu, max_tokens=max(new))
    assert rt.device_error() == 0
    for x, y in ((ko, kr), (vo, v[:total])):
        if fmt == "q4":
            c, s = quantised(y)
            y = (c.float() * s.float().repeat_interleave(32, dim=-1)).bfloat16()
        assert torch.equal(x[:total], y)
    # one of the two alone, and rows of nobody left as they were
    from sparse_kv_page_rank_gb300 import locks as L
    out = torch.full((total + spare, hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    for which, want in ((0, ko), (1, vo)):
        out.fill_(7)
        L.lockskv_read(rt.cache, L.make_tokens(cu, total + spare, max(new)), None if which else out, out if which else None)
        assert torch.equal(out[:total], want[:total]) and (out[total:] == 7).all()
    # in place, and without queries, the cache gets the same
    other = Case(lens, hq, hkv, P, fmt, seed=rot + P + len(lens))
    ort = other.runtime()
    wide = qkv.clone()
    wq, wk, wv = wide.split([hq, hkv, hkv], dim=1)
    ort.append(wk, wv, wq, rope=rope, interleaved=interleaved, cu_tokens=cu, q_out=wq)
    assert torch.equal(wq[:total], q_out[:total]) and torch.equal(wide[total:], qkv[total:])
    assert torch.equal(wide[:, hq:], qkv[:, hq:])
    assert torch.equal(other.k.view(torch.uint8), case.k.view(torch.uint8))


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_many_sequences_of_one_token(fmt):
    """More idle and live slots than a CTA per token is used for."""
    B = 1300
    lens = [(7 * b) % 40 for b in range(B)]
    case = Case(lens, 4, 2, 16, fmt, seed=4)
    rt = case.runtime()
    q, k, v = (torch.randn(B, h, D, generator=case.gen).bfloat16().cuda() for h in (4, 2, 2))
    rope = table(50, 128)
    before = (case.k.clone(), None if case.v is None else case.v.clone())
    q_in = q.clone()
    rt.append(k, v, q, rope=rope, q_out=q)
    assert rt.device_error() == 0
    n = torch.tensor(lens, device="cuda")
    live, idle = n.nonzero().flatten(), (n == 0).nonzero().flatten()
    at = n[live] - 1
    assert torch.equal(q[live], rotated(q_in[live], rope, at, 128, False).bfloat16())
    assert torch.equal(q[idle], q_in[idle])
    check_cache(case, before, rotated(k[live], rope, at, 128, False).bfloat16(), v[live], live, at)


def test_what_only_the_device_can_see_of_many_rows():
    from sparse_kv_page_rank_gb300 import locks as L
    case = Case([1400, 20], 4, 2, 16, "bf16", seed=6)
    rt = case.runtime()
    k, v = (torch.randn(1410, 2, D, generator=case.gen).bfloat16().cuda() for _ in range(2))
    rope = table(1399, 64)

    def call(cu, **kw):
        rt.append(k, v, cu_tokens=torch.tensor(cu, dtype=torch.int32).cuda(), **kw)
        return rt.device_error()

    assert call([0, 1390, 1410]) == 0
    assert call([0, 1390, 1410], rope=rope) == L.LOCKS_DEVERR_POSITION
    assert call([0, 1380, 1410]) == L.LOCKS_DEVERR_LENGTHS
    assert call([0, 1390, 1410], max_tokens=1300) == L.LOCKS_DEVERR_LENGTHS
    case.table[0, 70] = 1 << 20
    assert call([0, 1390, 1410]) == L.LOCKS_DEVERR_BLOCK_TABLE
