"""What the softmax weights of the 4-bit decode keep of tokens far below the largest,
and of value scales of any size.

Tolerances, besides those of an ordinary decode.  A warp's largest weight is at least 2^11
once it has seen its largest token, its largest value scale at least 1/4 of their limit.  Each of
the two roundings of a weight is off by 2^-11 of it or by 2^-25: by 2^-36 of the largest
weight, and by 2^-36 of the largest weight times the limit, which is at most four times
the largest scale; with codes up to 7 that is 2^-36 (1 + 4) per token, times the largest
value, relative to the largest token's share of the sum."""

import math

import pytest
import torch

from tests.kv_cases import D, Case, attend64, pack
from tests.test_gpu_kv_q4 import tolerances

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


def shared_cache(n, P, hkv, batch, seed):
    """`batch` sequences of n tokens that all hold the same pages, so that there are more
    problems than CTAs and one warp holds many tokens of a problem."""
    case = Case([n], 1, hkv, P, "q4", seed=seed, extra_cols=0)
    case.table = case.table.expand(batch, -1).contiguous()
    case.seq = case.seq.expand(batch).contiguous()
    case.nsum = case.nsum.expand(batch).contiguous()
    case.lens, case.B = [n] * batch, batch
    return case


def fill(case, kq, ks, vq, vs):
    """Codes and scales [hkv][n][...] of the one sequence's tokens into its pages."""
    n, P, hkv = kq.shape[1], case.P, case.hkv
    used = -(-n // P)
    parts = []
    for x in (kq, ks, vq, vs):
        y = torch.zeros(hkv, used * P, x.shape[-1])
        y[:, :n] = x
        parts.append(y.view(hkv, used, P, -1).transpose(0, 1))
    case.k[case.table[0, :used].long()] = pack(*parts).cuda()


def far_tokens(case, nats, vscale, seed):
    """A sink of value zero `nats` above the rest (its logit against a constant query)."""
    n, hkv = case.lens[0], case.hkv
    g = torch.Generator().manual_seed(seed)
    kq = torch.randint(-1, 2, (hkv, n, D), generator=g).float()
    ks = torch.full((hkv, n, 4), 0.05)
    vq = torch.randint(1, 8, (hkv, n, D), generator=g).float()
    vs = vscale * (0.5 + torch.rand(hkv, n, 4, generator=g))
    kq[:, 0] = 7
    ks[:, 0] = 1.0
    vq[:, 0] = 0
    fill(case, kq, ks.half(), vq, vs.half())
    return torch.full((case.B, case.hq, D), nats * math.sqrt(D) / (7 * D)).bfloat16().cuda()


def check_far(case, q, out, lse, keys=None):
    """Sequence 0's results against 64 bits, and every other sequence's against the same."""
    G = case.hq // case.hkv
    k, v = case.kv64(0)
    sc = case.scale64(0)
    for h in range(case.hkv):
        sl = slice(h * G, (h + 1) * G)
        kk, vv, ss = (x[h][slice(None) if keys is None else keys] for x in (k, v, sc))
        ro, rl, av, mag, _ = attend64(q[0, sl], kk, vv, ksc=ss)
        to, tl = tolerances(ro, rl, av, mag, kk.shape[0])
        top = (q[0, sl].double() @ kk.T / math.sqrt(D)).amax(dim=1)
        share = (top - rl).exp()[:, None]  # the largest token's
        to = to + 5 * kk.shape[0] * 2.0 ** -36 * share * vv.abs().max()
        assert ((out[:, sl].double() - ro).abs() <= to).all(), float(((out[:, sl].double() - ro).abs() / to).max())
        assert ((lse[:, sl].double() - rl).abs() <= tl).all()


@pytest.mark.parametrize("vscale", [2.0 ** -2, 2.0 ** -6, 2.0 ** -9, 2.0 ** -12, 2.0 ** -17])
@pytest.mark.parametrize("nats", [12, 15, 20])
@pytest.mark.parametrize("P,hq", [(64, 4), (16, 4), (64, 12)])
def test_tokens_far_below_a_sink_keep_their_weight(P, hq, nats, vscale):
    case = shared_cache(1500, P, 1, 320, seed=nats)
    case.hq = hq
    q = far_tokens(case, nats, vscale, seed=nats)
    rt = case.runtime(budget=1024)
    check_far(case, q, *rt.dense_decode(q))
    # listed pages: the first 1024 / P of the full ones, and the rest of the sequence behind them
    count = 1024 // P
    rt.sel_pages.copy_(torch.arange(count, dtype=torch.int32).expand(case.B, 1, -1))
    rt.sel_count.fill_(count)
    out, lse = rt.sparse_attend(q)
    full = 1500 // P * P
    keys = torch.cat([torch.arange(count * P), torch.arange(full, 1500)]).cuda()
    check_far(case, q, out, lse, keys)
    assert rt.device_error() == 0


@pytest.mark.parametrize("nats,vscale", [(12, 2.0 ** -9), (15, 2.0 ** -12), (20, 2.0 ** -8)])
@pytest.mark.parametrize("P", [64, 16])
def test_draft_tokens_far_below_a_sink(P, nats, vscale):
    case = shared_cache(1500, P, 1, 320, seed=nats)
    case.hq, new = 4, 2
    far_tokens(case, nats, vscale, seed=nats)
    rt = case.runtime()
    q = torch.full((case.B * new, 4, D), nats * math.sqrt(D) / (7 * D)).bfloat16().cuda()
    cu = torch.arange(0, case.B * new + 1, new, dtype=torch.int32).cuda()
    out, lse = rt.prompt_attend(q, cu_tokens=cu, max_tokens=new)
    assert rt.device_error() == 0
    for i in range(new):
        check_far(case, q[i::new], out[i::new], lse[i::new], torch.arange(1500 - new + 1 + i).cuda())


@pytest.mark.parametrize("steps", ["rise", "fall", "zeros first", "all tiny", "bound"])
@pytest.mark.parametrize("P,hq", [(64, 4), (16, 4), (16, 16)])
def test_value_scales_of_every_size(P, hq, steps):
    """Scales from the smallest half to the largest that a page may hold, in every order."""
    n = 1100
    case = shared_cache(n, P, 1, 310, seed=5)
    case.hq = hq
    g = torch.Generator().manual_seed(7)
    kq, vq = (torch.randint(-7, 8, (1, n, D), generator=g).float() for _ in range(2))
    ks = torch.full((1, n, 4), 0.2)
    at = torch.arange(n)
    exponent = {"rise": -24 + 37 * at // n, "fall": 13 - 37 * at // n, "zeros first": -12 + at // 200,
                "all tiny": -24 + 8 * at // n, "bound": torch.full((n,), 13)}[steps]
    vs = (2.0 ** exponent.double())[None, :, None].expand(1, n, 4).clone()
    if steps == "zeros first":
        vs[:, :300] = 0
    if steps == "bound":
        vs[:] = 9352
        vq[:] = 7
    fill(case, kq, ks.half(), vq, vs.half())
    q = case.query(1).expand(case.B, -1, -1).contiguous()
    rt = case.runtime()
    out, lse = rt.dense_decode(q)
    assert rt.device_error() == 0 and torch.isfinite(out.float()).all()
    check_far(case, q, out, lse)


def nan_scale(case, at, j, part):
    """The scale of group j of token `at` of the one sequence becomes NaN."""
    P, slot, u = case.P, at % case.P, at % 16
    off = (64 * P + 8 * slot + 2 * j if part == "k" else
           136 * P + 128 * (slot // 16) + 32 * (u % 8 // 2) + 16 * (u // 8) + 4 * j + 2 * (u % 2))
    case.k[int(case.table[0, at // P]), 0, off:off + 2] = torch.tensor([0xff, 0x7f], dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("P,hq", [(64, 4), (16, 4), (64, 12)])
def test_a_nan_scale_takes_no_digits_from_the_other_dimensions(P, hq):
    case = shared_cache(1500, P, 1, 320, seed=3)
    case.hq = hq
    q = far_tokens(case, 12, 2.0 ** -9, seed=3)
    rt = case.runtime()
    k, v = (x[0].clone() for x in case.kv64(0))
    for at in (390, 1499):
        nan_scale(case, at, 1, "v")
    out, lse = rt.dense_decode(q)
    ro, rl, av, mag, _ = attend64(q[0], k, v, ksc=case.scale64(0)[0])
    to, _ = tolerances(ro, rl, av, mag, 1500)
    share = ((q[0].double() @ k.T / math.sqrt(D)).amax(dim=1) - rl).exp()[:, None]
    to = to + 5 * 1500 * 2.0 ** -36 * share * v.abs().max()
    rest = torch.arange(D, device="cuda") // 32 != 1
    assert torch.isnan(out[..., ~rest]).all()
    assert ((out.double() - ro).abs() <= to)[..., rest].all()
    assert rt.device_error() == 0


@pytest.mark.parametrize("P", [64, 16])
def test_a_later_drafts_nan_scale_takes_no_digits_from_the_rows_before_it(P):
    case = shared_cache(1500, P, 1, 320, seed=4)
    case.hq, new = 4, 3
    far_tokens(case, 12, 2.0 ** -9, seed=4)
    rt = case.runtime()
    q = torch.full((case.B * new, 4, D), 12 * math.sqrt(D) / (7 * D)).bfloat16().cuda()
    nan_scale(case, 1499, 2, "v")
    cu = torch.arange(0, case.B * new + 1, new, dtype=torch.int32).cuda()
    out, lse = rt.prompt_attend(q, cu_tokens=cu, max_tokens=new)
    assert rt.device_error() == 0
    for i in range(new - 1):
        check_far(case, q[i::new], out[i::new], lse[i::new], torch.arange(1500 - new + 1 + i).cuda())
    assert torch.isnan(out[new - 1::new, :, 64:96]).all()
