"""Attention of one query token over a cache held in 4 bits: every page, listed
pages, the exact page log-sum-exp, the whole decode step and the summary builder,
against 64-bit references.

Tolerances.  A weight is rounded to fp16 twice (2^-11 each, before and after its
value scale) and an output once to bf16 (2^-8).  A logit is a sum of exact products
in fp32: 32 terms through the tensor core (at most 2^-23 of the running magnitude
each, the codes' offset of 72 scales included) and 4 scaled additions, under 2^-17 of
sum |q|(|k| + 80 s); its exponent's argument is rounded at 2^-24 of up to
|logit| + 16, and the hardware exponential adds 2^-22.  A logit error e changes
normalised weights by at most 2 e.  The sum of n weights in fp32 is off by at most
n 2^-24."""

import math

import pytest
import torch

from tests.kv_cases import Case, attend64, dequant64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


def tolerances(out, lse, absv, mag, n):
    e = 2.0 ** -17 * mag + 2.0 ** -22 * (mag + 16) + 2.0 ** -22
    return (2.0 ** -8 * out.abs() + (2.0 ** -10 + 2 * e + n * 2.0 ** -23)[:, None] * absv + 1e-30,
            e + n * 2.0 ** -24 + 2.0 ** -22 * (lse.abs() + 16))


def check(case, q, out, lse, tokens_of=None):
    """out, lse of one query per sequence; tokens_of(b, h): the token indices attended."""
    G = case.hq // case.hkv
    for b in range(case.B):
        k, v = case.kv64(b)
        sc = case.scale64(b)
        for h in range(case.hkv):
            idx = slice(None) if tokens_of is None else tokens_of(b, h)
            kk, vv, ss = k[h][idx], v[h][idx], sc[h][idx]
            sl = slice(h * G, (h + 1) * G)
            ro, rl, av, mag, _ = attend64(q[b, sl], kk, vv, ksc=ss)
            if kk.shape[0] == 0:
                assert (out[b, sl] == 0).all() and (lse[b, sl] == -math.inf).all()
                continue
            to, tl = tolerances(ro, rl, av, mag, kk.shape[0])
            assert ((out[b, sl].double() - ro).abs() <= to).all(), (b, h)
            assert ((lse[b, sl].double() - rl).abs() <= tl).all(), (b, h)


@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("hq,hkv,lens", [
    (1, 1, [1]), (1, 1, [4096]), (4, 1, [0, 1, 15, 16, 17, 63, 64, 65, 127, 128]),
    (32, 8, [1000, 3]), (3, 1, [777]), (8, 1, [2049]), (9, 1, [100, 2000]), (32, 2, [5000, 0, 17]),
    (6, 2, [333, 4444]), (8, 8, [12345]),
])
def test_every_page(P, hq, hkv, lens):
    case = Case(lens, hq, hkv, P, "q4", seed=P + hq + len(lens))
    rt, q = case.runtime(), case.query(len(lens))
    out, lse = rt.dense_decode(q)
    assert rt.device_error() == 0
    check(case, q, out, lse)
    # a second call finds its counters where the first left them
    out1 = out.clone()
    out2, _ = rt.dense_decode(q)
    assert torch.equal(out1, out2)


@pytest.mark.parametrize("P,hq,hkv,n", [(64, 32, 8, 40001), (16, 4, 1, 70001), (64, 16, 1, 100001)])
def test_every_page_of_a_long_cache(P, hq, hkv, n):
    case = Case([n], hq, hkv, P, "q4", seed=n)
    rt, q = case.runtime(), case.query(1)
    out, lse = rt.dense_decode(q)
    assert rt.device_error() == 0
    check(case, q, out, lse)


def test_many_sequences():
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 700, (97,), generator=g).tolist()
    case = Case(lens, 8, 2, 16, "q4", seed=9)
    rt, q = case.runtime(), case.query(97)
    out, lse = rt.dense_decode(q)
    assert rt.device_error() == 0
    check(case, q, out, lse)


@pytest.mark.parametrize("spread", [1e-4, 1.0, 1e3])
def test_small_and_large_values(spread):
    """Value scales from 3e-5 (subnormal halves) to 300, and one dominant token whose
    weight is 2^30 times the others'."""
    case = Case([3000], 4, 1, 64, "q4", seed=3, spread=spread)
    q = case.query(1, spread=min(2.0, 2.0 / spread))
    rt = case.runtime()
    out, lse = rt.dense_decode(q)
    check(case, q, out, lse)


def test_a_few_heavy_tokens_do_not_hide_the_rest():
    """A sink 20 nats above 60,000 tokens of equal logit, with values near zero: the
    result is made by weights of 2^-29 of the largest."""
    n, P = 60001, 64
    case = Case([n], 1, 1, P, "q4", seed=4)
    kq = torch.zeros(case.k.shape[0], 1, P, 128)
    ks = torch.ones(case.k.shape[0], 1, P, 4).half()
    vq = torch.full_like(kq, 3.0)
    vs = torch.full((case.k.shape[0], 1, P, 4), 0.25).half()
    first = int(case.table[0, 0])
    kq[first, 0, 0] = 7
    vq[first, 0, 0] = 0
    from tests.kv_cases import pack
    case.k.copy_(pack(kq, ks, vq, vs))
    q = torch.full((1, 1, 128), 20 * math.sqrt(128) / (7 * 128)).bfloat16().cuda()
    rt = case.runtime()
    out, lse = rt.dense_decode(q)
    k, v = case.kv64(0)
    ro, rl, av, mag, _ = attend64(q[0], k[0], v[0], ksc=case.scale64(0)[0])
    # every ordinary token has the same logit 0, so only the two fp16 roundings of its
    # weight and the sums count
    assert ((out[0].double() - ro).abs() <= (2.0 ** -8 + 2.0 ** -10 + n * 2.0 ** -23 + 1e-3) * ro.abs()).all()
    assert abs(lse[0, 0].item() - rl.item()) <= 1e-4


def test_nan_scale_reaches_exactly_its_head():
    case = Case([200, 300], 8, 2, 64, "q4", seed=8)
    rt, q = case.runtime(), case.query(2)
    page = int(case.table[1, 2])
    block = case.k[page, 1].clone()
    block[136 * 64:136 * 64 + 2] = torch.tensor([0xff, 0x7f], dtype=torch.uint8)  # token 128, dimensions 0-31
    case.k[page, 1] = block
    out, lse = rt.dense_decode(q)
    assert torch.isnan(out[1, 4:, :32]).all() and not torch.isnan(out[1, 4:, 32:]).any()
    assert not torch.isnan(out[0]).any() and not torch.isnan(out[1, :4]).any() and not torch.isnan(lse).any()


def _page_list(case, k_max, seed):
    g = torch.Generator().manual_seed(seed)
    lists = torch.zeros(case.B, case.hkv, max(k_max, 1), dtype=torch.int32)
    count = torch.zeros(case.B, case.hkv, dtype=torch.int32)
    for b in range(case.B):
        ns = int(case.nsum[b])
        for h in range(case.hkv):
            c = min(k_max, ns)
            lists[b, h, :c] = torch.randperm(ns, generator=g)[:c].sort().values.int()
            count[b, h] = c
    return lists, count


@pytest.mark.parametrize("P,hq,hkv,lens,short,budget", [
    (64, 32, 8, [4000], 1, 512), (16, 8, 2, [1000, 33, 16, 0, 5], 2, 128), (64, 16, 1, [3000, 640], 0, 256),
    (64, 4, 4, [64, 63, 700], 3, 0), (16, 12, 1, [9000], 40, 4096), (64, 1, 1, [9001], 0, 8192),
])
def test_listed_pages(P, hq, hkv, lens, short, budget):
    case = Case(lens, hq, hkv, P, "q4", seed=budget, nsum=[max(0, n // P - short) for n in lens])
    rt, q = case.runtime(budget=budget), case.query(len(lens))
    lists, count = _page_list(case, budget // P, 7)
    rt.sel_pages.copy_(lists)
    rt.sel_count.copy_(count)
    out, lse = rt.sparse_attend(q)
    assert rt.device_error() == 0

    def tokens_of(b, h):
        pages = lists[b, h, :count[b, h]].tolist()
        at = [t for p in pages for t in range(p * P, (p + 1) * P)] + list(range(int(case.nsum[b]) * P, lens[b]))
        return torch.tensor(at, dtype=torch.long, device="cuda")

    check(case, q, out, lse, tokens_of)


def test_bad_pages_are_reported_and_left_out():
    case = Case([640, 640], 4, 1, 64, "q4", seed=1)
    rt, q = case.runtime(budget=256), case.query(2)
    case.table[0, 3] = 10 ** 6
    out, lse = rt.dense_decode(q)
    from sparse_kv_page_rank_gb300 import locks as L
    assert rt.device_error() == L.LOCKS_DEVERR_BLOCK_TABLE
    good = torch.tensor([t for t in range(640) if not 192 <= t < 256], device="cuda")
    saved = case.table[0, 3].clone()
    case.table[0, 3] = case.table[0, 2]
    check(case, q, out, lse, lambda b, h: good if b == 0 else slice(None))
    case.table[0, 3] = saved
    rt.sel_pages.zero_()
    rt.sel_pages[..., :2] = torch.tensor([99, 1], dtype=torch.int32)
    rt.sel_count.fill_(2)
    case.table[0, 3] = case.table[0, 2]
    rt.sparse_attend(q)
    assert rt.device_error() == L.LOCKS_DEVERR_SEL_PAGE


@pytest.mark.parametrize("P,hq,hkv", [(64, 8, 2), (16, 4, 1), (64, 16, 1), (16, 12, 1)])
def test_exact_page_lse(P, hq, hkv):
    lens = [0, 1, 500, 777]
    case = Case(lens, hq, hkv, P, "q4", seed=21)
    rt, q = case.runtime(), case.query(len(lens))
    got = rt.exact_page_lse(q)
    G = hq // hkv
    for b, n in enumerate(lens):
        k, v = case.kv64(b)
        sc = case.scale64(b)
        for h in range(hkv):
            for p in range(got.shape[2]):
                x = got[b, h * G:(h + 1) * G, p].double()
                if p * P >= n:
                    assert torch.isnan(x).all()
                    continue
                at = slice(p * P, min(n, p * P + P))
                _, rl, av, mag, _ = attend64(q[b, h * G:(h + 1) * G], k[h, at], v[h, at], ksc=sc[h, at])
                _, tl = tolerances(av, rl, av, mag, P)
                assert ((x - rl).abs() <= tl).all()


@pytest.mark.parametrize("P", [16, 64])
def test_summaries_are_those_of_the_stored_keys(P):
    """The builder on 4-bit pages gives what it gives on bf16 pages that hold the same
    keys rounded to bf16."""
    from sparse_kv_page_rank_gb300.runtime import LocksRuntime
    case = Case([P * 12], 8, 2, P, "q4", seed=31)
    rt = case.runtime(rank=8)
    k, v = dequant64(case.k)
    rb = LocksRuntime(k.bfloat16(), v.bfloat16(), case.table, case.seq, case.nsum, 8, 8, 0)
    pages = case.table[0, :12]
    for r in (rt, rb):
        r.build_summaries(pages)
    assert rt.device_error() == 0
    assert torch.equal(rt.basis_t[pages.long()], rb.basis_t[pages.long()])
    assert torch.equal(rt.coeffs[pages.long()], rb.coeffs[pages.long()])


@pytest.mark.parametrize("P", [16, 64])
def test_decode_step_equals_its_parts(P):
    """The whole step on 4-bit pages: the selection of a bf16 cache with the same
    summaries, then the attention over the listed pages, bit for bit."""
    case = Case([P * 40 + 5, P * 33], 8, 2, P, "q4", seed=33)
    rt = case.runtime(rank=8, budget=P * 6)
    q = case.query(2)
    pages = torch.cat([case.table[b, :n // P] for b, n in enumerate(case.lens)])
    rt.build_summaries(pages)
    out, lse = rt.decode_step(q)
    out, lse, sel, cnt = out.clone(), lse.clone(), rt.sel_pages.clone(), rt.sel_count.clone()
    assert (cnt == 6).all() and rt.decode_step_launches() == 3
    rt.select(q)
    assert torch.equal(rt.sel_pages, sel) and torch.equal(rt.sel_count, cnt)
    out2, lse2 = rt.sparse_attend(q)
    assert rt.device_error() == 0
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    lists, count = sel.cpu(), cnt.cpu()

    def tokens_of(b, h):
        at = [t for p in lists[b, h, :count[b, h]].tolist() for t in range(p * P, (p + 1) * P)]
        return torch.tensor(at + list(range(int(case.nsum[b]) * P, case.lens[b])), device="cuda")

    check(case, q, out, lse, tokens_of)


def test_captured_and_replayed_while_the_cache_grows():
    case = Case([1000, 500], 8, 2, 64, "q4", seed=41, extra_cols=0)
    rt, q = case.runtime(), case.query(2)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        rt.dense_decode(q, stream=stream)
        with torch.cuda.graph(graph, stream=stream):
            rt.dense_decode(q, stream=stream)
    torch.cuda.synchronize()
    for lens in ([1000, 500], [700, 1], [0, 320]):
        case.lens = lens
        case.seq.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(case.query(2))
        graph.replay()
        torch.cuda.synchronize()
        check(case, q, rt.out, rt.lse)
    assert rt.device_error() == 0
