"""Causal attention of the newest tokens over the paged cache, bf16 and 4-bit pages,
against a 64-bit reference.

Tolerances.  bf16 pages: weights rounded to bf16 (2^-8), outputs to bf16 (2^-8),
logits sums of 128 exact products in fp32 (at most 2^-23 of the running magnitude
each: 2^-16 of sum |q||k|).  4-bit pages: keys exact, in two halves (256 products,
2^-15), values s * code rounded to fp16 (2^-11), weights to fp16 (2^-11).  A logit
error e changes normalised weights by at most 2 e.  fp16 is no finer than 2^-24 below
2^-14: weights are held times 2^6 relative to a reference that is at most the row's
maximum, so the largest is at least 2^6 and each weight is off by another 2^-25 / 2^6
of it, over m keys by m 2^-31 of the largest value."""

import math

import pytest
import torch

from tests.kv_cases import D, Case, attend64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


def cu_of(new):
    return torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32).cuda()


def check(case, new, q, out, lse, first_bad=None):
    """first_bad: (sequence, position) of a token that is not finite: the rows before it
    are compared, the rows that see it must show it."""
    G = case.hq // case.hkv
    q4 = case.fmt == "q4"
    row = 0
    for b, n in enumerate(new):
        k, v = case.kv64(b)
        at = torch.arange(case.lens[b], device="cuda")
        hidden = at[None, :] > (case.lens[b] - n + torch.arange(n, device="cuda"))[:, None]
        for h in range(case.hkv):
            kk, vv = k[h], v[h]
            rows = torch.arange(n, device="cuda")
            if first_bad is not None and first_bad[0] == b:
                before = case.lens[b] - n + rows < first_bad[1]
                assert not torch.isfinite(out[row:row + n][~before][:, h * G:(h + 1) * G].float()).all(dim=-1).any()
                kk, vv = kk[:first_bad[1]], vv[:first_bad[1]]
                rows = rows[before]
            for g in range(h * G, (h + 1) * G):
                if len(rows) == 0:
                    continue
                qq = q[row:row + n, g][rows]
                ro, rl, av, mag, _ = attend64(qq, kk, vv, hidden[rows][:, :kk.shape[0]])
                m = kk.shape[0]
                e = 2.0 ** (-15 if q4 else -16) * mag + 2.0 ** -22 * (mag + 16)
                to = 2.0 ** -8 * ro.abs() + ((2.0 ** -10 if q4 else 2.0 ** -8) + 2 * e + m * 2.0 ** -23)[:, None] * av
                if q4:
                    to = to + m * 2.0 ** -31 * vv.abs().max()
                tl = e + m * 2.0 ** -24 + 2.0 ** -22 * (rl.abs() + 16)
                go, gl = out[row:row + n, g][rows].double(), lse[row:row + n, g][rows].double()
                assert ((go - ro).abs() <= to + 1e-30).all(), (b, h, g, float(((go - ro).abs() / to).max()))
                assert ((gl - rl).abs() <= tl).all(), (b, h, g)
        row += n


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("P,hq,hkv,lens,new", [
    (64, 1, 1, [1], [1]),
    (64, 4, 1, [128], [128]),
    (64, 4, 1, [200], [200]),
    (16, 4, 1, [37, 16, 300], [37, 5, 299]),
    (64, 8, 2, [1000, 700], [513, 64]),
    (64, 3, 1, [400], [400]),
    (16, 32, 2, [77, 1, 250], [77, 1, 250]),
    (64, 10, 2, [513, 129, 64, 65], [513, 1, 0, 65]),
    (16, 8, 8, [600], [333]),
    (64, 32, 8, [2000], [2000]),
])
def test_prompts(fmt, P, hq, hkv, lens, new):
    case = Case(lens, hq, hkv, P, fmt, seed=P + sum(lens))
    rt, total = case.runtime(), sum(new)
    q = case.query(total + 2, spread=1.5)
    out = torch.full((total + 2, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((total + 2, hq), 7.0, device="cuda")
    rt.prompt_attend(q, cu_tokens=cu_of(new), max_tokens=max(new), out=out, lse=lse)
    assert rt.device_error() == 0
    check(case, new, q, out, lse)
    assert (out[total:] == 7).all() and (lse[total:] == 7).all()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("P,hq,hkv,lens,new", [
    (16, 32, 8, [3001], [5]), (64, 4, 1, [20000, 1, 9000], [3, 1, 64]), (64, 16, 1, [5000], [40]),
    (16, 2, 2, [4097], [1]),
])
def test_few_tokens_over_a_long_cache(fmt, P, hq, hkv, lens, new):
    """The keys cut among several CTAs; twice, since the second call needs the
    counters that the first leaves, and then another shape on the same workspace."""
    case = Case(lens, hq, hkv, P, fmt, seed=sum(lens))
    rt, total = case.runtime(), sum(new)
    for _ in range(2):
        q = case.query(total)
        out, lse = rt.prompt_attend(q, cu_tokens=cu_of(new), max_tokens=max(new))
        check(case, new, q, out, lse)
    one = [min(1, n) for n in new]
    q = case.query(sum(one))
    out, lse = rt.prompt_attend(q, cu_tokens=cu_of(one), max_tokens=1)
    check(case, one, q, out, lse)
    q = case.query(total)
    out, lse = rt.prompt_attend(q, cu_tokens=cu_of(new))  # max_tokens defaults to all rows
    check(case, new, q, out, lse)
    assert rt.device_error() == 0


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_one_token_per_sequence_equals_the_decode(fmt):
    lens = [100, 0, 700, 1]
    case = Case(lens, 8, 2, 64, fmt, seed=12)
    rt, q = case.runtime(), case.query(4)
    out = torch.full((4, 8, D), 7.0, dtype=torch.bfloat16, device="cuda")
    out, lse = rt.prompt_attend(q, out=out)
    live = [0, 2, 3]
    ref, rlse = rt.dense_decode(q)
    assert rt.device_error() == 0
    # both are within one bf16 rounding and the weights' rounding of the same number
    assert ((out[live].float() - ref[live].float()).abs() <= 2.0 ** -6 * (1 + ref[live].float().abs())).all()
    assert ((lse[live] - rlse[live]).abs() <= 2e-2 * (1 + rlse[live].abs())).all()
    assert (out[1] == 7).all()
    check(Case(lens, 8, 2, 64, fmt, seed=12), [1, 0, 1, 1], q[live], out[live], lse[live])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("P,new,at", [(64, 300, 250), (16, 300, 130), (64, 20, 390), (64, 300, 399)])
def test_a_later_token_that_is_not_finite_stays_out_of_earlier_rows(value, where, P, new, at):
    case = Case([400], 4, 1, P, "bf16", seed=3)
    pool = case.k if where == "k" else case.v
    pool[int(case.table[0, at // P]), 0, at % P] = value
    rt, q = case.runtime(), case.query(new)
    out, lse = rt.prompt_attend(q, cu_tokens=cu_of([new]))
    assert rt.device_error() == 0
    if where == "k" and value > 0:
        # an infinite key's logits are infinite or not numbers: only the rows before it are defined
        q, out, lse = q[:at - 400 + new], out[:at - 400 + new], lse[:at - 400 + new]
        case.lens = [at]
        check(case, [len(q)], q, out, lse)
    else:
        check(case, [new], q, out, lse, first_bad=(0, at))


@pytest.mark.parametrize("value", [float("nan"), float("-inf")])
@pytest.mark.parametrize("dim", [0, 77, 127])
def test_one_value_that_is_not_finite_reaches_one_column(value, dim):
    """One dimension of one token's value: the rows that see the token have it there and
    are right everywhere else."""
    case = Case([400], 4, 1, 64, "bf16", seed=3)
    at, new = 250, 300
    page, slot = int(case.table[0, at // 64]), at % 64
    was = case.v[page, 0, slot, dim].clone()
    rt, q = case.runtime(), case.query(new)
    good, _ = rt.prompt_attend(q, cu_tokens=cu_of([new]))
    case.v[page, 0, slot, dim] = value
    out, lse = rt.prompt_attend(q, cu_tokens=cu_of([new]))
    case.v[page, 0, slot, dim] = was
    sees = torch.arange(new, device="cuda") + 100 >= at
    assert torch.equal(out[~sees], good[~sees])
    col = out[sees][..., dim].float()
    assert (torch.isnan(col) if math.isnan(value) else col == value).all()
    rest = torch.arange(D, device="cuda") != dim
    assert torch.equal(out[sees][..., rest], good[sees][..., rest])
    assert rt.device_error() == 0


def test_a_nan_scale_of_a_later_token_stays_out_of_earlier_rows():
    case = Case([400], 4, 1, 64, "q4", seed=3)
    at = 333
    block = case.k[int(case.table[0, at // 64]), 0].clone()
    u = (at % 64) % 16
    for j in range(4):
        off = 136 * 64 + 128 * (at % 64 // 16) + 32 * (u % 8 // 2) + 16 * (u // 8) + 4 * j + 2 * (u % 2)
        block[off:off + 2] = torch.tensor([0xff, 0x7f], dtype=torch.uint8)
    case.k[int(case.table[0, at // 64]), 0] = block
    rt, q = case.runtime(), case.query(200)
    out, lse = rt.prompt_attend(q, cu_tokens=cu_of([200]))
    check(case, [200], q, out, lse, first_bad=(0, at))


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_large_logits(fmt):
    """Maxima that keep growing along the keys, so that O is rescaled often."""
    case = Case([1500], 2, 1, 64, fmt, seed=8, spread=3.0)
    rt, q = case.runtime(), case.query(1500, spread=4.0)
    out, lse = rt.prompt_attend(q, cu_tokens=cu_of([1500]))
    assert rt.device_error() == 0
    check(case, [1500], q, out, lse)


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_bad_pages_and_lengths(fmt):
    from sparse_kv_page_rank_gb300 import locks as L
    case = Case([640, 320], 4, 1, 64, fmt, seed=1)
    rt, new = case.runtime(), [100, 50]
    q = case.query(150)
    good, _ = (x.clone() for x in rt.prompt_attend(q, cu_tokens=cu_of(new)))
    assert rt.device_error() == 0
    case.table[0, 3] = 10 ** 6
    out, lse = rt.prompt_attend(q, cu_tokens=cu_of(new))
    assert rt.device_error() == L.LOCKS_DEVERR_BLOCK_TABLE
    assert torch.equal(out[100:], good[100:]) and torch.isfinite(out.float()).all()
    # the page's tokens are left out
    case.table[0, 3] = case.table[0, 2]
    k, v = case.kv64(0)
    keep = torch.tensor([t for t in range(640) if not 192 <= t < 256], device="cuda")
    hidden = keep[None, :] > (540 + torch.arange(100, device="cuda"))[:, None]
    for g in range(4):
        ro, rl, av, mag, _ = attend64(q[:100, g], k[0][keep], v[0][keep], hidden)
        tol = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -9 * mag + 1e-4)[:, None] * av
        assert ((out[:100, g].double() - ro).abs() <= tol).all()
    # more new tokens than the host said, and more than the sequence has
    out = torch.full_like(out, 7.0)
    rt.prompt_attend(q, cu_tokens=cu_of(new), max_tokens=60, out=out)
    assert rt.device_error() == L.LOCKS_DEVERR_LENGTHS
    rt.prompt_attend(case.query(400), cu_tokens=cu_of([10, 330]))
    assert rt.device_error() == L.LOCKS_DEVERR_LENGTHS


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_captured_and_replayed(fmt):
    case = Case([900, 400], 8, 2, 64, fmt, seed=41, extra_cols=0)
    rt = case.runtime()
    q = case.query(24)
    cu = cu_of([16, 8])
    out, lse = torch.empty(24, 8, D, dtype=torch.bfloat16, device="cuda"), torch.empty(24, 8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        rt.prompt_attend(q, cu_tokens=cu, max_tokens=20, out=out, lse=lse, stream=stream)
        with torch.cuda.graph(graph, stream=stream):
            rt.prompt_attend(q, cu_tokens=cu, max_tokens=20, out=out, lse=lse, stream=stream)
    torch.cuda.synchronize()
    for lens, new in (([900, 400], [16, 8]), ([600, 30], [4, 20]), ([20, 333], [20, 1])):
        case.lens = lens
        case.seq.copy_(torch.tensor(lens, dtype=torch.int32))
        cu.copy_(cu_of(new))
        q.copy_(case.query(24))
        graph.replay()
        torch.cuda.synchronize()
        check(case, new, q, out, lse)
    assert rt.device_error() == 0


def test_strided_queries():
    case = Case([300], 4, 2, 64, "bf16", seed=5)
    rt = case.runtime()
    wide = torch.randn(300, 8, D, generator=case.gen).bfloat16().cuda()
    out, lse = rt.prompt_attend(wide[:, 2:6], cu_tokens=cu_of([300]))
    check(case, [300], wide[:, 2:6], out, lse)


@pytest.mark.parametrize("P,hq,hkv,lens,new", [
    # the last 64 tokens hold keys of the newest rows only: a part of the work in which
    # the other rows see nothing
    (64, 8, 2, [64 * 40 + 3], [5]),
    (16, 8, 2, [64 * 3 + 1, 17, 5], [8, 2, 5]),
    (64, 1, 1, [32], [32]),
    (16, 1, 1, [31, 64, 0, 33], [31, 1, 0, 32]),
    (64, 6, 2, [500] * 37, [1, 2, 3, 4, 5, 6, 7, 8, 9, 10] * 3 + [0, 10, 1, 9, 2, 8, 3]),
    (16, 16, 1, [30000], [2]),
    (64, 12, 1, [9000, 65], [1, 2]),
])
def test_few_rows_of_4_bit_pages(P, hq, hkv, lens, new):
    """A few (token, head) rows of a KV head, in blocks of eight columns."""
    case = Case(lens, hq, hkv, P, "q4", seed=P + sum(lens))
    rt, total = case.runtime(), sum(new)
    for _ in range(2):
        q = case.query(total + 1, spread=1.5)
        out = torch.full((total + 1, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((total + 1, hq), 7.0, device="cuda")
        rt.prompt_attend(q, cu_tokens=cu_of(new), max_tokens=max(new), out=out, lse=lse)
        assert rt.device_error() == 0
        check(case, new, q, out, lse)
        assert (out[total:] == 7).all() and (lse[total:] == 7).all()


@pytest.mark.parametrize("P,at", [(64, 397), (16, 399), (64, 395), (16, 384)])
@pytest.mark.parametrize("part", ["k", "v"])
def test_a_nan_scale_of_a_draft_token_stays_out_of_earlier_rows(P, at, part):
    case = Case([400], 2, 1, P, "q4", seed=3)
    block = case.k[int(case.table[0, at // P]), 0]
    slot, u = at % P, at % 16
    for j in range(4):
        off = (64 * P + 128 * (slot // 16) + 8 * u + 2 * j if part == "k" else
               136 * P + 128 * (slot // 16) + 32 * (u % 8 // 2) + 16 * (u // 8) + 4 * j + 2 * (u % 2))
        block[off:off + 2] = torch.tensor([0xff, 0x7f], dtype=torch.uint8)
    rt, q = case.runtime(), case.query(16)
    out, lse = rt.prompt_attend(q, cu_tokens=cu_of([16]))
    assert rt.device_error() == 0
    check(case, [16], q, out, lse, first_bad=(0, at))


@pytest.mark.parametrize("new", [3, 16])
def test_strided_queries_of_few_rows(new):
    """Query rows of a wider matrix, as a fused projection writes them."""
    case = Case([777], 2, 1, 64, "q4", seed=new)
    wide = torch.randn(new, 4 * D, device="cuda").bfloat16()
    q = wide[:, D:3 * D].view(new, 2, D)
    rt = case.runtime()
    out, lse = rt.prompt_attend(q, cu_tokens=cu_of([new]))
    assert rt.device_error() == 0
    check(case, [new], q, out, lse)
    same, _ = rt.prompt_attend(q.contiguous(), cu_tokens=cu_of([new]))
    assert torch.equal(out, same)


@pytest.mark.parametrize("fmt,P,hq,hkv,new", [("bf16", 16, 4, 1, 300), ("bf16", 16, 16, 1, 100), ("bf16", 16, 8, 2, 20),
                                              ("q4", 16, 8, 2, 5), ("q4", 64, 4, 1, 40)])
def test_a_page_outside_the_pool_is_left_out(fmt, P, hq, hkv, new):
    """Its tokens are reported and take no part; the rest is as if they were not there,
    whatever the path: pages, planes, few rows."""
    from sparse_kv_page_rank_gb300 import locks as L
    case = Case([400], hq, hkv, P, fmt, seed=21)
    rt, q = case.runtime(), case.query(new)
    lp = 48 // P
    case.table[0, lp] = case.k.shape[0] + 3
    out, lse = rt.prompt_attend(q, cu_tokens=cu_of([new]), max_tokens=new)
    assert rt.device_error() == L.LOCKS_DEVERR_BLOCK_TABLE
    case.table[0, lp] = case.table[0, lp + 1]  # for the reference: any page that holds numbers
    gone = torch.zeros(400, dtype=torch.bool, device="cuda")
    gone[lp * P:(lp + 1) * P] = True
    at = torch.arange(400, device="cuda")
    hidden = gone[None, :] | (at[None, :] > (400 - new + torch.arange(new, device="cuda"))[:, None])
    k, v = case.kv64(0)
    for g in range(hq):
        h = g * hkv // hq
        ro, rl, av, mag, _ = attend64(q[:, g], k[h], v[h], hidden, ksc=case.scale64(0)[h])
        e = 2.0 ** -15 * mag + 2.0 ** -22 * (mag + 16)
        to = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2 * e + 400 * 2.0 ** -23)[:, None] * av + 400 * 2.0 ** -31 * v.abs().max()
        assert ((out[:, g].double() - ro).abs() <= to).all(), g
        assert ((lse[:, g].double() - rl).abs() <= e + 400 * 2.0 ** -24 + 2.0 ** -22 * (rl.abs() + 16)).all(), g


@pytest.mark.parametrize("fmt,P,hq,hkv,lens,new", [
    # whole waves of tiles, and some left over whose keys are cut
    ("bf16", 64, 32, 8, [3000], [1300]), ("q4", 64, 32, 8, [3000], [1300]),
    # fewer tiles than SMs, more than half as many
    ("bf16", 64, 16, 8, [5000, 2000], [700, 1000]), ("q4", 16, 16, 8, [5000, 300], [900, 300]),
])
def test_left_over_tiles(fmt, P, hq, hkv, lens, new):
    case = Case(lens, hq, hkv, P, fmt, seed=sum(lens), extra_cols=5)
    rt, q = case.runtime(), case.query(sum(new))
    first = None
    for _ in range(2):
        out, lse = rt.prompt_attend(q, cu_tokens=cu_of(new), max_tokens=max(new))
        assert rt.device_error() == 0
        assert first is None or torch.equal(out, first)
        first = out
    check(case, new, q, out, lse)
