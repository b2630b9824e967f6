"""The generation calls at the ends of what they allow: many requests, long vocabularies, pages beyond
4 GiB, the largest scales of 4-bit pages, several streams, other devices. Tolerances are those of
the files that are imported."""


import pytest
import torch

from sparse_kv_page_rank_gb300 import locks as L
from sparse_kv_page_rank_gb300.beams import LocksBeams
from sparse_kv_page_rank_gb300.runtime import LocksRuntime
from tests.gen_cases import shared_case
from tests.kv_cases import D, pack
from tests.test_gpu_gen_attend import check as check_attend
from tests.test_gpu_gen_reorder import Rows
from tests.test_gpu_gen_select import check as check_select, make
from tests.test_gpu_kv_append import table
from tests.test_gpu_kv_bounds import max_scale
from tests.test_gpu_kv_devices import Elsewhere

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("requests,W", [(9, 2), (33, 3), (129, 2), (300, 1), (260, 2)])
def test_attend_of_many_requests(fmt, requests, W):
    g = torch.Generator().manual_seed(requests)
    prompts = torch.randint(1, 200, (requests,), generator=g).tolist()
    tails = [[None if x == 0 else x for x in row] for row in torch.randint(0, 40, (requests, W), generator=g).tolist()]
    tails[requests // 2] = [None] * W
    case, _, shared = shared_case(prompts, tails, 2, 1, 16, fmt, seed=requests)
    beams = LocksBeams([case.runtime()], width=W)
    q = case.query(case.B)
    out, lse = beams.attend(q, shared)
    assert beams.device_error() == 0
    check_attend(case, q, out, lse)


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("W,hq,hkv,P", [(32, 16, 1, 64), (32, 32, 2, 16), (31, 15, 1, 64)])
def test_attend_of_the_widest_requests(fmt, W, hq, hkv, P):
    """Up to 512 (row, head) pairs over one KV head's shared pages."""
    tails = [[(7 * w) % 90 for w in range(W)], [None if w % 3 else w for w in range(W)]]
    case, _, shared = shared_case([260, 100], tails, hq, hkv, P, fmt, seed=W + P)
    beams = LocksBeams([case.runtime()], width=W)
    q = case.query(case.B)
    out, lse = beams.attend(q, shared)
    assert beams.device_error() == 0
    check_attend(case, q, out, lse)


@pytest.mark.parametrize("requests", [1, 3, 20, 140])
def test_a_bad_length_among_idle_rows_is_told(requests):
    case, W, shared = shared_case([50] + [20] * (requests - 1), [[1, 2]] + [[None, None]] * (requests - 1), 2, 1, 16, "bf16", seed=3)
    beams = LocksBeams([case.runtime()], width=W)
    q = case.query(case.B)
    case.seq[-1 if requests > 1 else 0] = -9
    if requests == 1:
        case.lens[0] = 0
    out, lse = beams.attend(q, shared)
    assert beams.device_error() == L.LOCKS_DEVERR_LENGTHS
    check_attend(case, q, out, lse)


def test_attend_at_the_largest_scale():
    case, W, shared = shared_case([700], [[33, 40, 1]], 4, 1, 64, "q4", seed=3)
    g = torch.Generator().manual_seed(1)
    pages = case.k.shape[0]
    kq, vq = (torch.randint(-7, 8, (pages, 1, 64, D), generator=g).float() for _ in range(2))
    bound = torch.full((pages, 1, 64, 4), max_scale())
    case.k.copy_(pack(kq, bound, vq, bound))
    beams = LocksBeams([case.runtime()], width=W)
    q = case.query(case.B, spread=0.1 / max_scale())
    out, lse = beams.attend(q, shared)
    assert torch.isfinite(out.float()).all()
    check_attend(case, q, out, lse)


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_lengths_that_the_table_cannot_hold(fmt):
    case, W, shared = shared_case([300], [[10, 10]], 4, 2, 64, fmt, seed=5)
    beams = LocksBeams([case.runtime()], width=W)
    q = case.query(case.B)
    good = beams.attend(q, shared)[0].clone()
    cols = case.table.shape[1]
    case.seq[1] = 1 << 30
    case.table[1].clamp_(min=0)
    out, _ = beams.attend(q, shared)
    assert beams.device_error() == L.LOCKS_DEVERR_LENGTHS and cols * 64 < 1 << 30
    # (shared pages and its own part are as before, in another cut of the line)
    assert (out[0].float() - good[0].float()).abs().max() < 0.02


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_pages_beyond_4_gib(fmt):
    """The same cache in the first pages of a pool and behind 4 GiB of it: the same bits."""
    hkv, P = 8, 64
    page_bytes = hkv * (144 * P if fmt == "q4" else P * D * 2)
    far = (1 << 32) // page_bytes + 5
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GiB")
    case, W, shared = shared_case([200], [[9, 9, 9]], 16, hkv, P, fmt, seed=8)
    n = case.k.shape[0]
    if fmt == "q4":
        k, v = torch.empty(far + n, hkv, 144 * P, dtype=torch.uint8, device="cuda"), None
    else:
        k, v = (torch.empty(far + n, hkv, P, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[far:] = case.k
    if v is not None:
        v[far:] = case.v
    tab = (case.table + far * (case.table >= 0)).int()
    lens = case.seq.clone()
    q = case.query(case.B)
    near = LocksBeams([case.runtime()], width=W)
    a = near.attend(q, shared)
    rt = LocksRuntime(k, v, tab, lens, case.nsum.clone(), 16, 2, 0)
    there = LocksBeams([rt], width=W)
    b = there.attend(q, shared)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    parents = torch.tensor([[2, 2, 0]], dtype=torch.int32).cuda()
    near.reorder(parents)
    there.reorder(parents)
    qkv = torch.randn(3, 16 + 2 * hkv, D, generator=case.gen).bfloat16().cuda()
    pos = torch.randint(0, 300, (2, 3), generator=case.gen).int().cuda()
    for r in (near.runtimes[0], rt):
        r.seq_lens.add_(1)
        q, kk, vv = qkv.split([16, hkv, hkv], dim=1)
        r.append(kk, vv, q, rope=table(300, 128), positions=pos, axes=L.make_axes([0, 1] * 32))
    assert torch.equal(k[far:].view(torch.uint8), case.k.view(torch.uint8))
    assert v is None or torch.equal(v[far:].view(torch.uint8), case.v.view(torch.uint8))
    a, b = near.attend(qkv[:, :16].contiguous(), shared), there.attend(qkv[:, :16].contiguous(), shared)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert near.device_error() == there.device_error() == rt.device_error() == 0


@pytest.mark.parametrize("B,W,V,keep,dtype", [(3000, 20, 64, 20, torch.bfloat16), (700, 3, 5000, 7, torch.float32),
                                              (1, 2, 1 << 22, 16, torch.bfloat16), (2, 32, 200000, 64, torch.float32)])
def test_select_of_many_rows_and_long_ones(B, W, V, keep, dtype):
    g = torch.Generator(device="cuda").manual_seed(B)
    logits = torch.randn(B, W, V, generator=g, device="cuda").mul_(3).to(dtype)
    scores = -torch.rand(B, W, generator=g, device="cuda") - 3
    beams = LocksBeams(width=W)
    got = beams.select(logits, scores, keep=keep)
    assert beams.device_error() == 0
    some = list(range(B)) if B < 100 else [0, 1, B // 2, B - 1]
    check_select([None if x is None else x[some] for x in got], logits[some], scores[some], None, -1, keep)


def test_select_of_rising_logits():
    """Every chunk exceeds the one before it: the lists overflow again and again."""
    for keep in (3, 16, 40):
        x = (torch.arange(100000).float() / 8000).expand(1, 2, -1).contiguous()
        x = torch.cat([x, x.flip(-1)]).cuda()
        scores = torch.tensor([[-1.0, -1.5]] * 2).cuda()
        got = LocksBeams(width=2).select(x, scores, keep=keep)
        check_select(got, x, scores, None, -1, keep)


def test_two_searches_on_two_streams():
    """Each with workspaces of its own, at the same time."""
    cases = [shared_case([3000], [[40, 41, 42, 43]], 16, 4, 64, fmt, seed=i) for i, fmt in enumerate(("bf16", "q4"))]
    searches = [LocksBeams([c.runtime()], width=W) for c, W, _ in cases]
    qs = [c.query(c.B) for c, _, _ in cases]
    logits, scores, _ = make(16, 4, 50000, torch.bfloat16, seed=4)
    want = [[x.clone() for x in s.attend(q, c[2])] for s, q, c in zip(searches, qs, cases)]
    pick = [LocksBeams(width=4) for _ in range(2)]
    best = [[x.clone() for x in p.select(logits, scores)[:3]] for p in pick]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs = dict(out=torch.empty_like(qs[i]), lse=torch.empty(4, 16, device="cuda"))
                some = dict(out_scores=torch.empty(16, 4, device="cuda"),
                            out_tokens=torch.empty(16, 4, dtype=torch.int32, device="cuda"),
                            out_parents=torch.empty(16, 4, dtype=torch.int32, device="cuda"))
            got.append((i, searches[i].attend(qs[i], cases[i][2], stream=st, **outs),
                        pick[i].select(logits, scores, stream=st, **some)))
    torch.cuda.synchronize()
    for i, a, b in got:
        assert all(torch.equal(x, y) for x, y in zip(a, want[i])) and all(torch.equal(x, y) for x, y in zip(b[:3], best[i]))


def test_tensors_of_another_device_are_refused(monkeypatch):
    case, W, shared = shared_case([100], [[3, 3]], 4, 1, 64, "bf16", seed=5)
    beams, q = LocksBeams([case.runtime()], width=W, end_token=1), case.query(case.B)
    logits, scores, _ = make(1, 2, 50, torch.float32, seed=1)
    ints = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    good = dict(logits=logits, scores=scores, ended=ints, out_scores=scores.clone(), out_parents=ints.clone(),
                out_tokens=ints.clone(), out_ended=ints.clone())
    for name in good:
        with pytest.raises(ValueError, match="on the device"):
            beams.select(**{**good, name: Elsewhere(good[name])})
    good = dict(q=q, shared_pages=shared, out=torch.empty_like(q), lse=torch.empty(2, 4, device="cuda"))
    for name in good:
        with pytest.raises(ValueError, match="on the device"):
            beams.attend(**{**good, name: Elsewhere(good[name])})
    with pytest.raises(ValueError, match="on the device"):
        beams.reorder(Elsewhere(ints))
    rt, kv = beams.runtimes[0], torch.zeros(2, 1, D, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="on the device"):
        rt.append(kv, kv, rope=table(100, 128), positions=Elsewhere(torch.zeros(2, 2, dtype=torch.int32, device="cuda")),
                  axes=L.make_axes([0, 1] * 32))
    here = torch.cuda.current_device()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: here + 1)
    for call in (lambda: beams.select(logits, scores, ints, stream=0), lambda: beams.attend(q, shared, stream=0),
                 lambda: beams.reorder(ints, stream=0)):
        with pytest.raises(ValueError, match="not the current device"):
            call()
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert beams.device_error() == 0 and case.seq.tolist() == [103, 103]


def test_many_rows_move():
    rows = Rows([33] * 600, 3, 1, 16, "bf16", 4, layers=2, seed=6)
    g = torch.Generator().manual_seed(2)
    rows.run(torch.randint(0, 3, (200, 3), generator=g).tolist())
    assert rows.beams.device_error() == 0


def test_own_outputs_on_another_stream():
    """Outputs that a call on another stream makes are not memory that work on the current one still writes."""
    logits, scores, _ = make(2, 4, 500, torch.float32, 5)
    beams, side = LocksBeams(width=4), torch.cuda.Stream()
    beams.select(logits, scores, keep=3, stream=side)  # the workspace
    torch.cuda.synchronize()
    before = [torch.zeros(2, 4, dtype=torch.int32, device="cuda") for _ in range(8)]
    torch.cuda._sleep(200_000_000)
    for x in before:
        x.fill_(7)
    del x, before
    got = beams.select(logits, scores, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    check_select(got, logits, scores, None, -1, 4)


@pytest.mark.parametrize("fmt,P", [("bf16", 64), ("bf16", 16), ("q4", 64), ("q4", 16)])
@pytest.mark.parametrize("prompts,W,hq,hkv", [([3000, 5, 1111], 8, 16, 4), ([9000], 16, 16, 2)])
def test_attend_gives_the_same_bits_every_time(fmt, P, prompts, W, hq, hkv):
    """The split follows the lengths alone, and nothing depends on which warp comes first."""
    tails = [[(11 * w + 3 * r) % 70 for w in range(W)] for r in range(len(prompts))]
    case, _, shared = shared_case(prompts, tails, hq, hkv, P, fmt, seed=W + P)
    beams = LocksBeams([case.runtime()], width=W)
    q = case.query(case.B)
    first = [x.clone() for x in beams.attend(q, shared)]
    check_attend(case, q, *first)
    differs = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        out, lse = beams.attend(q, shared)
        differs += (out.view(torch.int16) != first[0].view(torch.int16)).sum() + (lse != first[1]).sum()
    assert differs.item() == 0 and beams.device_error() == 0
