"""Writing tokens into the cache and reading them back, bit for bit.

The rotation is defined operation by operation in float32 (each product and the sum
rounded once), so torch's own float32 products and sums give the same bits; the
4-bit codes follow from those bf16 numbers exactly.  No tolerance is needed, but for
the rotation's meaning, which is compared with 64 bits: three float32 roundings
(3 * 2^-24 of |a c| + |b s|) and one to bf16 (2^-8 of the result)."""

import pytest
import torch

from tests.kv_cases import D, Case, unpack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


def table(rows, rot, base=10000.0):
    inv = base ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / max(rot, 1))
    at = torch.arange(rows, dtype=torch.float64)[:, None] * inv
    return torch.cat([at.cos(), at.sin()], dim=1).float().cuda()


def rotated(x, rope, row, rot, interleaved, dtype=torch.float32):
    """x bf16 [t][h][128] -> rotated, in `dtype` arithmetic, before the last rounding."""
    y = x.to(dtype)
    if rot == 0:
        return y
    cs = rope[row.long()].to(dtype)[:, None]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    i = torch.arange(rot // 2, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = y[..., ia], y[..., ib]
    out = y.clone()
    out[..., ia] = a * c - b * s
    out[..., ib] = b * c + a * s
    return out


def quantised(x):
    """bf16 [..., 128] -> codes int32 [..., 128], half scales [..., 4]."""
    g = x.float().unflatten(-1, (4, 32))
    s = (g.abs().amax(dim=-1) / 7).clamp(max=9352).half()
    q = torch.where(s[..., None] > 0, g / s.float()[..., None], torch.zeros_like(g)).round().clamp(-7, 7)
    return q.flatten(-2).int(), s


def rows_of(lens, new):
    seq = torch.tensor([b for b, n in enumerate(new) for _ in range(n)], dtype=torch.long)
    at = torch.tensor([lens[b] - n + i for b, n in enumerate(new) for i in range(n)], dtype=torch.long)
    cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32).cuda()
    return seq.cuda(), at.cuda(), cu


def check_cache(case, before, k, v, seq, at):
    """The pools hold k, v (bf16) at the tokens' slots and are untouched elsewhere."""
    page, slot = case.table[seq, at // case.P].long(), at % case.P
    if case.fmt == "bf16":
        for pool, old, x in ((case.k, before[0], k), (case.v, before[1], v)):
            want = old.clone()
            want[page, :, slot] = x
            assert torch.equal(pool.view(torch.int16), want.view(torch.int16))
        return
    got, old = unpack(case.k), unpack(before[0])
    for i, x in ((0, k), (2, v)):
        q, s = quantised(x)
        old[i][page, :, slot] = q
        old[i + 1][page, :, slot] = s
        assert torch.equal(got[i], old[i])
        assert torch.equal(got[i + 1].view(torch.int16), old[i + 1].view(torch.int16))


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("P,hq,hkv,lens,new,rot,interleaved", [
    (64, 32, 8, [100, 7, 64, 65], [1, 1, 1, 1], 128, False),
    (16, 4, 1, [33, 1, 500], [33, 0, 17], 64, False),
    (16, 6, 2, [33, 1, 500], [5, 1, 499], 96, True),
    (64, 1, 1, [1], [1], 16, False),
    (64, 16, 1, [1000, 0, 129], [900, 0, 129], 128, True),
    (16, 3, 3, [250, 251, 252, 253, 254], [16, 15, 1, 31, 32], 32, False),
    (64, 8, 2, [300], [200], 0, False),
])
def test_append_and_read(fmt, P, hq, hkv, lens, new, rot, interleaved):
    case = Case(lens, hq, hkv, P, fmt, seed=rot + P + len(lens))
    rt = case.runtime()
    seq, at, cu = rows_of(lens, new)
    total, spare = sum(new), 3  # rows behind the last sequence
    qkv = (torch.randn(total + spare, hq + 2 * hkv, D, generator=case.gen) * 3).bfloat16().cuda()
    qkv[:, :, 40] *= 20
    q, k, v = qkv.split([hq, hkv, hkv], dim=1)
    rope = table(max(lens) + 1, rot) if rot else None
    before = (case.k.clone(), None if case.v is None else case.v.clone())
    q_out = torch.full((total + spare, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got = rt.append(k, v, q, rope=rope, interleaved=interleaved, cu_tokens=cu, max_tokens=max(new), q_out=q_out)
    assert got is q_out and rt.device_error() == 0
    want = rotated(q[:total], rope, at, rot, interleaved).bfloat16()
    assert torch.equal(q_out[:total], want) and (q_out[total:] == 7).all()
    kr = rotated(k[:total], rope, at, rot, interleaved).bfloat16()
    check_cache(case, before, kr, v[:total], seq, at)
    if rot:
        exact = rotated(k[:total], rope, at, rot, interleaved, torch.float64)
        mag = rotated(k[:total].abs(), rope.abs(), at, rot, interleaved, torch.float64).abs()
        mag = torch.maximum(mag, 2 * k[:total].double().abs().amax(dim=-1, keepdim=True))
        assert ((kr.double() - exact).abs() <= 2.0 ** -8 * exact.abs() + 3 * 2.0 ** -24 * mag).all()
    # reading gives the numbers that attention sees
    ko, vo = rt.read_tokens(total + spare, cu_tokens=cu, max_tokens=max(new))
    if fmt == "bf16":
        assert torch.equal(ko[:total], kr) and torch.equal(vo[:total], v[:total])
    else:
        for x, y in ((ko, kr), (vo, v[:total])):
            c, s = quantised(y)
            assert torch.equal(x[:total], (c.float() * s.float().repeat_interleave(32, dim=-1)).bfloat16())
    # without queries the cache gets the same
    other = Case(lens, hq, hkv, P, fmt, seed=rot + P + len(lens))
    other.runtime().append(k, v, rope=rope, interleaved=interleaved, cu_tokens=cu)
    assert torch.equal(other.k.view(torch.uint8), case.k.view(torch.uint8))


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_one_token_per_sequence_and_idle_slots(fmt):
    lens = [5, 0, 64, 65, 0, 130]
    case = Case(lens, 8, 2, 64, fmt, seed=4)
    rt = case.runtime()
    q, k, v = (torch.randn(6, h, D, generator=case.gen).bfloat16().cuda() for h in (8, 2, 2))
    rope = table(200, 128)
    before = (case.k.clone(), None if case.v is None else case.v.clone())
    q_in = q.clone()
    rt.append(k, v, q, rope=rope, q_out=q)  # in place
    assert rt.device_error() == 0
    live = torch.tensor([b for b, n in enumerate(lens) if n], device="cuda")
    at = torch.tensor([n - 1 for n in lens if n], device="cuda")
    assert torch.equal(q[live], rotated(q_in[live], rope, at, 128, False).bfloat16())
    assert torch.equal(q[[1, 4]], q_in[[1, 4]])
    check_cache(case, before, rotated(k[live], rope, at, 128, False).bfloat16(), v[live], live, at)


def test_positions_of_the_callers_own():
    lens, new = [50, 20], [10, 20]
    case = Case(lens, 4, 2, 16, "q4", seed=6)
    rt = case.runtime()
    seq, at, cu = rows_of(lens, new)
    k, v = (torch.randn(30, 2, D, generator=case.gen).bfloat16().cuda() for _ in range(2))
    pos = torch.randint(0, 4000, (30,), generator=case.gen).int().cuda()
    rope = table(4000, 64)
    before = (case.k.clone(), None)
    rt.append(k, v, rope=rope, positions=pos, cu_tokens=cu)
    check_cache(case, before, rotated(k, rope, pos, 64, False).bfloat16(), v, seq, at)
    assert rt.device_error() == 0


def test_extreme_groups_in_4_bits():
    """Zeros, subnormal scales, ties, numbers beyond what a scale can hold, infinities and NaN."""
    case = Case([16], 1, 1, 16, "q4", seed=2)
    rt = case.runtime()
    x = torch.zeros(16, 1, D)
    x[1, 0, :32] = 2.0 ** -30
    x[2, 0, :32] = torch.arange(32) * 2.0 ** -22
    x[3, 0, :32] = torch.arange(32).float() * 0.25 - 4  # scale 4/7 in half, many near-ties
    x[4, 0, :32] = torch.linspace(-3.5, 3.5, 32)
    x[4, 0, 0] = 7.0  # scale 1: halves are ties
    x[5, 0, :32] = 1e6
    x[6, 0, 3], x[7, 0, 40] = float("inf"), float("nan")
    x[8, 0, :32] = -65000.0
    x = x.bfloat16().cuda()
    before = (case.k.clone(), None)
    rt.append(x, x, cu_tokens=torch.tensor([0, 16], dtype=torch.int32).cuda())
    kq, ks, vq, vs = unpack(case.k)
    page = int(case.table[0, 0])
    for q, s in ((kq, ks), (vq, vs)):
        q, s = q[page, 0], s[page, 0]
        assert torch.isnan(s[6, 0]) and torch.isnan(s[7, 1]) and torch.isfinite(s[7, 0]) and torch.isfinite(s[6, 1])
        keep = torch.ones(16, 4, dtype=torch.bool, device="cuda")
        keep[6, 0] = keep[7, 1] = False
        wq, ws = quantised(torch.where(torch.isfinite(x), x, torch.zeros_like(x))[:, 0])
        assert torch.equal(s[keep], ws[keep])
        assert torch.equal(q.unflatten(-1, (4, 32))[keep], wq.unflatten(-1, (4, 32))[keep])
        assert s[5, 0] == 9352 and (q[5, :32] == 7).all()
    assert rt.device_error() == 0


def test_what_only_the_device_can_see():
    from sparse_kv_page_rank_gb300 import locks as L
    case = Case([50, 20], 4, 2, 16, "bf16", seed=6)
    rt = case.runtime()
    k, v = (torch.randn(30, 2, D, generator=case.gen).bfloat16().cuda() for _ in range(2))
    rope = table(30, 64)

    def call(cu, **kw):
        before = case.k.clone()
        rt.append(k, v, cu_tokens=torch.tensor(cu, dtype=torch.int32).cuda(), **kw)
        err = rt.device_error()
        return err, int((case.k.view(torch.int16) != before.view(torch.int16)).any(dim=(1, 3)).sum())

    assert call([0, 5, 30], rope=rope)[0] == L.LOCKS_DEVERR_POSITION | L.LOCKS_DEVERR_LENGTHS  # 25 new of 20; position 49
    assert call([0, 0, 30])[0] == L.LOCKS_DEVERR_LENGTHS
    # sequence 0 writes 10 of its 20; sequence 1's rows 20-29 at positions 10-19 are what the call before left there
    assert call([0, 20, 30], max_tokens=10) == (L.LOCKS_DEVERR_LENGTHS, 10)
    case.table[0, 3] = 1 << 20
    case.table[1, 1] = -1
    assert call([0, 10, 20])[0] == L.LOCKS_DEVERR_BLOCK_TABLE
    assert call([30, 10, 20])[0] & ~L.LOCKS_DEVERR_BLOCK_TABLE in (0, L.LOCKS_DEVERR_LENGTHS)


def test_strides_and_captured_append():
    case = Case([40, 41], 4, 2, 16, "q4", seed=16, extra_cols=0)
    rt = case.runtime()
    wide = torch.randn(2, 64, D, generator=case.gen).bfloat16().cuda()
    q, k, v = wide[:, 3:7], wide[:, 20:22], wide[:, 50:52]
    rope = table(50, 128)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    q_out = torch.empty(2, 4, D, dtype=torch.bfloat16, device="cuda")
    with torch.cuda.stream(stream):
        rt.append(k, v, q, rope=rope, q_out=q_out, stream=stream)
        with torch.cuda.graph(graph, stream=stream):
            rt.append(k, v, q, rope=rope, q_out=q_out, stream=stream)
    torch.cuda.synchronize()
    for lens in ([40, 41], [17, 48]):
        case.seq.copy_(torch.tensor(lens, dtype=torch.int32))
        wide.copy_(torch.randn(2, 64, D, generator=case.gen).bfloat16())
        before = (case.k.clone(), None)
        graph.replay()
        torch.cuda.synchronize()
        seq, at = torch.tensor([0, 1], device="cuda"), torch.tensor(lens, device="cuda") - 1
        check_cache(case, before, rotated(k, rope, at, 128, False).bfloat16(), v, seq, at)
        assert torch.equal(q_out, rotated(q, rope, at, 128, False).bfloat16())
    assert rt.device_error() == 0
