"""Appending tokens whose positions have several axes, bit for bit (the rotation is defined
operation by operation in float32, so no tolerance is needed)."""

import pytest
import torch

from sparse_kv_page_rank_gb300 import locks as L
from tests.kv_cases import D, Case
from tests.test_gpu_kv_append import check_cache, rows_of, table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


def rotated(x, rope, positions, axes, interleaved, dtype=torch.float32):
    """x bf16 [t][h][128], a pair after another -> in `dtype` arithmetic, before the last rounding."""
    y, half = x.to(dtype), len(axes)
    out = y.clone()
    for i, axis in enumerate(axes):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        row = rope[positions[axis].long()].to(dtype)
        c, s = row[:, i, None], row[:, i + half, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
    return out


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("P,hq,hkv,lens,new,axes,interleaved", [
    (64, 32, 8, [100, 7, 64, 65], [1, 1, 1, 1], L.rope_axes([16, 24, 24]), False),
    (64, 32, 8, [3000], [2999], L.rope_axes([24, 20, 20], cyclic=True), False),
    (16, 4, 1, [33, 1, 500], [33, 0, 17], L.rope_axes([15, 17]), False),
    (16, 6, 2, [33, 1, 500], [5, 1, 499], L.rope_axes([16, 16, 16], cyclic=True), True),
    (64, 1, 1, [1], [1], [3, 0, 2, 1, 1, 2, 0, 3], False),
    (64, 16, 1, [1000, 0, 129], [900, 0, 129], L.rope_axes([0, 1, 63]), True),
    (16, 3, 3, [250, 251, 252, 253, 254], [16, 15, 1, 31, 32], [0] * 16, False),
    (64, 4, 2, [700, 900], [650, 900], [i % 4 for i in range(48)], False),
])
def test_append(fmt, P, hq, hkv, lens, new, axes, interleaved):
    case = Case(lens, hq, hkv, P, fmt, seed=len(axes) + P + len(lens))
    rt = case.runtime()
    seq, at, cu = rows_of(lens, new)
    total, spare = sum(new), 3  # rows behind the last sequence
    qkv = (torch.randn(total + spare, hq + 2 * hkv, D, generator=case.gen) * 3).bfloat16().cuda()
    q, k, v = qkv.split([hq, hkv, hkv], dim=1)
    rope = table(500, 2 * len(axes))
    n = max(axes) + 1
    wide = torch.randint(0, 500, (n, total + spare + 5), generator=case.gen).int().cuda()
    wide[:, total:] = -1  # positions of nobody
    pos = wide[:, :total + spare]
    before = (case.k.clone(), None if case.v is None else case.v.clone())
    q_out = torch.full((total + spare, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got = rt.append(k, v, q, rope=rope, interleaved=interleaved, positions=pos, axes=L.make_axes(axes), cu_tokens=cu,
                    max_tokens=max(new), q_out=q_out)
    assert got is q_out and rt.device_error() == 0
    want = rotated(q[:total], rope, pos[:, :total], axes, interleaved).bfloat16()
    assert torch.equal(q_out[:total], want) and (q_out[total:] == 7).all()
    kr = rotated(k[:total], rope, pos[:, :total], axes, interleaved).bfloat16()
    check_cache(case, before, kr, v[:total], seq, at)
    # its meaning: three float32 roundings (2^-24 of |a c| + |b s| each) and one to bf16 (2^-8 of the result)
    exact = rotated(q[:total], rope, pos[:, :total], axes, interleaved, torch.float64)
    mag = 2 * q[:total].double().abs().amax(dim=-1, keepdim=True)
    assert ((want.double() - exact).abs() <= 2.0 ** -8 * exact.abs() + 3 * 2.0 ** -24 * mag).all()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_one_row_on_every_axis_is_append(fmt, interleaved):
    lens, new = [900, 70, 64], [900, 1, 30]
    pair = [Case(lens, 8, 2, 16, fmt, seed=9) for _ in range(2)]
    _, _, cu = rows_of(lens, new)
    total = sum(new)
    q, k, v = (torch.randn(total, h, D, generator=pair[0].gen).bfloat16().cuda() for h in (8, 2, 2))
    rope = table(1000, 128)
    pos = torch.randint(0, 1000, (total,), generator=pair[0].gen).int().cuda()
    a = pair[0].runtime().append(k, v, q, rope=rope, interleaved=interleaved, positions=pos, cu_tokens=cu)
    b = pair[1].runtime().append(k, v, q, rope=rope, interleaved=interleaved, positions=pos.repeat(3, 1),
                                 axes=L.make_axes(L.rope_axes([22, 21, 21], cyclic=True)), cu_tokens=cu)
    assert torch.equal(a, b)
    for x, y in ((pair[0].k, pair[1].k), (pair[0].v, pair[1].v)):
        assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_a_token_with_a_row_outside_on_one_axis_is_skipped():
    case = Case([40, 41], 4, 2, 16, "bf16", seed=3)
    rt = case.runtime()
    q, k, v = (torch.randn(2, h, D, generator=case.gen).bfloat16().cuda() for h in (4, 2, 2))
    rope, axes = table(30, 128), [0, 1] * 32
    for bad in (30, -1):
        pos = torch.tensor([[3, 4], [5, bad]], dtype=torch.int32).cuda()
        before = (case.k.clone(), case.v.clone())
        q_out = torch.full_like(q, 7.0)
        rt.append(k, v, q, rope=rope, positions=pos, axes=L.make_axes(axes), q_out=q_out)
        assert rt.device_error() == L.LOCKS_DEVERR_POSITION
        assert (q_out[1] == 7).all() and torch.equal(q_out[:1], rotated(q[:1], rope, pos[:, :1], axes, False).bfloat16())
        seq, at = torch.tensor([0], device="cuda"), torch.tensor([39], device="cuda")
        check_cache(case, before, rotated(k[:1], rope, pos[:, :1], axes, False).bfloat16(), v[:1], seq, at)


def test_captured_on_a_stream_of_its_own():
    case = Case([40, 41], 4, 2, 16, "q4", seed=16, extra_cols=0)
    rt = case.runtime()
    q, k, v = (torch.randn(2, h, D, generator=case.gen).bfloat16().cuda() for h in (4, 2, 2))
    rope, axes = table(50, 128), L.rope_axes([16, 24, 24])
    pos = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    stream, graph, ax = torch.cuda.Stream(), torch.cuda.CUDAGraph(), L.make_axes(axes)
    stream.wait_stream(torch.cuda.current_stream())
    q_out = torch.empty_like(q)
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            rt.append(k, v, q, rope=rope, positions=pos, axes=ax, q_out=q_out, stream=stream)
    for rows in ([[0, 1], [2, 3], [4, 5]], [[49, 0], [7, 7], [8, 30]]):
        pos.copy_(torch.tensor(rows, dtype=torch.int32))
        before = (case.k.clone(), None)
        graph.replay()
        torch.cuda.synchronize()
        seq, at = torch.tensor([0, 1], device="cuda"), torch.tensor([39, 40], device="cuda")
        assert torch.equal(q_out, rotated(q, rope, pos, axes, False).bfloat16())
        check_cache(case, before, rotated(k, rope, pos, axes, False).bfloat16(), v, seq, at)
    assert rt.device_error() == 0


def test_refusals():
    case = Case([40, 41], 4, 2, 16, "bf16", seed=3)
    rt = case.runtime()
    q, k, v = (torch.randn(2, h, D, generator=case.gen).bfloat16().cuda() for h in (4, 2, 2))
    rope, pos, axes = table(30, 128), torch.zeros(2, 2, dtype=torch.int32, device="cuda"), L.make_axes([0, 1] * 32)
    before = case.k.clone()
    for kw in (dict(rope=None), dict(positions=None), dict(positions=pos.long()), dict(positions=pos[:, :1]),
               dict(positions=pos[:1]), dict(positions=pos.repeat(3, 1)[:5]), dict(positions=pos[0]), dict(rope=table(30, 64)),
               dict(positions=pos.T.contiguous().T), dict(positions=pos[:1].expand(2, 2)), dict(positions=pos.cpu())):
        with pytest.raises(ValueError):
            rt.append(k, v, q, **{**dict(rope=rope, positions=pos, axes=axes), **kw})
    for bad in ([], [0] * 65, [0, 4], [-1]):
        with pytest.raises(ValueError):
            L.make_axes(bad)
    for bad in (([], False), ([3, -1], False), ([1, 5], True)):
        with pytest.raises(ValueError):
            L.rope_axes(*bad)
    torch.cuda.synchronize()
    assert torch.equal(case.k.view(torch.int16), before.view(torch.int16)) and rt.device_error() == 0
