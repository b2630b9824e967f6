"""A cache's whole life: prompts appended and attended, their full pages summarised,
then decode steps and draft tokens that each append to what the last left behind.
Cache contents are compared with a history kept beside it, attention with 64 bits."""

import pytest
import torch

from tests.kv_cases import D, Case
from tests.test_gpu_kv_append import rotated, table
from tests.test_gpu_kv_q4 import check as check_decode_q4
from tests.test_gpu_prompt import check as check_rows
from tests.test_gpu_prompt import cu_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


class Served:
    def __init__(self, fmt, P, final, hq, hkv, budget):
        self.case = Case(final, hq, hkv, P, fmt, seed=P + sum(final))
        for pool in (self.case.k, self.case.v):
            if pool is not None:  # nothing is in the cache yet
                pool.view(torch.uint8).fill_(0xff)
        self.case.lens = [0] * len(final)
        self.case.seq.zero_()
        self.case.nsum.zero_()
        self.rt = self.case.runtime(budget=budget)
        self.rope = table(max(final), D)
        self.k = [torch.zeros(0, hkv, D, device="cuda") for _ in final]
        self.v = [torch.zeros(0, hkv, D, device="cuda") for _ in final]

    def tokens(self, new):
        """New tokens' projections, and their positions."""
        c, n = self.case, sum(new)
        qkv = torch.randn(n, c.hq + 2 * c.hkv, D, generator=c.gen).bfloat16().cuda()
        at = torch.cat([torch.arange(c.lens[b], c.lens[b] + m) for b, m in enumerate(new)]).cuda()
        return qkv, at

    def record(self, new, qkv, at):
        """The history of the tokens, and the new lengths."""
        c = self.case
        _, k, v = qkv.split([c.hq, c.hkv, c.hkv], dim=1)
        k = rotated(k, self.rope, at, D, False).bfloat16().float()
        row = 0
        for b, m in enumerate(new):
            self.k[b] = torch.cat([self.k[b], k[row:row + m]])
            self.v[b] = torch.cat([self.v[b], v[row:row + m].float()])
            row += m
            c.lens[b] += m

    def append(self, new):
        qkv, at = self.tokens(new)
        c = self.case
        q, k, v = qkv.split([c.hq, c.hkv, c.hkv], dim=1)
        want = rotated(q, self.rope, at, D, False).bfloat16()
        self.record(new, qkv, at)
        c.seq.copy_(torch.tensor(c.lens, dtype=torch.int32))
        q = self.rt.append(k, v, q, rope=self.rope, cu_tokens=cu_of(new), max_tokens=max(new))
        assert torch.equal(q, want)
        return q

    def summarise(self):
        """The pages that are full and not summarised yet."""
        c = self.case
        had = c.nsum.tolist()
        now = [n // c.P for n in c.lens]
        ids = torch.cat([c.table[b, had[b]:now[b]] for b in range(c.B)])
        if len(ids):
            self.rt.build_summaries(ids)
        c.nsum.copy_(torch.tensor(now, dtype=torch.int32))

    def check_cache(self):
        c = self.case
        for b in range(c.B):
            for got, want in zip(c.kv64(b), (self.k[b], self.v[b])):
                want = want.transpose(0, 1).double()
                if c.fmt == "bf16":
                    assert torch.equal(got, want)
                else:
                    # half a step of the group, whose scale is off by 2^-11 at most
                    top = want.abs().unflatten(-1, (4, 32)).amax(-1, keepdim=True).expand(*want.shape[:2], 4, 32)
                    assert ((got - want).abs() <= top.flatten(-2) * (0.5 / 7) * 1.02).all()

    def check_decode(self, q, out, lse):
        if self.case.fmt == "q4":
            check_decode_q4(self.case, q, out, lse)
        else:
            check_rows(self.case, [1] * self.case.B, q, out, lse)


@pytest.mark.parametrize("fmt,P,hq,hkv", [("bf16", 64, 8, 2), ("q4", 64, 8, 2), ("q4", 16, 12, 4), ("bf16", 16, 4, 4),
                                          ("q4", 64, 16, 1)])
def test_prompts_then_steps(fmt, P, hq, hkv):
    prompts = [130, 64, 301, 1]
    s = Served(fmt, P, [n + 40 for n in prompts], hq, hkv, budget=1024)
    q = s.append(prompts)
    out, lse = s.rt.prompt_attend(q, cu_tokens=cu_of(prompts), max_tokens=max(prompts))
    check_rows(s.case, prompts, q, out, lse)
    s.check_cache()
    s.summarise()
    for step in range(3):
        # one token each: every page, then the selected pages (the budget holds them all)
        q = s.append([1] * 4)
        s.check_decode(q, *s.rt.dense_decode(q))
        s.check_decode(q, *s.rt.decode_step(q))
        # drafts of different lengths, none for one sequence
        new = [3, 0, 5, 2]
        q = s.append(new)
        out, lse = s.rt.prompt_attend(q, cu_tokens=cu_of(new), max_tokens=5)
        check_rows(s.case, new, q, out, lse)
        s.summarise()
    # another prompt for one sequence beside single tokens of the others
    new = [1, 1, 9, 1]
    q = s.append(new)
    out, lse = s.rt.prompt_attend(q, cu_tokens=cu_of(new), max_tokens=9)
    check_rows(s.case, new, q, out, lse)
    s.check_cache()
    assert s.rt.device_error() == 0


@pytest.mark.parametrize("fmt,P", [("bf16", 64), ("q4", 16)])
def test_a_captured_step_appends_and_attends(fmt, P):
    """Lengths, append, drafts' attention and decode in one graph, replayed as the cache grows."""
    s = Served(fmt, P, [200, 90], 8, 2, budget=1024)
    prompts = [150, 40]
    q = s.append(prompts)
    s.rt.prompt_attend(q, cu_tokens=cu_of(prompts), max_tokens=150)
    new, cu, c = [2, 2], cu_of([2, 2]), s.case
    qkv, at = s.tokens(new)
    parts = qkv.split([c.hq, c.hkv, c.hkv], dim=1)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()

    def step():
        c.seq.add_(2)
        rows = s.rt.append(parts[1], parts[2], parts[0], rope=s.rope, cu_tokens=cu, max_tokens=2)
        out, lse = s.rt.prompt_attend(rows, cu_tokens=cu, max_tokens=2)
        last = rows[1::2].contiguous()
        s.rt.dense_decode(last)
        return rows, out, lse, last

    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()  # grows the workspace; its two tokens are written again by the first replay
        c.seq.sub_(2)
        with torch.cuda.graph(graph, stream=stream):
            rows, out, lse, last = step()
    torch.cuda.synchronize()
    for _ in range(4):
        fresh, at = s.tokens(new)
        qkv.copy_(fresh)
        graph.replay()
        torch.cuda.synchronize()
        s.record(new, qkv, at)
        assert c.seq.tolist() == c.lens
        assert torch.equal(rows, rotated(qkv[:, :c.hq], s.rope, at, D, False).bfloat16())
        check_rows(c, new, rows, out, lse)
        s.check_decode(last, s.rt.out, s.rt.lse)
    s.check_cache()
    assert s.rt.device_error() == 0


def test_a_captured_call_keeps_its_workspace_when_a_later_one_outgrows_it():
    case = Case([9000], 4, 1, 64, "bf16", seed=5)
    rt, q, cu = case.runtime(), case.query(3), cu_of([3])
    first, _ = rt.prompt_attend(q, cu_tokens=cu, max_tokens=3)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        out, _ = rt.prompt_attend(q, cu_tokens=cu, max_tokens=3)
    was = rt.prompt_ws.data_ptr()
    many = case.query(400)
    rt.prompt_attend(many, cu_tokens=cu_of([400]), max_tokens=400)
    assert rt.prompt_ws.data_ptr() != was
    junk = torch.full((64 << 20,), 0xff, dtype=torch.uint8, device="cuda")  # memory given back would be here
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and (junk == 0xff).all()
    assert rt.device_error() == 0


def test_a_capture_does_not_grow_the_workspace():
    case = Case([9000], 4, 1, 64, "bf16", seed=5)
    rt, q, cu = case.runtime(), case.query(3), cu_of([3])
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        with pytest.raises(RuntimeError, match="before the capture"):
            rt.prompt_attend(q, cu_tokens=cu, max_tokens=3)


def test_nothing_to_do():
    case = Case([100], 4, 1, 64, "q4", seed=5)
    rt = case.runtime()
    none = torch.zeros(0, 4, D, dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    was = case.k.clone()
    assert rt.append(none[:, :1], none[:, :1], none, cu_tokens=cu).shape == (0, 4, D)
    assert [x.shape for x in rt.read_tokens(0, cu_tokens=cu)] == [(0, 1, D)] * 2
    out, lse = rt.prompt_attend(none, cu_tokens=cu)
    assert out.shape == (0, 4, D) and lse.shape == (0, 4)
    assert rt.device_error() == 0 and torch.equal(case.k, was)


def test_wrong_places_and_shapes_are_refused():
    case = Case([100], 4, 1, 64, "bf16", seed=5)
    rt, q = case.runtime(), case.query(2)
    cu, kv = cu_of([2]), torch.zeros(2, 1, D, dtype=torch.bfloat16, device="cuda")
    for bad in (cu.cpu(), cu.long(), cu_of([1, 1]), torch.cat([cu, cu])[::2]):
        with pytest.raises(ValueError, match="cu_tokens"):
            rt.prompt_attend(q, cu_tokens=bad, max_tokens=2)
    for out in (torch.empty(3, 4, D, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 4, D, device="cuda"),
                torch.empty(2, 4, D, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="out must be"):
            rt.prompt_attend(q, cu_tokens=cu, max_tokens=2, out=out)
    for lse in (torch.empty(4, 2, device="cuda"), torch.empty(2, 4), torch.empty(2, 4, device="cuda").bfloat16()):
        with pytest.raises(ValueError, match="lse must be"):
            rt.prompt_attend(q, cu_tokens=cu, max_tokens=2, lse=lse)
    with pytest.raises(ValueError, match="on the device"):
        rt.prompt_attend(q.cpu(), cu_tokens=cu, max_tokens=2)
    for args, kw in (((kv.cpu(), kv), {}), ((kv, kv, q.cpu()), {}), ((kv, kv, q), {"q_out": q.cpu()}),
                     ((kv, kv), {"rope": table(100, 128).cpu()}),
                     ((kv, kv), {"rope": table(100, 128), "positions": torch.zeros(2, dtype=torch.int32)})):
        with pytest.raises(ValueError, match="on the device"):
            rt.append(*args, cu_tokens=cu, max_tokens=2, **kw)
    assert rt.device_error() == 0


@pytest.mark.parametrize("P", [64, 16])
def test_the_growing_loop_over_4_bit_pages(P):
    """Captured segments of decode steps, filled pages summarised beside them."""
    from sparse_kv_page_rank_gb300.growing import GrowingLoop
    segments = 3
    case = Case([P * (4 + segments), P * (2 + segments)], 8, 2, P, "q4", seed=P, nsum=[4, 2])
    case.seq.copy_(torch.tensor([4 * P, 2 * P], dtype=torch.int32))
    rt, q = case.runtime(budget=1024), case.query(2)
    for b in range(2):
        rt.build_summaries(case.table[b, :case.nsum[b]])
    loop = GrowingLoop(rt, q)
    loop.run(segments)
    torch.cuda.synchronize()
    assert case.seq.tolist() == case.lens and rt.device_error() == 0
    check_decode_q4(case, q, rt.out, rt.lse)  # the budget holds every page


@pytest.mark.parametrize("raw", [False, True])
def test_calls_on_another_stream(raw):
    """Outputs that a call makes belong to the stream it is given."""
    s = Served("q4", 64, [300, 100], 8, 2, budget=0)
    other = torch.cuda.Stream()
    qkv, at = s.tokens([300, 100])
    q, k, v = qkv.split([8, 2, 2], dim=1)
    s.record([300, 100], qkv, at)
    s.case.seq.copy_(torch.tensor(s.case.lens, dtype=torch.int32))
    cu = cu_of([300, 100])
    torch.cuda.synchronize()
    on = other.cuda_stream if raw else other
    rows = s.rt.append(k, v, q, rope=s.rope, cu_tokens=cu, max_tokens=300, stream=on)
    out, lse = s.rt.prompt_attend(rows, cu_tokens=cu, max_tokens=300, stream=on)
    kr, vr = s.rt.read_tokens(400, cu_tokens=cu, max_tokens=300, stream=on)
    other.synchronize()
    assert s.rt.device_error() == 0
    assert torch.equal(rows, rotated(q, s.rope, at, D, False).bfloat16())
    check_rows(s.case, [300, 100], rows, out, lse)
    want = [torch.cat([x.transpose(0, 1) for x in pair]) for pair in zip(s.case.kv64(0), s.case.kv64(1))]
    for got, x in zip((kr, vr), want):
        assert torch.equal(got, x.float().bfloat16())


def test_the_step_without_a_workspace_over_4_bit_pages():
    from sparse_kv_page_rank_gb300 import locks as L
    case = Case([1000, 130], 8, 2, 64, "q4", seed=9, nsum=[14, 1])
    rt, q = case.runtime(budget=256), case.query(2)
    for b in range(2):
        rt.build_summaries(case.table[b, :case.nsum[b]])
    out, lse = (x.clone() for x in rt.decode_step(q))
    got, glse = torch.zeros_like(out), torch.zeros_like(lse)
    err = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    L.locks_decode_step_static(rt.cache, rt.summary, rt.params, q, got, glse, None, None, err)
    assert int(err) == 0 and torch.equal(got, out) and torch.equal(glse, lse)


@pytest.mark.parametrize("fmt,P", [("bf16", 64), ("bf16", 16), ("q4", 64), ("q4", 16)])
def test_pages_beyond_4_gib_of_a_pool(fmt, P):
    """The same pages in a small pool and at the end of a large one give the same bits."""
    from sparse_kv_page_rank_gb300.runtime import LocksRuntime
    small = Case([700, 90], 16, 8, P, fmt, seed=P)
    page_bytes = small.k[0].numel() * small.k.element_size()
    pages = (9 << 30) // 2 // page_bytes
    shift = pages - small.k.shape[0]
    pools = []
    for x in (small.k, small.v):
        if x is not None:
            big = torch.empty((pages,) + tuple(x.shape[1:]), dtype=x.dtype, device="cuda")
            big[shift:] = x
            pools.append(big)
    high_table = small.table + shift
    rt = small.runtime()
    high = LocksRuntime(pools[0], pools[1] if len(pools) == 2 else None, high_table, small.seq, small.nsum, 16, 2, 0)
    rope, gen = table(800, D), torch.Generator().manual_seed(1)
    for new in ([3, 1], [400, 80]):
        cu = cu_of(new)
        qkv = torch.randn(sum(new), 32, D, generator=gen).bfloat16().cuda()
        got = []
        for r in (rt, high):
            q = r.append(qkv[:, 16:24], qkv[:, 24:], qkv[:, :16], rope=rope, cu_tokens=cu, max_tokens=max(new))
            k, v = r.read_tokens(sum(new), cu_tokens=cu, max_tokens=max(new))
            out, lse = r.prompt_attend(q, cu_tokens=cu, max_tokens=max(new))
            dec, dlse = r.dense_decode(q[:2].contiguous())
            got.append([q, k, v, out, lse, dec.clone(), dlse.clone()])
            assert r.device_error() == 0
        for a, b in zip(*got):
            assert torch.equal(a, b)
