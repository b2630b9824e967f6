"""Reorders and everything that reads what they write, one directly behind the other in one graph: the
same bits as with a wait after every call. Rows have different lengths and the parents permute them, so each
reorder changes lengths, tables and counts."""

import pytest
import torch

from sparse_kv_page_rank_gb300.beams import LocksBeams
from tests.gen_cases import shared_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("requests,W,P,hq,hkv", [(1, 4, 64, 4, 1), (3, 5, 16, 4, 2), (8, 4, 16, 2, 1), (20, 3, 16, 2, 1), (140, 2, 16, 2, 1)])
def test_behind_reorders(fmt, requests, W, P, hq, hkv):
    g = torch.Generator().manual_seed(requests + W)
    prompts = torch.randint(1, 300, (requests,), generator=g).tolist()
    tails = torch.randint(0, 120, (requests, W), generator=g).tolist()
    case, _, shared = shared_case(prompts, tails, hq, hkv, P, fmt, seed=requests, nsum=[0] * (requests * W))
    rt = case.runtime(budget=64)
    case.table.clamp_(min=0)  # entries past a row's end move with it
    beams, q = LocksBeams([rt], width=W), case.query(case.B)
    n, steps = case.B, 12
    parents = [torch.stack([torch.randperm(W, generator=g) for _ in range(requests)]).int().cuda() for _ in range(steps)]
    state = [x.clone() for x in (case.table, case.seq, case.nsum)]

    def pass_(wait):
        outs = []

        def keep(*xs):
            wait()
            outs.extend(x.clone() for x in xs)
            wait()

        for p in parents:
            beams.reorder(p)
            wait()
            keep(*beams.attend(q, shared, out=torch.empty_like(q), lse=torch.empty(n, hq, device="cuda")))
            beams.reorder(p)
            wait()
            keep(*rt.dense_decode(q, out=torch.empty_like(q), lse=torch.empty(n, hq, device="cuda")))
            beams.reorder(p)
            wait()
            keep(*rt.decode_step(q, out=torch.empty_like(q), lse=torch.empty(n, hq, device="cuda")))
            beams.reorder(p)
            wait()
            keep(*rt.prompt_attend(q))
            beams.reorder(p)
            wait()
            keep(*rt.read_tokens(n))
            keep(case.table, case.seq)
        return outs

    want = pass_(torch.cuda.synchronize)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = pass_(lambda: None)
    for _ in range(20):
        for x, y in zip((case.table, case.seq, case.nsum), state):
            x.copy_(y)
        for x in got:
            x.view(torch.uint8).fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
    assert beams.device_error() == 0 and rt.device_error() == 0
