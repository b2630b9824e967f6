"""The prompt attention's workspace when the call goes to a stream that is not the current one."""

import weakref

import pytest
import torch

from tests.kv_cases import D, Case
from tests.test_gpu_prompt import check, cu_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


@pytest.mark.parametrize("raw", [False, True])
def test_a_call_captured_on_another_stream_keeps_its_workspace(raw):
    case = Case([9000], 4, 1, 64, "bf16", seed=5)
    rt, q, cu = case.runtime(), case.query(3), cu_of([3])
    first, _ = rt.prompt_attend(q, cu_tokens=cu, max_tokens=3)
    out, lse = torch.empty_like(q), torch.empty(3, 4, device="cuda")
    graph, stream, other = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream, capture_error_mode="thread_local"):
        with torch.cuda.stream(other):  # not captured
            rt.prompt_attend(q, cu_tokens=cu, max_tokens=3, out=out, lse=lse,
                             stream=stream.cuda_stream if raw else stream)
    used = weakref.ref(rt.prompt_ws)
    rt.prompt_attend(case.query(400), cu_tokens=cu_of([400]), max_tokens=400)
    assert rt.prompt_ws is not used()
    assert used() is not None, "the graph's workspace was given back"
    junk = torch.full((64 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and (junk == 0xff).all()
    assert rt.device_error() == 0


def test_a_capture_on_another_stream_does_not_grow_the_workspace():
    case = Case([9000], 4, 1, 64, "bf16", seed=5)
    rt, q, cu = case.runtime(), case.query(3), cu_of([3])
    out, lse = torch.empty_like(q), torch.empty(3, 4, device="cuda")
    graph, stream, other = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream, capture_error_mode="thread_local"):
        with torch.cuda.stream(other):
            with pytest.raises(RuntimeError, match="before the capture"):
                rt.prompt_attend(q, cu_tokens=cu, max_tokens=3, out=out, lse=lse, stream=stream)
    # the capture was not disturbed, and calls outside of one work
    out, lse = rt.prompt_attend(q, cu_tokens=cu, max_tokens=3, stream=stream)
    torch.cuda.synchronize()
    check(case, [3], q, out, lse)
    assert rt.device_error() == 0 and out.shape == (3, 4, D)


def test_the_default_streams_handle():
    case = Case([300], 4, 1, 64, "q4", seed=5)
    rt, q, cu = case.runtime(), case.query(3), cu_of([3])
    out, lse = rt.prompt_attend(q, cu_tokens=cu, max_tokens=3, stream=0)
    torch.cuda.synchronize()
    check(case, [3], q, out, lse)
