"""Calls on tokens and prompts refuse tensors of another device than the cache's, and to
run while another device is the current one (where they would launch)."""

import pytest
import torch

from tests.kv_cases import D, Case
from tests.test_gpu_kv_append import table
from tests.test_gpu_prompt import cu_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


class Elsewhere:
    """A tensor that says that it is on the next device."""

    def __init__(self, x):
        self._x = x

    def __getattr__(self, name):
        return getattr(self._x, name)

    @property
    def device(self):
        return torch.device("cuda", self._x.device.index + 1)

    def get_device(self):
        return self._x.device.index + 1


def test_tensors_of_another_device_are_refused():
    case = Case([100], 4, 1, 64, "bf16", seed=5)
    rt, q = case.runtime(), case.query(2)
    cu, kv = cu_of([2]), torch.zeros(2, 1, D, dtype=torch.bfloat16, device="cuda")
    before = case.k.clone()
    rope, pos = table(100, 128), torch.zeros(2, dtype=torch.int32, device="cuda")
    good = dict(k=kv, v=kv, q=q, q_out=torch.empty_like(q), rope=rope, positions=pos, cu_tokens=cu)
    for name in good:
        with pytest.raises(ValueError, match="on the device"):
            rt.append(**{**good, name: Elsewhere(good[name])}, max_tokens=2)
    good = dict(q=q, cu_tokens=cu, out=torch.empty_like(q), lse=torch.empty(2, 4, device="cuda"))
    for name in good:
        with pytest.raises(ValueError, match="on the device"):
            rt.prompt_attend(**{**good, name: Elsewhere(good[name])}, max_tokens=2)
    with pytest.raises(ValueError, match="on the device"):
        rt.read_tokens(2, cu_tokens=Elsewhere(cu), max_tokens=2)
    torch.cuda.synchronize()
    assert torch.equal(case.k.view(torch.int16), before.view(torch.int16)) and rt.device_error() == 0


def test_another_current_device_is_refused(monkeypatch):
    case = Case([100], 4, 1, 64, "q4", seed=5)
    rt, q = case.runtime(), case.query(2)
    cu, kv = cu_of([2]), torch.zeros(2, 1, D, dtype=torch.bfloat16, device="cuda")
    before = case.k.clone()
    here = torch.cuda.current_device()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: here + 1)
    for call in (lambda: rt.append(kv, kv, cu_tokens=cu, max_tokens=2, stream=0),
                 lambda: rt.read_tokens(2, cu_tokens=cu, max_tokens=2, stream=0),
                 lambda: rt.prompt_attend(q, cu_tokens=cu, max_tokens=2, stream=0)):
        with pytest.raises(ValueError, match="not the current device"):
            call()
    monkeypatch.undo()
    assert torch.equal(case.k, before) and rt.device_error() == 0
