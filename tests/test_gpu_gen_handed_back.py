"""Outputs of a choice handed back as the next one's hypotheses, and kept over steps."""

import pytest
import torch

from sparse_kv_page_rank_gb300 import locks as L
from sparse_kv_page_rank_gb300.beams import LocksBeams
from tests.test_gpu_gen_select import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


@pytest.mark.parametrize("keep", [2, 8, 64])
def test_the_first_of_one_request(keep):
    """One request keeps another number than its beams: a view of the object's own outputs is
    contiguous then, and may be given back."""
    W, V, end = 4, 5000, 9
    beams = LocksBeams(width=W, end_token=end)
    logits, scores, _ = make(1, W, V, torch.float32, seed=keep)
    ended = torch.zeros(1, W, dtype=torch.int32, device="cuda")
    out = beams.select(logits, scores, ended, keep=max(keep, W))
    for step in range(3):
        s, e = out[0][:, :W], out[3][:, :W]
        old_s, old_e = s.clone(), e.clone()
        logits = make(1, W, V, torch.float32, seed=step)[0]
        fresh = LocksBeams(width=W, end_token=end).select(logits, old_s, old_e, keep=keep)
        fresh = [x.clone() for x in fresh]
        out = beams.select(logits, s, e, keep=keep)
        assert all(torch.equal(a, b) for a, b in zip(out, fresh))
        check(out, logits, old_s, old_e, end, keep)
        if keep < W:
            out = beams.select(logits, old_s, old_e, keep=W)
    assert beams.device_error() == 0


def test_several_requests_are_refused():
    W, V = 3, 200
    beams = LocksBeams(width=W, end_token=1)
    logits, scores, _ = make(2, W, V, torch.float32, seed=1)
    ended = torch.zeros(2, W, dtype=torch.int32, device="cuda")
    for name, x in (("out_scores", scores), ("out_ended", ended)):
        wide = torch.cat([x, x], dim=1).contiguous()
        with pytest.raises(L.LocksError):
            beams.select(logits, wide.flatten()[:2 * W].view(2, W) if name == "out_scores" else scores,
                         wide.flatten()[:2 * W].view(2, W) if name == "out_ended" else ended, keep=2 * W, **{name: wide})
    torch.cuda.synchronize()
    assert beams.device_error() == 0


def test_back_pointers_are_copied_to_be_kept():
    """As in the module's example: the object's own outputs are the next call's too, copies are not."""
    W, V, steps = 3, 400, 5
    beams = LocksBeams(width=W)
    scores = torch.zeros(2, W, device="cuda")
    trail, own, want = [], [], []
    for step in range(steps):
        logits, _, _ = make(2, W, V, torch.float32, seed=step)
        want.append([x.clone() for x in LocksBeams(width=W).select(logits, scores.clone())[1:3]])
        scores, parents, tokens, _ = beams.select(logits, scores)
        trail.append((parents.clone(), tokens.clone()))
        own.append((parents, tokens))
    assert all(torch.equal(a, b) for t, w in zip(trail, want) for a, b in zip(t, w))
    assert all(a is b for t in own for a, b in zip(t, own[0]))
