"""Calls that the generation entry points allow beside the usual ones: without the optional arguments, over
workspaces full of whatever memory held, at tables that are full, with idle rows' positions left as they
were."""

import math

import pytest
import torch

from sparse_kv_page_rank_gb300 import locks as L
from sparse_kv_page_rank_gb300.beams import LocksBeams
from tests.gen_cases import shared_case
from tests.kv_cases import D, Case
from tests.test_gpu_gen_attend import check as check_attend
from tests.test_gpu_gen_axes import rotated
from tests.test_gpu_gen_reorder import Rows
from tests.test_gpu_gen_select import check as check_select, make
from tests.test_gpu_kv_append import check_cache, rows_of, table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_kv_page_rank_gb300.build_lib import build
    build()


def poison(ws, byte):
    """All of a workspace but its error word."""
    ws[4:] = byte
    torch.cuda.synchronize()


@pytest.mark.parametrize("byte", [0, 0x7f, 0xff])
def test_workspaces_may_hold_anything(byte):
    case, W, shared = shared_case([3000, 70, 1], [[9, 60, None, 9], [None] * 4, [0, 1, 2, 3]], 8, 2, 64, "bf16", seed=4)
    beams = LocksBeams([case.runtime()], width=W)
    q = case.query(case.B)
    poison(beams._attend_ws, byte)
    out, lse = beams.attend(q, shared)
    check_attend(case, q, out, lse)
    logits, scores, _ = make(3, W, 40000, torch.float32, seed=2)
    scores[1, 2] = -math.inf
    logits[0, 1] = -math.inf
    for keep in (4, 40):
        pick = LocksBeams(width=W)
        pick.select(logits, scores, keep=keep)
        poison(pick._select_ws, byte)
        check_select(pick.select(logits, scores, keep=keep), logits, scores, None, -1, keep)
        assert pick.device_error() == 0
    rows = Rows([100] * 8, 4, 1, 64, "bf16", 4, seed=3)
    poison(rows.beams._reorder_ws, byte)
    rows.run([[1, 1, 3, 0], [2, 2, 2, -1]])
    assert beams.device_error() == rows.beams.device_error() == 0


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_attend_without_lse(fmt):
    case, W, shared = shared_case([300], [[10, None, 70]], 4, 2, 16, fmt, seed=5)
    rt = case.runtime()
    beams, q = LocksBeams([rt], width=W), case.query(case.B)
    want = beams.attend(q, shared)[0].clone()
    out = torch.empty_like(q)
    L.locksgen_attend(rt.cache, rt.params, W, shared, q, out, None, beams._attend_ws, beams._attend_ws.numel())
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("P", [16, 64])
def test_rows_that_fill_their_tables(fmt, P):
    """Lengths of all that the table holds: append, attend, and the reorder of rows without an open page."""
    n = 6 * P
    case = Case([n] * 3, 4, 2, P, fmt, seed=P, extra_cols=0)
    case.table[1:, :4] = case.table[0, :4]
    beams = LocksBeams([case.runtime()], width=3)
    q = case.query(3)
    for s in (0, 4, 6):
        out, lse = beams.attend(q, torch.tensor([min(s, 4)], dtype=torch.int32, device="cuda"))
        check_attend(case, q, out, lse)
    before = case.table.clone()
    beams.reorder(torch.tensor([[2, 2, 0]], dtype=torch.int32, device="cuda"))
    assert torch.equal(case.table, before[[2, 2, 0]]) and case.seq.tolist() == [n] * 3 and beams.device_error() == 0


def test_choice_without_the_optional_arrays():
    """An end_token without `ended`, and the C call without `out_ended`."""
    W, V, end = 3, 700, 5
    logits, scores, _ = make(2, W, V, torch.bfloat16, seed=8)
    logits[1, 2, end] = 30
    beams = LocksBeams(width=W, end_token=end)
    got = [x.clone() for x in beams.select(logits, scores)]
    check_select(got, logits, scores, None, end, W)
    assert int(got[3].sum()) >= 1
    outs = [torch.empty_like(x) for x in got[:3]]
    choice = L.locksgen_choice_t(logits.data_ptr(), scores.data_ptr(), None, *(x.data_ptr() for x in outs), None, V, 2, W, V, W,
                                 L.LOCKS_DTYPE_BF16, end)
    need = L.locksgen_select_workspace_size(choice)
    ws = torch.zeros(need + 256, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:]
    L.locksgen_select(choice, ws, need)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, got))
    # and out_ended without an end_token
    ended = torch.full((2, W), 7, dtype=torch.int32, device="cuda")
    assert LocksBeams(width=W).select(logits, scores, out_ended=ended)[3] is ended and (ended == 0).all()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_a_step_with_idle_rows_and_spare_axes(fmt, interleaved):
    """One token per row, idle rows' positions unset, more axes of positions than pairs have, no queries."""
    lens = [33, 0, 64, 0, 1]
    case = Case(lens, 4, 2, 16, fmt, seed=6)
    rt = case.runtime()
    live = [b for b, n in enumerate(lens) if n]
    k, v = (torch.randn(5, 2, D, generator=case.gen).bfloat16().cuda() for _ in range(2))
    rope, axes = table(80, 128), [0, 2] * 32
    pos = torch.full((4, 5), -9, dtype=torch.int32)
    pos[:3, live] = torch.randint(0, 80, (3, len(live)), generator=case.gen).int()
    pos[1::2] = pos[1::2].clamp(min=0)
    pos[3] = 3
    pos[1] = 79
    pos = pos.cuda()
    before = (case.k.clone(), None if case.v is None else case.v.clone())
    assert rt.append(k, v, rope=rope, interleaved=interleaved, positions=pos, axes=L.make_axes(axes)) is None
    assert rt.device_error() == 0
    seq = torch.tensor(live, device="cuda")
    at = torch.tensor([lens[b] - 1 for b in live], device="cuda")
    kr = rotated(k[live], rope, pos[:, live], axes, interleaved).bfloat16()
    check_cache(case, before, kr, v[live], seq, at)


def test_no_tokens_at_all():
    case = Case([33, 5], 4, 2, 16, "bf16", seed=6)
    rt = case.runtime()
    none = torch.empty(0, 2, D, dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    before = case.k.clone()
    rt.append(none, none, rope=table(80, 128), positions=torch.empty(2, 0, dtype=torch.int32, device="cuda"),
              axes=L.make_axes([0, 1] * 32), cu_tokens=cu)
    torch.cuda.synchronize()
    assert torch.equal(case.k.view(torch.int16), before.view(torch.int16)) and rt.device_error() == 0
    assert rows_of([33, 5], [0, 0])[2].tolist() == [0, 0, 0]
