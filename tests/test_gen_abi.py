"""The host-side checks of locksgen.h, without a GPU."""

import re
import subprocess
from pathlib import Path

import pytest

from sparse_kv_page_rank_gb300 import locks as L
from sparse_kv_page_rank_gb300.build_lib import LIB, build
from tests.test_kv_layout import _append, _cache, _status

ROOT = Path(__file__).resolve().parents[1]


@pytest.fixture(scope="module")
def lib():
    build()
    return L.lib()


def test_declared_calls_are_exported(lib):
    text = (ROOT / "include" / "locksgen.h").read_text()
    names = set(re.findall(r"LOCKS_API\s+[\w\s\*]+?\b(locksgen_\w+)\s*\(", text))
    assert len(names) == 7
    out = subprocess.run(["nm", "-D", "--defined-only", LIB], capture_output=True, text=True).stdout
    assert {line.split()[-1] for line in out.splitlines() if "locksgen_" in line} == names
    assert all(hasattr(lib, n) for n in names)


def test_header_compiles_as_c_and_agrees_with_the_binding(tmp_path, lib):
    import ctypes
    import shutil
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "h.c", tmp_path / "h"
    src.write_text('#include "locksgen.h"\n#include <stdio.h>\n#include <stddef.h>\nint main(void) { printf("%d %d %d %d %d %d %d %d", '
                   "(int)sizeof(locksgen_axes_t), (int)offsetof(locksgen_axes_t, axis_of_pair), (int)sizeof(locksgen_choice_t), "
                   "(int)offsetof(locksgen_choice_t, end_token), LOCKSGEN_MAX_BEAMS, LOCKSGEN_MAX_KEEP, LOCKSGEN_DEVERR_LOGITS, "
                   "LOCKSGEN_DEVERR_PARENT); return 0; }\n")
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", f"-I{ROOT / 'include'}", str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(L.locksgen_axes_t), L.locksgen_axes_t.axis_of_pair.offset, ctypes.sizeof(L.locksgen_choice_t),
                   L.locksgen_choice_t.end_token.offset, L.LOCKSGEN_MAX_BEAMS, L.LOCKSGEN_MAX_KEEP, L.LOCKSGEN_DEVERR_LOGITS,
                   L.LOCKSGEN_DEVERR_PARENT]


def _axes(pairs=64, **kw):
    axes = L.make_axes([0, 1] * (pairs // 2))
    axes.positions, axes.axis_stride = 0xB000, 2
    for k, v in kw.items():
        setattr(axes, k, v)
    return axes


@pytest.mark.parametrize("append,axes,status", [
    (dict(rope=None, rotary_dim=0), {}, L.LOCKS_ERR_INVALID_ARG),
    (dict(positions=0xC000), {}, L.LOCKS_ERR_INVALID_ARG),
    ({}, dict(positions=None), L.LOCKS_ERR_INVALID_ARG),
    ({}, dict(num_axes=0), L.LOCKS_ERR_INVALID_ARG),
    ({}, dict(num_axes=1), L.LOCKS_ERR_INVALID_ARG),  # a pair of an axis that is not there
    ({}, dict(num_axes=5), L.LOCKS_ERR_UNSUPPORTED),
    ({}, dict(axis_stride=1), L.LOCKS_ERR_INVALID_ARG),
    (dict(rotary_dim=24), {}, L.LOCKS_ERR_UNSUPPORTED),
    (dict(k=0x6001), {}, L.LOCKS_ERR_INVALID_ARG),
    (dict(q_out=None), {}, L.LOCKS_ERR_INVALID_ARG),
])
def test_axes(lib, append, axes, status):
    tokens = L.make_tokens(None, 2, 1)
    assert _status(lambda: L.locksgen_append_axes(_cache(), tokens, _append(**append), _axes(**axes), stream=0)) == status


def test_axes_without_tokens(lib):
    L.locksgen_append_axes(_cache(), L.make_tokens(0x100, 0, 0), _append(), _axes(), stream=0)
    L.locksgen_append_axes(_cache(), L.make_tokens(0x100, 2, 0), _append(), _axes(), stream=0)


def _choice(**kw):
    d = dict(logits=0x1000, scores=0x2000, ended=None, out_scores=0x3000, out_parents=0x4000, out_tokens=0x5000, out_ended=None,
             row_stride=100, batch=2, beams=4, vocab=100, keep=4, dtype=L.LOCKS_DTYPE_F32, end_token=-1)
    d.update(kw)
    return L.locksgen_choice_t(**d)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), 1), (dict(scores=None), 1), (dict(out_scores=None), 1), (dict(out_parents=None), 1),
    (dict(out_tokens=None), 1), (dict(batch=0), 1), (dict(beams=0), 1), (dict(beams=33), 2), (dict(vocab=0), 1),
    (dict(vocab=(1 << 22) + 1, row_stride=1 << 23), 2), (dict(keep=0), 1), (dict(keep=65), 2), (dict(dtype=L.LOCKS_DTYPE_Q4), 1),
    (dict(row_stride=99), 1), (dict(logits=0x1002), 1), (dict(logits=0x1001, dtype=L.LOCKS_DTYPE_BF16), 1),
    (dict(end_token=-2), 1), (dict(end_token=100), 1), (dict(ended=0x6000), 1), (dict(batch=20000), 2),
    (dict(keep=3, out_scores=0x2000), 1), (dict(keep=3, ended=0x6000, out_ended=0x6000, end_token=1), 1),
])
def test_choice(lib, kw, status):
    assert _status(lambda: L.locksgen_select(_choice(**kw), 0x100, 1 << 30, stream=0)) == status


def test_choice_workspace(lib):
    need = L.locksgen_select_workspace_size(_choice())
    assert need % 256 == 0 and need > 256
    for ws, n in ((None, 1 << 30), (0x100, need - 1), (0x180, 1 << 30)):
        assert _status(lambda: L.locksgen_select(_choice(), ws, n, stream=0)) == L.LOCKS_ERR_WORKSPACE
    assert L.locksgen_select_workspace_size(_choice(vocab=100000, row_stride=100000, keep=8)) > 8 * need
    assert _status(lambda: L.locksgen_select_workspace_size(_choice(keep=65))) == L.LOCKS_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,beams,status", [
    (dict(), 0, 1), (dict(), 3, 1), (dict(batch=66), 33, 2), (dict(block_table=None), 2, 1), (dict(k_pool=None), 2, 1),
    (dict(v_pool=0x2008), 2, 1), (dict(head_dim=64), 2, 2), (dict(page_size=32), 2, 2),
])
def test_caches(lib, kw, beams, status):
    one = (L.locks_cache_t * 1)(_cache(**kw))
    assert _status(lambda: L.locksgen_reorder(one, 1, beams, 0x9000, 0x100, 1 << 30, stream=0)) == status
    params = L.make_params(4, 0)
    assert _status(lambda: L.locksgen_attend(one[0], params, beams, 0x9000, 0xA000, 0xB000, None, 0x100, 1 << 40, stream=0)) == status


@pytest.mark.parametrize("kw", [dict(block_table=0x3100), dict(seq_lens=0x4100), dict(n_summarized=None), dict(batch=4),
                                dict(num_kv_heads=1), dict(page_size=16), dict(pages_total=11), dict(max_pages=9), dict(kv_format=1)])
def test_layers_differ_in_their_pools_only(lib, kw):
    two = (L.locks_cache_t * 2)(_cache(), _cache(**kw))
    assert _status(lambda: L.locksgen_reorder(two, 2, 2, 0x9000, 0x100, 1 << 30, stream=0)) == L.LOCKS_ERR_INVALID_ARG


def test_reorder_and_attend_arguments(lib):
    one, params = (L.locks_cache_t * 1)(_cache()), L.make_params(4, 0)
    need = L.locksgen_reorder_workspace_size(one[0], 2)
    for n, parents, ws, size, status in ((0, 0x9000, 0x100, need, 1), (1, None, 0x100, need, 1), (1, 0x9000, None, need, 4),
                                         (1, 0x9000, 0x100, need - 1, 4), (1, 0x9000, 0x80, need, 4)):
        assert _status(lambda: L.locksgen_reorder(one, n, 2, parents, ws, size, stream=0)) == status
    need = L.locksgen_attend_workspace_size(one[0], params, 2)
    assert need % 256 == 0
    good = dict(shared_pages=0x9000, q=0xA000, out=0xB000, lse=None, ws=0x100, ws_bytes=need)
    for kw, status in ((dict(shared_pages=None), 1), (dict(q=None), 1), (dict(q=0xA008), 1), (dict(out=None), 1),
                       (dict(ws=None), 4), (dict(ws=0x40), 4), (dict(ws_bytes=need - 1), 4)):
        args = {**good, **kw}
        assert _status(lambda: L.locksgen_attend(one[0], params, 2, *args.values(), stream=0)) == status
    assert _status(lambda: L.locksgen_attend(one[0], L.make_params(34, 0), 2, *good.values(), stream=0)) == 2


def test_axes_of_pairs():
    assert L.rope_axes([2, 1, 3]) == [0, 0, 1, 2, 2, 2]
    assert L.rope_axes([4, 2, 2], cyclic=True) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert L.rope_axes([5]) == L.rope_axes([5], cyclic=True) == [0] * 5
    axes = L.make_axes([2, 0, 1])
    assert axes.num_axes == 3 and axes.pairs == 3 and list(axes.axis_of_pair[:4]) == [2, 0, 1, 0]
