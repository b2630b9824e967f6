"""The limits of locksgen.h: declared, the same in the binding, and held at their ends. Without a GPU."""

import re
from pathlib import Path

import pytest

from sparse_kv_page_rank_gb300 import locks as L
from tests.test_gen_abi import _choice, lib  # noqa: F401
from tests.test_kv_layout import _cache, _status

HEADER = (Path(__file__).resolve().parents[1] / "include" / "locksgen.h").read_text()


def test_every_limit_is_declared_and_bound():
    found = {n: eval(v) for n, v in re.findall(r"#define (LOCKSGEN_MAX_\w+) (.+)", HEADER)}
    assert {"LOCKSGEN_MAX_BEAMS", "LOCKSGEN_MAX_KEEP", "LOCKSGEN_MAX_AXES", "LOCKSGEN_MAX_ROWS", "LOCKSGEN_MAX_VOCAB"} == set(found)
    assert all(getattr(L, n) == v for n, v in found.items())


def _sizes(batch, beams, vocab, keep):
    return L.locksgen_select_workspace_size(_choice(batch=batch, beams=beams, vocab=vocab, row_stride=vocab, keep=keep))


@pytest.mark.parametrize("batch,beams,vocab,keep", [
    (L.LOCKSGEN_MAX_ROWS, 1, 100, 4), (L.LOCKSGEN_MAX_ROWS // 5, 5, 100, 4), (1, 1, L.LOCKSGEN_MAX_VOCAB, 1),
    (1, L.LOCKSGEN_MAX_BEAMS, 100, L.LOCKSGEN_MAX_KEEP),
])
def test_the_largest(lib, batch, beams, vocab, keep):  # noqa: F811
    assert _sizes(batch, beams, vocab, keep) > 0
    for more in ((batch + 1 if batch * beams > 60000 else batch, beams, vocab, keep),
                 (batch, beams, vocab + 1 if vocab > 100 else vocab, keep),
                 (batch, beams + 1 if beams > 5 else beams, vocab, keep), (batch, beams, vocab, keep + 1 if keep > 4 else keep)):
        if more != (batch, beams, vocab, keep):
            assert _status(lambda: _sizes(*more)) == L.LOCKS_ERR_UNSUPPORTED


def test_a_workspace_is_for_its_sizes(lib):  # noqa: F811
    """Fewer rows may need more: one that is too small is refused, whatever it was made for."""
    sizes = [_sizes(b, 1, 50000, 64) for b in range(1, 400)]
    later = [b for b in range(1, len(sizes)) if sizes[b] < sizes[b - 1]]
    assert later
    b = later[0]
    choice = _choice(batch=b, beams=1, vocab=50000, row_stride=50000, keep=64)
    assert _status(lambda: L.locksgen_select(choice, 0x100, sizes[b], stream=0)) == L.LOCKS_ERR_WORKSPACE


def test_the_line_of_shared_pages_fits_32_bits(lib):  # noqa: F811
    """Every row's part is a segment of its tiles and a few places more, and there is one more per request."""
    csrc = Path(L.__file__).parent / "csrc"
    found = [int(n) for f in csrc.iterdir() for n in re.findall(r"constexpr int kSegment = (\d+);", f.read_text())]
    assert len(found) == 1  # one place says how many
    params = L.make_params(1, 0)
    for rows in (1 << 10, 1 << 15):
        tiles = (1 << 31) // (2 * rows) - found[0]  # 2 rows segments of so many: 2^31 places
        def size(n, rows=rows):
            return L.locksgen_attend_workspace_size(_cache(batch=rows, num_kv_heads=1, max_pages=n, page_size=64, pages_total=10), params, 1)
        assert size(tiles - 1) > 0
        assert _status(lambda: size(tiles)) == L.LOCKS_ERR_UNSUPPORTED
