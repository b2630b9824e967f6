"""Read-only loads in kernels that begin before the kernel ahead of them has ended.

Such a kernel (griddepcontrol.wait) lives while lengths, block tables, queries and pages are still being
written: locksgen_reorder and lockskv_append let their successors begin early. A read-only load requires that
its data does not change while the kernel lives, so these files hold none."""

import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "sparse_kv_page_rank_gb300" / "csrc"


def _code(path):
    text = re.sub(r"/\*.*?\*/", " ", path.read_text(), flags=re.S)
    return re.sub(r"//[^\n]*", " ", text)


EARLY = sorted(p.name for p in CSRC.glob("*.cu") if re.search(r"\bpdl_wait\s*\(", _code(p)))


def test_the_files_are_found():
    assert {"kv_append.cu", "prompt.cu", "attend.cu", "attend_q4.cu", "scan.cu", "topk.cu"} <= set(EARLY)


@pytest.mark.parametrize("name", EARLY + ["common.cuh", "kv_q4.cuh"])
def test_no_read_only_loads(name):
    lines = [line.strip() for line in _code(CSRC / name).splitlines()
             if re.search(r"__ldg\b|ld\.global(\.\w+)*\.nc|__restrict__", line)]
    assert not lines, lines
