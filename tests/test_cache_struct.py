"""locks_cache_t keeps the size and layout that it had before it named a page format, so
that a caller built against the earlier header is served as before."""

import ctypes
import shutil
import subprocess
from pathlib import Path

import pytest

from sparse_kv_page_rank_gb300 import locks as L
from sparse_kv_page_rank_gb300.build_lib import build

ROOT = Path(__file__).resolve().parents[1]


class EarlierCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_pool", "v_pool", "block_table", "seq_lens", "n_summarized")] + [
        (n, ctypes.c_int32) for n in ("batch", "num_kv_heads", "head_dim", "page_size", "pages_total", "max_pages")]


def test_sizes_agree():
    assert ctypes.sizeof(L.locks_cache_t) == ctypes.sizeof(EarlierCache) == 64
    c = L.locks_cache_t(max_pages=2 ** 27 - 1, kv_format=L.LOCKS_KV_Q4)
    assert (c.max_pages, c.kv_format) == (2 ** 27 - 1, L.LOCKS_KV_Q4)
    # no table that the limits allow is wider: 16-token pages, 2^31 tokens
    assert (2 ** 31 - 1) // 16 <= 2 ** 27 - 1


def test_the_binding_and_the_header_agree(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "c.c", tmp_path / "c"
    src.write_text("""
#include <stdio.h>
#include <string.h>
#include "locks.h"
int main(void) {
  locks_cache_t c = {(void*)1, (void*)2, (void*)3, (void*)4, (void*)5, 6, 7, 8, 9, 10, 11};  /* as before formats */
  unsigned char b[sizeof c];
  if (sizeof c != 64 || c.kv_format != 0 || c.max_pages != 11) return 1;
  c.kv_format = LOCKS_KV_Q4;
  c.max_pages = (1 << 27) - 1;
  memcpy(b, &c, sizeof c);
  for (unsigned i = 0; i < sizeof c; ++i) printf("%02x", b[i]);
  return 0;
}
""")
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", f"-I{ROOT / 'include'}", str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    c = L.locks_cache_t(1, 2, 3, 4, 5, 6, 7, 8, 9, 10, (1 << 27) - 1, L.LOCKS_KV_Q4)
    assert bytes(c).hex() == got


@pytest.mark.parametrize("behind", [0x00, 0x01, 0x55, 0xff])
def test_an_earlier_callers_struct_is_read_to_its_end_only(behind):
    build()
    raw = (ctypes.c_ubyte * 128)(*([behind] * 128))
    old = EarlierCache.from_buffer(raw)
    for n, x in dict(k_pool=0x1000, v_pool=0x2000, block_table=0x3000, seq_lens=0x4000, n_summarized=0x5000, batch=2,
                     num_kv_heads=2, head_dim=128, page_size=64, pages_total=10, max_pages=10).items():
        setattr(old, n, x)
    p = L.make_params(8, 512)
    new = L.locks_cache_t(0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 2, 2, 128, 64, 10, 10, 0)
    n = ctypes.c_size_t(0)
    status = L.lib().locks_workspace_size(ctypes.cast(ctypes.byref(old), ctypes.POINTER(L.locks_cache_t)), None,
                                          ctypes.byref(p), ctypes.byref(n))
    assert status == L.LOCKS_OK and n.value == L.locks_workspace_size(new, None, p)


def test_a_table_wider_than_the_field_is_refused():
    import torch
    build()
    k, lens = torch.zeros(2, 1, 64, 128, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    one = torch.zeros(1, 1, dtype=torch.int32)
    for cols in (1 << 27, (1 << 28) + 5, 1 << 31):
        with pytest.raises(L.LocksError) as e:
            L.make_cache(k, k, one.expand(1, cols), lens)
        assert e.value.status == L.LOCKS_ERR_UNSUPPORTED
    c = L.make_cache(k, k, one.expand(1, (1 << 27) - 1), lens)
    assert c.max_pages == (1 << 27) - 1
    # what the field holds but the limits on tokens do not allow
    with pytest.raises(L.LocksError) as e:
        L.locks_workspace_size(c, None, L.make_params(4, 0))
    assert e.value.status == L.LOCKS_ERR_UNSUPPORTED
