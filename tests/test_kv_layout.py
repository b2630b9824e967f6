"""The 4-bit page layout and the host-side checks of lockskv.h, without a GPU."""

import re
from pathlib import Path

import pytest
import torch

from sparse_kv_page_rank_gb300 import locks as L
from sparse_kv_page_rank_gb300.build_lib import LIB, build
from tests.kv_cases import pack, q4_places, unpack

ROOT = Path(__file__).resolve().parents[1]


@pytest.fixture(scope="module")
def lib():
    build()
    return L.lib()


@pytest.mark.parametrize("P", [16, 64])
def test_every_nibble_and_scale_has_one_place(P):
    kb, kn, ks, vb, vn, vs = q4_places(P)
    nibbles = torch.cat([(b * 2 + n // 4).reshape(-1) for b, n in ((kb, kn), (vb, vn))])
    scales = torch.cat([s[:, ::32].reshape(-1) for s in (ks, vs)])
    taken = torch.cat([nibbles, (scales[:, None] * 2 + torch.arange(4)).reshape(-1)])
    assert taken.unique().numel() == taken.numel() == 2 * L.kv_q4_block_bytes(P)
    assert (scales % 2 == 0).all()
    # a dimension's scale is that of its 32
    assert (ks.view(P, 4, 32) == ks.view(P, 4, 32)[..., :1]).all()
    # the block size of the header
    text = (ROOT / "include" / "locks.h").read_text()
    expr = re.search(r"#define LOCKS_KV_Q4_BLOCK_BYTES\(P\) (.+)", text).group(1).replace("(P)", str(P))
    assert eval(expr) == L.kv_q4_block_bytes(P)


@pytest.mark.parametrize("P", [16, 64])
def test_pack_and_unpack(P):
    g = torch.Generator().manual_seed(P)
    kq, vq = (torch.randint(-7, 8, (3, 2, P, 128), generator=g) for _ in range(2))
    ks, vs = (torch.rand(3, 2, P, 4, generator=g).half() for _ in range(2))
    got = unpack(pack(kq, ks, vq, vs))
    for a, b in zip(got, (kq, ks, vq, vs)):
        assert torch.equal(a, b.to(a.dtype))


def test_declared_calls_are_exported(lib):
    import subprocess
    text = (ROOT / "include" / "lockskv.h").read_text()
    names = set(re.findall(r"LOCKS_API\s+[\w\s\*]+?\b(lockskv_\w+)\s*\(", text))
    assert len(names) == 4
    out = subprocess.run(["nm", "-D", "--defined-only", LIB], capture_output=True, text=True).stdout
    assert {line.split()[-1] for line in out.splitlines() if "lockskv_" in line} == names
    for n in names:
        assert hasattr(lib, n)


def test_headers_compile_as_c(tmp_path):
    import shutil
    import subprocess
    src = tmp_path / "h.c"
    src.write_text('#include "lockskv.h"\nint main(void) { locks_cache_t c = {0}; return (int)(c.kv_format + '
                   'sizeof(lockskv_append_t) - sizeof(lockskv_append_t)); }\n')
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", f"-I{ROOT / 'include'}", "-c", str(src), "-o",
                    str(tmp_path / "h.o")], check=True)


def _cache(**kw):
    d = dict(k_pool=0x1000, v_pool=0x2000, block_table=0x3000, seq_lens=0x4000, n_summarized=0x5000, batch=2,
             num_kv_heads=2, head_dim=128, page_size=64, pages_total=10, max_pages=10, kv_format=0)
    d.update(kw)
    return L.locks_cache_t(**d)


def _append(**kw):
    d = dict(k=0x6000, v=0x7000, q=0x8000, q_out=0x9000, rope=0xA000, positions=None, k_stride=256, v_stride=256,
             q_stride=1024, q_out_stride=1024, num_q_heads=8, rope_rows=100, rotary_dim=128, interleaved=0)
    d.update(kw)
    return L.lockskv_append_t(**d)


def _status(call):
    with pytest.raises(L.LocksError) as e:
        call()
    return e.value.status


INVALID, UNSUPPORTED, WORKSPACE = L.LOCKS_ERR_INVALID_ARG, L.LOCKS_ERR_UNSUPPORTED, L.LOCKS_ERR_WORKSPACE


@pytest.mark.parametrize("cache,status", [
    (dict(kv_format=2), INVALID), (dict(kv_format=-1), INVALID), (dict(k_pool=None), INVALID),
    (dict(v_pool=None), INVALID), (dict(k_pool=0x1008), INVALID), (dict(head_dim=64), UNSUPPORTED),
    (dict(page_size=32), UNSUPPORTED), (dict(block_table=None), INVALID), (dict(seq_lens=None), INVALID),
    (dict(kv_format=1, v_pool=None, k_pool=0x1004), INVALID),
])
def test_caches_refused(lib, cache, status):
    c, t, p = _cache(**cache), L.make_tokens(0xB000, 5, 5), L.make_params(8, 0)
    assert _status(lambda: L.lockskv_append(c, t, _append(), None, 0, 0)) == status
    assert _status(lambda: L.lockskv_read(c, t, 0x8000, 0x9000, None, 0, 0)) == status
    assert _status(lambda: L.lockskv_prompt_attend(c, p, t, 0x8000, 1024, 0x9000, None, 0x100000, 1 << 30, 0)) == status


@pytest.mark.parametrize("tokens", [(0xB000, -1, 5), (0xB000, 5, -1), (None, 3, 1), (None, 2, 2)])
def test_token_rows_refused(lib, tokens):
    t, p = L.make_tokens(*tokens), L.make_params(8, 0)
    assert _status(lambda: L.lockskv_append(_cache(), t, _append(), None, 0, 0)) == INVALID
    assert _status(lambda: L.lockskv_read(_cache(), t, 0x8000, 0x9000, None, 0, 0)) == INVALID
    assert _status(lambda: L.lockskv_prompt_attend(_cache(), p, t, 0x8000, 1024, 0x9000, None, 0x100000, 1 << 30, 0)) == INVALID
    assert _status(lambda: L.lockskv_prompt_workspace_size(_cache(), p, t)) == INVALID


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q_out=None), INVALID), (dict(q=None), INVALID),
    (dict(k=0x6002), INVALID), (dict(q_out=0x9008), INVALID), (dict(k_stride=255), INVALID),
    (dict(k_stride=260), INVALID), (dict(v_stride=128), INVALID), (dict(q_stride=1000), INVALID),
    (dict(q_out=0x8000, q_out_stride=2048), INVALID), (dict(num_q_heads=0), INVALID),
    (dict(rotary_dim=24), UNSUPPORTED), (dict(rotary_dim=144), UNSUPPORTED), (dict(rotary_dim=-16), INVALID),
    (dict(rope=None), INVALID), (dict(rotary_dim=0), INVALID), (dict(rope_rows=0), INVALID),
    (dict(rope=0xA004), INVALID), (dict(interleaved=2), INVALID),
])
@pytest.mark.parametrize("fmt", [0, 1])
def test_appends_refused(lib, kw, status, fmt):
    t = L.make_tokens(0xB000, 5, 5)
    assert _status(lambda: L.lockskv_append(_cache(kv_format=fmt), t, _append(**kw), None, 0, 0)) == status


def test_workspaces_and_reads_refused(lib):
    t, p, c = L.make_tokens(0xB000, 5, 5), L.make_params(8, 0), _cache()
    assert _status(lambda: L.lockskv_append(c, t, _append(), 0x100010, 256, 0)) == WORKSPACE
    assert _status(lambda: L.lockskv_append(c, t, _append(), 0x100000, 2, 0)) == WORKSPACE
    assert _status(lambda: L.lockskv_read(c, t, None, None, None, 0, 0)) == INVALID
    assert _status(lambda: L.lockskv_read(c, t, 0x8008, None, None, 0, 0)) == INVALID
    need = L.lockskv_prompt_workspace_size(c, p, t)
    assert need >= 256 and need % 256 == 0
    for ws, n in ((None, need), (0x100010, need), (0x100000, need - 1)):
        assert _status(lambda: L.lockskv_prompt_attend(c, p, t, 0x8000, 1024, 0x9000, None, ws, n, 0)) == WORKSPACE
    assert _status(lambda: L.lockskv_prompt_attend(c, p, t, None, 1024, 0x9000, None, 0x100000, need, 0)) == INVALID
    assert _status(lambda: L.lockskv_prompt_attend(c, p, t, 0x8000, 1000, 0x9000, None, 0x100000, need, 0)) == INVALID
    assert _status(lambda: L.lockskv_prompt_attend(c, p, t, 0x8000, 1024, 0x9008, None, 0x100000, need, 0)) == INVALID
    assert _status(lambda: L.lockskv_prompt_attend(c, L.make_params(34, 0), t, 0x8000, 8192, 0x9000, None, 0x100000,
                                                   1 << 30, 0)) == UNSUPPORTED


def test_nothing_to_do_is_no_error(lib):
    p, c = L.make_params(8, 0), _cache()
    for t in (L.make_tokens(0xB000, 0, 5), L.make_tokens(0xB000, 5, 0)):
        L.lockskv_append(c, t, _append(), None, 0, 0)
        L.lockskv_read(c, t, 0x8000, 0x9000, None, 0, 0)
        need = L.lockskv_prompt_workspace_size(c, p, t)
        L.lockskv_prompt_attend(c, p, t, 0x8000, 1024, 0x9000, None, 0x100000, need, 0)


def test_four_bit_caches_have_workspaces_and_keep_the_three_kernel_step(lib):
    p = L.make_params(8, 512, flags=L.LOCKS_FLAG_FUSED)
    c = _cache(kv_format=1, v_pool=None)
    assert L.locks_workspace_size(c, None, p) % 256 == 0
    assert L.locks_decode_step_launches(c, L.make_summary(16, 16, 8), p) == 3


def test_make_cache_reads_the_format_off_the_tensor():
    t, s = torch.zeros(2, 5, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for P in (16, 64):
        c = L.make_cache(torch.zeros(7, 3, 144 * P, dtype=torch.uint8), None, t, s)
        assert (c.kv_format, c.page_size, c.num_kv_heads, c.pages_total, c.v_pool) == (L.LOCKS_KV_Q4, P, 3, 7, None)
    c = L.make_cache(torch.zeros(7, 3, 16, 128, dtype=torch.bfloat16), torch.zeros(7, 3, 16, 128).bfloat16(), t, s)
    assert c.kv_format == L.LOCKS_KV_BF16
    with pytest.raises(ValueError):
        L.make_cache(torch.zeros(7, 3, 1000, dtype=torch.uint8), None, t, s)


def test_rows_that_are_no_token_rows_are_refused():
    x = torch.zeros(4, 6, 128, dtype=torch.bfloat16)
    assert L._row_stride(x[:, 1:3], "k") == 768
    assert L._row_stride(x[:1, 1:3], "k") % 8 == 0
    for bad in (x.float(), x[..., :64], x.transpose(0, 1)[:, :3], x[:, ::2], x[0]):
        with pytest.raises(ValueError):
            L._row_stride(bad, "k")
