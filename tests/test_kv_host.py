"""Host-only checks of the paged-cache entry points: bad arguments are refused with the
documented status before anything is launched, and the binding checks types and shapes."""
import ctypes
import math

import pytest
import torch

import fp8_block_scaled_12_b200 as F
from fp8_block_scaled_12_b200.kv import _CacheStruct

OK, INVALID, SHAPE, ALIGN, UNSUP = range(5)
FAKE = 0x7F0000000000       # 16-byte aligned, never dereferenced
S = None


def cache(**kw):
    d = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, num_pages=10, page_size=16, heads=2, head_dim=128,
             page_stride=2 * 16 * 128, head_stride=16 * 128, token_stride=128, fmt=0, scale_fmt=0)
    d.update(kw)
    return _CacheStruct(**d)


BAD_CACHES = [
    (dict(k=None), INVALID), (dict(v_scale=None), INVALID), (dict(num_pages=0), INVALID), (dict(heads=0), INVALID),
    (dict(head_dim=0), INVALID), (dict(page_size=0), INVALID), (dict(fmt=2), INVALID), (dict(scale_fmt=-1), INVALID),
    (dict(head_dim=120), SHAPE), (dict(head_dim=272, token_stride=272, head_stride=272 * 16), SHAPE),
    (dict(page_size=12), SHAPE), (dict(page_size=4), SHAPE), (dict(num_pages=2 ** 31 - 1), SHAPE),
    (dict(token_stride=112), INVALID), (dict(token_stride=136), ALIGN), (dict(page_stride=2 ** 41), SHAPE),
    (dict(k=FAKE + 8), ALIGN), (dict(k_scale=FAKE + 4), ALIGN), (dict(head_stride=-2048), INVALID),
]


@pytest.mark.parametrize("change,status", BAD_CACHES, ids=[str(c) for c, _ in BAD_CACHES])
def test_bad_caches_are_refused_by_every_call(change, status):
    c = ctypes.byref(cache(**change))
    w = F.lib.fp8_kv_write(FAKE, 256, 128, FAKE, 256, 128, 4, FAKE, c, S)
    r = F.lib.fp8_kv_read(c, FAKE, 4, 4, FAKE, 1, 4, FAKE, FAKE, S)
    a = F.lib.fp8_paged_attention(FAKE, 1024, 128, 1, 8, c, FAKE, 4, 4, FAKE, 0.1, 0, FAKE, None, FAKE, 1 << 30, S)
    assert (w, r, a) == (status,) * 3
    assert F.lib.fp8_paged_attention_ws_bytes(1, 8, c) == 0


def test_null_cache():
    assert F.lib.fp8_kv_write(FAKE, 256, 128, FAKE, 256, 128, 4, FAKE, None, S) == INVALID
    assert F.lib.fp8_paged_attention_ws_bytes(1, 8, None) == 0


def norm_rope(q=(FAKE, 1024, 128), k=(FAKE, 256, 128), T=4, Hq=8, Hk=2, D=128, wq=FAKE, wk=FAKE, eps=1e-6, cs=FAKE,
              max_pos=100, R=128, inter=0, pos=FAKE, qo=(FAKE, 1024, 128), ko=(FAKE, 256, 128)):
    return F.lib.fp8_qk_norm_rope(*q, *k, T, Hq, Hk, D, wq, wk, eps, cs, max_pos, R, inter, pos, *qo, *ko, S)


def test_norm_rope_validation():
    assert norm_rope(T=-1) == INVALID
    assert norm_rope(D=120, R=96) == SHAPE
    assert norm_rope(D=512) == SHAPE
    assert norm_rope(R=40) == SHAPE
    assert norm_rope(R=144) == INVALID                     # more than the head has
    assert norm_rope(R=-16) == INVALID
    assert norm_rope(eps=-1.0) == INVALID
    assert norm_rope(eps=math.nan) == INVALID
    assert norm_rope(inter=2) == INVALID
    assert norm_rope(cs=None) == INVALID
    assert norm_rope(pos=None) == INVALID
    assert norm_rope(max_pos=0) == INVALID
    assert norm_rope(pos=FAKE + 4) == ALIGN
    assert norm_rope(q=(None, 1024, 128)) == INVALID
    assert norm_rope(qo=(None, 1024, 128)) == INVALID
    assert norm_rope(k=(FAKE + 8, 256, 128)) == ALIGN
    assert norm_rope(q=(FAKE, 1028, 128)) == ALIGN
    assert norm_rope(q=(FAKE, 1024, 64)) == INVALID        # heads that overlap
    assert norm_rope(qo=(FAKE, 0, 128)) == INVALID         # outputs whose tokens overlap
    assert norm_rope(qo=(FAKE, 512, 128)) == INVALID
    assert norm_rope(ko=(FAKE, 128, 128)) == INVALID
    assert norm_rope(ko=(FAKE, 128, 384)) == INVALID       # heads first: 4 tokens of 128 channels
    assert norm_rope(Hk=1, ko=(FAKE, 64, 128)) == INVALID
    assert norm_rope(wq=FAKE + 2) == ALIGN
    assert norm_rope(T=0, q=(None, 0, 0), k=(None, 0, 0), qo=(None, 0, 0), ko=(None, 0, 0), cs=None, pos=None) == OK
    assert norm_rope(Hq=0, Hk=0) == OK


def fused(q=(FAKE, 1024, 128), k=(FAKE, 256, 128), v=(FAKE, 256, 128), T=4, Hq=8, wq=None, wk=None, eps=1e-6, cs=FAKE,
          max_pos=100, R=64, inter=1, pos=FAKE, slots=FAKE, c=None, qo=(FAKE, 1024, 128)):
    c = cache() if c is None else c
    return F.lib.fp8_qk_norm_rope_kv_write(*q, *k, *v, T, Hq, wq, wk, eps, cs, max_pos, R, inter, pos, slots,
                                           ctypes.byref(c), *qo, S)


def test_fused_validation():
    assert fused(T=-1) == INVALID
    assert fused(Hq=-1) == INVALID
    assert fused(slots=None) == INVALID
    assert fused(slots=FAKE + 4) == ALIGN
    assert fused(v=(None, 256, 128)) == INVALID
    assert fused(v=(FAKE, 256, 100)) == INVALID
    assert fused(q=(None, 1024, 128)) == INVALID
    assert fused(R=136) == INVALID
    assert fused(R=24) == SHAPE
    assert fused(wk=FAKE + 8) == ALIGN
    assert fused(qo=(FAKE, 896, 128)) == INVALID
    assert fused(T=2 ** 31) == SHAPE
    assert fused(T=0) == OK
    assert F.lib.fp8_kv_write(FAKE, 256, 128, FAKE, 256, 128, -4, FAKE, ctypes.byref(cache()), S) == INVALID
    assert F.lib.fp8_kv_write(FAKE, 252, 128, FAKE, 256, 128, 4, FAKE, ctypes.byref(cache()), S) == ALIGN


def test_read_validation():
    c = ctypes.byref(cache())
    rd = F.lib.fp8_kv_read
    assert rd(c, FAKE, 4, 4, FAKE, -1, 4, FAKE, FAKE, S) == INVALID
    assert rd(c, FAKE, 3, 4, FAKE, 1, 4, FAKE, FAKE, S) == INVALID     # table rows that overlap
    assert rd(c, None, 4, 4, FAKE, 1, 4, FAKE, FAKE, S) == INVALID
    assert rd(c, FAKE, 4, 4, None, 1, 4, FAKE, FAKE, S) == INVALID
    assert rd(c, FAKE, 4, 4, FAKE, 1, 4, FAKE, FAKE + 8, S) == ALIGN
    assert rd(c, FAKE, 4, 4, FAKE + 2, 1, 4, FAKE, FAKE, S) == ALIGN
    assert rd(c, FAKE, 4, 4, FAKE, 1, 2 ** 31, FAKE, FAKE, S) == SHAPE
    assert rd(c, FAKE, 4, 4, FAKE, 0, 4, FAKE, FAKE, S) == OK
    assert rd(c, FAKE, 4, 4, FAKE, 1, 0, None, None, S) == OK


def attn(q=(FAKE, 1024, 128), B=3, Hq=8, c=None, table=FAKE, ts=8, mp=8, lens=FAKE, scale=0.1, window=0, out=FAKE,
         lse=None, ws=FAKE, n=None):
    c = cache() if c is None else c
    n = F.lib.fp8_paged_attention_ws_bytes(B, Hq, ctypes.byref(c)) if n is None else n
    return F.lib.fp8_paged_attention(*q, B, Hq, ctypes.byref(c), table, ts, mp, lens, scale, window, out, lse, ws, n, S)


def test_attention_validation():
    assert attn(B=-1) == INVALID
    assert attn(Hq=0) == INVALID
    assert attn(Hq=7) == SHAPE                             # not a multiple of the kv heads
    assert attn(ts=7) == INVALID
    assert attn(window=-1) == INVALID
    assert attn(scale=math.inf) == INVALID
    assert attn(scale=math.nan) == INVALID
    assert attn(table=None) == INVALID
    assert attn(lens=None) == INVALID
    assert attn(out=None) == INVALID
    assert attn(ws=None) == INVALID
    assert attn(q=(None, 1024, 128)) == INVALID
    assert attn(q=(FAKE, 1020, 128)) == ALIGN
    assert attn(q=(FAKE, 1024, 96)) == INVALID
    assert attn(lens=FAKE + 2) == ALIGN
    assert attn(lse=FAKE + 1) == ALIGN
    assert attn(ws=FAKE + 8) == ALIGN
    assert attn(n=0) == SHAPE
    assert attn(n=F.lib.fp8_paged_attention_ws_bytes(3, 8, ctypes.byref(cache())) - 1) == SHAPE
    assert attn(ts=2 ** 40, mp=2 ** 30) == SHAPE           # more tokens than 32 bits count
    assert attn(B=2 ** 20, ts=2 ** 20, mp=2 ** 20, n=1 << 60) == SHAPE
    assert attn(B=0, q=(None, 0, 0), table=None, lens=None, out=None, ws=None) == OK


def test_workspace_grows_with_what_it_holds():
    c = F.KVCache(4, 16, 2, 64, device="cpu")
    n = F.paged_attention_ws_bytes(3, 8, c)
    assert n % 8 == 0 and F.paged_attention_ws_bytes(4, 8, c) > n
    assert F.paged_attention_ws_bytes(3, 32, c) > n        # 16 heads a kv head: larger partial sums
    with pytest.raises(ValueError):
        F.paged_attention_ws_bytes(3, 7, c)


def test_binding_checks():
    c = F.KVCache(4, 16, 2, 64, device="cpu")
    bf = dict(dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        F.kv_write(torch.zeros(3, 2, 64, **bf), torch.zeros(3, 2, 64, **bf), torch.zeros(3, dtype=torch.int64), c)
    with pytest.raises(ValueError):
        F.KVCache(4, 16, 2, 64, layout="DHN", device="cpu")
    with pytest.raises(ValueError):                        # strides that differ
        F.KVCache.wrap(c.k, c.v.transpose(1, 2).contiguous().transpose(1, 2), c.k_scale, c.v_scale)
    with pytest.raises(ValueError):
        F.KVCache.wrap(c.k, c.v[:2], c.k_scale, c.v_scale)
    with pytest.raises(TypeError):
        F.KVCache.wrap(c.k.float(), c.v, c.k_scale, c.v_scale)
    with pytest.raises(TypeError):
        F.KVCache.wrap(c.k, c.v, c.k_scale.double(), c.v_scale)
    with pytest.raises(ValueError):
        F.KVCache.wrap(c.k, c.v, c.k_scale.transpose(1, 2).contiguous().transpose(1, 2), c.v_scale)
    with pytest.raises(ValueError):
        F.KVCache.wrap(c.k, c.v, c.k_scale, c.v_scale, fmt=7)
    from fp8_block_scaled_12_b200 import kv
    x = torch.zeros(3, 2, 64, **bf)
    assert kv._rows(x.transpose(0, 1), "x", (2, 3, 64)) == (x.data_ptr(), 64, 128)
    with pytest.raises(TypeError):
        kv._rows(x.float(), "x", (3, 2, 64))
    with pytest.raises(ValueError):
        kv._rows(x, "x", (3, 3, 64))
    with pytest.raises(ValueError):
        kv._rows(x.transpose(1, 2), "x", (3, 64, 2))
    with pytest.raises(TypeError):
        kv._table(torch.zeros(3, 4, dtype=torch.int64), 3)
    with pytest.raises(ValueError):
        kv._table(torch.zeros(3, 4, dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        kv._table(torch.zeros(4, 3, dtype=torch.int32).T, 3)
    with pytest.raises(ValueError):
        kv._rope(None, torch.zeros(8, 16), 3)
    with pytest.raises(TypeError):
        kv._rope(torch.zeros(3, dtype=torch.int32), torch.zeros(8, 16), 3)


def test_layouts_of_a_cache():
    h, n = F.KVCache(4, 16, 2, 64, device="cpu"), F.KVCache(4, 16, 2, 64, layout="NHD", device="cpu")
    assert h.k.shape == n.k.shape == (4, 2, 16, 64)
    assert h.k.stride() == (2048, 1024, 64, 1) and n.k.stride() == (2048, 64, 128, 1)


def test_rope_table_angles_keep_far_positions():
    t = F.rope_table(131072, 64, device="cpu")
    assert t.shape == (131072, 64) and t.dtype == torch.float32
    for p in (0, 1, 4097, 131071):
        for i in (0, 3, 31):
            a = p * 10000.0 ** (-2 * i / 64)
            assert abs(float(t[p, i]) - math.cos(a)) < 1e-7
            assert abs(float(t[p, 32 + i]) - math.sin(a)) < 1e-7


def test_c_client_and_structure_layout(tmp_path):
    """A C99 program built against the header; the binding's structure has the same layout."""
    import os
    import shutil
    import subprocess
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    here = os.path.dirname(os.path.abspath(__file__))
    libdir = os.path.dirname(F.LIB_PATH)
    exe = str(tmp_path / "c_kv_check")
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                    os.path.join(os.path.dirname(here), "include"), "-o", exe, os.path.join(here, "c_kv_check.c"),
                    "-L", libdir, "-lfp8lin", "-Wl,-rpath," + libdir], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr)
    s = _CacheStruct
    assert [int(x) for x in r.stdout.split()] == [ctypes.sizeof(s), s.v_scale.offset, s.num_pages.offset,
                                                  s.token_stride.offset, s.scale_fmt.offset]


@pytest.mark.parametrize("B,Hq", [(2 ** 31, 8), (2 ** 62, 8), (1, 65536), (-1, 8), (1, 0), (1, 3)])
def test_no_workspace_for_counts_that_the_call_refuses(B, Hq):
    assert F.lib.fp8_paged_attention_ws_bytes(B, Hq, ctypes.byref(cache())) == 0


@pytest.mark.parametrize("B", [1, 2 ** 20, 2 ** 28, (2 ** 31 - 1) // 6, (2 ** 31 - 1) // 6 + 1, 2 ** 30, 2 ** 31 - 1])
@pytest.mark.parametrize("Hq", [2, 8, 34, 65534, 65536])
@pytest.mark.parametrize("D", [128, 256])
def test_workspace_and_call_refuse_the_same_counts(B, Hq, D):
    """The narrowest table there is, so the counts alone decide; the call stops at its missing outputs."""
    c = cache(head_dim=D, token_stride=D, head_stride=16 * D, page_stride=32 * D)
    n = F.lib.fp8_paged_attention_ws_bytes(B, Hq, ctypes.byref(c))
    status = F.lib.fp8_paged_attention(FAKE, Hq * D, D, B, Hq, ctypes.byref(c), None, 0, 0, None, 0.1, 0, None, None,
                                       None, 1 << 62, S)
    assert status in (INVALID, SHAPE)
    assert (n > 0) == (status == INVALID)
