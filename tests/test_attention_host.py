"""Refusals of the rotary, cache and attention calls (no GPU, nothing is launched)."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest

import bit_gemv_amd as rf

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000          # an aligned fake device address: never dereferenced
NULL, SHAPE, ALIGN = rf.RFP2_E_NULL, rf.RFP2_E_SHAPE, rf.RFP2_E_ALIGN


def cache(**kw):
    f = dict(k=P, v=P, k_scale=P, v_scale=P, page_table=P, seqs=4, max_pages=8, pages=16,
             page_size=64, kv_heads=8, head_dim=128, format=rf.KV_I8)
    f.update(kw)
    return ctypes.byref(rf._KvCacheStruct(*[f[n] for n, _ in rf._KvCacheStruct._fields_]))


BAD_CACHES = [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(page_table=None), NULL),
    (dict(k_scale=None), NULL), (dict(v_scale=None), NULL),
    (dict(format=2), SHAPE), (dict(format=-1), SHAPE),
    (dict(page_size=0), SHAPE), (dict(page_size=4), SHAPE), (dict(page_size=48), SHAPE),
    (dict(page_size=8192), SHAPE), (dict(page_size=-64), SHAPE),
    (dict(head_dim=0), SHAPE), (dict(head_dim=80), SHAPE), (dict(head_dim=288), SHAPE),
    (dict(kv_heads=0), SHAPE), (dict(kv_heads=1025), SHAPE),
    (dict(pages=0), SHAPE), (dict(pages=1 << 31), SHAPE),
    (dict(seqs=0), SHAPE), (dict(seqs=(1 << 20) + 1), SHAPE),
    (dict(max_pages=0), SHAPE), (dict(max_pages=1 << 25), SHAPE),
    (dict(k=P + 8), ALIGN), (dict(v=P + 8), ALIGN), (dict(k_scale=P + 8), ALIGN),
    (dict(v_scale=P + 4), ALIGN), (dict(page_table=P + 2), ALIGN),
]


def write(c, k=P, v=P, T=2, ks=1024, vs=1024, seq=P, pos=P, err=None):
    return rf.lib().rfp2_kv_write(c, k, v, T, ks, vs, seq, pos, err, None)


def read(c, k=P, v=P, T=2, ks=1024, vs=1024, seq=P, pos=P, err=None):
    return rf.lib().rfp2_kv_read(c, T, seq, pos, k, v, ks, vs, err, None)


def fused(c, q=P, k=P, v=P, T=2, H=32, qs=4096, ks=1024, vs=1024, seq=P, pos=P, freqs=P,
          rot=128, style=0, mscale=1.0, out=P, os_=4096, err=None):
    return rf.lib().rfp2_rope_kv_write(c, q, k, v, T, H, qs, ks, vs, seq, pos, freqs, rot, style,
                                       mscale, out, os_, err, None)


def attn(c, q=P, B=2, T=1, H=32, qs=4096, lens=P, scale=0.1, window=0, y=P, err=None, ws=P,
         ws_bytes=1 << 40):
    return rf.lib().rfp2_paged_attn(c, q, B, T, H, qs, lens, scale, window, y, err, ws, ws_bytes,
                                    None)


@pytest.mark.parametrize("fields,status", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(fields, status):
    for call in (write, read, fused, attn):
        assert call(cache(**fields)) == status, call.__name__
    assert rf.lib().rfp2_paged_attn_workspace_bytes(cache(**fields), 1, 1, 32) == 0


def test_a_half_cache_needs_no_scales():
    # everything but the stride is in order: the scales were not what was refused
    c = dict(format=rf.KV_F16, k_scale=None, v_scale=None)
    assert write(cache(**c), ks=8) == SHAPE
    assert rf.lib().rfp2_paged_attn_workspace_bytes(cache(**c), 1, 1, 32) > 0


@pytest.mark.parametrize("call", [write, read, fused])
def test_token_rows(call):
    for n in ("k", "v", "seq", "pos"):
        assert call(cache(), **{n: None}) == NULL
    for n in ("k", "v"):
        assert call(cache(), **{n: P + 4}) == ALIGN
    for n in ("seq", "pos", "err"):
        assert call(cache(), **{n: P + 2}) == ALIGN
    for bad in (dict(T=0), dict(T=(1 << 30) + 1), dict(ks=1020), dict(vs=1020), dict(ks=1026),
                dict(vs=-1024)):
        assert call(cache(), **bad) == SHAPE
    assert call(None) == NULL


def test_fused_write():
    for n in ("q", "out", "freqs"):
        assert fused(cache(), **{n: None}) == NULL
    for bad in (dict(rot=0), dict(rot=3), dict(rot=130), dict(style=2), dict(mscale=math.inf),
                dict(mscale=math.nan), dict(H=-1), dict(qs=4092), dict(os_=4094),
                dict(H=1 << 20)):
        assert fused(cache(), **bad) == SHAPE, bad
    for bad in (dict(q=P + 4), dict(out=P + 8), dict(freqs=P + 4)):
        assert fused(cache(), **bad) == ALIGN


def test_rope():
    def rope(x=P, T=2, H=4, D=64, xs=256, pos=P, freqs=P, rot=64, style=0, mscale=1.0, y=2 * P,
             ys=256):
        return rf.lib().rfp2_rope(x, T, H, D, xs, pos, freqs, rot, style, mscale, y, ys, None)
    for n in ("x", "pos", "freqs", "y"):
        assert rope(**{n: None}) == NULL
    for bad in (dict(T=0), dict(H=0), dict(D=2), dict(D=66), dict(D=1028), dict(xs=252),
                dict(ys=258), dict(rot=0), dict(rot=5), dict(rot=66), dict(style=-1),
                dict(mscale=math.nan), dict(y=P, ys=512), dict(H=1 << 20, xs=1 << 26, ys=1 << 26)):
        assert rope(**bad) == SHAPE, bad
    for bad in (dict(x=P + 4), dict(y=P + 8), dict(pos=P + 2), dict(freqs=P + 4)):
        assert rope(**bad) == ALIGN, bad

    def freqs(rot=64, base=1e4, factor=1.0, orig=0.0, low=1.0, high=32.0, out=P):
        return rf.lib().rfp2_rope_freqs(rot, base, factor, orig, low, high, out, None)
    assert freqs(out=None) == NULL and freqs(out=P + 4) == ALIGN
    for bad in (dict(rot=0), dict(rot=7), dict(rot=1026), dict(base=1.0), dict(base=math.nan),
                dict(base=math.inf), dict(factor=0.5), dict(factor=math.nan), dict(orig=-1.0),
                dict(orig=math.nan), dict(orig=4096.0, low=32.0), dict(orig=4096.0, low=-1.0),
                dict(orig=4096.0, high=math.inf), dict(orig=4096.0, low=math.nan)):
        assert freqs(**bad) == SHAPE, bad


def test_paged_attn():
    need = rf.lib().rfp2_paged_attn_workspace_bytes(cache(), 2, 1, 32)
    assert need > 0 and need % 256 == 0
    for n in ("q", "lens", "y", "ws"):
        assert attn(cache(), **{n: None}) == NULL
    for bad in (dict(B=0), dict(B=5), dict(T=0), dict(T=9), dict(H=0), dict(H=12), dict(H=1032),
                dict(qs=4092), dict(qs=4098), dict(window=-1), dict(scale=math.inf),
                dict(scale=math.nan), dict(ws_bytes=need - 1)):
        assert attn(cache(), **bad) == SHAPE, bad
    assert attn(cache(seqs=2000), B=1025) == SHAPE
    # the tiles of all sequences together are counted in 32 bits
    far = dict(seqs=1024, max_pages=(1 << 31) // 64 - 1)
    assert attn(cache(**far), B=33) == SHAPE
    assert rf.lib().rfp2_paged_attn_workspace_bytes(cache(**far), 32, 1, 32) > 0
    for bad in (dict(q=P + 4), dict(y=P + 4), dict(lens=P + 2), dict(err=P + 1), dict(ws=P + 64)):
        assert attn(cache(), **bad) == ALIGN, bad
    assert attn(None) == NULL


def test_binding_refuses_what_the_calls_would_overrun():
    torch = pytest.importorskip("torch")
    host = torch.zeros(4, 8, 64, 128, dtype=torch.int8)
    with pytest.raises(ValueError):
        rf.KvCache(host, host, None, None, torch.zeros(1, 1, dtype=torch.int32))   # not on a GPU
    with pytest.raises(TypeError):
        rf.KvCache(host.float(), host, None, None, None)
    with pytest.raises(TypeError):
        rf._cache_ref(object())
    with pytest.raises(ValueError):
        rf._rows(torch.zeros(2, 4), 2, 4, "x")
    with pytest.raises(ValueError):
        rf.KvCache.allocate(7, 1, 64, 1, 64, torch.zeros(1, 1, dtype=torch.int32))


PROGRAM = r"""
#include "rfp2.h"
#include <stdio.h>
int main(void) {
  char dummy[64];
  void* p = (void*)(((unsigned long)dummy + 15) & ~15ul);  /* never dereferenced */
  rfp2_kv_cache c = {0};
  hipStream_t st = (hipStream_t)0;
  int ok = rfp2_rope_freqs(64, 1e4, 1.0, 0.0, 0.0, 0.0, NULL, st) == RFP2_E_NULL &&
           rfp2_rope(NULL, 1, 1, 64, 64, p, p, 64, RFP2_ROPE_HALF, 1.0, p, 64, st) == RFP2_E_NULL &&
           rfp2_kv_write(NULL, p, p, 1, 64, 64, p, p, NULL, st) == RFP2_E_NULL &&
           rfp2_kv_write(&c, p, p, 1, 64, 64, p, p, NULL, st) == RFP2_E_NULL &&
           rfp2_kv_read(&c, 1, p, p, p, p, 64, 64, NULL, st) == RFP2_E_NULL &&
           rfp2_rope_kv_write(&c, p, p, p, 1, 1, 64, 64, 64, p, p, p, 64, RFP2_ROPE_INTERLEAVED,
                              1.0, p, 64, NULL, st) == RFP2_E_NULL &&
           rfp2_paged_attn_workspace_bytes(&c, 1, 1, 1) == 0 &&
           rfp2_paged_attn(&c, p, 1, 1, 1, 64, p, 1.0f, 0, p, NULL, p, 0, st) == RFP2_E_NULL;
  c.k = c.v = p; c.page_table = (const int32_t*)p;
  c.seqs = c.max_pages = c.pages = c.kv_heads = 1; c.page_size = 16; c.head_dim = 64;
  c.format = RFP2_KV_F16;
  ok = ok && rfp2_paged_attn_workspace_bytes(&c, 1, 1, 1) > 0 &&
       rfp2_kv_write(&c, p, p, 0, 64, 64, p, p, NULL, st) == RFP2_E_SHAPE;
  puts(ok ? "ok" : "FAILED");
  return !ok;
}
"""


def test_the_calls_from_c(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe, lib = tmp_path / "a.c", tmp_path / "a", rf.LIB_PATH
    src.write_text(PROGRAM)
    cmd = [cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-D__HIP_PLATFORM_AMD__",
           "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"), str(src), "-o",
           str(exe), lib, "-Wl,-rpath," + os.path.dirname(lib)]
    built = subprocess.run(cmd, capture_output=True, text=True, timeout=120)
    assert built.returncode == 0, built.stderr[-2000:]
    ran = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert ran.returncode == 0 and ran.stdout.strip() == "ok", ran.stdout + ran.stderr
