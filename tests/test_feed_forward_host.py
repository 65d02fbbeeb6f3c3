"""Refusals of the norm, routing, gate and combine calls (no GPU, nothing is launched)."""
import math
import os
import shutil
import subprocess

import pytest

import bit_gemv_amd as rf

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, P2, P3 = 0x10000, 0x20000, 0x30000          # aligned fake device addresses: never dereferenced
NULL, SHAPE, ALIGN = rf.RFP2_E_NULL, rf.RFP2_E_SHAPE, rf.RFP2_E_ALIGN


def heads(x=P, T=2, H=4, D=64, xs=256, gain=P, eps=1e-6, y=P2, ys=256):
    return rf.lib().rfp2_rms_norm(x, T, H, D, xs, gain, eps, y, ys, None)


def norm(x=P, add=P2, T=2, K=64, xs=64, as_=64, gain=P, eps=1e-6, h=P3, hs=64, y=None, ys=0, q=P,
         d=P):
    return rf.lib().rfp2_add_rms_norm(x, add, T, K, xs, as_, gain, eps, h, hs, y, ys, q, d, None)


def combine(x=P, rows=P2, weights=P, T=2, k=4, K=64, xs=64, gain=P, eps=1e-6, h=P3, hs=64, y=None,
            ys=0, q=P, d=P):
    return rf.lib().rfp2_moe_combine(x, rows, weights, T, k, K, xs, gain, eps, h, hs, y, ys, q, d,
                                     None)


def route(l=P, T=2, E=16, stride=16, bias=P, score=0, groups=4, group_top=1, top_groups=2, top_k=4,
          renorm=1, scale=1.0, ids=P, weights=P, err=None):
    return rf.lib().rfp2_moe_route(l, T, E, stride, bias, score, groups, group_top, top_groups,
                                   top_k, renorm, scale, ids, weights, err, None)


def gated(g=P, u=P, M=2, K=64, gs=64, us=64, act=0, q=P, d=P):
    return rf.lib().rfp2_quantize_gated_acts(g, u, M, K, gs, us, act, q, d, None)


def dequant(q=P, d=P, M=2, K=64, a=P):
    return rf.lib().rfp2_dequantize_acts(q, d, M, K, a, None)


def test_heads():
    for n in ("x", "gain", "y"):
        assert heads(**{n: None}) == NULL
    for bad in (dict(T=0), dict(H=0), dict(D=2), dict(D=66), dict(D=1028, xs=8192, ys=8192),
                dict(xs=252), dict(ys=258), dict(T=(1 << 30) + 1), dict(H=1 << 20, xs=1 << 26, ys=1 << 26),
                dict(y=P, ys=512), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf)):
        assert heads(**bad) == SHAPE, bad
    for bad in (dict(x=P + 4), dict(y=P + 8), dict(gain=P + 4)):
        assert heads(**bad) == ALIGN, bad


@pytest.mark.parametrize("call", [norm, combine])
def test_rows(call):
    assert call(q=None) == NULL and call(d=None) == NULL           # one of the pair alone
    assert call(q=None, d=None) == NULL                            # nothing of the norm is wanted
    for bad in (dict(T=0), dict(T=(1 << 30) + 1), dict(K=0), dict(K=62), dict(K=60), dict(K=(1 << 24) + 32),
                dict(K=2, q=None, d=None, y=P, ys=64), dict(K=6, q=None, d=None, y=P2 + 64, ys=64),
                dict(xs=60), dict(xs=66), dict(hs=60), dict(hs=66), dict(y=P, ys=60), dict(y=P, ys=66),
                dict(eps=0.0), dict(eps=math.nan), dict(eps=math.inf),
                dict(h=P, xs=128), dict(y=P, ys=64, xs=128), dict(h=P3, y=P3, ys=64)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(x=P + 4), dict(gain=P + 4), dict(h=P3 + 8), dict(y=P2 + 68, ys=64), dict(q=P + 2),
                dict(d=P + 1)):
        assert call(**bad) == ALIGN, bad


def test_add_norm():
    assert norm(x=None) == NULL and norm(gain=None) == NULL
    assert norm(add=None) == SHAPE                                 # h without an addition
    for bad in (dict(as_=60), dict(as_=66), dict(h=P2, as_=128), dict(y=P2, ys=64, as_=128)):
        assert norm(**bad) == SHAPE, bad
    assert norm(add=P2 + 4) == ALIGN


def test_combine():
    assert combine(rows=None) == NULL and combine(weights=None) == NULL
    for kw in (dict(), dict(y=P, ys=64, q=None, d=None), dict(h=None, q=None, d=None)):
        assert combine(gain=None, **kw) == NULL                    # a norm's output, or no output
    for bad in (dict(k=0), dict(k=1025), dict(T=1 << 21, k=1024), dict(h=P2), dict(y=P2, ys=64)):
        assert combine(**bad) == SHAPE, bad
    assert combine(rows=P2 + 4) == ALIGN and combine(weights=P + 2) == ALIGN
    # without a norm eps is not read: what is refused here is the stride
    assert combine(gain=None, q=None, d=None, eps=math.nan, hs=60) == SHAPE


def test_route():
    for n in ("l", "ids", "weights"):
        assert route(**{n: None}) == NULL
    assert route(bias=None, group_top=2) == NULL
    for bad in (dict(T=0), dict(T=(1 << 30) + 1), dict(E=0), dict(E=2049, stride=4096, groups=1, top_groups=1),
                dict(stride=15), dict(score=2), dict(score=-1), dict(groups=0), dict(groups=3),
                dict(groups=5), dict(E=130, stride=130, groups=65), dict(top_groups=0), dict(top_groups=5),
                dict(top_k=0), dict(top_k=9), dict(top_k=65, E=2048, stride=2048),
                dict(group_top=0), dict(group_top=3), dict(groups=16, group_top=2, top_groups=8),
                dict(scale=math.inf), dict(scale=math.nan)):
        assert route(**bad) == SHAPE, bad
    for n in ("l", "bias", "ids", "weights", "err"):
        assert route(**{n: P + 2}) == ALIGN


def test_gate():
    for n in ("g", "u", "q", "d"):
        assert gated(**{n: None}) == NULL
    for bad in (dict(M=0), dict(M=(1 << 30) + 1), dict(K=0), dict(K=48), dict(K=(1 << 24) + 32), dict(gs=60),
                dict(us=60), dict(gs=66), dict(us=66), dict(act=2), dict(act=-1)):
        assert gated(**bad) == SHAPE, bad
    for bad in (dict(g=P + 4), dict(u=P + 8), dict(q=P + 2), dict(d=P + 2)):
        assert gated(**bad) == ALIGN, bad


def test_values_of_codes():
    for n in ("q", "d", "a"):
        assert dequant(**{n: None}) == NULL
    for bad in (dict(M=0), dict(M=(1 << 30) + 1), dict(K=0), dict(K=40), dict(K=1 << 31)):
        assert dequant(**bad) == SHAPE, bad
    for bad in (dict(q=P + 2), dict(d=P + 2), dict(a=P + 4)):
        assert dequant(**bad) == ALIGN, bad


PROGRAM = r"""
#include "rfp2.h"
#include <stdio.h>
int main(void) {
  char dummy[64];
  void* p = (void*)(((unsigned long)dummy + 15) & ~15ul);  /* never dereferenced */
  hipStream_t st = (hipStream_t)0;
  int ok = rfp2_rms_norm(NULL, 1, 1, 64, 64, p, 1e-6, p, 64, st) == RFP2_E_NULL &&
           rfp2_add_rms_norm(NULL, p, 1, 64, 64, 64, p, 1e-6, p, 64, NULL, 0, p, p, st) == RFP2_E_NULL &&
           rfp2_moe_combine(p, NULL, p, 1, 1, 64, 64, NULL, 0.0, p, 64, NULL, 0, NULL, NULL, st) ==
               RFP2_E_NULL &&
           rfp2_moe_route(p, 1, 8, 8, NULL, RFP2_ROUTE_SOFTMAX, 1, 1, 1, 9, 1, 1.0, p, p, NULL, st) ==
               RFP2_E_SHAPE &&
           rfp2_moe_route(p, 1, 8, 8, NULL, RFP2_ROUTE_SIGMOID, 1, 1, 1, 2, 0, 1.0, NULL, p, p, st) ==
               RFP2_E_NULL &&
           rfp2_quantize_gated_acts(p, p, 1, 32, 32, 32, RFP2_GATE_SILU, NULL, p, st) == RFP2_E_NULL &&
           rfp2_quantize_gated_acts(p, p, 1, 33, 36, 36, RFP2_GATE_GELU, p, p, st) == RFP2_E_SHAPE &&
           rfp2_dequantize_acts(p, p, 1, 16, p, st) == RFP2_E_SHAPE;
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


def test_binding_refuses_what_is_not_on_the_gpu():
    torch = pytest.importorskip("torch")
    x, q, i = torch.zeros(2, 64), torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2, 4, dtype=torch.int32)
    for call in (lambda: rf.rfp2_rms_norm(x, 2, 1, 64, x[0], 1e-6, x),
                 lambda: rf.rfp2_add_rms_norm(x, x, 2, 64, x[0], 1e-6, x, None, q, x),
                 lambda: rf.rfp2_moe_combine(None, x, x, 2, 1, 64, x),
                 lambda: rf.rfp2_moe_route(x, 2, 64, None, 0, 1, 1, 1, 4, True, 1.0, i, x),
                 lambda: rf.rfp2_quantize_gated_acts(x, x, 2, 64, 0, q, x),
                 lambda: rf.rfp2_dequantize_acts(q, x, 2, 64, x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        rf.rfp2_rms_norm([[0.0] * 64], 1, 1, 64, x[0], 1e-6, x)
