"""The exponential and the logistic function of the routing and gate kernels, compiled for the
host with the chip's reciprocal estimate modelled by its bound (CPU only).

Bounds, of the value: 2^f by its polynomial (ln 2)^10 / 10! * 2^(1/2) / 2^9 / 2^10 = 1.9e-14; the
constant log2(e) is 2.0e-17 off, times 690 and ln 2 9.6e-15; some ten roundings of at most 2^-53
each, 1.2e-15: in all 3.0e-14 < 2^-44.  The reciprocal's estimate is off by 2^-24 or less, and
so the corrected one by 2^-48 and two roundings: 3.4e-14 < 2^-44 for the logistic function."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_gemv_amd", "csrc")
SOURCE = r"""
#include <cmath>
#include <cstdint>
using std::fma;
static double off = 0.0;                      // of the estimate, relative
static double estimate(double d) { return (1.0 / d) * (1.0 + off); }
#define __device__
#define __forceinline__ inline
#define __builtin_amdgcn_rcp estimate
#define __builtin_bit_cast(T, x) bits<T>(x)
template <class T, class F> static T bits(F x) { T t; __builtin_memcpy(&t, &x, sizeof t); return t; }
#include "scores_device.h"
extern "C" void exps(const double* x, double* y, long n) { for (long i = 0; i < n; ++i) y[i] = rfp2::exp_f64(x[i]); }
extern "C" void logistics(const double* x, double* y, long n, double e) {
  off = e;
  for (long i = 0; i < n; ++i) y[i] = rfp2::logistic(x[i]);
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    d = tmp_path_factory.mktemp("scores")
    (d / "hip").mkdir()
    (d / "hip" / "hip_runtime.h").write_text("")
    (d / "scores.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-fPIC", "-shared", "-I", str(d), "-I", CSRC,
                    str(d / "scores.cpp"), "-o", str(d / "scores.so")], check=True, timeout=120)
    return ctypes.CDLL(str(d / "scores.so"))


def call(f, x, *more):
    y = np.empty_like(x)
    f(x.ctypes.data_as(ctypes.c_void_p), y.ctypes.data_as(ctypes.c_void_p), ctypes.c_long(len(x)), *more)
    return y


def inputs():
    rng = np.random.default_rng(0)
    halves = (np.arange(-1990, 1991) / 2 / 1.4426950408889634)       # where n + f goes to the next n
    x = np.concatenate([rng.uniform(-690, 690, 200000), rng.uniform(-2, 2, 100000), rng.uniform(-40, 40, 100000),
                        halves, np.nextafter(halves, 1000), -np.logspace(-300, 0, 600), np.logspace(-300, 0, 600),
                        [0.0, -0.0, 690.0, -690.0]])
    return x[np.abs(x) <= 690.0]


def test_exponential(host):
    x = inputs()
    want = np.exp(x.astype(np.longdouble))
    assert np.abs(call(host.exps, x) / want - 1).max() <= 2.0 ** -44


@pytest.mark.parametrize("off", [0.0, 2.0 ** -24, -2.0 ** -24, 2.0 ** -25])
def test_logistic(host, off):
    x = inputs()
    want = 1 / (1 + np.exp(-x.astype(np.longdouble)))
    assert np.abs(call(host.logistics, x, ctypes.c_double(off)) / want - 1).max() <= 2.0 ** -44
