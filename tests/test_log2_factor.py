"""The split of scale * log2(e) into two floats (csrc/log2_factor.h), compiled for the host, over all fp32 scales of
an octave: powers of two change nothing but the exponent."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "host_memory_streamed_stream_gb300",
                    "csrc")
SOURCE = """
#include "log2_factor.h"
extern "C" void split(const float* scale, long n, float* one, float* hi, float* lo) {
  for (long i = 0; i < n; ++i) {
    const mt::Factor f = mt::factor(scale[i]);
    one[i] = f.one, hi[i] = f.hi, lo[i] = f.lo;
  }
}
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("factor")
    src, lib = d / "split.cpp", d / "split.so"
    src.write_text(SOURCE)
    subprocess.run([gxx, "-O2", "-ffp-contract=off", "-shared", "-fPIC", "-I" + CSRC, str(src), "-o", str(lib)],
                   check=True)
    f = ctypes.CDLL(str(lib)).split
    f.argtypes = [ctypes.c_void_p, ctypes.c_long] + [ctypes.c_void_p] * 3

    def call(scale):
        out = [np.empty_like(scale) for _ in range(3)]
        f(scale.ctypes.data, scale.size, *(o.ctypes.data for o in out))
        return out

    return call


def test_every_scale_of_an_octave(split):
    scale = (np.arange(1 << 23, dtype=np.uint32) + np.uint32(0x3f800000)).view(np.float32)
    one, hi, lo = split(scale)
    # -inf * lo + (-inf * hi - m) is -inf, as the power of an impossible token has to be, only with both above 0
    assert hi.min() > 0 and lo.min() > 0
    assert not np.any(hi.view(np.uint32) & 0xfff)  # twelve bits: hi * z is a sum of at most 36
    c = scale.astype(np.float64) * np.log2(np.e)
    assert np.all(np.abs(one - c) <= 2.0 ** -24 * c * 1.5)  # rounded factor, rounded product
    assert np.all(np.abs(hi.astype(np.float64) + lo - c) <= 2.0 ** -34 * c)


def test_limits(split):
    scale = np.array([2.0 ** -64, 2.0 ** 64, 1 / 7.343, 1.6381017], np.float32)
    one, hi, lo = split(scale)
    assert np.all(np.isfinite(one)) and hi.min() > 0 and lo.min() > 0
