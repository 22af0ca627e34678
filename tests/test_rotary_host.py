"""Rotary frequencies (host only) and the refusals of the rotary and query/key-norm entries, which
are decided before anything is launched (the pointers handed over here are never read)."""
import ctypes
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def lib():
    from host_memory_streamed_stream_gb300 import _build, _lib

    _build.build()
    return _lib.load()


@pytest.fixture(scope="module")
def K(lib):
    pytest.importorskip("torch")
    from host_memory_streamed_stream_gb300 import kernels

    return kernels


@pytest.mark.parametrize("rot", [2, 16, 64, 128, 256])
@pytest.mark.parametrize("theta", [10000.0, 5e5])
def test_frequencies(K, rot, theta):
    i = np.arange(rot // 2)
    f = np.exp(-2.0 * i / rot * math.log(theta))
    # a power in 64 bits: a few rounding steps (2^-53) times its exponent's size (< 16)
    tol = dict(rtol=64 * 2.0 ** -53, atol=0)
    np.testing.assert_allclose(K.rotary_inv_freq(rot, theta), f, **tol)
    np.testing.assert_allclose(K.rotary_inv_freq(rot, theta, "linear", 8.0), f / 8, **tol)
    if rot > 2:
        got = K.rotary_inv_freq(rot, theta, "base", 8.0)
        # the ends of the scaled base: the highest frequency kept, the lowest divided by the factor
        np.testing.assert_allclose(got[[0, -1]], [1.0, f[-1] / 8], **tol)
    got = K.rotary_inv_freq(rot, theta, "bands", 4.0, original_positions=2048, low=1.0, high=32.0)
    turns = 2048 * f / (2 * math.pi)
    np.testing.assert_allclose(got[turns >= 32], f[turns >= 32], **tol)
    np.testing.assert_allclose(got[turns <= 1], f[turns <= 1] / 4, **tol)
    mid = (turns > 1) & (turns < 32)
    w = (turns[mid] - 1) / 31
    np.testing.assert_allclose(got[mid], f[mid] * (w + (1 - w) / 4), rtol=1e-13)


def test_frequency_refusals(lib):
    buf = (ctypes.c_double * 128)()
    nan, inf = float("nan"), float("inf")
    good = dict(rot=64, theta=1e4, scaling=3, factor=4.0, orig=2048.0, low=1.0, high=32.0)

    def call(out=buf, **kw):
        a = dict(good, **kw)
        return lib.mtk_rotary_inv_freq(a["rot"], a["theta"], a["scaling"], a["factor"], a["orig"], a["low"], a["high"],
                                       out)

    assert call() == 0
    for kw in (dict(rot=0), dict(rot=-2), dict(rot=7), dict(rot=258), dict(theta=0.0), dict(theta=nan),
               dict(theta=inf), dict(scaling=-1), dict(scaling=4), dict(factor=0.0), dict(factor=nan),
               dict(orig=0.0), dict(low=32.0), dict(high=nan), dict(rot=2, scaling=2), dict(out=None)):
        assert call(**kw) == -1, kw
    # what a scaling does not use is not checked
    assert call(scaling=0, factor=nan, orig=nan, low=nan, high=nan) == 0


def test_entry_refusals(lib):
    """Bad sizes, strides and alignments: MT_EINVAL without a launch (and so without a GPU)."""
    p, e = 1 << 20, 1 << 21  # aligned addresses that nothing reads
    f = (ctypes.c_double * 64)(*([1.0] * 64))
    bad = (ctypes.c_double * 64)(*([float("nan")] * 64))
    assert lib.mtk_rotary_table(None, 64, 16, 1.0, p, None) == -1
    assert lib.mtk_rotary_table(f, 64, 16, 1.0, None, None) == -1
    for rot, n, out, src in ((63, 16, p, f), (0, 16, p, f), (258, 16, p, f), (64, 0, p, f), (64, 16, p + 8, f),
                             (64, 16, p, bad)):
        assert lib.mtk_rotary_table(src, rot, n, 1.0, out, None) == -1
    for amp in (float("nan"), float("inf"), 1e39):
        assert lib.mtk_rotary_table(f, 64, 16, amp, p, None) == -1

    def rotary(x=p, ldx=256, y=e, ldy=256, T=4, heads=2, hd=128, rot=64, pos=None, cs=p, n_pos=8, err=p):
        return lib.mtk_rotary(x, ldx, y, ldy, T, heads, hd, rot, 0, pos, cs, n_pos, 0, err, None)

    for kw in (dict(x=None), dict(y=None), dict(x=p + 2), dict(y=e + 8), dict(ldx=252), dict(ldx=248), dict(ldy=0),
               dict(T=0), dict(T=-1), dict(heads=0), dict(hd=0), dict(hd=120), dict(hd=8192, ldx=16384, ldy=16384),
               dict(rot=0), dict(rot=24), dict(rot=144), dict(rot=-16), dict(cs=None), dict(cs=p + 4), dict(n_pos=0),
               dict(err=None), dict(err=p + 2), dict(pos=p + 2), dict(y=p, ldy=512), dict(y=p + 512),
               dict(y=p + 496, ldx=512, ldy=512), dict(y=p + 528, ldx=512, ldy=512), dict(y=p - 1024, ldy=512)):
        assert rotary(**kw) == -1, kw

    def norm(x=p, ldx=512, gq=p, gk=p, y=e, ldy=384, rstd=p, T=4, nh=2, nkv=1, hd=128, rot=64, eps=1e-5, cs=p, n_pos=8,
             err=p):
        return lib.mtk_qk_norm_rope(x, ldx, gq, gk, y, ldy, rstd, T, nh, nkv, hd, rot, 0, eps, None, cs, n_pos, err,
                                    None)

    for kw in (dict(x=None), dict(gq=None), dict(gk=None), dict(y=None), dict(gq=p + 2), dict(gk=p + 8), dict(ldx=376),
               dict(ldy=380), dict(T=0), dict(nh=0), dict(nkv=0), dict(hd=96), dict(hd=256, ldx=1024, ldy=1024),
               dict(rot=8), dict(rot=160), dict(eps=-1.0), dict(eps=float("nan")), dict(cs=None), dict(n_pos=0),
               dict(err=None), dict(y=p), dict(rstd=p + 2), dict(y=p + 1024, ldy=512)):
        assert norm(**kw) == -1, kw

    d = 1 << 22

    def back(dy=d, lddy=384, x=p, ldx=512, gq=p, gk=p, rstd=p, dx=e, lddx=384, part=p, dgq=p, dgk=p, T=4, hd=128,
             rot=64, cs=p):
        return lib.mtk_qk_norm_rope_bwd(dy, lddy, x, ldx, gq, gk, rstd, dx, lddx, part, dgq, dgk, T, 2, 1, hd, rot, 0,
                                        None, cs, 8, p, None)

    for kw in (dict(dy=None), dict(x=None), dict(rstd=None), dict(dx=None), dict(part=None), dict(dgq=None),
               dict(dgk=None), dict(lddy=376), dict(lddx=388), dict(T=0), dict(hd=32), dict(rot=40), dict(cs=None),
               dict(dx=p, lddx=384), dict(dx=d, lddx=512), dict(dx=d + 768), dict(dx=p + 1024, lddx=512),
               dict(rstd=p + 1), dict(part=p + 2), dict(dgq=p + 1), dict(dgk=p + 1)):
        assert back(**kw) == -1, kw
    assert lib.mtk_qk_norm_rope_bwd_parts(0, 2, 1, 128) == 0
    assert lib.mtk_qk_norm_rope_bwd_parts(5, 2, 1, 96) == 0
    assert 2 <= lib.mtk_qk_norm_rope_bwd_parts(5, 2, 1, 128) <= 304


def test_binding_refusals(K):
    """The binding refuses types and shapes that the C entry cannot see."""
    import torch

    from host_memory_streamed_stream_gb300 import MTError

    with pytest.raises(MTError):
        K.rotary_inv_freq(64, scaling="cubic")
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(MTError):  # not on a GPU
        K.rotary(x, 2, 128, torch.zeros(8, 32, 2))
    with pytest.raises(MTError):
        K.rotary(x.float(), 2, 128, torch.zeros(8, 32, 2))
    with pytest.raises(MTError):
        K.rotary(x, 3, 128, torch.zeros(8, 32, 2))
