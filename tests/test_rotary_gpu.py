"""Rotary positions and query/key norms with the rotation, against float64.

Tolerances: a bf16 result is off by at most half a step (2^-8 of its size) plus the fp32 arithmetic
in front of the rounding: a few steps of 2^-24 of the terms that are added, times the length of the
sums (128 squares and products at most: below 2^-16 in all).
"""
import math

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8   # half a bf16 step
ACC = 2.0 ** -16   # fp32 arithmetic on up to 128 terms, see above


@pytest.fixture(scope="module")
def K():
    from host_memory_streamed_stream_gb300 import _build

    _build.build()
    from host_memory_streamed_stream_gb300 import kernels

    return kernels


def _bf16(rng, shape, scale=1.0):
    x = oracle.bf16_bits_to_float(oracle.float_to_bf16_bits(rng.standard_normal(shape) * scale))
    return x, torch.tensor(x, dtype=torch.float32).to(torch.bfloat16).cuda()


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _pairs(rot, inter):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)


def _turn(x, cs, pos, inter, sign=1.0):
    """Rotation of the last axis of x [T, H, hd] in float64, and the size of the terms added."""
    rot = 2 * cs.shape[1]
    ia, ib = _pairs(rot, inter)
    c, s = cs[pos][:, None, :, 0], sign * cs[pos][:, None, :, 1]
    y, size = x.copy(), np.abs(x)
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    both = np.abs(x[..., ia]) + np.abs(x[..., ib])
    size[..., ia] = size[..., ib] = both
    return y, size


def _table(K, rot, n_pos):
    t = K.rotary_table(K.rotary_inv_freq(rot), n_pos)
    return t, _np(t)


@pytest.mark.parametrize("n_pos,rot,scaling,amp", [(1, 2, "plain", 1.0), (4096, 128, "plain", 1.0), (70, 6, "linear", 1.0),
                                                  (131072, 64, "bands", 1.3), (333, 256, "base", 0.5)])
def test_table(K, n_pos, rot, scaling, amp):
    f = K.rotary_inv_freq(rot, 10000.0, scaling, 4.0, original_positions=2048)
    got = K.rotary_table(f, n_pos, amplitude=amp).cpu().numpy().astype(np.float64)
    a = np.arange(n_pos)[:, None] * f  # float64: below 2^18 radians, so within 2^-34
    ref = amp * np.stack([np.cos(a), np.sin(a)], -1)
    # the angle's fp32 form is off by 2^-26 turns at most, the function and the product by two steps
    assert np.max(np.abs(got - ref)) <= amp * (2 * math.pi * 2.0 ** -26 + 3 * 2.0 ** -24)


def test_table_negative_and_large_frequencies(K):
    f = np.array([-0.3, 17.5, -1e-12, 0.0, 2 * math.pi, -2 * math.pi])
    got = K.rotary_table(f, 1000).cpu().numpy().astype(np.float64)
    a = np.arange(1000)[:, None] * f
    # a frequency above one turn keeps 2^-53 of its size: 1000 * 17.5 * 2^-53 is nothing here
    assert np.max(np.abs(got - np.stack([np.cos(a), np.sin(a)], -1))) <= 2 * math.pi * 2.0 ** -26 + 3 * 2.0 ** -24


@pytest.mark.parametrize("T,heads,hd,rot", [(1, 1, 16, 16), (1, 48, 128, 128), (37, 5, 64, 16), (200, 8, 128, 64),
                                            (333, 3, 112, 96), (5, 64, 256, 256), (3, 300, 16, 16)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary(K, T, heads, hd, rot, inter, inverse):
    rng = np.random.default_rng(T + heads + hd + rot)
    n_pos = 50
    tab, cs = _table(K, rot, n_pos)
    # a column slice of a wider buffer, as q | k of a fused projection
    full, ft = _bf16(rng, (T, heads * hd + 24))
    x, xt = full[:, 8:8 + heads * hd], ft[:, 8:8 + heads * hd]
    pos = rng.integers(0, n_pos, T).astype(np.int32)
    post = torch.tensor(pos).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = ft.clone()
    y = K.rotary(xt, heads, hd, tab, positions=post, interleaved=inter, inverse=inverse, err=err)
    assert torch.equal(ft, before)
    ref, size = _turn(x.reshape(T, heads, hd), cs, pos, inter, -1.0 if inverse else 1.0)
    got = _np(y).reshape(T, heads, hd)
    assert np.all(np.abs(got - ref) <= HALF * np.abs(ref) + ACC * size)
    np.testing.assert_array_equal(got[..., rot:], x.reshape(T, heads, hd)[..., rot:])
    # in place: the same bits, and the columns around the slice untouched
    z = K.rotary(xt, heads, hd, tab, positions=post, interleaved=inter, inverse=inverse, out=xt, err=err)
    assert z.data_ptr() == xt.data_ptr() and torch.equal(xt, y)
    assert torch.equal(ft[:, :8], before[:, :8]) and torch.equal(ft[:, 8 + heads * hd:], before[:, 8 + heads * hd:])
    # positions t % n_pos without an array
    a = K.rotary(y, heads, hd, tab, interleaved=inter, err=err)
    b = K.rotary(y, heads, hd, tab, positions=(torch.arange(T, dtype=torch.int32, device="cuda") % n_pos),
                 interleaved=inter, err=err)
    assert torch.equal(a, b) and int(err.item()) == 0


def test_into_other_columns_of_the_same_buffer(K):
    """The input's own buffer may hold the output, next to it."""
    rng = np.random.default_rng(4)
    T, hd, nh, nkv = 70, 64, 3, 2
    cols = (nh + nkv) * hd
    tab, _ = _table(K, hd, 100)
    x, buf = _bf16(rng, (T, 2 * cols + 8))
    gain = torch.ones(hd, dtype=torch.bfloat16, device="cuda")
    a, b = buf[:, :cols], buf[:, cols + 8:]
    keep = a.clone()
    want = K.rotary(a, nh + nkv, hd, tab)
    assert torch.equal(K.rotary(a, nh + nkv, hd, tab, out=b), want) and torch.equal(a, keep)
    wy, wr = K.qk_norm_rope(a, gain, gain, nh, nkv, hd, tab)
    y, r = K.qk_norm_rope(a, gain, gain, nh, nkv, hd, tab, out=b)
    assert torch.equal(y, wy) and torch.equal(r, wr) and torch.equal(a, keep)
    from host_memory_streamed_stream_gb300 import MTError

    for out in (buf[:, 8:8 + cols], buf[:, cols - 64:2 * cols - 64]):
        with pytest.raises(MTError):
            K.rotary(a, nh + nkv, hd, tab, out=out)


def test_rotary_bad_position_is_flagged_and_left(K):
    rng = np.random.default_rng(3)
    tab, cs = _table(K, 32, 20)
    x, xt = _bf16(rng, (6, 2 * 64))
    pos = np.array([0, 19, 20, -1, 2 ** 31 - 1, 7], dtype=np.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = _np(K.rotary(xt, 2, 64, tab, positions=torch.tensor(pos).cuda(), err=err))
    assert int(err.item()) == 8
    np.testing.assert_array_equal(y[2:5], x[2:5])
    good = np.array([0, 1, 5])
    ref, size = _turn(x[good].reshape(3, 2, 64), cs, pos[good], False)
    assert np.all(np.abs(y[good].reshape(3, 2, 64) - ref) <= HALF * np.abs(ref) + ACC * size)


NORMS = [(1, 4, 4, 64, 64), (1, 40, 8, 128, 128), (37, 4, 1, 64, 16), (200, 8, 2, 128, 64), (333, 4, 4, 64, 0),
         (1500, 3, 3, 128, 128), (3, 40, 40, 128, 32), (20000, 2, 1, 64, 48)]


def _norm_case(K, T, nh, nkv, hd, rot, seed):
    rng = np.random.default_rng(seed)
    tab, cs = _table(K, rot, 77) if rot else (None, None)
    _, ft = _bf16(rng, (T, (nh + 2 * nkv) * hd), 2.0)
    ft[0, :hd] = 0  # a row of zeros: rstd = 1/sqrt(eps)
    x = _np(ft)[:, :(nh + nkv) * hd].reshape(T, nh + nkv, hd)
    gq, gqt = _bf16(rng, (hd,))
    gk, gkt = _bf16(rng, (hd,))
    pos = rng.integers(0, 77, T).astype(np.int32)
    g = np.concatenate([np.tile(gq, (nh, 1)), np.tile(gk, (nkv, 1))])
    return rng, tab, cs, ft, x, gqt, gkt, g, pos


@pytest.mark.parametrize("T,nh,nkv,hd,rot", NORMS)
@pytest.mark.parametrize("inter", [False, True])
def test_qk_norm_rope(K, T, nh, nkv, hd, rot, inter):
    rng, tab, cs, ft, x, gqt, gkt, g, pos = _norm_case(K, T, nh, nkv, hd, rot, T + nh + hd + rot)
    post = torch.tensor(pos).cuda()
    before = ft.clone()
    y, rstd = K.qk_norm_rope(ft, gqt, gkt, nh, nkv, hd, tab, positions=post, interleaved=inter)
    assert torch.equal(ft, before)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
    n = x * r * g
    ref, size = _turn(n, cs, pos, inter) if rot else (n, np.abs(n))
    got = _np(y).reshape(T, nh + nkv, hd)
    assert np.all(np.abs(got - ref) <= HALF * np.abs(ref) + ACC * size)
    assert np.all(np.abs(_np(rstd) / r[..., 0] - 1) <= ACC)
    # in place: the same bits; v's columns are left
    z, r2 = K.qk_norm_rope(ft, gqt, gkt, nh, nkv, hd, tab, positions=post, interleaved=inter, out=ft)
    assert torch.equal(ft[:, :(nh + nkv) * hd], y) and torch.equal(r2, rstd)
    assert torch.equal(ft[:, (nh + nkv) * hd:], before[:, (nh + nkv) * hd:])


@pytest.mark.parametrize("T,nh,nkv,hd,rot", NORMS)
@pytest.mark.parametrize("inter", [False, True])
def test_qk_norm_rope_backward(K, T, nh, nkv, hd, rot, inter):
    rng, tab, cs, ft, x, gqt, gkt, g, pos = _norm_case(K, T, nh, nkv, hd, rot, T + nh + hd + rot)
    post = torch.tensor(pos).cuda()
    _, rstd = K.qk_norm_rope(ft, gqt, gkt, nh, nkv, hd, tab, positions=post, interleaved=inter)
    dy, dyt = _bf16(rng, (T, (nh + nkv) * hd))
    dx, dgq, dgk = K.qk_norm_rope_bwd(dyt, ft, gqt, gkt, rstd, nh, nkv, hd, tab, positions=post, interleaved=inter)
    d = dy.reshape(T, nh + nkv, hd)
    u, usize = _turn(d, cs, pos, inter, -1.0) if rot else (d, np.abs(d))
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
    n = x * r
    m = (u * g * n).mean(-1, keepdims=True)
    ref = r * (u * g - n * m)
    size = r * (usize * np.abs(g) + np.abs(n) * (usize * np.abs(g * n)).mean(-1, keepdims=True))
    assert np.all(np.abs(_np(dx).reshape(ref.shape) - ref) <= HALF * np.abs(ref) + 2 * ACC * size)
    # gains: fp32 sums; a thread adds its rows one after the other, then at most 64 slots, and the
    # parts in two steps: the number of additions in a row times 2^-24 of the terms' sum, on top of
    # the terms' own error
    parts = min(T, 608)
    adds = -(-T // parts) * (nh + nkv) + 64 + parts + 32
    for got, heads in ((dgq, slice(0, nh)), (dgk, slice(nh, None))):
        ref_g = (u * n)[:, heads].sum((0, 1))
        terms = (usize * np.abs(n))[:, heads].sum((0, 1))
        assert np.all(np.abs(_np(got) - ref_g) <= HALF * np.abs(ref_g) + (adds * 2.0 ** -24 + ACC) * terms)
    # twice: the same bits; dx over dy and over x: the same bits, v's columns left
    dx2, dgq2, dgk2 = K.qk_norm_rope_bwd(dyt, ft, gqt, gkt, rstd, nh, nkv, hd, tab, positions=post, interleaved=inter)
    assert torch.equal(dx, dx2) and torch.equal(dgq, dgq2) and torch.equal(dgk, dgk2)
    v = ft[:, (nh + nkv) * hd:].clone()
    for o in (dyt.clone(), ft):
        src = o if o is not ft else dyt
        dx2, dgq2, dgk2 = K.qk_norm_rope_bwd(src, ft, gqt, gkt, rstd, nh, nkv, hd, tab, positions=post,
                                             interleaved=inter, out=o)
        assert torch.equal(o[:, :(nh + nkv) * hd], dx) and torch.equal(dgq, dgq2) and torch.equal(dgk, dgk2)
    assert torch.equal(ft[:, (nh + nkv) * hd:], v)


def test_qk_norm_backward_against_differences(K):
    """The formula itself: central differences of a float64 forward."""
    rng = np.random.default_rng(9)
    hd, eps = 64, 1e-5
    x, g, w = rng.standard_normal(hd), rng.standard_normal(hd), rng.standard_normal(hd)

    def f(x, g):
        return float((w * x / np.sqrt((x * x).mean() + eps) * g).sum())

    r = 1 / np.sqrt((x * x).mean() + eps)
    dx = r * (w * g - x * r * (w * g * x * r).mean())
    dg = w * x * r
    step = 1e-6
    for i in range(0, hd, 7):
        e = np.zeros(hd)
        e[i] = step
        # a central difference is off by step^2 of the third derivative and 2^-53 / step: below 1e-8
        assert abs((f(x + e, g) - f(x - e, g)) / (2 * step) - dx[i]) < 1e-7
        assert abs((f(x, g + e) - f(x, g - e)) / (2 * step) - dg[i]) < 1e-7


def test_on_another_stream_and_captured(K):
    rng = np.random.default_rng(4)
    nh, nkv, hd, T = 8, 2, 128, 300
    tab, _ = _table(K, hd, T)
    _, xt = _bf16(rng, (T, (nh + 2 * nkv) * hd))
    _, gt = _bf16(rng, (hd,))
    _, dyt = _bf16(rng, (T, (nh + nkv) * hd))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        y, r = K.qk_norm_rope(xt, gt, gt, nh, nkv, hd, tab, err=err)
        return (y, r) + tuple(K.qk_norm_rope_bwd(dyt, xt, gt, gt, r, nh, nkv, hd, tab, err=err)) + (
            K.rotary(y, nh + nkv, hd, tab, inverse=True, err=err), K.rotary_table(K.rotary_inv_freq(hd), T))

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t in got:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and int(err.item()) == 0
