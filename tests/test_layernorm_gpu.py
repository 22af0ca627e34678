"""Layer norm, forward and backward, against float64.

Tolerances. A sum over a row runs in chains of at most 32 terms a thread, 5 shuffles and 32 warps: 2^-24 * 128 = 2^-17
of the sum of sizes bounds it, with what is done with it (a few steps). With C = 2^-17: mean within C mean|x|; n = (x -
mean) rstd within C (|n| + mean|x| rstd) (rstd's own error is that of n's sum of squares). bf16 results add half a
step, 2^-8.
"""
import numpy as np
import pytest

from oracle import tune

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF, C, F = 2.0 ** -8, 2.0 ** -17, 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def K():
    from host_memory_streamed_stream_gb300 import _build

    _build.build()
    from host_memory_streamed_stream_gb300 import kernels

    return kernels


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _rows(rng, T, h, kind, pad=0, size=1.5, offset=0.3):
    buf = torch.full((T, h + pad), float("nan"), dtype=TYPES[kind], device="cuda")
    buf[:, :h] = torch.tensor(rng.standard_normal((T, h)) * size + offset, dtype=torch.float32).cuda().to(TYPES[kind])
    return buf[:, :h]


def _gain(rng, h, about=1.0):
    return torch.tensor(about + 0.3 * rng.standard_normal(h), dtype=torch.float32).bfloat16().cuda()


SIZES = [(1, 8), (5, 16), (3, 256), (700, 64), (1, 5120), (33, 1160), (9, 4096), (4, 8200), (3, 16384), (2000, 520),
         (400, 1024), (650, 4096)]


@pytest.mark.parametrize("T,h", SIZES)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("bias,pad", [(True, 0), (False, 24)])
def test_forward(K, T, h, kind, bias, pad):
    rng = np.random.default_rng(T + h)
    x = _rows(rng, T, h, kind, pad)
    g, b = _gain(rng, h), _gain(rng, h, 0.0) if bias else None
    out = torch.full((T, h + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = K.layernorm_fwd(x, g, b, eps=1e-5, out=out[:, :h])
    xa, ga = _np(x), _np(g)
    Y, M, R = tune.layernorm_fwd(xa, ga, _np(b) if bias else None)
    size = np.abs(xa).mean(1)
    assert np.all(np.abs(_np(mean) - M) <= C * size)
    assert np.all(np.abs(_np(rstd) - R) <= C * R * (1 + size * R))
    nerr = C * (np.abs(xa - M[:, None]) * R[:, None] * (2 + size * R)[:, None] + (size * R)[:, None])
    assert np.all(np.abs(_np(y) - Y) <= HALF * np.abs(Y) + nerr * np.abs(ga) + F * np.abs(_np(b) if bias else 0.0))
    assert torch.all(out[:, h:] == 3.0)
    assert torch.equal(K.layernorm_fwd(x, g, b)[0], y)


def test_forward_far_from_zero(K):
    """A mean 2^12 times the spread: the squares are of centred values, which costs 2^-12 of it, not 2^-24."""
    rng = np.random.default_rng(3)
    x = _rows(rng, 5, 4096, "f32", size=0.25, offset=1024.0)
    g = torch.ones(4096, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = K.layernorm_fwd(x, g)
    Y, M, R = tune.layernorm_fwd(_np(x), np.ones(4096))
    assert np.all(np.abs(_np(rstd) - R) <= C * R * (1 + 1024 * R) ** 1)
    assert np.all(np.abs(_np(y) - Y) <= HALF * np.abs(Y) + C * 4100 * (1 + np.abs(Y)))


def test_constant_rows(K):
    """No spread: rstd = 1 / sqrt(eps), y = beta; with eps 0 it is infinite, as by the formula."""
    x = torch.full((3, 512), 2.5, device="cuda")
    g = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    b = torch.full((512,), 0.5, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = K.layernorm_fwd(x, g, b, eps=1e-4)
    assert torch.all(y == 0.5) and torch.all(mean == 2.5) and torch.allclose(rstd, torch.full_like(rstd, 100.0))
    assert bool(torch.isinf(K.layernorm_fwd(x, g, b, eps=0.0)[2]).all())


@pytest.mark.parametrize("T,h", SIZES)
@pytest.mark.parametrize("kind,dy_kind", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("res,bias,pad", [(True, True, 0), (False, False, 24), (True, True, 8)])
def test_backward(K, T, h, kind, dy_kind, res, bias, pad):
    rng = np.random.default_rng(T * 3 + h)
    x, dy = _rows(rng, T, h, kind, pad), _rows(rng, T, h, dy_kind, pad, size=0.5, offset=0.05)
    dres = _rows(rng, T, h, kind, pad, size=0.5) if res else None
    g = _gain(rng, h)
    _, mean, rstd = K.layernorm_fwd(x, g)
    dx, dxb, dg, db = K.layernorm_bwd(dy, x, g, mean, rstd, dres=dres, bias=bias)
    xa, da, ga, ma, ra = _np(x), _np(dy), _np(g), _np(mean), _np(rstd)
    DX, DG, DB = tune.layernorm_bwd(da, xa, ga, ma, ra, _np(dres) if res else None)
    n = (xa - ma[:, None]) * ra[:, None]
    nerr = 4 * F * (np.abs(xa) + np.abs(ma)[:, None]) * ra[:, None]
    u = np.abs(da * ga)
    # the two means, each within C of the mean of its terms' sizes (and n's error), times 1 and n
    m1 = C * u.mean(1, keepdims=True)
    m2 = (C * u * np.abs(n) + u * nerr).mean(1, keepdims=True)
    M2 = np.abs((da * ga * n).mean(1, keepdims=True))
    derr = ra[:, None] * (4 * F * u + m1 + np.abs(n) * m2 + nerr * M2 + 4 * F * np.abs(n) * M2)
    derr = derr + 4 * F * np.abs(DX) + (2 * F * np.abs(_np(dres)) if res else 0)
    assert dx.dtype == x.dtype
    assert np.all(np.abs(_np(dx) - DX) <= derr + (HALF * np.abs(DX) if kind == "bf16" else 0))
    if kind == "f32":
        assert torch.equal(dxb, dx.bfloat16())
    else:
        assert dxb is None
    # sums over T rows: chains of rows a block, groups, 16 and T / 304 / 16 parts: below T + 64 steps of the sizes
    chain = F * (min(T, 2000) / 100 + 80)
    gerr = chain * (np.abs(da) * np.abs(n)).sum(0) + (np.abs(da) * nerr).sum(0)
    assert np.all(np.abs(_np(dg) - DG) <= HALF * np.abs(DG) + 1.01 * gerr)
    if bias:
        assert np.all(np.abs(_np(db) - DB) <= HALF * np.abs(DB) + 1.01 * chain * np.abs(da).sum(0))
    else:
        assert db is None
    again = K.layernorm_bwd(dy, x, g, mean, rstd, dres=dres, bias=bias)
    assert all(a is b or torch.equal(a, b) for a, b in zip(again, (dx, dxb, dg, db)))


def test_residual_in_place(K):
    """The C entry takes dx = dres: the gradient is added where it lies."""
    from host_memory_streamed_stream_gb300 import _lib

    rng = np.random.default_rng(4)
    T, h = 70, 1032
    x, dy, dres = (_rows(rng, T, h, "f32") for _ in range(3))
    g = _gain(rng, h)
    _, mean, rstd = K.layernorm_fwd(x, g)
    want, wb, _, _ = K.layernorm_bwd(dy, x, g, mean, rstd, dres=dres)
    lib = _lib.load()
    part = torch.empty(2 * h * lib.mtk_layernorm_bwd_parts(T, h), device="cuda")
    dg = torch.empty(h, dtype=torch.bfloat16, device="cuda")
    rc = lib.mtk_layernorm_bwd(dy.data_ptr(), 0, h, x.data_ptr(), 0, h, g.data_ptr(), mean.data_ptr(),
                               rstd.data_ptr(), dres.data_ptr(), h, dres.data_ptr(), None, part.data_ptr(),
                               dg.data_ptr(), None, T, h, torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(dres, want)


@pytest.mark.parametrize("T,h", [(300, 2056), (7, 12000), (900, 96)])
def test_stream_and_graph(K, T, h):
    """Forward and backward on a stream of their own, and captured and replayed on other rows."""
    rng = np.random.default_rng(5)
    x, dy = _rows(rng, T, h, "f32"), _rows(rng, T, h, "bf16", size=0.2)
    g, b = _gain(rng, h), _gain(rng, h, 0.0)

    def step():
        y, mean, rstd = K.layernorm_fwd(x, g, b)
        return (y, *K.layernorm_bwd(dy, x, g, mean, rstd))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    x.copy_(_rows(rng, T, h, "f32"))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(step(), held))


def test_refusals(K):
    from host_memory_streamed_stream_gb300 import MTError

    x = torch.zeros(4, 64, device="cuda")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    f = torch.zeros(4, device="cuda")
    bad = [lambda: K.layernorm_fwd(x.double(), g), lambda: K.layernorm_fwd(x.half(), g),
           lambda: K.layernorm_fwd(x.t(), g), lambda: K.layernorm_fwd(x, g.float()), lambda: K.layernorm_fwd(x, g[:32]),
           lambda: K.layernorm_fwd(x[:, :60].contiguous(), g[:60]), lambda: K.layernorm_fwd(x[:, 2:34], g[:32]),
           lambda: K.layernorm_fwd(x, g, g.float()), lambda: K.layernorm_fwd(x, g, eps=-1.0),
           lambda: K.layernorm_fwd(x, g, out=x), lambda: K.layernorm_fwd(x.bfloat16(), g, out=x.bfloat16()[:3]),
           lambda: K.layernorm_bwd(x, x, g, f, f.double()), lambda: K.layernorm_bwd(x[:3], x, g, f, f),
           lambda: K.layernorm_bwd(x, x, g, f, f, dres=x.bfloat16()), lambda: K.layernorm_bwd(x, x, g, f[:3], f)]
    for i, call in enumerate(bad):
        with pytest.raises(MTError):
            call()
            pytest.fail(f"call {i} was taken")
    y = x.bfloat16()
    with pytest.raises(MTError):  # over its input
        K.layernorm_fwd(y, g, out=y)
