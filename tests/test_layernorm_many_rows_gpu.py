"""Layer norm where a block takes many rows in turn, several times what its ring holds, against float64: refilled
slots, the sums that two blocks of a cluster exchange row after row, gains' sums over many rows.

Tolerances. A sum over a row runs in chains of at most 32 terms a thread, 5 shuffles and 32 warps: C = 2^-17 of the
sum of sizes bounds it. mean is within C mean|x|, n = (x - mean) rstd within C (|n| + mean|x| rstd), a bf16 result
2^-8 of its size. A gain's sum over T rows has chains of T / 76 rows (a block), at most 8 groups of a block, T / 76 /
16 blocks a warp and 16 warps: below T / 64 + 64 steps of 2^-24 of the sum of sizes.
"""
import numpy as np
import pytest

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


def _rows(g, T, h, kind, size=1.5, offset=0.3):
    return (torch.randn(T, h, device="cuda", generator=g) * size + offset).to(TYPES[kind])


def _below(err, bound):
    return bool((err.abs() <= bound).all())


# 6 to 20 rows a group, whose ring holds 4 at most; WIDE: two blocks of a cluster share a row
SIZES = [(30000, 64), (25001, 1000), (4001, 4096), (2003, 8192)]
WIDE = [(601, 8200), (1000, 12000), (500, 16384)]


@pytest.mark.parametrize("T,h", SIZES + [(1400, 12000), (1300, 16384)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_forward(K, T, h, kind):
    g = torch.Generator(device="cuda").manual_seed(T)
    x = _rows(g, T, h, kind)
    ga, be = _rows(g, 1, h, "bf16", 0.3, 1.0)[0], _rows(g, 1, h, "bf16", 0.3, 0.0)[0]
    y, mean, rstd = K.layernorm_fwd(x, ga, be)
    xd, gd, bd = x.double(), ga.double(), be.double()
    M = xd.mean(1)
    R = 1 / ((xd - M[:, None]).square().mean(1) + 1e-5).sqrt()
    size = xd.abs().mean(1)
    assert _below(mean.double() - M, C * size)
    assert _below(rstd.double() - R, C * R * (1 + size * R))
    n = (xd - M[:, None]) * R[:, None]
    Y = n * gd + bd
    nerr = C * (n.abs() * (2 + size * R)[:, None] + (size * R)[:, None])
    assert _below(y.double() - Y, HALF * Y.abs() + nerr * gd.abs() + F * bd.abs())
    again = K.layernorm_fwd(x, ga, be)
    assert all(torch.equal(a, b) for a, b in zip(again, (y, mean, rstd)))


@pytest.mark.parametrize("T,h", SIZES + WIDE)
@pytest.mark.parametrize("kind,dy_kind", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("res", [True, False])
def test_backward(K, T, h, kind, dy_kind, res):
    g = torch.Generator(device="cuda").manual_seed(T + 1)
    x, dy = _rows(g, T, h, kind), _rows(g, T, h, dy_kind, 0.5, 0.05)
    dres = _rows(g, T, h, kind, 0.5) if res else None
    ga = _rows(g, 1, h, "bf16", 0.3, 1.0)[0]
    _, mean, rstd = K.layernorm_fwd(x, ga)
    dx, dxb, dg, db = K.layernorm_bwd(dy, x, ga, mean, rstd, dres=dres)
    xd, dd, gd, m, r = x.double(), dy.double(), ga.double(), mean.double()[:, None], rstd.double()[:, None]
    n = (xd - m) * r
    u = dd * gd
    m1, m2 = u.mean(1, keepdim=True), (u * n).mean(1, keepdim=True)
    DX = r * (u - m1 - n * m2)
    if res:
        DX = DX + dres.double()
    nerr = 4 * F * (xd.abs() + m.abs()) * r
    e1 = C * u.abs().mean(1, keepdim=True)
    e2 = (C * (u * n).abs() + u.abs() * nerr).mean(1, keepdim=True)
    derr = r * (4 * F * u.abs() + e1 + n.abs() * e2 + nerr * m2.abs() + 4 * F * (n * m2).abs()) + 4 * F * DX.abs()
    if res:
        derr = derr + 2 * F * dres.double().abs()
    assert _below(dx.double() - DX, derr + (HALF * DX.abs() if kind == "bf16" else 0.0))
    assert dxb is None if kind == "bf16" else torch.equal(dxb, dx.bfloat16())
    chain = F * (T / 64 + 64)
    DG, DB = (dd * n).sum(0), dd.sum(0)
    assert _below(dg.double() - DG, HALF * DG.abs() + 1.01 * (chain * (dd * n).abs() + dd.abs() * nerr).sum(0))
    assert _below(db.double() - DB, HALF * DB.abs() + 1.01 * chain * dd.abs().sum(0))
    again = K.layernorm_bwd(dy, x, ga, mean, rstd, dres=dres)
    assert all(a is b or torch.equal(a, b) for a, b in zip(again, (dx, dxb, dg, db)))
