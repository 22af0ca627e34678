"""The gradient of the log-probabilities where a row's logits are far from 0 and its lse has lost the sum's logarithm,
against float64 of the same logits.

Tolerances. p is a ratio: its own power has a rounded factor and exponent, 2^-24 of the distance each, and the power's
2^-22; the sum's chain has at most V / 256 + 16 terms. Distances are from the row's largest logit where the row is far
(beyond 110 a term is below 2^-149), and from lse, itself rounded, changed in base and compared (3 * 2^-24 |lse|),
where |lse| <= 1024. Rounding to bf16 adds 2^-8, and the label's column is a difference of two numbers of size 1 (2 *
2^-24).
"""
import numpy as np
import pytest

from oracle import tune

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF, F, NEAR = 2.0 ** -8, 2.0 ** -24, 1024.0
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def K():
    from host_memory_streamed_stream_gb300 import _build

    _build.build()
    from host_memory_streamed_stream_gb300 import kernels

    return kernels


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _far_rows(T, V, kind):
    g = torch.Generator(device="cuda").manual_seed(V + T)
    z = torch.zeros(T, (V + 7) // 8 * 8 + 8, device="cuda")
    z[:, :V] = torch.randn(T, V, device="cuda", generator=g)
    z[0, :V] = -1.0e9
    z[1, :V] = 3.0e12
    z[1, :V:3] = 2.9e12
    z[2, :V] += 60000.0
    z[3, 5:V] = -1.0e9       # a mask beside ordinary ones
    z[4, :V] -= 1.0e5
    z[5, :V] *= 3.0e4
    z[6, :V] += 1.0e7
    z[7, :V] = -3.0e38
    z[8, 1:V] = -float("inf")
    z[8, 0] = 5.0e6          # the label alone
    z[9, :V] += 1020.0       # on both sides of the border
    z[10, :V] -= 1040.0
    z[11, V - 1] = 3.3e38
    return z.to(TYPES[kind])


@pytest.mark.parametrize("T,V", [(16, 72), (13, 5003), (12, 40001), (12, 170000)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1.0, 0.7, 1.4])
def test_far_gradient(K, T, V, kind, scale):
    rng = np.random.default_rng(V)
    a = float(np.float32(scale))
    buf = _far_rows(T, V, kind)
    z = buf[:, :V]
    lab = (np.arange(T) % 5).astype(np.int32)
    lab[1], lab[8], lab[-1] = 1, 0, V - 1
    lt = torch.tensor(lab).cuda()
    dlogp = rng.standard_normal(T).astype(np.float32)
    dt = torch.tensor(dlogp).cuda()
    logp, lse = K.token_logprobs(z, lt, scale=a)
    out = torch.full(buf.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    K.token_logprobs_bwd(z, lt, lse, dt, scale=a, out=out[:, :V])
    x = _np(z)
    ref = tune.token_logprobs_bwd(x, lab, dlogp, a)
    rs = tune.token_logprobs(x, lab, a)[1]
    size = np.minimum(np.abs(rs), NEAR)
    rel = (F * (3 * 110 + 16 + V / 256) + 3 * F * size)[:, None]
    y = x * a
    p = np.exp(y - y.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    k = np.abs(a * dlogp)[:, None]
    assert np.all(np.abs(_np(out[:, :V]) - ref) <= HALF * np.abs(ref) + k * (p * rel + 2 * F) + 1e-38)
    assert torch.all(out[:, V:] == 7.0)
    if kind == "bf16":  # in place
        K.token_logprobs_bwd(z, lt, lse, dt, scale=a, out=z)
        assert torch.equal(z, out[:, :V])


@pytest.mark.parametrize("V", [72, 40001])
def test_rows_without_a_sum(K, V):
    """NaN, +inf and nothing but -inf give NaN in the whole row; masked rows of them zeros."""
    z = torch.zeros(6, (V + 7) // 8 * 8, device="cuda")[:, :V]
    z[0, 3], z[1, V - 1], z[2] = float("nan"), float("inf"), -float("inf")
    z[3], z[4], z[5] = z[0], z[1], z[2]
    lab = torch.tensor([1, 1, 1, -1, -1, -1], dtype=torch.int32).cuda()
    _, lse = K.token_logprobs(z, lab)
    d = K.token_logprobs_bwd(z, lab, lse, torch.ones(6, device="cuda"))
    assert bool(torch.isnan(d[:3]).all()) and torch.all(d[3:] == 0)


def test_far_rows_among_near_ones(K):
    """A batch in which every third row is far, in a graph and eagerly: each row as it is alone."""
    rng = np.random.default_rng(3)
    T, V = 300, 33000
    z = torch.tensor(rng.standard_normal((T, V)), dtype=torch.float32).cuda()
    z[::3] += 2.0e4
    lab = torch.tensor(rng.integers(-20, V, T), dtype=torch.int32).cuda()
    dlogp = torch.tensor(rng.standard_normal(T), dtype=torch.float32).cuda()
    _, lse = K.token_logprobs(z, lab)
    d = K.token_logprobs_bwd(z, lab, lse, dlogp)
    for t in (0, 1, 2, 3, 297, 299):
        assert torch.equal(K.token_logprobs_bwd(z[t:t + 1], lab[t:t + 1], lse[t:t + 1], dlogp[t:t + 1])[0], d[t])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = K.token_logprobs_bwd(z, lab, lse, dlogp)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, d)
