"""The policy loss's gradient where logits have an offset: p keeps its scale. Against float64 of the same logits.

Tolerance. A bf16 result is rounded by at most 2^-8 of its size, in the mean of squares by 2^-8 / sqrt(3), and so the
mean relative error of N columns by 2^-8 / sqrt(3 N); six of those are allowed. What all columns of a row have in common
is to stay below 2^-13: the subtracted part of an exponent of up to 2^16 as known in two floats, 2^-18, and the row's
sum, 2^-18 at most; what the columns do not share, distances of up to 16 times a factor rounded by 2^-25, is below it.
"""
import numpy as np
import pytest

from oracle import tune

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    from host_memory_streamed_stream_gb300 import _build

    _build.build()
    from host_memory_streamed_stream_gb300 import kernels

    return kernels


@pytest.mark.parametrize("V", [1000, 9000, 60000])
@pytest.mark.parametrize("scale", [1.0, 0.7, 1.4])
@pytest.mark.parametrize("offset", [0.0, 1500.0, -2500.0, 4000.0, 12000.0, -40000.0])
def test_common_factor(K, V, scale, offset):
    rng = np.random.default_rng(V)
    T, a = max(6, 60000 // V), float(np.float32(scale))
    z = torch.tensor(rng.standard_normal((T, V)) + offset, dtype=torch.float32).cuda()
    lab = rng.integers(0, V, T).astype(np.int32)
    x = z.cpu().numpy().astype(np.float64)
    logp = tune.token_logprobs(x, lab, a)[0]
    old = logp.astype(np.float32)
    adv = np.ones(T, np.float32)
    d = K.policy_loss(z, torch.tensor(lab).cuda(), torch.tensor(old).cuda(), torch.tensor(adv).cuda(), scale=a)[3]
    ref = tune.policy_loss(x, lab, old, adv, scale=a)[3]
    rel = d.float().cpu().numpy().astype(np.float64) / ref - 1
    rel[np.arange(T), lab] = 0.0
    assert np.abs(rel).max() <= 2.0 ** -8 + 2.0 ** -13
    assert abs(rel.sum() / (T * (V - 1))) <= 2.0 ** -13 + 6 * 2.0 ** -8 / np.sqrt(3.0 * T * V)


@pytest.mark.parametrize("T,V", [(9, 1000), (300, 9000), (5, 60000), (3, 200000)])
def test_far_rows_in_place(K, T, V):
    """Rows that are summed again, beside near and masked ones: the gradient over bf16 logits is the one beside them."""
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn(T, V, device="cuda", generator=g) * 3
    z[::2] = z[::2] * 2000 + 2.0e5
    z = z.to(torch.bfloat16)
    lab = torch.randint(0, V, (T,), device="cuda", generator=g, dtype=torch.int32)
    lab[T // 2] = -1
    adv = torch.randn(T, device="cuda", generator=g)
    # advantages below 0 at a ratio of 1: no row is clipped
    old = K.token_logprobs(z, lab)[0]
    want = K.policy_loss(z, lab, old, -adv.abs())
    assert bool(torch.isfinite(want[3].float()).all()) and bool((want[3] != 0).any())
    got = K.policy_loss(z, lab, old, -adv.abs(), out=z)
    assert got[3] is z and all(torch.equal(a, b) for a, b in zip(want, got))
