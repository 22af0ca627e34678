"""The policy loss where a ratio or a KL term passes the range of fp32: rows that weigh nothing or have no advantage
add nothing, as in float64, where the exponential is finite.

Tolerances as for near rows: logp is within 2^-24 (2 R + 20 + V / 128) with R <= 16 here, which exp and a few
roundings pass on: 1e-4 of a row's size bounds it; bf16 gradients add 2^-8.
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


def _dev(a):
    return torch.tensor(np.asarray(a, np.float32)).cuda()


@pytest.mark.parametrize("V", [72, 5000, 40000])
@pytest.mark.parametrize("kl", [0.0, 0.1])
def test_rows_that_count_nothing(K, V, kl):
    rng = np.random.default_rng(V)
    T = 8
    z = rng.standard_normal((T, V)).astype(np.float32)
    lab = rng.integers(0, V, T).astype(np.int32)
    logp, _ = tune.token_logprobs(z, lab)
    old = (logp + 0.05).astype(np.float32)
    ref = (logp - 0.1).astype(np.float32)
    adv, w = rng.standard_normal(T).astype(np.float32), rng.random(T).astype(np.float32)
    old[:4] = -150.0              # a ratio of e^140
    adv[0], adv[1] = 0.0, 2.0     # no advantage; one whose clip holds
    w[2:5], adv[2], adv[3] = 0.0, -3.0, 3.0
    if kl:
        ref[4] = 200.0
    loss, row, lp, d = K.policy_loss(_dev(z), torch.tensor(lab).cuda(), _dev(old), _dev(adv),
                                     ref_logp=_dev(ref) if kl else None, weights=_dev(w), kl=kl)
    L, R, _, D = tune.policy_loss(z, lab, old, adv, ref if kl else None, w.astype(np.float64), kl=kl)
    row, d = row.cpu().numpy().astype(np.float64), d.float().cpu().numpy().astype(np.float64)
    assert np.all(row[2:5] == 0) and np.all(d[2:5] == 0)
    size = np.abs(w) * (1.3 * np.abs(adv) + kl * 3)
    assert np.all(np.abs(row - R) <= 1e-4 * size) and abs(float(loss) - L) <= 1e-4 * size.sum()
    assert np.all(np.abs(d - D) <= 2.0 ** -8 * np.abs(D) + 1e-4 * size[:, None])


def test_what_is_beyond_stays_beyond(K):
    """A weighted loss of that size is as large as fp32 holds, and NaN is not hidden by a weight of 0."""
    z = torch.zeros(3, 64, device="cuda")
    z[2, 5] = float("nan")
    lab = torch.tensor([1, 1, 1], dtype=torch.int32).cuda()
    loss, row, _, d = K.policy_loss(z, lab, _dev([-150, -4, -4]), _dev([-2, 1, 1]), weights=_dev([1, 1, 0]))
    assert float(row[0]) > 3e38 and bool(torch.isnan(row[2])) and bool(torch.isnan(d[2]).all())
    assert bool(torch.isfinite(row[1])) and bool(torch.isnan(loss))
