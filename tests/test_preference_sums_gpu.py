"""Preference loss of long sequences: scores of thousands whose difference decides, against float64 of the same numbers.

Tolerances. Sums are held in pairs of floats, which are good to 2^-40 of the sums here, so that the difference of two
scores is rounded once, and h = beta (s_0 - s_1) - margin takes three roundings of numbers below |h| + margin: 4 *
2^-24 (|h| + 1). A mean divides each sum first, by a rounded reciprocal: 2 * 2^-24 of either mean. The loss (h -
1/2)^2 / beta^2 and its derivative are smooth in h; what is computed from h takes eight roundings more.
"""
import numpy as np
import pytest

from oracle import tune

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F = 2.0 ** -24


@pytest.fixture(scope="module")
def K():
    from host_memory_streamed_stream_gb300 import _build

    _build.build()
    from host_memory_streamed_stream_gb300 import kernels

    return kernels


def _dev(a, dtype=torch.float32):
    return torch.tensor(np.asarray(a), dtype=dtype).cuda()


# one launch for all of it, with several warps a sequence and with one, up to its largest; a block a pair
@pytest.mark.parametrize("lengths", [[2000, 2001], [250] * 16, [40] * 100, [30000, 30011], [2500] * 6, [128] * 32,
                                     [100] * 34, [0, 4096], [2048, 2049], [700] * 5 + [1]])
@pytest.mark.parametrize("ref,masked,average", [(False, False, False), (True, True, False), (True, False, True)])
def test_long_sums(K, lengths, ref, masked, average):
    rng = np.random.default_rng(len(lengths))
    bounds = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    T, n = int(bounds[-1]), len(lengths)
    logp = (-3 - 3 * rng.random(T)).astype(np.float32)
    rl = (-3 - 3 * rng.random(T)).astype(np.float32) if ref else None
    lab = np.where(rng.random(T) < 0.3, -1, 1).astype(np.int32) if masked else None
    beta, margin = 0.25, 0.125
    loss, rew, d = K.preference_loss(_dev(logp), _dev(bounds, torch.int32),
                                     labels=None if lab is None else _dev(lab, torch.int32),
                                     ref_logp=None if rl is None else _dev(rl), kind="square", beta=beta, margin=margin,
                                     average=average)
    x, r = logp.astype(np.float64), 0.0 if rl is None else rl.astype(np.float64)
    L, RW, D = tune.preference_loss(x, bounds, lab, r, kind="square", beta=beta, margin=margin, average=average)
    rew, d = (v.cpu().numpy().astype(np.float64) for v in (rew, d))
    assert np.all(np.abs(rew - RW) <= 4 * F * np.abs(RW))
    h = RW[0::2] - RW[1::2] - margin
    herr = 4 * F * (np.abs(h) + 1) + (2 * F * (np.abs(RW[0::2]) + np.abs(RW[1::2])) if average else 0.0)
    u = np.abs(h - 0.5) / beta
    lerr = 2 * u * herr / beta + (herr / beta) ** 2 + 8 * F * (u ** 2)
    assert abs(float(loss) - L) <= np.mean(lerr) + 2 * F * abs(L)
    derr = np.repeat(2 * herr / beta + 8 * F * 2 * u, 2) / (n // 2)
    each = np.concatenate([np.full(k, e) for k, e in zip(lengths, derr)])
    if average:
        on = np.ones(T, bool) if lab is None else lab >= 0
        each /= np.concatenate([np.full(k, max(1, on[a:a + k].sum())) for a, k in zip(bounds, lengths)])
    assert np.all(np.abs(d - D) <= each)
