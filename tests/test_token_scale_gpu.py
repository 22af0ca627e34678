"""Log-probabilities and the policy loss with -inf among the logits, at scales where the rounded scale * log2(e) has
no bits beyond its twelfth, against float64.

Tolerances. Each term 2^(c z - max) has a rounded factor and exponent (2^-24 of |a z - lse| each, 2 R, R the largest
|a z - lse| of the row) and the exponential's own error (2^-22); a sum of at most V / 128 + 16 terms in a chain, 2^-24
each: lse is within L = 2^-24 (2 R + 20 + V / 128). fp32 results add half a step (2^-24), bf16 ones 2^-8; p has twice L,
lse's rounding and change of base (3 * 2^-24 |lse|) and eight roundings.
"""
import numpy as np
import pytest

from oracle import tune

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF, F = 2.0 ** -8, 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
TEMPERATURES = [0.4831, 0.9662, 1.0349, 1.9324, 2.0698, 7.343, 1 / 1.6381017, 4151 ** 0.5, 1.0, 0.7]


@pytest.fixture(scope="module")
def K():
    from host_memory_streamed_stream_gb300 import _build

    _build.build()
    from host_memory_streamed_stream_gb300 import kernels

    return kernels


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _dev(a, dtype=torch.float32):
    return torch.tensor(np.asarray(a), dtype=dtype).cuda()


# a warp a row, a block a row, and clusters: few rows, and rows wider than a block's share
@pytest.mark.parametrize("T,V", [(7, 1021), (200, 9001), (3, 60001), (160, 90003)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_banned_columns_at_any_scale(K, T, V, kind):
    rng = np.random.default_rng(V)
    z = torch.zeros(T, (V + 7) // 8 * 8, dtype=TYPES[kind], device="cuda")[:, :V]
    z[:] = torch.randn(T, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(V)) * 3
    z[:, V - 5:] = -float("inf")  # a ragged end of padding columns
    z[::2, 1::3] = -float("inf")
    z[T - 1, 1:] = -float("inf")  # the label alone is left
    lab = (rng.integers(0, (V - 5) // 3, T) * 3).astype(np.int32)
    lab[0], lab[T - 1] = -1, 0
    lt, on, at = _dev(lab, torch.int32), lab >= 0, np.arange(T)
    x = _np(z)
    adv = rng.standard_normal(T).astype(np.float32)
    for temperature in TEMPERATURES:
        a = float(np.float32(1 / temperature))
        rl, rs = tune.token_logprobs(x, lab, a)
        y = np.where(np.isfinite(x), x, x[at, np.maximum(lab, 0)][:, None]) * a
        tol = F * (2 * np.abs(y - rs[:, None]).max(1) + 20 + V / 128)
        logp, lse = K.token_logprobs(z, lt, scale=a)
        assert np.all(np.abs(_np(logp) - rl) <= np.where(on, tol + F * np.abs(rl), 0)), temperature
        assert np.all(np.abs(_np(lse) - rs) <= np.where(on, tol + F * np.abs(rs), 0)), temperature
        # p of columns beside the label's at their full size: dlogp of 1
        d = _np(K.token_logprobs_bwd(z, lt, lse, torch.ones(T, device="cuda"), scale=a))
        ref = tune.token_logprobs_bwd(x, lab, np.ones(T), a)
        rel = (2 * tol + 3 * F * np.abs(rs) + 8 * F)[:, None]
        p = np.exp(x * a - rs[:, None])
        assert np.all(np.abs(d - ref) <= HALF * np.abs(ref) + a * (p * rel + 2 * F) * on[:, None]), temperature
        old = (rl + 0.05).astype(np.float32)  # inside the clip
        loss, row, lp, g = K.policy_loss(z, lt, _dev(old), _dev(adv), scale=a)
        L, R, _, D = tune.policy_loss(x, lab, old, adv, scale=a)
        size = np.abs(adv) / T * np.exp(rl - old) * on
        assert np.all(np.abs(_np(lp) - rl) <= np.where(on, tol + F * np.abs(rl), 0)), temperature
        assert np.all(np.abs(_np(row) - R) <= size * (tol + F * np.abs(rl) + 8 * F)), temperature
        assert abs(float(loss) - L) <= np.sum(size * (tol + F * np.abs(rl) + 9 * F)) + F * abs(L), temperature
        room = (a * size * (2 * tol + F * np.abs(rl) + 16 * F))[:, None]
        assert np.all(np.abs(_np(g) - D) <= HALF * np.abs(D) * (1 + HALF) + 2 * room + 1e-38), temperature
