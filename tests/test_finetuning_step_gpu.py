"""Embedding, layer norm, the head's GEMM and the policy loss together, with ratios well away from the clip's borders:
every row falls on the side that it falls on in float64, and the loss is compared.

Tolerances. y is rounded to bf16 (2^-8 of its size, at most) and meets W in a sum of h products, whose error has a
deviation below sqrt(h) 2^-8 / 2 |y| |W| = D; over all T V logits the largest of them stays below 6 D, in lse as well,
and logp has two of them: 12 D. A row's loss is A r (held: A times the border): it errs by exp(12 D) - 1 of its size.
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


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("kl", [0.0, 0.05])
def test_loss_of_a_step(K, kl):
    rng = np.random.default_rng(8)
    T, h, V, size = 320, 128, 1000, 0.1

    def bf16(*shape, scale=1.0):
        return torch.tensor(rng.standard_normal(shape) * scale, dtype=torch.float32).bfloat16().cuda()

    E, W, b = bf16(V, h, scale=0.5), bf16(V, h, scale=size), bf16(h, scale=0.2)
    G = bf16(h, scale=0.1) + 1
    tok = rng.integers(-1, V, T).astype(np.int32)
    lab = rng.integers(0, V, T).astype(np.int32)
    lab[rng.random(T) < 0.2] = -1
    x = tune.embed_lookup(tok, _np(E), 4.0)
    y = tune.layernorm_fwd(x, _np(G), _np(b))[0]
    z = y @ _np(W).T
    logp = tune.token_logprobs(z, lab)[0]
    on = lab >= 0
    # ratios on either side of 0.8 and 1.3, none nearer than 0.1 in their logarithm
    ratio = rng.choice([0.5, 0.7, 0.95, 1.0, 1.1, 1.5, 2.0], T)
    old = (logp - np.log(ratio)).astype(np.float32)
    ref = (logp + 0.3 * rng.standard_normal(T)).astype(np.float32)
    adv = rng.standard_normal(T).astype(np.float32)
    room = 12 * np.sqrt(h) * 2.0 ** -9 * np.abs(y).mean() * size
    r = np.exp(logp - old)[on]
    assert min(np.abs(np.log(r / 0.8)).min(), np.abs(np.log(r / 1.3)).min()) > 3 * room
    L, R, _, _ = tune.policy_loss(z, lab, old, adv, ref if kl else None, None, 0.2, 0.3, kl)

    tt, lt = torch.tensor(tok).cuda(), torch.tensor(lab).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    X = K.embed_lookup(tt, E, scale=4.0, err=err)
    Y = K.layernorm_fwd(X, G, b)[0]
    Z = K.gemm(Y, False, W, False, T, V, h, epi=K.EPI_STORE_F32, err=err)
    loss, row, lp, _ = K.policy_loss(Z, lt, torch.tensor(old).cuda(), torch.tensor(adv).cuda(),
                                     ref_logp=torch.tensor(ref).cuda() if kl else None, clip_low=0.2, clip_high=0.3,
                                     kl=kl, err=err)
    K.check(err)
    assert np.all(np.abs(_np(lp) - logp)[on] <= room)
    far = np.abs(ref - logp)
    terr = (np.maximum(ratio, 1.3) * np.abs(adv) + kl * (np.exp(far) + far)) * (np.exp(room) - 1) / T * on
    assert np.all(np.abs(_np(row) - R) <= terr + 1e-12)
    assert abs(float(loss) - L) <= terr.sum()
    assert abs(L) > 3 * terr.sum()  # so that another loss would be seen
