"""The oracle of the fine-tuning operators against finite differences, and the entries' refusals (nothing is launched:
the pointers handed over are never read)."""
import numpy as np
import pytest

from oracle import tune


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


def _differences(f, x, g, rtol):
    """d f / d x by central differences of step 1e-6 (step^2 and 2^-53 / step), each against g."""
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + 1e-6
        up = f()
        x[i] = keep - 1e-6
        down = f()
        x[i] = keep
        assert abs((up - down) / 2e-6 - g[i]) < rtol, (i, g[i])


@pytest.mark.parametrize("kl", [0.0, 0.3])
@pytest.mark.parametrize("scale", [1.0, 1.7])
def test_policy_gradient(kl, scale):
    rng = np.random.default_rng(5)
    T, V = 9, 7
    z = rng.standard_normal((T, V))
    labels = rng.integers(0, V, T)
    labels[[2, 8]] = -1
    adv, w = rng.standard_normal(T), rng.random(T)
    logp, _ = tune.token_logprobs(z, labels, scale)
    old, ref = logp + 0.3 * rng.standard_normal(T), logp + 0.5 * rng.standard_normal(T)
    args = (labels, old, adv, ref, w, 0.2, 0.28, kl, scale)
    *_, d = tune.policy_loss(z, *args)
    held = np.exp(logp - old)
    assert (held > 1.28).any() and (held < 0.8).any()  # the clip is reached on both sides
    _differences(lambda: tune.policy_loss(z, *args)[0], z, d, 1e-8)


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "square"])
@pytest.mark.parametrize("average", [False, True])
def test_preference_gradient(kind, average):
    rng = np.random.default_rng(6)
    bounds = np.array([1, 4, 4, 9, 15])
    T = 17
    logp, ref = -rng.random(T) * 3, -rng.random(T) * 3
    labels = np.where(rng.random(T) < 0.3, -1, 1)
    kw = dict(bounds=bounds, labels=labels, ref=ref, kind=kind, beta=0.7, margin=0.2, average=average,
              smoothing=0.1 if kind == "sigmoid" else 0.0)
    loss, rewards, d = tune.preference_loss(logp, **kw)
    assert rewards[1] == 0.0 and (d[[0, 15, 16]] == 0).all() and (d[labels < 0] == 0).all()
    _differences(lambda: tune.preference_loss(logp, **kw)[0], logp, d, 1e-8)


def test_layernorm_gradient():
    rng = np.random.default_rng(7)
    x, gamma, beta, dy, dres = (rng.standard_normal(s) for s in ((3, 8), 8, 8, (3, 8), (3, 8)))

    def f():
        return float((tune.layernorm_fwd(x, gamma, beta)[0] * dy).sum() + (x * dres).sum())

    _, mean, rstd = tune.layernorm_fwd(x, gamma, beta)
    dx, dg, db = tune.layernorm_bwd(dy, x, gamma, mean, rstd, dres)
    for a, g in ((x, dx), (gamma, dg), (beta, db)):
        _differences(f, a, g, 1e-8)


def test_embedding_gradient():
    rng = np.random.default_rng(8)
    E, dx, tok = rng.standard_normal((5, 3)), rng.standard_normal((6, 3)), np.array([4, 0, -1, 4, 2, 7])
    dE = tune.embed_lookup_bwd(tok, dx, 5, 2.5)
    _differences(lambda: float((tune.embed_lookup(tok, E, 2.5) * dx).sum()), E, dE, 1e-8)


P, Q = 1 << 20, 1 << 24  # aligned addresses that nothing reads


def test_loss_refusals(lib):
    nan, inf = float("nan"), float("inf")

    def rows(z=P, type=1, ld=104, lab=P, logp=P, lse=P, T=4, V=101, scale=1.0, err=None):
        return lib.mtk_token_logprobs(z, type, ld, lab, logp, lse, T, V, scale, err, None)

    common = [dict(z=None), dict(z=P + 2), dict(z=P + 8), dict(type=2), dict(type=-1), dict(ld=96), dict(ld=101),
              dict(ld=108), dict(lab=None), dict(lab=P + 2), dict(T=0), dict(T=-1), dict(V=0), dict(V=105),
              dict(scale=0.0), dict(scale=-1.0), dict(scale=nan), dict(scale=inf), dict(scale=1e-20), dict(scale=2e19),
              dict(T=(1 << 30) + 1), dict(V=(1 << 28) + 1, ld=(1 << 28) + 8, ldd=(1 << 28) + 8)]
    for kw in common + [dict(logp=None), dict(lse=P + 1), dict(err=P + 1)]:
        assert rows(**{k: v for k, v in kw.items() if k != "ldd"}) == -1, kw

    def grad(z=P, type=1, ld=104, lab=P, lse=P, dlogp=P, d=Q, ldd=104, T=4, V=101, scale=1.0):
        return lib.mtk_token_logprobs_bwd(z, type, ld, lab, lse, dlogp, d, ldd, T, V, scale, None)

    out = [dict(d=None), dict(d=Q + 8), dict(ldd=96), dict(ldd=100), dict(d=P, ldd=112), dict(d=P, type=0),
           dict(d=P + 208), dict(d=P - 208), dict(d=P + 816)]
    for kw in common + out + [dict(lse=None), dict(dlogp=P + 3)]:
        assert grad(**kw) == -1, kw

    def policy(z=P, type=1, ld=104, lab=P, old=P, adv=P, ref=None, w=None, lo=0.2, hi=0.2, kl=0.0, scale=1.0, d=Q,
               ldd=104, logp=P, row=P, loss=P, T=4, V=101, err=None):
        return lib.mtk_policy_loss(z, type, ld, lab, old, adv, ref, w, lo, hi, kl, scale, d, ldd, logp, row, loss, T,
                                   V, err, None)

    for kw in common + out + [dict(old=None), dict(adv=P + 2), dict(ref=P + 2), dict(w=P + 1), dict(lo=-0.1),
                              dict(lo=1.1), dict(lo=nan), dict(hi=-0.1), dict(hi=inf), dict(kl=-1.0), dict(kl=nan),
                              dict(kl=0.1), dict(logp=None), dict(row=None), dict(loss=None), dict(err=P + 2)]:
        assert policy(**kw) == -1, kw

    def pref(logp=P, ref=None, lab=None, bounds=P, pairs=2, T=8, kind=0, beta=0.1, margin=0.0, smooth=0.0, pl=P,
             loss=P, rew=P, d=P):
        return lib.mtk_preference_loss(logp, ref, lab, bounds, pairs, T, kind, beta, margin, smooth, 0, pl, loss, rew,
                                       d, None)

    for kw in (dict(logp=None), dict(ref=P + 2), dict(lab=P + 2), dict(bounds=None), dict(pairs=0),
               dict(pairs=(1 << 20) + 1), dict(T=0), dict(T=(1 << 30) + 1), dict(kind=3), dict(kind=-1), dict(beta=0.0),
               dict(beta=inf),
               dict(margin=nan), dict(smooth=-0.1), dict(smooth=0.6), dict(smooth=nan), dict(pl=None), dict(loss=None),
               dict(rew=P + 2), dict(d=None)):
        assert pref(**kw) == -1, kw


def test_norm_and_embedding_refusals(lib):
    def fwd(x=P, type=0, ldx=64, g=P, b=None, y=Q, ldy=64, mean=P, rstd=P, T=4, h=64, eps=1e-5):
        return lib.mtk_layernorm_fwd(x, type, ldx, g, b, y, ldy, mean, rstd, T, h, eps, None)

    for kw in (dict(x=None), dict(x=P + 8), dict(type=3), dict(ldx=56), dict(ldx=68), dict(g=None), dict(g=P + 8),
               dict(b=P + 2), dict(y=None), dict(y=Q + 4), dict(ldy=60), dict(mean=None), dict(rstd=P + 2), dict(T=0),
               dict(T=(1 << 30) + 1),
               dict(h=0), dict(h=60), dict(h=16392, ldx=16392, ldy=16392), dict(eps=-1.0), dict(eps=float("nan")),
               dict(y=P), dict(y=P + 512)):
        assert fwd(**kw) == -1, kw

    R = 1 << 26

    def bwd(dy=P, dt=0, lddy=64, x=Q, type=0, ldx=64, g=P, mean=P, rstd=P, res=None, ldr=0, dx=R, dxb=None, part=P,
            dg=P, db=P, T=4, h=64):
        return lib.mtk_layernorm_bwd(dy, dt, lddy, x, type, ldx, g, mean, rstd, res, ldr, dx, dxb, part, dg, db, T, h,
                                     None)

    for kw in (dict(dy=None), dict(dt=2), dict(lddy=60), dict(x=None), dict(type=2), dict(ldx=32), dict(g=P + 4),
               dict(mean=None), dict(rstd=None), dict(res=P, ldr=60), dict(res=P + 4, ldr=64), dict(dx=None),
               dict(dx=R + 8), dict(dxb=R + 16384, type=1), dict(dxb=R + 64), dict(part=None), dict(part=P + 4),
               dict(dg=None), dict(db=P + 1), dict(T=0), dict(T=(1 << 30) + 1), dict(h=12), dict(dx=Q), dict(dx=P),
               dict(dx=P + 512),
               dict(res=R, ldr=72), dict(res=R + 256, ldr=64)):
        assert bwd(**kw) == -1, kw
    assert lib.mtk_layernorm_bwd_parts(0, 64) == 0 and lib.mtk_layernorm_bwd_parts(4, 60) == 0
    assert lib.mtk_layernorm_bwd_parts(4, 16392) == 0
    for T in (1, 5, 10000):
        for h in (8, 1160, 16384):
            assert 1 <= lib.mtk_layernorm_bwd_parts(T, h) <= T

    def look(tok=P, E=P, x=Q, type=0, T=4, h=64, V=100, scale=1.0, err=None):
        return lib.mtk_embed_lookup(tok, E, x, type, T, h, V, scale, err, None)

    common = [dict(tok=None), dict(tok=P + 2), dict(type=2), dict(T=0), dict(T=(1 << 26) + 1), dict(h=0), dict(h=60),
              dict(h=65544), dict(V=0), dict(V=(1 << 24) + 1), dict(scale=float("inf")), dict(err=P + 2)]
    for kw in common + [dict(E=None), dict(E=P + 8), dict(x=None), dict(x=Q + 8), dict(x=P), dict(x=P + 12784)]:
        assert look(**kw) == -1, kw

    def back(tok=P, dx=P, type=0, dE=Q, scratch=R, T=4, h=64, V=100, scale=1.0, err=None):
        return lib.mtk_embed_lookup_bwd(tok, dx, type, dE, scratch, T, h, V, scale, 0, err, None)

    for kw in common + [dict(dx=None), dict(dx=P + 8), dict(dE=None), dict(dE=Q + 2), dict(scratch=None),
                        dict(scratch=R + 8), dict(dE=P), dict(dx=Q + 12784), dict(scratch=Q), dict(scratch=P)]:
        assert back(**kw) == -1, kw
    assert lib.mtk_embed_lookup_bwd_scratch_bytes(0, 64) == 0
    assert lib.mtk_embed_lookup_bwd_scratch_bytes(4, 0) == 0


def test_binding_refusals(K):
    """The binding refuses what the C entry cannot see; a tensor that is not on the GPU is refused first."""
    import torch

    from host_memory_streamed_stream_gb300 import MTError

    z, lab, f = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    b = torch.zeros(3, dtype=torch.int32)
    g = torch.zeros(8, dtype=torch.bfloat16)
    for call in (lambda: K.token_logprobs(z, lab), lambda: K.token_logprobs(z[0], lab),
                 lambda: K.token_logprobs_bwd(z, lab, f, f), lambda: K.policy_loss(z, lab, f, f),
                 lambda: K.preference_loss(f, b), lambda: K.preference_loss(f, b, kind="other"),
                 lambda: K.layernorm_fwd(z, g), lambda: K.layernorm_bwd(z, z, g, f, f),
                 lambda: K.embed_lookup(lab, z.bfloat16()), lambda: K.embed_lookup_bwd(lab, z, 10)):
        with pytest.raises(MTError):
            call()
    K.check(torch.zeros(1, dtype=torch.int32))
    with pytest.raises(MTError, match="token"):
        K.check(torch.tensor([16], dtype=torch.int32))
