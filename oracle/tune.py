"""The ends of a fine-tuning step in numpy float64: log-probabilities of given tokens, the policy and preference losses on
them, layer norm, and the embedding with a scale, each with its gradient."""
import numpy as np


def token_logprobs(z, labels, scale=1.0):
    """(logp, lse) of z [T, V]; rows with labels < 0 give 0."""
    y = np.asarray(z, np.float64) * scale
    on = labels >= 0
    with np.errstate(invalid="ignore", divide="ignore"):
        m = y.max(1)
        log_sum = np.log(np.exp(y - m[:, None]).sum(1))
        lse = m + log_sum
        logp = y[np.arange(len(y)), np.where(on, labels, 0)] - m - log_sum  # exact differences of far logits
    return np.where(on, logp, 0.0), np.where(on, lse, 0.0)


def token_logprobs_bwd(z, labels, dlogp, scale=1.0):
    y = np.asarray(z, np.float64) * scale
    y = y - y.max(1, keepdims=True)
    p = np.exp(y) / np.exp(y).sum(1, keepdims=True)
    hot = np.zeros_like(p)
    on = labels >= 0
    hot[on, labels[on]] = 1.0
    return np.where(on[:, None], (scale * dlogp)[:, None] * (hot - p), 0.0)


def policy_terms(logp, old, adv, ref=None, clip_low=0.2, clip_high=0.2, kl=0.0):
    """Each row's loss and its derivative by logp."""
    r = np.exp(logp - old)
    cut = np.clip(r, 1 - clip_low, 1 + clip_high)
    loss = -np.minimum(r * adv, cut * adv)
    d = np.where(r * adv > cut * adv, 0.0, -r * adv)
    if kl:
        far = ref - logp
        loss = loss + kl * (np.exp(far) - far - 1)
        d = d + kl * (1 - np.exp(far))
    return loss, d


def policy_loss(z, labels, old, adv, ref=None, weights=None, clip_low=0.2, clip_high=0.2, kl=0.0, scale=1.0):
    """(loss, row losses, logp, dlogits)"""
    logp, _ = token_logprobs(z, labels, scale)
    loss, d = policy_terms(logp, old, adv, ref, clip_low, clip_high, kl)
    w = np.where(labels >= 0, 1.0 / len(labels) if weights is None else weights, 0.0)
    return (w * loss).sum(), w * loss, logp, token_logprobs_bwd(z, labels, w * d, scale)


def preference_loss(logp, bounds, labels=None, ref=None, kind="sigmoid", beta=0.1, margin=0.0, smoothing=0.0,
                    average=False):
    """(loss, rewards, dlogp)"""
    n = len(bounds) - 1
    on = np.ones(len(logp), bool) if labels is None else labels >= 0
    term = np.where(on, logp - (0.0 if ref is None else ref), 0.0)
    s, share = np.zeros(n), np.ones(n)
    for j in range(n):
        rows = slice(bounds[j], bounds[j + 1])
        if average:
            share[j] = 1.0 / max(1, on[rows].sum())
        s[j] = term[rows].sum() * share[j]
    h = beta * (s[0::2] - s[1::2]) - margin
    if kind == "sigmoid":
        loss = (1 - smoothing) * np.logaddexp(0, -h) + smoothing * np.logaddexp(0, h)
        d = smoothing - np.exp(-np.logaddexp(0, h))
    elif kind == "hinge":
        loss, d = np.maximum(0, 1 - h), -(h < 1).astype(float)
    else:
        loss, d = ((h - 0.5) / beta) ** 2, 2 * (h - 0.5) / beta ** 2
    d = beta * d / len(h)
    dlogp = np.zeros(len(logp))
    for j in range(n):
        rows = slice(bounds[j], bounds[j + 1])
        dlogp[rows] = np.where(on[rows], (d[j // 2] if j % 2 == 0 else -d[j // 2]) * share[j], 0.0)
    return loss.mean(), beta * s, dlogp


def layernorm_fwd(x, gamma, beta=None, eps=1e-5):
    """(y, mean, rstd)"""
    mean = x.mean(1)
    rstd = 1 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None] * gamma
    return y if beta is None else y + beta, mean, rstd


def layernorm_bwd(dy, x, gamma, mean, rstd, dres=None):
    """(dx, dgamma, dbeta)"""
    n = (x - mean[:, None]) * rstd[:, None]
    u = dy * gamma
    dx = rstd[:, None] * (u - u.mean(1, keepdims=True) - n * (u * n).mean(1, keepdims=True))
    return dx if dres is None else dx + dres, (dy * n).sum(0), dy.sum(0)


def embed_lookup(tok, E, scale=1.0):
    on = (tok >= 0) & (tok < len(E))
    return np.where(on[:, None], E[np.where(on, tok, 0)] * scale, 0.0)


def embed_lookup_bwd(tok, dx, V, scale=1.0):
    dE = np.zeros((V, dx.shape[1]))
    on = (tok >= 0) & (tok < V)
    np.add.at(dE, tok[on], dx[on])
    return dE * scale
