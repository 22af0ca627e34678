"""Log-probabilities of given tokens and the losses on them, against float64.

Tolerances. A bf16 result is off by half a step at most (2^-8 of its size). A row's lse: each term 2^(c z - max) has a
rounded factor c and a rounded exponent (2^-24 of |a z - lse| each, 2 R) and the exponential's own error (2^-22), and
the sum is of at most V / 128 + 16 terms in a chain, 2^-24 each: LSE(V, R) = 2^-24 (2 R + 4 + V / 128 + 16), R the
largest |a z - lse| that matters, bounded by the largest |a z - lse| of the row. A result adds half a step of its own,
2^-24.
"""
import numpy as np
import pytest

from oracle import tune

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF, F = 2.0 ** -8, 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


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


def _logits(rng, T, V, kind, pad=8, size=3.0, banned=0):
    """Rows inside a buffer with other columns (NaN) behind them."""
    ld = (V + 7) // 8 * 8 + pad
    buf = torch.full((T, ld), float("nan"), dtype=TYPES[kind], device="cuda")
    buf[:, :V] = _dev(rng.standard_normal((T, V)) * size).to(TYPES[kind])
    if banned:
        buf[:, V - banned:V] = -float("inf")
    return buf[:, :V]


def _labels(rng, T, V, masked=0.3):
    lab = rng.integers(0, V, T).astype(np.int32)
    lab[rng.random(T) < masked] = -1
    return lab


def _lse_tol(z, labels, scale, lse):
    y = np.where(np.isfinite(z), z, 0) * scale
    R = np.abs(y - lse[:, None]).max(1)
    return F * (2 * R + 4 + z.shape[1] / 128 + 16)


SIZES = [(1, 1), (3, 5), (1, 64), (7, 1021), (5, 1024), (40, 4096), (9, 8200), (6, 32003), (4, 50001), (3, 152064),
         (2, 262147), (300, 257)]


@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_logprobs_and_gradient(K, T, V, kind):
    rng = np.random.default_rng(T * 7 + V)
    scale = 1.0 if V % 2 else 1.4
    z = _logits(rng, T, V, kind, banned=2 if V > 100 else 0)
    lab = _labels(rng, T, V - (2 if V > 100 else 0))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    logp, lse = K.token_logprobs(z, _dev(lab, torch.int32), scale=scale, err=err)
    x = _np(z)
    rl, rs = tune.token_logprobs(x, lab, scale)
    tol = _lse_tol(x, lab, scale, rs)
    on = lab >= 0
    assert np.all(np.abs(_np(lse) - rs)[on] <= (tol + F * np.abs(rs))[on])
    assert np.all(np.abs(_np(logp) - rl)[on] <= (tol + F * np.abs(rl))[on])
    assert np.all(_np(logp)[~on] == 0) and np.all(_np(lse)[~on] == 0)
    dlogp = rng.standard_normal(T).astype(np.float32)
    out = torch.full((T, z.stride(0) if T > 1 else (V + 7) // 8 * 8 + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    d = K.token_logprobs_bwd(z, _dev(lab, torch.int32), lse, _dev(dlogp), scale=scale, out=out[:, :V])
    ref = tune.token_logprobs_bwd(x, lab, dlogp, scale)
    # p has lse's error, its rounding and its change of base (2^-24 |lse| each), and its own exponential's
    k = np.abs(scale * dlogp)[:, None]
    p = np.exp(np.where(on[:, None], x * scale - rs[:, None], -np.inf))
    rel = (2 * tol + 3 * F * np.abs(rs) + 8 * F)[:, None]
    assert np.all(np.abs(_np(d) - ref) <= HALF * np.abs(ref) + k * (p * rel + 2 * F * (np.abs(ref) > 0)) + 1e-38)
    assert torch.all(out[:, V:] == 7.0)
    assert int(err.item()) == 0
    fresh = K.token_logprobs_bwd(z, _dev(lab, torch.int32), lse, _dev(dlogp), scale=scale)
    assert torch.equal(fresh, d)
    if kind == "bf16":  # in place, the columns behind the rows as they were
        z2 = torch.full_like(out, 5.0)
        z2[:, :V] = z
        K.token_logprobs_bwd(z2[:, :V], _dev(lab, torch.int32), lse, _dev(dlogp), scale=scale, out=z2[:, :V])
        assert torch.equal(z2[:, :V], d) and torch.all(z2[:, V:] == 5.0)


def _policy_inputs(rng, T, logp):
    old = (logp + 0.3 * rng.standard_normal(T)).astype(np.float32)
    # away from the clip's borders, where the gradient jumps
    for b in (0.8, 1.28):
        old = np.where(np.abs(np.exp(logp - old) - b) < 1e-3, old + np.float32(0.01), old).astype(np.float32)
    adv = rng.standard_normal(T).astype(np.float32)
    ref = (logp + 0.5 * rng.standard_normal(T)).astype(np.float32)
    w = rng.random(T).astype(np.float32)
    return old, adv, ref, w


@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("kl,weighted", [(0.0, False), (0.2, True)])
def test_policy(K, T, V, kind, kl, weighted):
    rng = np.random.default_rng(T * 5 + V)
    scale = 1.0 if V % 2 else 1.4
    banned = 2 if V > 100 else 0
    z = _logits(rng, T, V, kind, banned=banned)
    lab = _labels(rng, T, V - banned)
    x = _np(z)
    rl, rs = tune.token_logprobs(x, lab, scale)
    old, adv, ref, w = _policy_inputs(rng, T, rl)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((T, (V + 7) // 8 * 8 + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    args = [_dev(lab, torch.int32), _dev(old), _dev(adv)]
    kw = dict(ref_logp=_dev(ref) if kl else None, weights=_dev(w) if weighted else None, clip_low=0.2, clip_high=0.28,
              kl=kl, scale=scale, err=err)
    loss, row, logp, d = K.policy_loss(z, *args, out=out[:, :V], **kw)
    wr = w.astype(np.float64) if weighted else np.full(T, 1 / T)
    L, R, _, D = tune.policy_loss(x, lab, old, adv, ref if kl else None, wr, 0.2, 0.28, kl, scale)
    on = lab >= 0
    tol = _lse_tol(x, lab, scale, rs) + F * np.abs(rl)  # of logp, and so of log r and log(ref / p)
    assert np.all(np.abs(_np(logp) - rl)[on] <= tol[on]) and np.all(_np(logp)[~on] == 0)
    r = np.where(on, np.exp(rl - old), 0)
    q = np.where(on, np.exp(ref - rl), 0) if kl else np.zeros(T)
    far = np.abs(np.where(on, ref - rl, 0)) if kl else np.zeros(T)
    # exp of a sum with error tol, a few roundings after it; the KL term's parts are of the sizes q, 1 and |far|
    terr = np.abs(wr) * ((np.maximum(r, 1.3) * np.abs(adv)) * (tol + 8 * F) + kl * (q + 1 + far) * (tol + 8 * F))
    assert np.all(np.abs(_np(row) - R) <= terr + F * np.abs(R))
    assert abs(float(loss) - L) <= np.sum(terr) + F * (np.abs(R).sum() + abs(L))
    kerr = scale * np.abs(wr) * (r * np.abs(adv) * (tol + 8 * F) + kl * (q + 1) * (tol + 8 * F))
    perr = np.abs(D) * (tol[:, None] + 8 * F)
    assert np.all(np.abs(_np(d) - D) <= HALF * np.abs(D) * (1 + HALF) + 2 * kerr[:, None] + perr + 1e-38)
    assert np.all(_np(d)[~on] == 0) and torch.all(out[:, V:] == 7.0) and int(err.item()) == 0
    if T > 1:  # the fixed order: the same bits again
        again = K.policy_loss(z, *args, **kw)
        assert torch.equal(again[0], loss) and torch.equal(again[3], d)
    if kind == "bf16":
        z2 = torch.full_like(out, 5.0)
        z2[:, :V] = z
        K.policy_loss(z2[:, :V], *args, out=z2[:, :V], **kw)
        assert torch.equal(z2[:, :V], d) and torch.all(z2[:, V:] == 5.0)


def test_many_rows(K):
    """More rows than a launch has blocks at a time, of one vector each and a ragged end, most of them masked."""
    rng = np.random.default_rng(9)
    T, V = 70001, 13
    z = _logits(rng, T, V, "f32", pad=0)
    lab = _labels(rng, T, V, masked=0.6)
    lt = _dev(lab, torch.int32)
    x = _np(z)
    rl, rs = tune.token_logprobs(x, lab)
    logp, lse = K.token_logprobs(z, lt)
    on = lab >= 0
    tol = _lse_tol(x, lab, 1.0, rs) + F * np.abs(rl)
    assert np.all(np.abs(_np(logp) - rl)[on] <= tol[on])
    w = rng.standard_normal(T).astype(np.float32)
    d = _np(K.token_logprobs_bwd(z, lt, lse, _dev(w)))
    ref = tune.token_logprobs_bwd(x, lab, w)
    assert np.all(np.abs(d - ref) <= HALF * np.abs(ref) + np.abs(w)[:, None] * (2 * tol + 16 * F)[:, None])
    loss, row, lp, dl = K.policy_loss(z, lt, logp, _dev(w))
    assert torch.equal(lp, logp)
    assert torch.all(dl[~torch.tensor(on).cuda()] == 0)
    # at ratio 1 neither side of the clip holds: the gradient is that of -A logp / T
    want = tune.token_logprobs_bwd(x, lab, -w.astype(np.float64) / T)
    room = (np.abs(w) / T * (4 * tol + 32 * F))[:, None]
    assert np.all(np.abs(_np(dl) - want) <= HALF * np.abs(want) + room)


@pytest.mark.parametrize("V", [40, 2000, 33000, 152064])
def test_values_at_the_ends(K, V):
    """-inf columns, a label on one, a row of nothing else, the type's largest values, NaN; NaN in masked rows."""
    inf, big = float("inf"), 3.0e38
    z = torch.zeros(8, V, dtype=torch.float32, device="cuda")
    z[0, :-1] = -inf                      # the label alone is left
    z[1, 5] = -inf                        # the label cannot be
    z[2] = -inf
    z[3] = -big
    z[4, V // 2] = big                    # far above all others
    z[5, 7] = float("nan")
    z[6] = float("nan")                   # masked
    z[7, ::2] = -big
    lab = _dev([V - 1, 5, 3, 3, V // 2, 1, -1, 1], torch.int32)
    for zz in (z, z.bfloat16()):
        logp, lse = K.token_logprobs(zz, lab)
        a = logp.cpu().tolist()
        assert a[0] == 0.0 and a[1] == -inf and a[2] != a[2] and a[4] == 0.0 and a[5] != a[5] and a[6] == 0.0
        assert abs(a[7] + np.log(V // 2)) < 1e-5
        # -big * log2(e) is -inf in fp32: a row of nothing but the lowest values counts as one of -inf
        assert a[3] != a[3] or abs(a[3] + np.log(V)) < 1e-5
        one = torch.ones(8, device="cuda")
        d = K.token_logprobs_bwd(zz, lab, lse, one)
        assert torch.all(d[0] == 0) and torch.all(d[4] == 0) and torch.all(d[6] == 0)
        assert float(d[7, 0]) == 0.0 and abs(float(d[7, 1]) - 1 + 1 / (V // 2)) < 0.01
        loss, row, lp, g = K.policy_loss(zz, lab, torch.zeros(8, device="cuda"), one)
        assert torch.all(g[0] == 0) and torch.all(g[6] == 0) and float(row[6]) == 0.0
        assert bool(torch.isnan(row[5])) and bool(torch.isnan(g[5]).all()) and bool(torch.isnan(loss))
        # ratio 0 for the impossible label: nothing to gain, no gradient through it
        assert float(row[1]) == 0.0


@pytest.mark.parametrize("V", [72, 5000, 40000, 170000])
@pytest.mark.parametrize("T", [3, 200])
def test_far_logits(K, V, T):
    """Logits far from 0, where c z loses its fraction: rows of nothing but a mask's value, equal huge ones, a mask
    beside ordinary ones, an offset that leaves the fp32 logits 2^-8. Against float64 of the same fp32 values: with the
    largest logit subtracted first, what remains is the tolerance of near rows."""
    rng = np.random.default_rng(V + T)
    z = torch.tensor(rng.standard_normal((T, V)), dtype=torch.float32).cuda()
    z[0] = -1.0e9
    z[1] = 3.0e12
    z[1, ::3] = 2.9e12
    z[2, :] += 60000.0
    if T > 3:
        z[3, 5:] = -1.0e9
        z[4] -= 1.0e5
        z[5] *= 3.0e4
    lab = (np.arange(T) % 5).astype(np.int32)
    lab[1] = 1
    lt = _dev(lab, torch.int32)
    x = _np(z)
    rl, rs = tune.token_logprobs(x, lab)
    logp, lse = K.token_logprobs(z, lt)
    spread = np.where(np.abs(x - x.max(1, keepdims=True)) < 100, np.abs(x - rs[:, None]), 0).max(1)
    # a rounded factor on distances up to |z - max| <= 100 (beyond, a term is 0), the row's size in lse itself
    tol = F * (2 * (spread + 110) + 4 + V / 128 + 16)
    assert np.all(np.abs(_np(logp) - rl) <= tol + 2 * F * np.abs(rl))
    assert np.all(np.abs(_np(lse) - rs) <= tol + F * np.abs(rs))
    adv = rng.standard_normal(T).astype(np.float32)
    old = _dev(rl + 0.01)
    loss, row, lp, d = K.policy_loss(z, lt, old, _dev(adv))
    ref = tune.policy_loss(x, lab, _np(old), adv)[3]
    k = np.abs(adv / T * np.exp(rl - _np(old)))[:, None]
    room = k * (2 * tol + 3 * F * np.abs(rl) + 16 * F)[:, None]
    assert np.all(np.abs(_np(lp) - rl) <= tol + 2 * F * np.abs(rl))  # summed over other blocks than logp
    assert np.all(np.abs(_np(d) - ref) <= HALF * np.abs(ref) + 2 * room + 1e-38)


def test_preference_of_impossible_tokens(K):
    """A rejected answer with a token of probability 0: nothing left to gain; a preferred one: an infinite loss."""
    inf = float("inf")
    b = _dev([0, 2, 4], torch.int32)
    for pad in (0, 5000):  # both forms of the kernel
        tail = [0.0] * pad
        for kind in ("sigmoid", "hinge"):
            loss, rew, d = K.preference_loss(_dev([-1.0, -2.0, -inf, -1.0] + tail), b, kind=kind)
            assert float(loss) == 0.0 and float(rew[1]) == -inf and torch.all(d == 0)
            loss, _, d = K.preference_loss(_dev([-1.0, -inf, -2.0, -1.0] + tail), b, kind=kind, beta=0.5)
            assert float(loss) == inf and d[:4].tolist() == [-0.5, -0.5, 0.5, 0.5]
            loss, _, d = K.preference_loss(_dev([-1.0, float("nan"), -2.0, -1.0] + tail), b, kind=kind)
            assert bool(torch.isnan(loss)) and bool(torch.isnan(d[:4]).all())


def test_label_outside_the_vocabulary(K):
    from host_memory_streamed_stream_gb300 import MTError

    rng = np.random.default_rng(1)
    z = _logits(rng, 4, 100, "f32")
    lab = _dev([3, 100, 2 ** 31 - 1, -2 ** 31], torch.int32)
    one = torch.ones(4, device="cuda")
    for call in (lambda e: K.token_logprobs(z, lab, err=e), lambda e: K.policy_loss(z, lab, one, one, err=e)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = call(err)
        with pytest.raises(MTError, match="token"):
            K.check(err)
        assert torch.all((out[0] if len(out) == 2 else out[2])[1:] == 0)
        if len(out) == 4:
            assert torch.all(out[3][1:] == 0)
        waits = torch.full((1,), 5, dtype=torch.int32, device="cuda")  # another code stays
        call(waits)
        assert int(waits.item()) == 5
        call(None)
    lse = torch.zeros(4, device="cuda")
    assert torch.all(K.token_logprobs_bwd(z, lab, lse, one)[1:] == 0)


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "square"])
@pytest.mark.parametrize("average,ref,masked", [(False, True, True), (True, False, True), (True, True, False)])
@pytest.mark.parametrize("lengths,first,tail", [([1, 1], 0, 0), ([5, 0, 0, 0, 300, 700], 3, 11), ([4000, 3500], 0, 1),
                                                ([17] * 90, 2, 0)])
def test_preference(K, kind, average, ref, masked, lengths, first, tail):
    rng = np.random.default_rng(len(lengths) + first)
    bounds = np.concatenate([[first], first + np.cumsum(lengths)]).astype(np.int32)
    T = int(bounds[-1]) + tail
    logp = (-3 * rng.random(T)).astype(np.float32)
    rl = (-3 * rng.random(T)).astype(np.float32) if ref else None
    lab = _labels(rng, T, 50) if masked else None
    kw = dict(kind=kind, beta=0.3, margin=0.1, smoothing=0.1 if kind == "sigmoid" else 0.0, average=average)
    loss, rew, d = K.preference_loss(_dev(logp), _dev(bounds, torch.int32),
                                     labels=None if lab is None else _dev(lab, torch.int32),
                                     ref_logp=None if rl is None else _dev(rl), **kw)
    L, RW, D = tune.preference_loss(logp.astype(np.float64), bounds, lab, rl, **kw)
    # a score: differences of numbers up to 3 and a chain of T / 512 + 32 additions of the running sums' size
    n = len(lengths)
    size = np.array([3.0 * max(1, k) for k in lengths])
    share = 1 / np.maximum(1, np.array(lengths) * 0.4) if average else np.ones(n)
    serr = F * size * (T / 512 + 34) * share
    assert np.all(np.abs(_np(rew) - RW) <= 0.3 * serr + 2 * F * np.abs(RW))
    herr = 0.3 * (serr[0::2] + serr[1::2]) + 4 * F * (1 + np.abs(RW[0::2]) + np.abs(RW[1::2]))
    h = RW[0::2] - RW[1::2] - 0.1
    steep = {"sigmoid": 1.0, "hinge": 1.0, "square": (2 * np.abs(h) + 1) / 0.09}[kind]
    assert abs(float(loss) - L) <= np.mean(steep * herr) + 16 * F * (1 + abs(L))
    curve = {"sigmoid": 0.25, "hinge": 0.0, "square": 2 / 0.09}[kind]
    derr = 0.3 / (n // 2) * (curve * herr + 16 * F * steep)
    each = np.zeros(T)
    for j in range(n):
        each[bounds[j]:bounds[j + 1]] = derr[j // 2] * share[j]
    assert np.all(np.abs(_np(d) - D) <= each + 1e-38)
    assert np.all(_np(d)[:first] == 0) and np.all(_np(d)[int(bounds[-1]):] == 0)


def test_preference_far_from_the_border(K):
    """Margins of hundreds: the loss is linear or 0, nothing overflows."""
    for h in (300.0, -300.0):
        logp = _dev([h, 0.0])
        loss, rew, d = K.preference_loss(logp, _dev([0, 1, 2], torch.int32), beta=1.0)
        assert abs(float(loss) - max(0.0, -h)) <= 1e-4 and float(rew[0]) == h
        assert float(d[0]) == (0.0 if h > 0 else -1.0) and float(d[1]) == -float(d[0])


def test_preference_step(K):
    """Log-probabilities, loss and gradient of the logits together, as a step uses them, on a stream of its own and
    captured into a graph that is replayed with other logits."""
    rng = np.random.default_rng(11)
    lengths, V, kind = [30, 41, 0, 25], 1003, "bf16"
    bounds = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    T = int(bounds[-1]) + 6
    z = _logits(rng, T, V, kind)
    lab = _labels(rng, T, V)
    rl = (-7 - rng.random(T)).astype(np.float32)
    lt, bt, rt = _dev(lab, torch.int32), _dev(bounds, torch.int32), _dev(rl)

    def step():
        logp, lse = K.token_logprobs(z, lt)
        loss, rew, dlogp = K.preference_loss(logp, bt, labels=lt, ref_logp=rt, beta=0.2)
        return loss, rew, K.token_logprobs_bwd(z, lt, lse, dlogp)

    def check(out):
        x = _np(z)
        logp, _ = tune.token_logprobs(x, lab)
        L, RW, D = tune.preference_loss(logp, bounds, lab, rl, beta=0.2)
        D = tune.token_logprobs_bwd(x, lab, D)
        # sums of 41 terms of size 10, each off by 2^-19 at most
        assert abs(float(out[0]) - L) <= 1e-4 and np.all(np.abs(_np(out[1]) - RW) <= 1e-4)
        assert np.all(np.abs(_np(out[2]) - D) <= HALF * np.abs(D) + 1e-4 * np.abs(D).max() + 1e-38)
        # rows behind the last sequence (logp of a label there is no part of the loss)
        assert torch.all(out[2][int(bounds[-1]):] == 0)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        check(step())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(2):
        z.copy_(_dev(rng.standard_normal((T, V)) * 2).to(z.dtype))
        graph.replay()
        torch.cuda.synchronize()
        check(held)


@pytest.mark.parametrize("T,V", [(5, 60000), (170, 40000), (3, 170000)])
def test_wide_rows_in_a_graph(K, T, V):
    """Rows split over clusters, captured and replayed with other logits and labels: what an eager call gives."""
    rng = np.random.default_rng(T)
    z = _logits(rng, T, V, "bf16")
    lab = _dev(_labels(rng, T, V), torch.int32)
    old, adv = _dev(rng.standard_normal(T) - 11), _dev(rng.standard_normal(T))
    K.policy_loss(z, lab, old, adv)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = K.policy_loss(z, lab, old, adv)
        logp, lse = K.token_logprobs(z, lab)
        grad = K.token_logprobs_bwd(z, lab, lse, adv)
    for _ in range(2):
        z.copy_(_dev(rng.standard_normal((T, V)) * 2).to(z.dtype))
        lab.copy_(_dev(_labels(rng, T, V), torch.int32))
        adv.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, K.policy_loss(z, lab, old, adv)))
        again = K.token_logprobs(z, lab)
        assert torch.equal(again[0], logp) and torch.equal(again[1], lse)
        assert torch.equal(K.token_logprobs_bwd(z, lab, lse, adv), grad)


def test_two_calls_at_once(K):
    """Policy losses of different sizes on two streams at the same time give what they give alone."""
    rng = np.random.default_rng(12)
    sets = []
    for T, V in ((300, 32000), (500, 9001)):
        z = _logits(rng, T, V, "f32")
        lab = _dev(_labels(rng, T, V), torch.int32)
        sets.append((z, lab, _dev(rng.standard_normal(T) - 9), _dev(rng.standard_normal(T))))
    want = [K.policy_loss(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(K.policy_loss(*s))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_refusals(K):
    from host_memory_streamed_stream_gb300 import MTError

    z = torch.zeros(4, 64, device="cuda")
    lab = torch.zeros(4, dtype=torch.int32, device="cuda")
    f = torch.zeros(4, device="cuda")
    b = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    bad = [lambda: K.token_logprobs(z.double(), lab), lambda: K.token_logprobs(z.half(), lab),
           lambda: K.token_logprobs(z.t(), lab), lambda: K.token_logprobs(z, lab.long()),
           lambda: K.token_logprobs(z, lab[:3]), lambda: K.token_logprobs(z, lab.cpu()),
           lambda: K.token_logprobs(z[:, :63].contiguous(), lab), lambda: K.token_logprobs(z[:, 1:], lab),
           lambda: K.token_logprobs(z, lab, scale=0.0), lambda: K.token_logprobs(z, lab, err=f),
           lambda: K.token_logprobs_bwd(z, lab, f, f.double()), lambda: K.token_logprobs_bwd(z, lab, f[:3], f),
           lambda: K.token_logprobs_bwd(z, lab, f, f, out=z), lambda: K.token_logprobs_bwd(z, lab, f, f, out=z[:3]),
           lambda: K.policy_loss(z, lab, f, f, kl=0.1), lambda: K.policy_loss(z, lab, f, f, weights=f[:2]),
           lambda: K.policy_loss(z, lab, f.bfloat16(), f), lambda: K.policy_loss(z, lab, f, f, clip_low=1.5),
           lambda: K.preference_loss(f, b[:2]), lambda: K.preference_loss(f, b.long()),
           lambda: K.preference_loss(f, b, labels=lab[:2]), lambda: K.preference_loss(f, b, kind="softmax"),
           lambda: K.preference_loss(f, b, beta=0.0), lambda: K.preference_loss(f, b, smoothing=0.7)]
    for i, call in enumerate(bad):
        with pytest.raises(MTError):
            call()
            pytest.fail(f"call {i} was taken")
