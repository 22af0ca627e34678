"""Embedding lookup with a scale and its gradient by sorted tokens, against float64; the ends of a step together.

Tolerances. The lookup is one product, rounded once to its type (bf16: 2^-8, fp32: 2^-24). A gradient's row is an fp32
sum of n rows in some order: n 2^-24 of the sum of sizes, then one rounding to bf16.
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


def _matrix(rng, T, h, kind, size=1.0):
    return torch.tensor(rng.standard_normal((T, h)) * size, dtype=torch.float32).cuda().to(TYPES[kind])


def _tokens(rng, T, V, how):
    if how == "one":  # one token everywhere
        tok = np.full(T, V - 1)
    elif how == "none":
        tok = np.full(T, -1)
    elif how == "order":
        tok = np.arange(T) % V
    else:  # frequent and rare ones, some padding
        tok = np.minimum((V * rng.random(T) ** 4).astype(np.int64), V - 1)
        tok[rng.random(T) < 0.1] = -1 - rng.integers(0, 5)
    return tok.astype(np.int32)


@pytest.mark.parametrize("T,h,V", [(1, 8, 1), (1, 4096, 1000), (257, 264, 31), (4000, 64, 152064), (33, 8200, 70)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_lookup(K, T, h, V, kind):
    rng = np.random.default_rng(T + h)
    E = _matrix(rng, V, h, "bf16", 0.02)
    tok = _tokens(rng, T, V, "zipf")
    tok[0] = V - 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = K.embed_lookup(torch.tensor(tok).cuda(), E, scale=h ** 0.5, dtype=TYPES[kind], err=err)
    ref = tune.embed_lookup(tok, _np(E), np.float32(h ** 0.5).astype(np.float64))
    assert x.dtype == TYPES[kind] and int(err.item()) == 0
    assert np.all(np.abs(_np(x) - ref) <= (F if kind == "f32" else HALF) * np.abs(ref) + 1e-40)


@pytest.mark.parametrize("T,h,V", [(1, 8, 1), (31, 16, 7), (128, 1032, 5), (1000, 256, 300), (5000, 72, 32000),
                                   (4097, 2056, 100), (9000, 8, 152064), (40000, 40, 1000), (140000, 8, 70000),
                                   (600, 64, 300000)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("how", ["zipf", "one", "none", "order"])
def test_gradient(K, T, h, V, kind, how):
    rng = np.random.default_rng(T * 3 + h + V)
    tok = _tokens(rng, T, V, how)
    tt = torch.tensor(tok).cuda()
    dx = _matrix(rng, T, h, kind)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dE = K.embed_lookup_bwd(tt, dx, V, scale=1.5, err=err)
    x = _np(dx)
    ref, size = tune.embed_lookup_bwd(tok, x, V, 1.5), tune.embed_lookup_bwd(tok, np.abs(x), V, 1.5)
    n = np.bincount(tok[tok >= 0], minlength=V)[:, None]
    got = _np(dE)
    assert np.all(np.abs(got - ref) <= HALF * np.abs(ref) + 1.01 * F * (n + 2) * size)
    assert np.all(got[n[:, 0] == 0] == 0) and int(err.item()) == 0
    assert torch.equal(K.embed_lookup_bwd(tt, dx, V, scale=1.5), dE)
    # added to what is there: a row of no token keeps its bits
    if V * h <= 1 << 22:
        old = _matrix(rng, V, h, "bf16")
        acc = old.clone()
        assert K.embed_lookup_bwd(tt, dx, V, scale=1.5, accumulate=acc) is acc
        want = ref + _np(old)
        assert np.all(np.abs(_np(acc) - want) <= HALF * np.abs(want) + 1.01 * F * ((n + 2) * size + np.abs(want)))
        free = torch.tensor(n[:, 0] == 0).cuda()
        assert torch.equal(acc[free], old[free])


def test_infinities_stay_in_their_rows(K):
    """NaN in the gradient of a padding token, infinity in one token's: neither reaches another row."""
    T, h, V = 300, 136, 50
    rng = np.random.default_rng(2)
    tok = rng.integers(0, V - 1, T).astype(np.int32)
    tok[[3, 100, 299]] = -1
    tok[7] = V - 1
    dx = _matrix(rng, T, h, "f32")
    dx[[3, 100, 299]] = float("nan")
    dx[7] = float("inf")
    dE = K.embed_lookup_bwd(torch.tensor(tok).cuda(), dx, V)
    assert bool(torch.isfinite(dE[:V - 1].float()).all()) and bool((dE[V - 1] == float("inf")).all())


def test_ids_outside_the_table(K):
    from host_memory_streamed_stream_gb300 import MTError

    rng = np.random.default_rng(3)
    V, h = 40, 64
    tok = torch.tensor([0, 40, -3, 2 ** 31 - 1, 39, -2 ** 31], dtype=torch.int32).cuda()
    E, dx = _matrix(rng, V, h, "bf16"), _matrix(rng, 6, h, "f32")
    for call in (lambda e: K.embed_lookup(tok, E, err=e), lambda e: K.embed_lookup_bwd(tok, dx, V, err=e)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = call(err)
        with pytest.raises(MTError, match="token"):
            K.check(err)
        if len(out) == 6:
            assert torch.equal(out[[0, 4]], E[[0, 39]].float()) and torch.all(out[[1, 2, 3, 5]] == 0)
        else:
            assert torch.equal(out[[0, 39]], dx[[0, 4]].bfloat16()) and torch.all(out[1:39] == 0)


def test_at_once_and_captured(K):
    """Gradients on two streams at the same time, and in two graphs replayed at the same time: what they give alone."""
    rng = np.random.default_rng(4)
    sets = []
    for T, h, V in ((9000, 520, 32000), (40000, 264, 4000), (50, 1032, 9000)):
        sets.append((torch.tensor(_tokens(rng, T, V, "zipf")).cuda(), _matrix(rng, T, h, "f32"), V))
    want = [K.embed_lookup_bwd(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(K.embed_lookup_bwd(*s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs, held = [torch.cuda.CUDAGraph() for _ in sets], []
    for s, gr in zip(sets, graphs):
        with torch.cuda.graph(gr):
            held.append(K.embed_lookup_bwd(*s))
    for s in sets:
        s[1].mul_(-2.0)
    for _ in range(3):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, K.embed_lookup_bwd(*s)) for a, s in zip(held, sets))


def test_refusals(K):
    from host_memory_streamed_stream_gb300 import MTError

    tok = torch.zeros(4, dtype=torch.int32, device="cuda")
    E = torch.zeros(10, 64, dtype=torch.bfloat16, device="cuda")
    dx = torch.zeros(4, 64, device="cuda")
    bad = [lambda: K.embed_lookup(tok.long(), E), lambda: K.embed_lookup(tok, E.float()),
           lambda: K.embed_lookup(tok, E[:, :32]), lambda: K.embed_lookup(tok, E, dtype=torch.float16),
           lambda: K.embed_lookup(tok.cpu(), E), lambda: K.embed_lookup(tok, E[:, :60].contiguous()),
           lambda: K.embed_lookup(tok, E, scale=float("nan")), lambda: K.embed_lookup(tok, E, err=dx),
           lambda: K.embed_lookup(tok[:0], E), lambda: K.embed_lookup_bwd(tok, dx.double(), 10),
           lambda: K.embed_lookup_bwd(tok, dx[:3], 10), lambda: K.embed_lookup_bwd(tok, dx[:, :32], 10),
           lambda: K.embed_lookup_bwd(tok.long(), dx, 10), lambda: K.embed_lookup_bwd(tok, dx, 0),
           lambda: K.embed_lookup_bwd(tok, dx, 1 << 25), lambda: K.embed_lookup_bwd(tok, dx, 10, accumulate=E.float()),
           lambda: K.embed_lookup_bwd(tok, dx, 11, accumulate=E)]
    for i, call in enumerate(bad):
        with pytest.raises(MTError):
            call()
            pytest.fail(f"call {i} was taken")


def _chain(E, G, b, W, tok, lab, old, adv):
    """Embedding, norm, head and policy loss in float64, and the gradients of table, gain, bias and head."""
    x = tune.embed_lookup(tok, E, 4.0)
    y, mean, rstd = tune.layernorm_fwd(x, G, b)
    z = y @ W.T
    loss, _, logp, dz = tune.policy_loss(z, lab, old, adv)
    dx, dg, db = tune.layernorm_bwd(dz @ W, x, G, mean, rstd)
    return loss, logp, tune.embed_lookup_bwd(tok, dx, len(E), 4.0), dg, db, dz.T @ y


def test_step_of_them_together(K):
    """Embedding, layer norm, the GEMMs of the head, the policy loss and all gradients back to the table, twice as used
    and once replayed from a graph. bf16 holds y, dz and the gradients (2^-8 each), so the results are compared in
    norm, with room for the four roundings on the longest way (y, z's sums of y, dz, and the result): 4 * 2^-8."""
    rng = np.random.default_rng(6)
    T, h, V = 256, 128, 512
    tok = _tokens(rng, T, V, "zipf")
    lab = rng.integers(0, V, T).astype(np.int32)
    lab[:40] = -1
    E, W = _matrix(rng, V, h, "bf16", 0.5), _matrix(rng, V, h, "bf16", 0.2)
    G, b = _matrix(rng, 1, h, "bf16")[0] * 0.1 + 1, _matrix(rng, 1, h, "bf16")[0]
    tt, lt = torch.tensor(tok).cuda(), torch.tensor(lab).cuda()
    adv = rng.standard_normal(T).astype(np.float32)
    old = np.full(T, -6.0, np.float32)  # about the level of the log-probabilities: the clip holds some rows
    at, ot = torch.tensor(adv).cuda(), torch.tensor(old).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        x = K.embed_lookup(tt, E, scale=4.0, err=err)
        y, mean, rstd = K.layernorm_fwd(x, G, b)
        z = K.gemm(y, False, W, False, T, V, h, epi=K.EPI_STORE_F32, err=err)
        loss, _, logp, dz = K.policy_loss(z, lt, ot, at, clip_low=0.2, clip_high=0.2, err=err)
        dy = K.gemm(dz, False, W, True, T, h, V, epi=K.EPI_STORE_F32, err=err)
        dW = K.gemm(dz, True, y, True, V, h, T, epi=K.EPI_STORE_F32, err=err)
        dx, _, dg, db = K.layernorm_bwd(dy, x, G, mean, rstd)
        return loss, logp, K.embed_lookup_bwd(tt, dx, V, scale=4.0, err=err), dg, db, dW

    out = step()
    # the plain form sees the y that the kernels rounded, so that no row of it falls on the other side of the clip
    want = _chain(_np(E), _np(G), _np(b), _np(W), tok, lab, old, adv)
    ratio = np.exp(want[1] - old)[lab >= 0]
    near = np.minimum(np.abs(ratio - 0.8) / 0.8, np.abs(ratio - 1.2) / 1.2)
    assert near.min() > 0, "a row on the border"
    for got, ref in zip(out[1:], want[1:]):
        got = _np(got)
        assert got.shape == ref.shape
    lp = _np(out[1])
    # z: 128 products of rounded y: sqrt(128) * 0.2 * 2^-9 in the mean, six times that at most
    assert np.abs(lp - want[1]).max() <= 6 * 0.2 * np.sqrt(128) * 2.0 ** -9 * 2
    assert all(torch.equal(a, c) for a, c in zip(out, step()))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(out, held))
    K.check(err)
    # gradients against the formulas on the kernels' own rounded intermediates: each operator's error alone remains
    x = tune.embed_lookup(tok, _np(E), 4.0)
    _, mean, rstd = tune.layernorm_fwd(x, _np(G), _np(b))
    y = _np(K.layernorm_fwd(K.embed_lookup(tt, E, scale=4.0), G, b)[0])
    dz = tune.policy_loss(y @ _np(W).T, lab, old, adv)[3]
    dx, dg, db = tune.layernorm_bwd(dz @ _np(W), x, _np(G), mean, rstd)
    for got, ref in zip(out[2:], (tune.embed_lookup_bwd(tok, dx, V, 4.0), dg, db, dz.T @ y)):
        assert np.linalg.norm(_np(got) - ref) <= 4 * HALF * np.linalg.norm(ref)
