"""Attention over spans, forward and backward, against the float64 oracle head by head.

Tolerances, element by element. Half a bf16 step is 2^-8 of a value; scores are fp32 sums of at most
128 exact products, so the probabilities carry a relative error below 2^-11 (128 * 2^-24 of a sum of
magnitudes that scale and log2(e) bring below 2^7 here, the exponential's and the cap's 2^-22 times
scores below 2^7). P and dS are rounded to bf16 in front of their products, and the results once more.
The backward's oracle takes o and lse as the kernel does: row sums in fp32 of 128 products (2^-16).
"""
import numpy as np
import pytest

import oracle
from oracle import spans as osp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF, PROB, SUM = 2.0 ** -8, 2.0 ** -11, 2.0 ** -16


@pytest.fixture(scope="module")
def K():
    from host_memory_streamed_stream_gb300 import _build

    _build.build()
    from host_memory_streamed_stream_gb300 import kernels

    return kernels


def _bf16(rng, shape, scale=1.0):
    x = oracle.bf16_bits_to_float(oracle.float_to_bf16_bits(rng.standard_normal(shape) * scale))
    return x, torch.tensor(x, dtype=torch.float32).to(torch.bfloat16).cuda()


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _i32(x):
    return torch.tensor(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _spans(kind, rng, B, s):
    """(lo, hi) int32 [B*s] of a kind of mask; None, None for the built-in causal one."""
    i = np.tile(np.arange(s), B)
    if kind == "causal":
        return None, None
    if kind == "all":
        return np.zeros(B * s), np.full(B * s, s)
    if kind == "window":  # the last 70 keys
        return np.maximum(i - 69, 0), i + 1
    if kind == "any":  # any nonempty ranges, in no order
        a, b = rng.integers(0, s, B * s), rng.integers(0, s, B * s)
        return np.minimum(a, b), np.maximum(a, b) + 1
    if kind == "none":
        return np.zeros(B * s), np.zeros(B * s)
    pad = {"docs": 0, "docs_padded": s // 7, "prefix": s // 9, "gaps": s // 9}[kind]
    bounds, prefix = [], []
    lo, hi = np.zeros(B * s, dtype=np.int32), np.zeros(B * s, dtype=np.int32)
    for b in range(B):
        at = int(rng.integers(0, 4)) if kind == "gaps" and s > 8 else 0
        while at < s - pad:
            n = min(int(rng.integers(1, max(2, s // 3 + 2))), s - pad - at)
            p = n * 2 // 5 if kind == "prefix" else n if kind == "gaps" else 0
            r = np.arange(n)
            lo[b * s + at:b * s + at + n] = at
            hi[b * s + at:b * s + at + n] = at + np.maximum(r + 1, p)
            at += n + (int(rng.integers(0, 6)) if kind == "gaps" else 0)
    return lo, hi


# (B, s, nh, nkv, hd, mask, cap, bias)
CASES = [
    (1, 1, 2, 1, 64, "causal", 0.0, False), (2, 1, 4, 4, 128, "all", 20.0, True),
    (3, 5, 4, 2, 128, "docs", 0.0, True), (2, 64, 2, 2, 64, "prefix", 5.0, False),
    (1, 65, 2, 1, 128, "docs_padded", 0.0, False), (2, 128, 4, 4, 64, "docs", 30.0, True),
    (1, 129, 4, 1, 128, "causal", 50.0, False), (2, 200, 4, 2, 128, "causal", 0.0, True),
    (2, 200, 4, 2, 64, "docs_padded", 10.0, False), (2, 333, 4, 1, 64, "prefix", 0.0, True),
    (1, 333, 8, 2, 128, "gaps", 0.0, False), (1, 600, 8, 2, 128, "window", 0.0, False),
    (1, 600, 4, 4, 64, "any", 15.0, True), (2, 384, 2, 2, 128, "any", 0.0, False),
    (1, 512, 2, 1, 128, "all", 0.0, False), (1, 700, 2, 2, 128, "docs_padded", 30.0, True),
    (2, 150, 2, 2, 64, "none", 0.0, False), (1, 1000, 2, 1, 64, "docs", 0.0, False),
    (4, 127, 6, 3, 128, "gaps", 8.0, True), (1, 1300, 1, 1, 128, "prefix", 0.0, False),
]


def _check_forward(o, lse, x, vis, scale, cap, slopes, B, s, nh, nkv, hd):
    q, k, v = x
    lse = lse.cpu().numpy().astype(np.float64)
    for b in range(B):
        for h in range(nh):
            e = v[b, :, h // (nh // nkv)]
            ro, rl, p = osp.forward(q[b, :, h], k[b, :, h // (nh // nkv)], e, vis[b], scale, cap, slopes[h])
            assert np.all(np.abs(o[b, :, h] - ro) <= HALF * np.abs(ro) + (HALF + PROB) * (p @ np.abs(e))), (b, h)
            dead = ~vis[b].any(1)
            assert np.all(o[b, dead, h] == 0) and np.all(lse[b, h, dead] == -np.inf)
            # in log2 units: 2^-11 relative is 2^-11 log2(e) < 2^-10
            assert np.all(np.abs(lse[b, h, ~dead] - rl[~dead]) <= 2.0 ** -10)


def _check_backward(got, x, o, lse, do, vis, scale, cap, slopes, B, s, nh, nkv, hd):
    q, k, v = x
    dq, dk, dv = got
    G = nh // nkv
    lse = lse.cpu().numpy().astype(np.float64)
    for b in range(B):
        for g in range(nkv):
            rk, rv, ek, ev = (np.zeros((s, hd)) for _ in range(4))
            for h in range(g * G, (g + 1) * G):
                a, c, e, d, oh = q[b, :, h], k[b, :, g], v[b, :, g], do[b, :, h], o[b, :, h]
                fq, fk, fv, p, ds = osp.backward(a, c, e, vis[b], scale, d, cap, slopes[h], oh, lse[b, h])
                _, dz = osp.scores(a, c, vis[b], scale, cap, slopes[h])
                sums = np.abs(d) @ np.abs(e).T + (np.abs(d) * np.abs(oh)).sum(1, keepdims=True)
                err = (HALF + PROB) * np.abs(ds) + p * (dz * SUM + (PROB if cap else 0.0) * 2.0 ** -4) * sums
                assert np.all(np.abs(dq[b, :, h] - fq) <= HALF * np.abs(fq) + scale * (err @ np.abs(c))), (b, h)
                rk += fk
                rv += fv
                ek += scale * (err.T @ np.abs(a))
                ev += (HALF + PROB) * (p.T @ np.abs(d))
            assert np.all(np.abs(dk[b, :, g] - rk) <= HALF * np.abs(rk) + ek + 1e-30), (b, g)
            assert np.all(np.abs(dv[b, :, g] - rv) <= HALF * np.abs(rv) + ev + 1e-30), (b, g)


def _case(K, B, s, nh, nkv, hd, kind, cap, bias, seed):
    rng = np.random.default_rng(seed)
    T = B * s
    # q | k of one buffer, v of another, both with columns around them
    qk, qkt = _bf16(rng, (T, (nh + nkv) * hd + 16), 1.5 if cap else 1.0)
    vv, vt = _bf16(rng, (T, nkv * hd + 24))
    q, k, v = qkt[:, 8:8 + nh * hd], qkt[:, 8 + nh * hd:8 + (nh + nkv) * hd], vt[:, 16:16 + nkv * hd]
    x = (qk[:, 8:8 + nh * hd].reshape(B, s, nh, hd), qk[:, 8 + nh * hd:8 + (nh + nkv) * hd].reshape(B, s, nkv, hd),
         vv[:, 16:16 + nkv * hd].reshape(B, s, nkv, hd))
    lo, hi = _spans(kind, rng, B, s)
    i = np.tile(np.arange(s), B)
    vis = [osp.visible((np.zeros(T) if lo is None else lo)[b * s:(b + 1) * s],
                       (i + 1 if hi is None else hi)[b * s:(b + 1) * s], s) for b in range(B)]
    slopes = rng.uniform(-0.02, 0.3, nh).astype(np.float32) if bias else np.zeros(nh)
    kw = dict(lo=None if lo is None else _i32(lo), hi=None if hi is None else _i32(hi), cap=cap,
              slopes=torch.tensor(slopes).cuda() if bias else None,
              err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    return rng, (q, k, v), x, vis, slopes.astype(np.float64), kw


@pytest.mark.parametrize("B,s,nh,nkv,hd,kind,cap,bias", CASES)
def test_forward(K, B, s, nh, nkv, hd, kind, cap, bias):
    rng, qkv, x, vis, slopes, kw = _case(K, B, s, nh, nkv, hd, kind, cap, bias, 31 * s + nh)
    scale = 0.11 if s % 2 else hd ** -0.5
    o, lse = K.attn_span_fwd(*qkv, B, s, nh, nkv, hd, scale=scale, **kw)
    _check_forward(_np(o).reshape(B, s, nh, hd), lse, x, vis, scale, cap, slopes, B, s, nh, nkv, hd)
    # into a column range: the same bits, its surroundings untouched; twice the same
    wide = torch.full((B * s, nh * hd + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    o2, lse2 = K.attn_span_fwd(*qkv, B, s, nh, nkv, hd, scale=scale, out=wide[:, 8:8 + nh * hd], **kw)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    assert bool((wide[:, :8] == 7).all()) and bool((wide[:, 8 + nh * hd:] == 7).all())
    assert int(kw["err"].item()) == 0


@pytest.mark.parametrize("B,s,nh,nkv,hd,kind,cap,bias", CASES)
def test_backward(K, B, s, nh, nkv, hd, kind, cap, bias):
    rng, qkv, x, vis, slopes, kw = _case(K, B, s, nh, nkv, hd, kind, cap, bias, 31 * s + nh)
    scale = 0.11 if s % 2 else hd ** -0.5
    o, lse = K.attn_span_fwd(*qkv, B, s, nh, nkv, hd, scale=scale, **kw)
    do, dot = _bf16(rng, (B * s, nh * hd))
    got = K.attn_span_bwd(*qkv, o, lse, dot, B, s, nh, nkv, hd, scale=scale, **kw)
    _check_backward([_np(t).reshape(B, s, -1, hd) for t in got], x, _np(o).reshape(B, s, nh, hd), lse,
                    do.reshape(B, s, nh, hd), vis, scale, cap, slopes, B, s, nh, nkv, hd)
    # into the column ranges of one buffer: the same bits, its surroundings untouched
    wide = torch.full((B * s, (nh + 2 * nkv) * hd + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    a, b, c = 8 + nh * hd, 8 + (nh + nkv) * hd, 8 + (nh + 2 * nkv) * hd
    again = K.attn_span_bwd(*qkv, o, lse, dot, B, s, nh, nkv, hd, scale=scale,
                            out=(wide[:, 8:a], wide[:, a:b], wide[:, b:c]), **kw)
    assert all(torch.equal(u, w) for u, w in zip(got, again))
    assert bool((wide[:, :8] == 7).all()) and bool((wide[:, c:] == 7).all())
    assert int(kw["err"].item()) == 0


@pytest.mark.parametrize("s,nh,nkv,kind,cap", [(1100, 144, 9, "causal", 0.0), (1030, 120, 10, "docs_padded", 20.0),
                                               (3500, 152, 8, "prefix", 0.0)])
def test_long_walks_of_few_key_tiles(K, s, nh, nkv, kind, cap):
    """Many query heads on a key head: dK and dV from parts of the walk over them, key heads sampled."""
    B, hd, G = 1, 64, nh // nkv
    rng, qkv, x, vis, slopes, kw = _case(K, B, s, nh, nkv, hd, kind, cap, False, s)
    o, lse = K.attn_span_fwd(*qkv, B, s, nh, nkv, hd, **kw)
    do, dot = _bf16(rng, (s, nh * hd))
    got = [_np(t).reshape(B, s, -1, hd) for t in K.attn_span_bwd(*qkv, o, lse, dot, B, s, nh, nkv, hd, **kw)]
    assert int(kw["err"].item()) == 0
    on, do = _np(o).reshape(B, s, nh, hd), do.reshape(B, s, nh, hd)
    for g in (0, nkv - 1):
        h = slice(g * G, (g + 1) * G)
        k = slice(g, g + 1)
        _check_backward([got[0][:, :, h], got[1][:, :, k], got[2][:, :, k]], (x[0][:, :, h], x[1][:, :, k], x[2][:, :, k]),
                        on[:, :, h], lse[:, h], do[:, :, h], vis, hd ** -0.5, cap, np.zeros(G), B, s, G, 1, hd)
    again = K.attn_span_bwd(*qkv, o, lse, dot, B, s, nh, nkv, hd, **kw)
    for a, b in zip(again, got):
        assert np.array_equal(_np(a).reshape(b.shape), b)


@pytest.mark.parametrize("cap", [30.0, 50.0, 60.0])
@pytest.mark.parametrize("size", [2.0 ** -30, 1.0, 2.0 ** 30])
def test_scores_at_the_cap(K, cap, size):
    """Scores of +-1152 before the cap: documents whose scores are all at -cap, all at +cap, at both,
    with small and large values. One fused buffer holds q, k, v, the output and the gradients."""
    rng = np.random.default_rng(int(cap))
    B, s, nh, nkv, hd = 1, 330, 2, 1, 128
    row, key = np.where(np.arange(s) % 3 == 1, -1.0, 1.0), np.ones(s)
    row[:70], row[70:140] = -1.0, 1.0
    key[200:] = np.where(np.arange(s)[200:] % 5 < 2, -1.0, 1.0)
    u = np.where(rng.random(hd) < 0.5, -3.0, 3.0)
    q = np.broadcast_to((row[:, None] * u)[:, None], (s, nh, hd))
    k = (key[:, None] * u)[:, None]
    v, _ = _bf16(rng, (s, 1, hd))
    v = v * size
    do, dot = _bf16(rng, (s, nh * hd))
    buf = torch.zeros(s, 11 * hd, dtype=torch.bfloat16, device="cuda")
    buf[:, :4 * hd] = torch.tensor(np.concatenate([q, k, v], 1).reshape(s, 4 * hd)).to(torch.bfloat16).cuda()
    cols = [buf[:, a * hd:b * hd] for a, b in ((0, 2), (2, 3), (3, 4), (4, 6), (6, 8), (8, 9), (9, 10))]
    lo, hi, _ = K.doc_spans([0, 70, 140, 330], B, s)
    kw = dict(lo=_i32(lo), hi=_i32(hi), scale=1.0, cap=cap, err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    o, lse = K.attn_span_fwd(*cols[:3], B, s, nh, nkv, hd, out=cols[3], **kw)
    got = K.attn_span_bwd(*cols[:3], o, lse, dot, B, s, nh, nkv, hd, out=cols[4:], **kw)
    assert int(kw["err"].item()) == 0 and bool((buf[:, 10 * hd:] == 0).all())
    x, vis = (q[None], k[None], v[None]), [osp.visible(lo, hi, s)]
    on = _np(o).reshape(B, s, nh, hd)
    _check_forward(on, lse, x, vis, 1.0, cap, np.zeros(nh), B, s, nh, nkv, hd)
    _check_backward([_np(t).reshape(B, s, -1, hd) for t in got], x, on, lse, do.reshape(B, s, nh, hd), vis, 1.0, cap,
                    np.zeros(nh), B, s, nh, nkv, hd)


@pytest.mark.parametrize("kind", ["docs_padded", "gaps", "prefix"])
@pytest.mark.parametrize("hd,s", [(64, 333), (128, 300)])
def test_padding_may_hold_anything(K, kind, hd, s):
    """NaN and infinities in the padding rows of q, k, v, o and dout change no bit of the rest."""
    B, nh, nkv = 2, 4, 2
    rng, qkv, x, vis, slopes, kw = _case(K, B, s, nh, nkv, hd, kind, 0.0, True, 5)
    _, dot = _bf16(rng, (B * s, nh * hd))
    o, lse = K.attn_span_fwd(*qkv, B, s, nh, nkv, hd, **kw)
    want = K.attn_span_bwd(*qkv, o, lse, dot, B, s, nh, nkv, hd, **kw)
    dead = torch.tensor(np.concatenate([~m.any(1) for m in vis])).cuda()
    assert 0 < int(dead.sum()) < B * s
    junk = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").to(torch.bfloat16)
    for t in (*qkv, dot):
        fill = junk[torch.randint(0, 3, (int(dead.sum()), t.shape[1]), device="cuda")]
        t[dead] = fill
    o2, lse2 = K.attn_span_fwd(*qkv, B, s, nh, nkv, hd, **kw)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    o2 = o2.clone()
    o2[dead] = float("nan")
    got = K.attn_span_bwd(*qkv, o2, lse, dot, B, s, nh, nkv, hd, **kw)
    for a, b in zip(got, want):
        assert torch.equal(a, b) and bool((a[dead] == 0).all())


def test_spans_are_clamped(K):
    """Bounds far outside the sequence act as its ends."""
    B, s, nh, nkv, hd = 1, 200, 2, 2, 64
    rng, qkv, x, vis, _, kw = _case(K, B, s, nh, nkv, hd, "all", 0.0, False, 6)
    want = K.attn_span_fwd(*qkv, B, s, nh, nkv, hd, **kw)
    kw.update(lo=torch.full((s,), -2 ** 31, dtype=torch.int32, device="cuda"),
              hi=torch.full((s,), 2 ** 31 - 1, dtype=torch.int32, device="cuda"))
    got = K.attn_span_fwd(*qkv, B, s, nh, nkv, hd, **kw)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_causal_case_agrees_with_the_causal_kernel(K):
    """No spans, cap or bias: the layer template's attention, forward and backward."""
    rng = np.random.default_rng(8)
    B, s, nh, nkv, hd = 2, 300, 8, 2, 128
    _, t = _bf16(rng, (B * s, (nh + 2 * nkv) * hd))
    _, dot = _bf16(rng, (B * s, nh * hd))
    q, k, v = t[:, :nh * hd], t[:, nh * hd:(nh + nkv) * hd], t[:, (nh + nkv) * hd:]
    o, lse = K.attn_fwd(t, B, s, nh, nkv, hd)
    o2, lse2 = K.attn_span_fwd(q, k, v, B, s, nh, nkv, hd)
    # both within half a step of the same sums, whose fp32 parts are below 2^-11 of it
    assert float((o.float() - o2.float()).abs().max()) <= 2.0 ** -6 * float(o.float().abs().max())
    assert float((lse - lse2).abs().max()) <= 2.0 ** -10
    d = K.attn_bwd(t, o, lse, dot, B, s, nh, nkv, hd)
    d2 = torch.cat(K.attn_span_bwd(q, k, v, o, lse, dot, B, s, nh, nkv, hd), 1)
    assert float((d.float() - d2.float()).abs().max()) <= 2.0 ** -6 * float(d.float().abs().max())


def test_offsets_past_32_bits(K):
    """The last documents of a buffer whose element offsets pass 2^31 and 2^32."""
    s, nh, nkv, hd, wide = 131072, 2, 1, 128, 36864
    rng = np.random.default_rng(12)
    buf = torch.zeros(s, wide, dtype=torch.bfloat16, device="cuda")
    n, last = 300, s - 300
    x, xt = _bf16(rng, (n, 4 * hd))
    do, dot = _bf16(rng, (n, nh * hd))
    buf[last:, :4 * hd] = xt
    dout = torch.zeros(s, nh * hd, dtype=torch.bfloat16, device="cuda")
    dout[last:] = dot
    q, k, v = buf[:, :nh * hd], buf[:, nh * hd:3 * hd], buf[:, 3 * hd:4 * hd]
    bounds = np.concatenate([np.arange(0, last, 256), [last, s]])
    lo, hi, _ = K.doc_spans(bounds, 1, s)
    kw = dict(lo=_i32(lo), hi=_i32(hi))
    o, lse = K.attn_span_fwd(q, k, v, 1, s, nh, nkv, hd, **kw)
    out = tuple(buf[:, a * hd:b * hd] for a, b in ((8, 10), (10, 11), (11, 12)))
    K.attn_span_bwd(q, k, v, o, lse, dout, 1, s, nh, nkv, hd, out=out, **kw)
    xs = (x[:, :2 * hd].reshape(1, n, 2, hd), x[:, 2 * hd:3 * hd].reshape(1, n, 1, hd),
          x[:, 3 * hd:].reshape(1, n, 1, hd))
    vis = [osp.visible(np.zeros(n), np.arange(1, n + 1), n)]
    on = _np(o[last:]).reshape(1, n, nh, hd)
    tail = lse[:, :, last:].contiguous()
    _check_forward(on, tail, xs, vis, hd ** -0.5, 0.0, np.zeros(nh), 1, n, nh, nkv, hd)
    _check_backward([_np(t[last:]).reshape(1, n, -1, hd) for t in out], xs, on, tail, do.reshape(1, n, nh, hd), vis,
                    hd ** -0.5, 0.0, np.zeros(nh), 1, n, nh, nkv, hd)


def test_streams_and_graphs(K):
    """On another stream, and captured: two graphs whose replays alternate, each with its own scratch."""
    B, s, nh, nkv, hd = 2, 260, 4, 2, 128
    cases = [_case(K, B, s, nh, nkv, hd, kind, cap, bias, 3) for kind, cap, bias in
             (("docs_padded", 20.0, False), ("prefix", 0.0, True))]
    dots = [_bf16(c[0], (B * s, nh * hd))[1] for c in cases]

    def step(n):
        qkv, kw = cases[n][1], cases[n][5]
        o, lse = K.attn_span_fwd(*qkv, B, s, nh, nkv, hd, **kw)
        return (o, lse, *K.attn_span_bwd(*qkv, o, lse, dots[n], B, s, nh, nkv, hd, **kw))

    want = [step(n) for n in range(2)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [step(n) for n in range(2)]
    side.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, g))
    graphs, outs = [], []
    for n in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(n))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for w, g in zip(want, outs):
        assert all(torch.equal(a, b) for a, b in zip(w, g))


@pytest.mark.parametrize("cap,bias", [(0.0, False), (25.0, True)])
def test_attention_block_of_packed_documents(K, cap, bias):
    """The set together, as a layer runs it: boundaries -> spans and positions, scaled table, norms
    with rotation, attention, and back to the projection's gradient, against float64."""
    rng = np.random.default_rng(17)
    B, s, nh, nkv, hd, eps = 2, 190, 4, 2, 64, 1e-5
    T, G, H = B * s, nh // nkv, nh + nkv
    bounds, prefix = np.array([0, 40, 41, 150, 260, 370]), np.array([10, 0, 0, 30, 0])
    lo, hi, pos = K.doc_spans(bounds, B, s, prefix)
    tab = K.rotary_table(K.rotary_inv_freq(hd, scaling="bands", factor=4.0, original_positions=64), s, amplitude=1.1)
    cs = _np(tab)
    x, xt = _bf16(rng, (T, (nh + 2 * nkv) * hd))
    gq, gqt = _bf16(rng, (hd,))
    gk, gkt = _bf16(rng, (hd,))
    do, dot = _bf16(rng, (T, nh * hd))
    slopes = rng.uniform(0, 0.2, nh).astype(np.float32) if bias else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    post = _i32(pos)
    kw = dict(lo=_i32(lo), hi=_i32(hi), cap=cap, slopes=None if slopes is None else torch.tensor(slopes).cuda(),
              err=err)
    y, rstd = K.qk_norm_rope(xt, gqt, gkt, nh, nkv, hd, tab, positions=post, eps=eps, err=err)
    q, k, v = y[:, :nh * hd], y[:, nh * hd:], xt[:, H * hd:]
    o, lse = K.attn_span_fwd(q, k, v, B, s, nh, nkv, hd, **kw)
    dx = torch.empty_like(xt)
    K.attn_span_bwd(q, k, v, o, lse, dot, B, s, nh, nkv, hd,
                    out=(dx[:, :nh * hd], dx[:, nh * hd:H * hd], dx[:, H * hd:]), **kw)
    _, dgq, dgk = K.qk_norm_rope_bwd(dx, xt, gqt, gkt, rstd, nh, nkv, hd, tab, positions=post, out=dx, err=err)
    assert int(err.item()) == 0

    def turn(t, sign):
        c, sn = cs[pos][:, None, :, 0], sign * cs[pos][:, None, :, 1]
        a, b = t[..., :hd // 2], t[..., hd // 2:]
        return np.concatenate([a * c - b * sn, b * c + a * sn], -1)

    xs = x.reshape(T, nh + 2 * nkv, hd)
    r = 1 / np.sqrt((xs[:, :H] ** 2).mean(-1, keepdims=True) + eps)
    g = np.concatenate([np.tile(gq, (nh, 1)), np.tile(gk, (nkv, 1))])
    n = xs[:, :H] * r
    yr = turn(n * g, 1.0).reshape(B, s, H, hd)
    vr = xs[:, H:].reshape(B, s, nkv, hd)
    ro, d = np.zeros((B, s, nh, hd)), np.zeros((B, s, nh + 2 * nkv, hd))
    for b in range(B):
        vis = osp.visible(lo[b * s:(b + 1) * s], hi[b * s:(b + 1) * s], s)
        for h in range(nh):
            j, sl = h // G, 0.0 if slopes is None else float(slopes[h])
            args = (yr[b, :, h], yr[b, :, nh + j], vr[b, :, j], vis, hd ** -0.5)
            ro[b, :, h] = osp.forward(*args, cap, sl)[0]
            fq, fk, fv, _, _ = osp.backward(*args, do.reshape(B, s, nh, hd)[b, :, h], cap, sl)
            d[b, :, h] += fq
            d[b, :, nh + j] += fk
            d[b, :, H + j] += fv
    u = turn(d[:, :, :H].reshape(T, H, hd), -1.0)
    dn = u * g
    d[:, :, :H] = (r * (dn - n * (dn * n).mean(-1, keepdims=True))).reshape(B, s, H, hd)
    rg = (u * n).sum(0)
    # y, o, P, dS and the gradients between the kernels are rounded to bf16, each by 2^-8 at most,
    # independently: over a tensor the 2-norms add up to less than six such roundings, twice over
    # for what a query's or key's rounding does to its scores (of size sqrt(hd) / sqrt(hd) here)
    bound = 12 * HALF
    for got, ref in ((_np(o).reshape(B, s, nh, hd), ro), (_np(dx).reshape(d.shape), d), (_np(dgq), rg[:nh].sum(0)),
                     (_np(dgk), rg[nh:].sum(0))):
        assert np.linalg.norm(got - ref) <= bound * np.linalg.norm(ref)


@pytest.mark.parametrize("cap,bias", [(0.0, False), (30.0, True)])
def test_a_bad_position_in_the_flag_stops_no_kernel(K, cap, bias):
    """A flag that already holds a data error (code 8): the same bits as with a clean one, the code still there."""
    B, s, nh, nkv, hd = 2, 700, 8, 2, 128
    rng, qkv, _, _, _, kw = _case(K, B, s, nh, nkv, hd, "docs", cap, bias, 11)
    _, dot = _bf16(rng, (B * s, nh * hd))
    _, w = _bf16(rng, (1000, nh * hd))
    _, fused = _bf16(rng, (B * s, (nh + 2 * nkv) * hd))

    def step(code):
        err = torch.full((1,), code, dtype=torch.int32, device="cuda")
        args = dict(kw, err=err)
        o, lse = K.attn_span_fwd(*qkv, B, s, nh, nkv, hd, **args)
        out = [o, lse, *K.attn_span_bwd(*qkv, o, lse, dot, B, s, nh, nkv, hd, **args)]
        out.append(K.gemm(o, False, w, False, B * s, 1000, nh * hd, err=err))
        o, lse = K.attn_fwd(fused, B, s, nh, nkv, hd, err=err)
        out += [o, lse, K.attn_bwd(fused, o, lse, dot, B, s, nh, nkv, hd, err=err)]
        assert int(err.item()) == code
        return out

    want = step(0)
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(step(8), want))


def test_a_wait_that_gives_up_is_recorded_over_a_bad_position(K):
    from host_memory_streamed_stream_gb300 import _lib

    err = torch.full((1,), 8, dtype=torch.int32, device="cuda")
    gone = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert _lib.load().mtk_bounded_wait_check(err.data_ptr(), gone.data_ptr(), 1_000_000, None) == 0
    torch.cuda.synchronize()
    assert int(err.item()) == 6 and int(gone.item()) == 1
