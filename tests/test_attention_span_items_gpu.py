"""Attention over spans where every block of the backward works on several items, most of them walks of one and
two tiles: short documents, many heads. Sampled heads against the float64 oracle (with the tolerances derived in
test_attention_span_gpu.py), all of them against calls of a few heads, in which a block has one or two items.
"""
import numpy as np
import pytest

from oracle import spans as osp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_attention_span_gpu import K, _bf16, _check_backward, _check_forward, _i32, _np  # noqa: E402, F401

B, S, NH, CHUNK = 4, 700, 32, 4  # 768 query tiles; 4 key heads: 96 key tiles, one a block, none cut


def _bounds(kind, rng):
    """Documents of the B * S tokens; those of a sequence that end before it leave padding."""
    if kind == "tiles":  # every walk is one tile, the last tile's of 60 rows
        starts = [np.arange(b * S, (b + 1) * S, 128) for b in range(B)]
        return np.unique(np.concatenate([*starts, [B * S]])), []
    out, dead = [], []
    for b in range(B):
        at, end = b * S, (b + 1) * S
        if kind == "mixed":  # a long document among short ones, then padding over a whole tile and more
            end -= 290 + 13 * b
            out += [at, at + 250]
            at += 250
        while at < end:
            out.append(at)
            at = min(at + int(rng.integers(60, 201)), end)
        if end < (b + 1) * S:
            dead.append((end, (b + 1) * S))
        out.append(end)
    return np.unique(np.array(out + [B * S])), dead


@pytest.mark.parametrize("cap,bias", [(0.0, False), (30.0, False), (0.0, True), (60.0, True)])
@pytest.mark.parametrize("kind", ["tiles", "short", "mixed"])
@pytest.mark.parametrize("hd,nkv", [(64, 32), (128, 32), (128, 16)])
def test_many_short_walks(K, hd, nkv, kind, cap, bias):
    rng = np.random.default_rng(hd + nkv)
    T, G = B * S, NH // nkv
    bounds, dead = _bounds(kind, rng)
    lo, hi, _ = K.doc_spans(bounds, B, S)
    for a, b in dead:  # padding, not a document
        lo[a:b] = hi[a:b] = 0
    size = 1.5 if cap else 1.0
    q, qt = _bf16(rng, (T, NH * hd), size)
    k, kt = _bf16(rng, (T, nkv * hd), size)
    v, vt = _bf16(rng, (T, nkv * hd))
    do, dot = _bf16(rng, (T, NH * hd))
    for a, b in dead:
        for i, t in enumerate((qt, kt, vt, dot)):
            t[a:b] = (float("nan"), float("inf"), -float("inf"), float("nan"))[i]
    slopes = rng.uniform(-0.02, 0.3, NH).astype(np.float32) if bias else np.zeros(NH, np.float32)
    slt = torch.tensor(slopes).cuda() if bias else None
    kw = dict(lo=_i32(lo), hi=_i32(hi), cap=cap, err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    o, lse = K.attn_span_fwd(qt, kt, vt, B, S, NH, nkv, hd, slopes=slt, **kw)
    got = K.attn_span_bwd(qt, kt, vt, o, lse, dot, B, S, NH, nkv, hd, slopes=slt, **kw)
    for _ in range(10):
        again = K.attn_span_bwd(qt, kt, vt, o, lse, dot, B, S, NH, nkv, hd, slopes=slt, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
    for g in range(0, nkv, CHUNK):
        qs, ks, hs = (slice(g * G * hd, (g + CHUNK) * G * hd), slice(g * hd, (g + CHUNK) * hd),
                      slice(g * G, (g + CHUNK) * G))
        few = (qt[:, qs], kt[:, ks], vt[:, ks])
        args = (B, S, CHUNK * G, CHUNK, hd)
        o1, lse1 = K.attn_span_fwd(*few, *args, slopes=None if slt is None else slt[hs], **kw)
        assert torch.equal(o1, o[:, qs]) and torch.equal(lse1, lse[:, hs])
        few_got = K.attn_span_bwd(*few, o1, lse1, dot[:, qs], *args, slopes=None if slt is None else slt[hs], **kw)
        assert all(torch.equal(a, b) for a, b in zip(few_got, (got[0][:, qs], got[1][:, ks], got[2][:, ks])))
    assert int(kw["err"].item()) == 0
    vis = [osp.visible(lo[b * S:(b + 1) * S], hi[b * S:(b + 1) * S], S) for b in range(B)]
    heads = [a.reshape(B, S, -1, hd) for a in (q, k, v, do, _np(o), *(_np(t) for t in got))]
    for g in (0, nkv - 1):
        h, j = slice(g * G, (g + 1) * G), slice(g, g + 1)
        x = (heads[0][:, :, h], heads[1][:, :, j], heads[2][:, :, j])
        args = (vis, hd ** -0.5, cap, slopes[h].astype(np.float64), B, S, G, 1, hd)
        _check_forward(heads[4][:, :, h], lse[:, h].contiguous(), x, *args)
        _check_backward([heads[5][:, :, h], heads[6][:, :, j], heads[7][:, :, j]], x, heads[4][:, :, h],
                        lse[:, h].contiguous(), heads[3][:, :, h], *args)


@pytest.mark.parametrize("hd", [64, 128])
def test_two_streams_at_once(K, hd):
    """Calls that overlap on the device: the blocks of one wait for the other's tensor memory, results unchanged."""
    rng = np.random.default_rng(hd)
    b, s, nh = 2, 1000, 24
    streams, calls, want = [torch.cuda.Stream() for _ in range(2)], [], []
    for cap in (0.0, 20.0):
        q, k, v, d = (_bf16(rng, (b * s, nh * hd))[1] for _ in range(4))
        lo, hi, _ = K.doc_spans(np.unique(np.append(rng.integers(0, b * s, 15), [0, b * s])), b, s)
        kw = dict(lo=_i32(lo), hi=_i32(hi), cap=cap, err=torch.zeros(1, dtype=torch.int32, device="cuda"))

        def call(q=q, k=k, v=v, d=d, kw=kw):
            o, lse = K.attn_span_fwd(q, k, v, b, s, nh, nh, hd, **kw)
            return (o, lse, *K.attn_span_bwd(q, k, v, o, lse, d, b, s, nh, nh, hd, **kw))

        calls.append((call, kw["err"]))
        want.append(call())
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for n in range(2):
            with torch.cuda.stream(streams[n]):
                got[n].append(calls[n][0]())
    torch.cuda.synchronize()
    for n in range(2):
        K.check(calls[n][1])
        assert all(torch.equal(a, w) for g in got[n] for a, w in zip(g, want[n]))
