"""The span-attention oracle against finite differences and plain causal attention, the document
spans against the definition, and the entries' refusals (nothing is launched)."""
import numpy as np
import pytest

from oracle import model as om
from oracle import spans as osp


@pytest.fixture(scope="module")
def lib():
    from host_memory_streamed_stream_gb300 import _build, _lib

    _build.build()
    return _lib.load()


@pytest.mark.parametrize("cap,slope", [(0.0, 0.0), (3.0, 0.0), (0.0, 0.3), (2.0, 0.1)])
def test_backward_against_differences(cap, slope):
    rng = np.random.default_rng(int(10 * cap + 100 * slope))
    n, d = 7, 5
    q, k, v, w = (rng.standard_normal((n, d)) for _ in range(4))
    lo, hi = [0, 0, 0, 3, 3, 0, 3], [3, 3, 3, 7, 5, 0, 7]  # two documents, a prefix, an empty row
    vis = osp.visible(lo, hi, n)

    def f(q, k, v):
        return float((osp.forward(q, k, v, vis, 0.6, cap, slope)[0] * w).sum())

    grads = osp.backward(q, k, v, vis, 0.6, w, cap, slope)[:3]
    step = 1e-6
    for x, g in zip((q, k, v), grads):
        for i in np.ndindex(*x.shape):
            keep = x[i]
            x[i] = keep + step
            up = f(q, k, v)
            x[i] = keep - step
            down = f(q, k, v)
            x[i] = keep
            assert abs((up - down) / (2 * step) - g[i]) < 1e-8  # step^2 and 2^-53 / step
    o, lse, p = osp.forward(q, k, v, vis, 0.6, cap, slope)
    assert np.all(o[5] == 0) and lse[5] == -np.inf and np.all(grads[0][5] == 0)


def test_causal_case_is_the_models_attention():
    rng = np.random.default_rng(2)
    s, hd = 19, 8
    q, k, v = (rng.standard_normal((1, s, 1, hd)) for _ in range(3))
    ref, _ = om.causal_attention(q, k, v)
    vis = osp.visible(np.zeros(s), np.arange(1, s + 1), s)
    o, _, _ = osp.forward(q[0, :, 0], k[0, :, 0], v[0, :, 0], vis, hd ** -0.5)
    np.testing.assert_allclose(o, ref[0, :, 0], rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("seed", range(12))
def test_doc_spans_against_the_definition(lib, seed):
    from host_memory_streamed_stream_gb300 import kernels as K

    rng = np.random.default_rng(seed)
    B, s = int(rng.integers(1, 4)), int(rng.integers(1, 40))
    n = int(rng.integers(0, 9))
    bounds = np.sort(rng.integers(0, B * s + 1, n + 1)).astype(np.int32)
    prefix = rng.integers(0, 12, n).astype(np.int32) if seed % 2 else None
    got = K.doc_spans(bounds, B, s, prefix)
    for a, b in zip(got, osp.document_spans(bounds, B, s, prefix)):
        np.testing.assert_array_equal(a, b)
    lo, hi, _ = got
    assert np.all(lo >= 0) and np.all(hi <= s) and np.all(lo <= hi)


def test_doc_spans_refusals(lib):
    from host_memory_streamed_stream_gb300 import MTError, kernels as K

    for bounds, B, s, prefix in (([3, 1], 1, 8, None), ([-1, 4], 1, 8, None), ([0, 9], 1, 8, None), ([], 1, 8, None),
                                 ([0, 4], 0, 8, None), ([0, 4], 1, 0, None), ([0, 4], 1, 8, [-1]),
                                 ([0, 4], 1, 8, [1, 2]), ([[0, 4]], 1, 8, None)):
        with pytest.raises(MTError):
            K.doc_spans(np.array(bounds, dtype=np.int32), B, s, prefix)
    b = np.array([0, 4], dtype=np.int32)
    out = np.zeros(8, dtype=np.int32)
    p = out.ctypes.data
    assert lib.mtk_doc_spans(None, 1, None, 1, 8, p, p, None) == -1
    assert lib.mtk_doc_spans(b.ctypes.data, -1, None, 1, 8, p, p, None) == -1
    assert lib.mtk_doc_spans(b.ctypes.data, 1, None, 1, 8, None, p, None) == -1
    assert lib.mtk_doc_spans(b.ctypes.data, 1, None, 65536, 65536, p, p, None) == -1  # B*s past int32
    assert lib.mtk_doc_spans(b.ctypes.data, 1, None, 1, 8, p, p, None) == 0  # positions may be NULL


def test_attn_span_refusals(lib):
    p = 1 << 20  # an aligned address that nothing reads
    nan, inf = float("nan"), float("inf")
    fwd = dict(q=p, ldq=512, k=p, ldk=256, v=p, ldv=256, lo=p, hi=p, o=p, ldo=512, lse=p, B=2, s=64, nh=4, nkv=2,
               hd=128, scale=0.1, cap=0.0, slopes=None, err=p)
    bwd = dict(fwd, dout=p, lddo=512, dq=p, lddq=512, dk=p, lddk=256, dv=p, lddv=256, scratch=p)
    for i, name in enumerate(("q", "k", "v", "o", "dout", "dq", "dk", "dv")):  # no two overlap
        if name in fwd:
            fwd[name] = p + (i << 20)
        bwd[name] = p + (i << 20)

    def call_fwd(**kw):
        a = dict(fwd, **kw)
        return lib.mtk_attn_span_fwd(a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["lo"], a["hi"], a["o"],
                                     a["ldo"], a["lse"], a["B"], a["s"], a["nh"], a["nkv"], a["hd"], a["scale"],
                                     a["cap"], a["slopes"], a["err"], None)

    def call_bwd(**kw):
        a = dict(bwd, **kw)
        return lib.mtk_attn_span_bwd(a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["lo"], a["hi"], a["o"],
                                     a["ldo"], a["lse"], a["dout"], a["lddo"], a["dq"], a["lddq"], a["dk"], a["lddk"],
                                     a["dv"], a["lddv"], a["scratch"], a["B"], a["s"], a["nh"], a["nkv"], a["hd"],
                                     a["scale"], a["cap"], a["slopes"], a["err"], None)

    common = [dict(q=None), dict(k=None), dict(v=None), dict(q=p + 8), dict(k=p + 2), dict(v=p + 4), dict(ldq=504),
              dict(ldk=252), dict(ldv=0), dict(lo=p + 2), dict(hi=p + 1), dict(o=None), dict(o=p + 8), dict(ldo=508),
              dict(ldo=256), dict(lse=None), dict(B=0), dict(s=0), dict(s=-1), dict(s=4194305), dict(nh=0),
              dict(nkv=0), dict(nkv=3), dict(hd=96), dict(hd=32), dict(scale=0.0), dict(scale=-1.0), dict(scale=nan),
              dict(scale=inf), dict(cap=-1.0), dict(cap=nan), dict(cap=inf), dict(cap=1e-39), dict(slopes=p + 2),
              dict(err=None), dict(B=1 << 30), dict(ldq=1 << 31)]
    for kw in common:
        assert call_fwd(**kw) == -1, kw
        assert call_bwd(**kw) == -1, kw
    for kw in (dict(dout=None), dict(dout=p + 8), dict(lddo=256), dict(dq=None), dict(dk=None), dict(dv=None),
               dict(dq=p + 2), dict(lddq=256), dict(lddk=128), dict(lddv=254), dict(scratch=None),
               dict(scratch=p + 8)):
        assert call_bwd(**kw) == -1, kw
    # outputs over an input or another output: the same memory, shifted by a row, columns that meet in
    # rows of one stride (128 rows of 512 columns: 131072 bytes), and strides that differ
    for name in ("q", "k", "v"):
        for kw in (dict(o=fwd[name]), dict(o=fwd[name] + 1024), dict(o=fwd[name] - 131072 + 1024),
                   dict(o=fwd[name] + 496, ldo=1024, ldq=1024, ldk=1024, ldv=1024)):
            assert call_fwd(**kw) == -1, (name, kw)
    for out in ("dq", "dk", "dv"):
        for name in ("q", "k", "v", "o", "dout", "dq", "dk", "dv"):
            if name != out:
                assert call_bwd(**{out: bwd[name]}) == -1, (out, name)
                assert call_bwd(**{out: bwd[name] + 512}) == -1, (out, name)
    for kw in (dict(lse=p + 2), dict(err=p + 1)):
        assert call_fwd(**kw) == -1 and call_bwd(**kw) == -1, kw
    # the longest walk of a key tile
    assert call_bwd(B=1, s=1 << 22, nh=64, nkv=1, ldq=8192, ldo=8192, lddo=8192, lddq=8192) == -1
    assert lib.mtk_attn_span_bwd_scratch_bytes(0, 1, 1, 1, 64) == 0
    assert lib.mtk_attn_span_bwd_scratch_bytes(1, 4194305, 1, 1, 64) == 0
    assert lib.mtk_attn_span_bwd_scratch_bytes(2, 129, 4, 2, 64) >= 2 * 4 * 256 * 8


def test_attn_span_backward_refuses_walks_of_too_many_steps(lib):
    """The limit on a key tile's walk counts whole tiles: one token, 2^24 query heads on one key head."""
    at = [(i + 1) << 32 for i in range(8)]  # aligned addresses that nothing reads, no two rows overlap
    nh, hd = 1 << 24, 64
    q = nh * hd
    scratch, lse, err = 1 << 40, 1 << 36, 1 << 21
    assert lib.mtk_attn_span_bwd(at[0], q, at[1], hd, at[2], hd, None, None, at[3], q, lse, at[4], q, at[5], q, at[6], hd,
                                 at[7], hd, scratch, 1, 1, nh, 1, hd, 0.1, 0.0, None, err, None) == -1


def test_doc_spans_takes_whole_numbers_of_32_bits(lib):
    """Boundaries that a conversion to int32 would change are refused, not wrapped or cut."""
    from host_memory_streamed_stream_gb300 import MTError, kernels as K

    for bounds, prefix in ((np.array([0, 2 ** 32 + 4]), None), (np.array([0, 4], dtype=np.uint64) + 2 ** 32, None),
                           ([0.0, 4.7], None), ([0, 4], np.array([2 ** 32 + 1])), ([0, 4], [1.5]), ([0, 2 ** 31], None),
                           ([False, True], None)):
        with pytest.raises(MTError):
            K.doc_spans(bounds, 1, 8, prefix)
    want = K.doc_spans(np.array([0, 4, 8], dtype=np.int32), 1, 8, np.array([2, 0], dtype=np.int32))
    for dtype in (np.uint8, np.int16, np.int64):
        got = K.doc_spans(np.array([0, 4, 8], dtype=dtype), 1, 8, [2, 0])
        assert all(np.array_equal(a, b) for a, b in zip(got, want))
    assert not any(a.any() for a in K.doc_spans([3], 1, 8, []))  # no documents
