"""Per-kernel binding (``include/mt_kernels.h``) over torch CUDA tensors: marshalling only.

Each function passes the tensors' device pointers and the current torch stream
to one C entry point and raises on a nonzero status. What only the device sees goes into the flag `err`
that a call may be given; check(err) reads it.
"""
from __future__ import annotations

import ctypes
import functools

import numpy as np
import torch

from . import MTError, _lib

EPI_STORE_BF16, EPI_STORE_F32, EPI_ADD_F32 = 0, 1, 2
ROTARY_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "bands": 3}


def _p(t):
    return None if t is None else t.data_ptr()


def _s():
    return torch.cuda.current_stream().cuda_stream


def _stream(dev):
    """The current stream's handle on device number `dev` (the same as _s(), without making a Stream
    object: 0.3 us instead of 7 on the Grace host)."""
    return torch._C._cuda_getCurrentRawStream(dev)


def _ok(rc, what):
    if rc != 0:
        raise MTError(rc, what)


def gemm(A, a_mn, B, b_mn, M, N, K, epi=EPI_STORE_BF16, R=None, err=None, out=None):
    """C[M,N] = A * B (see mtk_gemm_bf16 for the operand storage orders)."""
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16 if epi == EPI_STORE_BF16 else torch.float32, device=A.device)
    err = _err(err, A.device)
    _ok(_lib.load().mtk_gemm_bf16(A.data_ptr(), A.stride(0), int(a_mn), B.data_ptr(), B.stride(0), int(b_mn),
                                  out.data_ptr(), out.stride(0), _p(R), R.stride(0) if R is not None else 0, M, N, K,
                                  epi, err.data_ptr(), _s()), "gemm")
    return out


def gemm_use_workspace(device=None):
    """Give the mtk_gemm_* calls a zeroed split workspace on `device` (None: turn the split off).
    Returns the workspace tensor, which must stay alive while it is in use."""
    lib = _lib.load()
    if device is None:
        _ok(lib.mtk_gemm_use_workspace(None), "gemm_use_workspace")
        return None
    ws = torch.zeros(int(lib.mtk_gemm_workspace_bytes()), dtype=torch.uint8, device=device)
    _ok(lib.mtk_gemm_use_workspace(ws.data_ptr()), "gemm_use_workspace")
    return ws


def _err(err, dev):
    """The flag's tensor: the caller's, or a new one that nobody reads."""
    if err is None:
        return torch.zeros(1, dtype=torch.int32, device=dev)
    if err.dtype is not torch.int32 or err.numel() < 1 or err.device != dev:
        raise MTError(-1, f"err: an int32 tensor on {dev}")
    return err


def check(err):
    """Wait for the calls that were given `err` (a zeroed int32 device tensor of one element) and raise
    MTError if one of them left a code there: a wait that gave up (outputs are then invalid), or a
    position outside its rotation table (that token is unrotated). Calls without `err` report neither.
    """
    code = int(err.item())
    if code != 0:
        raise MTError(-7, "a position outside the rotation table" if code == 8 else
                      f"a kernel's bounded wait gave up (code {code})")


def gemm_qkv_rope(a, w, cos_sin, seq, n_heads, n_kv_heads, head_dim, err=None):
    """qkv = a W^T with RoPE on the q and k heads, fused in the GEMM epilogue."""
    T, h = a.shape
    qkv = torch.empty(T, (n_heads + 2 * n_kv_heads) * head_dim, dtype=torch.bfloat16, device=a.device)
    err = _err(err, a.device)
    _ok(_lib.load().mtk_gemm_qkv_rope(a.data_ptr(), w.data_ptr(), qkv.data_ptr(), cos_sin.data_ptr(), T, h, n_heads,
                                      n_kv_heads, head_dim, seq, err.data_ptr(), _s()), "gemm_qkv_rope")
    return qkv


def gemm_swiglu(b, wgu, f, keep_gu=False, err=None):
    """act = silu(b Wg^T) * (b Wu^T) fused in the GEMM epilogue; optionally also [g | u]."""
    T, h = b.shape
    act = torch.empty(T, f, dtype=torch.bfloat16, device=b.device)
    gu = torch.empty(T, 2 * f, dtype=torch.bfloat16, device=b.device) if keep_gu else None
    err = _err(err, b.device)
    _ok(_lib.load().mtk_gemm_swiglu(b.data_ptr(), wgu.data_ptr(), act.data_ptr(), _p(gu), T, h, f, err.data_ptr(),
                                    _s()), "gemm_swiglu")
    return act, gu


def gemm_swiglu_bwd(dy, wd, gu, f, err=None):
    """dgu from dact = dy Wd and gu = [g | u], the SwiGLU backward fused in the GEMM epilogue."""
    T, h = dy.shape
    dgu = torch.empty(T, 2 * f, dtype=torch.bfloat16, device=dy.device)
    err = _err(err, dy.device)
    _ok(_lib.load().mtk_gemm_swiglu_bwd(dy.data_ptr(), wd.data_ptr(), gu.data_ptr(), dgu.data_ptr(), T, h, f,
                                        err.data_ptr(), _s()), "gemm_swiglu_bwd")
    return dgu


def rmsnorm_fwd(x, gamma, eps=1e-5):
    T, h = x.shape
    y = torch.empty(T, h, dtype=torch.bfloat16, device=x.device)
    rstd = torch.empty(T, dtype=torch.float32, device=x.device)
    _ok(_lib.load().mtk_rmsnorm_fwd(x.data_ptr(), gamma.data_ptr(), y.data_ptr(), rstd.data_ptr(), T, h, eps, _s()),
        "rmsnorm_fwd")
    return y, rstd


def rmsnorm_bwd(dy, x, gamma, rstd, dres=None):
    T, h = x.shape
    lib = _lib.load()
    parts = lib.mtk_rmsnorm_bwd_parts(T)
    partial = torch.empty(parts, h, dtype=torch.float32, device=x.device)
    dx = torch.empty(T, h, dtype=torch.float32, device=x.device)
    dxb = torch.empty(T, h, dtype=torch.bfloat16, device=x.device)
    dg = torch.empty(h, dtype=torch.bfloat16, device=x.device)
    _ok(lib.mtk_rmsnorm_bwd(dy.data_ptr(), x.data_ptr(), gamma.data_ptr(), rstd.data_ptr(), _p(dres), dx.data_ptr(),
                            dxb.data_ptr(), partial.data_ptr(), dg.data_ptr(), T, h, _s()), "rmsnorm_bwd")
    return dx, dxb, dg


def rope_(qkv, seq, n_heads, n_kv_heads, head_dim, cos_sin, inverse=False):
    T = qkv.shape[0]
    _ok(_lib.load().mtk_rope(qkv.data_ptr(), qkv.stride(0), T, seq, n_heads, n_kv_heads, head_dim, cos_sin.data_ptr(),
                             int(inverse), _s()), "rope")
    return qkv


# The calls below take views of larger buffers, so the types, shapes and strides that the C entry
# cannot see are checked here (MTError with MT_EINVAL, like the entry's own refusals).
def _need(ok, what):
    if not ok:
        raise MTError(-1, what)


def _device(t):
    """Number of the device of `t`, which has to be the current one (the kernels launch there)."""
    dev = t.get_device()
    _need(dev >= 0 and dev == torch._C._cuda_getDevice(), "tensors have to be on the current CUDA device")
    return dev


def _rows(t, n, cols, what, dev):
    """Row stride of a bf16 [n, >= cols] view on device `dev` with unit column stride."""
    shape, stride = t.shape, t.stride()
    if (t.dtype is not torch.bfloat16 or len(shape) != 2 or shape[0] != n or shape[1] < cols or stride[1] != 1
            or t.get_device() != dev):
        raise MTError(-1, f"{what}: a bf16 [{n}, >= {cols}] tensor with unit column stride on cuda:{dev}")
    return stride[0] if n > 1 else (cols + 7) // 8 * 8


def _vec(t, n, dtype, what, dev):
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or t.get_device() != dev:
        raise MTError(-1, f"{what}: a contiguous {dtype} tensor of {n} elements on cuda:{dev}")
    return t.data_ptr()


def _table(cos_sin, dev):
    """(pointer, positions, rotated columns) of a rotation table; no table: no rotation."""
    if cos_sin is None:
        return None, 0, 0
    shape = cos_sin.shape
    _need(len(shape) == 3 and shape[2] == 2, "cos_sin: [n_pos, rot_dim/2, 2]")
    return _vec(cos_sin, cos_sin.numel(), torch.float32, "cos_sin", dev), shape[0], 2 * shape[1]


def _host(a):
    """Address of a contiguous numpy array (ndarray.ctypes costs 2 us more after a launch)."""
    try:
        return ctypes.addressof(ctypes.c_char.from_buffer(a))
    except (TypeError, ValueError):  # read-only or empty
        return a.ctypes.data


def rotary_inv_freq(rot_dim, theta=10000.0, scaling="plain", factor=1.0, original_positions=0, low=1.0, high=32.0):
    """rot_dim/2 rotation frequencies (numpy float64, radians per position); see mtk_rotary_inv_freq
    for the scalings "plain", "linear", "base" and "bands"."""
    if scaling not in ROTARY_SCALINGS:
        raise MTError(-1, f"scaling: one of {sorted(ROTARY_SCALINGS)}")
    out = np.empty(max(int(rot_dim) // 2, 1), dtype=np.float64)
    _ok(_lib.load().mtk_rotary_inv_freq(rot_dim, theta, ROTARY_SCALINGS[scaling], factor, original_positions, low, high,
                                        _host(out)), "rotary_inv_freq")
    return out


def rotary_table(inv_freq, n_pos, amplitude=1.0, out=None):
    """fp32 [n_pos, rot_dim/2, 2] = amplitude * (cos, sin) of p * inv_freq[i] on the current device."""
    f = np.ascontiguousarray(inv_freq, dtype=np.float64)
    _need(f.ndim == 1, "inv_freq: one frequency for each pair")
    if out is None:
        out = torch.empty((n_pos, f.size, 2), dtype=torch.float32, device="cuda")
    _need(out.shape == (n_pos, f.size, 2), "out: fp32 [n_pos, rot_dim/2, 2]")
    dev = _device(out)
    _ok(_lib.load().mtk_rotary_table(_host(f), 2 * f.size, n_pos, amplitude,
                                     _vec(out, out.numel(), torch.float32, "out", dev), _stream(dev)), "rotary_table")
    return out


def rotary(x, heads, head_dim, cos_sin, positions=None, interleaved=False, inverse=False, out=None, err=None):
    """x [T, heads*head_dim] with the first rot_dim (the table's) columns of every head rotated at
    `positions` (int32 [T]; None: t % n_pos). out: a new tensor, another one, or x itself (in place).
    A position outside the table leaves its token unrotated and a code in `err` (see check)."""
    T, cols, dev = x.shape[0], heads * head_dim, _device(x)
    ldx = _rows(x, T, cols, "x", dev)
    tab, n_pos, rot = _table(cos_sin, dev)
    if out is None:
        out = torch.empty((T, cols), dtype=torch.bfloat16, device=x.device)
    pos = None if positions is None else _vec(positions, T, torch.int32, "positions", dev)
    err = _err(err, x.device)
    _ok(_lib.load().mtk_rotary(x.data_ptr(), ldx, out.data_ptr(), _rows(out, T, cols, "out", dev), T, heads, head_dim,
                               rot, interleaved, pos, tab, n_pos, inverse, err.data_ptr(), _stream(dev)), "rotary")
    return out


def qk_norm_rope(x, gq, gk, n_heads, n_kv_heads, head_dim, cos_sin=None, positions=None, interleaved=False, eps=1e-5,
                 out=None, err=None):
    """RMSNorm of each query and key head of x [T, >= (nh+nkv)*hd] and the rotation (cos_sin None:
    none): (y [T, (nh+nkv)*hd], rstd f32 [T, nh+nkv]). out: as for rotary."""
    T, heads, dev = x.shape[0], n_heads + n_kv_heads, _device(x)
    cols = heads * head_dim
    ldx = _rows(x, T, cols, "x", dev)
    tab, n_pos, rot = _table(cos_sin, dev)
    if out is None:
        out = torch.empty((T, cols), dtype=torch.bfloat16, device=x.device)
    rstd = torch.empty((T, heads), dtype=torch.float32, device=x.device)
    pos = None if positions is None else _vec(positions, T, torch.int32, "positions", dev)
    err = _err(err, x.device)
    _ok(_lib.load().mtk_qk_norm_rope(x.data_ptr(), ldx, _vec(gq, head_dim, torch.bfloat16, "gq", dev),
                                     _vec(gk, head_dim, torch.bfloat16, "gk", dev), out.data_ptr(),
                                     _rows(out, T, cols, "out", dev), rstd.data_ptr(), T, n_heads, n_kv_heads,
                                     head_dim, rot, interleaved, eps, pos, tab, n_pos, err.data_ptr(), _stream(dev)),
        "qk_norm_rope")
    return out, rstd


def qk_norm_rope_bwd(dy, x, gq, gk, rstd, n_heads, n_kv_heads, head_dim, cos_sin=None, positions=None,
                     interleaved=False, out=None, err=None):
    """(dx [T, (nh+nkv)*hd], dgq, dgk) of qk_norm_rope; out: a new tensor for dx, another one, dy or x."""
    T, heads, dev = x.shape[0], n_heads + n_kv_heads, _device(x)
    cols = heads * head_dim
    ldx, lddy = _rows(x, T, cols, "x", dev), _rows(dy, T, cols, "dy", dev)
    tab, n_pos, rot = _table(cos_sin, dev)
    if out is None:
        out = torch.empty((T, cols), dtype=torch.bfloat16, device=x.device)
    lib = _lib.load()
    parts = lib.mtk_qk_norm_rope_bwd_parts(T, n_heads, n_kv_heads, head_dim)
    partial = torch.empty((parts, head_dim), dtype=torch.float32, device=x.device)
    dgq, dgk = torch.empty_like(gq), torch.empty_like(gk)
    pos = None if positions is None else _vec(positions, T, torch.int32, "positions", dev)
    err = _err(err, x.device)
    _ok(lib.mtk_qk_norm_rope_bwd(dy.data_ptr(), lddy, x.data_ptr(), ldx,
                                 _vec(gq, head_dim, torch.bfloat16, "gq", dev),
                                 _vec(gk, head_dim, torch.bfloat16, "gk", dev),
                                 _vec(rstd, T * heads, torch.float32, "rstd", dev), out.data_ptr(),
                                 _rows(out, T, cols, "out", dev), partial.data_ptr(), dgq.data_ptr(), dgk.data_ptr(),
                                 T, n_heads, n_kv_heads, head_dim, rot, interleaved, pos, tab, n_pos, err.data_ptr(),
                                 _stream(dev)), "qk_norm_rope_bwd")
    return out, dgq, dgk


def swiglu_fwd(gu, f):
    T = gu.shape[0]
    act = torch.empty(T, f, dtype=torch.bfloat16, device=gu.device)
    _ok(_lib.load().mtk_swiglu_fwd(gu.data_ptr(), act.data_ptr(), T, f, _s()), "swiglu_fwd")
    return act


def swiglu_bwd(gu, dact, f):
    T = gu.shape[0]
    dgu = torch.empty(T, 2 * f, dtype=torch.bfloat16, device=gu.device)
    _ok(_lib.load().mtk_swiglu_bwd(gu.data_ptr(), dact.data_ptr(), dgu.data_ptr(), T, f, _s()), "swiglu_bwd")
    return dgu


def embed_fwd(tok, E):
    T = tok.numel()
    V, h = E.shape
    x = torch.empty(T, h, dtype=torch.float32, device=E.device)
    _ok(_lib.load().mtk_embed_fwd(tok.data_ptr(), E.data_ptr(), x.data_ptr(), T, h, _s()), "embed_fwd")
    return x


def embed_bwd(order, offsets, dx, V):
    h = dx.shape[1]
    dE = torch.empty(V, h, dtype=torch.bfloat16, device=dx.device)
    _ok(_lib.load().mtk_embed_bwd(order.data_ptr(), offsets.data_ptr(), dx.data_ptr(), dE.data_ptr(), V, h, _s()),
        "embed_bwd")
    return dE


def cross_entropy(logits, labels):
    T, V = logits.shape
    dl = torch.empty(T, V, dtype=torch.bfloat16, device=logits.device)
    rl = torch.empty(T, dtype=torch.float32, device=logits.device)
    loss = torch.empty(1, dtype=torch.float32, device=logits.device)
    _ok(_lib.load().mtk_cross_entropy(logits.data_ptr(), labels.data_ptr(), dl.data_ptr(), rl.data_ptr(),
                                      loss.data_ptr(), T, V, _s()), "cross_entropy")
    return loss, rl, dl


def attn_fwd(qkv, B, s, nh, nkv, hd, err=None):
    o = torch.empty(B * s, nh * hd, dtype=torch.bfloat16, device=qkv.device)
    lse = torch.empty(B, nh, s, dtype=torch.float32, device=qkv.device)
    err = _err(err, qkv.device)
    _ok(_lib.load().mtk_attn_fwd(qkv.data_ptr(), o.data_ptr(), lse.data_ptr(), B, s, nh, nkv, hd, err.data_ptr(),
                                 _s()), "attn_fwd")
    return o, lse


def attn_bwd(qkv, o, lse, dout, B, s, nh, nkv, hd, err=None, cos_sin=None):
    """dqkv; with cos_sin (fp32 [s][hd/2][2]) dq and dk get the transpose RoPE rotation."""
    dqkv = torch.empty_like(qkv)
    delta = torch.empty(B, nh, (s + 127) // 128 * 128, 2, dtype=torch.float32, device=qkv.device)
    err = _err(err, qkv.device)
    lib = _lib.load()
    if cos_sin is None:
        _ok(lib.mtk_attn_bwd(qkv.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(), dqkv.data_ptr(),
                             delta.data_ptr(), B, s, nh, nkv, hd, err.data_ptr(), _s()), "attn_bwd")
    else:
        _ok(lib.mtk_attn_bwd_rope(qkv.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(), dqkv.data_ptr(),
                                  delta.data_ptr(), cos_sin.data_ptr(), B, s, nh, nkv, hd, err.data_ptr(), _s()),
            "attn_bwd_rope")
    return dqkv


def _int32(a, what):
    """A contiguous int32 array of the same whole numbers."""
    a = np.asarray(a)
    _need(a.size == 0 or (a.dtype.kind in "iu" and a.min() >= -2 ** 31 and a.max() < 2 ** 31),
          f"{what}: 32-bit integers")
    return np.ascontiguousarray(a, dtype=np.int32)


def doc_spans(bounds, B, s, prefix=None):
    """(lo, hi, positions) numpy int32 [B*s] of packed documents: document d holds the tokens
    bounds[d] <= t < bounds[d+1]; prefix: how many of its first tokens all of it sees (None: causal)."""
    bounds = _int32(bounds, "bounds")
    _need(bounds.ndim == 1 and bounds.size >= 1, "bounds: n_docs + 1 token indices")
    if prefix is not None:
        prefix = _int32(prefix, "prefix")
        _need(prefix.shape == (bounds.size - 1,), "prefix: one length for each document")
    _need(B > 0 and s > 0, "B and s: positive")
    out = np.empty((3, B * s), dtype=np.int32)
    _ok(_lib.load().mtk_doc_spans(bounds.ctypes.data, bounds.size - 1, None if prefix is None else prefix.ctypes.data,
                                  B, s, out[0].ctypes.data, out[1].ctypes.data, out[2].ctypes.data), "doc_spans")
    return out[0], out[1], out[2]


def _span_args(q, k, v, B, s, nh, nkv, hd, lo, hi, slopes, dev):
    T = B * s
    return (q.data_ptr(), _rows(q, T, nh * hd, "q", dev), k.data_ptr(), _rows(k, T, nkv * hd, "k", dev), v.data_ptr(),
            _rows(v, T, nkv * hd, "v", dev), None if lo is None else _vec(lo, T, torch.int32, "lo", dev),
            None if hi is None else _vec(hi, T, torch.int32, "hi", dev),
            None if slopes is None else _vec(slopes, nh, torch.float32, "slopes", dev))


def attn_span_fwd(q, k, v, B, s, nh, nkv, hd, lo=None, hi=None, scale=None, cap=0.0, slopes=None, out=None, err=None):
    """(o, lse) of attention in which row i sees the keys lo[i] <= j < hi[i] (int32 [B*s], see
    doc_spans; None: causal). scale: 1/sqrt(hd) if None; cap: tanh cap of the scores (0: none);
    slopes: fp32 [nh], lowers the scores by slopes[h] |i - j|. q, k, v may be column ranges of
    wider tensors. With a cap up to 50.5 and no slopes, v has to lie between 2^-40 and 2^40 in size, or be 0."""
    dev = _device(q)
    *ptrs, sl = _span_args(q, k, v, B, s, nh, nkv, hd, lo, hi, slopes, dev)
    if out is None:
        out = torch.empty((B * s, nh * hd), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((B, nh, s), dtype=torch.float32, device=q.device)
    err = _err(err, q.device)
    _ok(_lib.load().mtk_attn_span_fwd(*ptrs, out.data_ptr(), _rows(out, B * s, nh * hd, "out", dev), lse.data_ptr(), B,
                                      s, nh, nkv, hd, hd ** -0.5 if scale is None else scale, cap, sl, err.data_ptr(),
                                      _stream(dev)), "attn_span_fwd")
    return out, lse


@functools.lru_cache(maxsize=256)
def _span_scratch(B, s, nh, nkv, hd):
    return _lib.load().mtk_attn_span_bwd_scratch_bytes(B, s, nh, nkv, hd)


def attn_span_bwd(q, k, v, o, lse, dout, B, s, nh, nkv, hd, lo=None, hi=None, scale=None, cap=0.0, slopes=None,
                  out=None, err=None):
    """(dq, dk, dv) of attn_span_fwd; out: three tensors to write, such as the column ranges of a fused
    projection's gradient; None: new ones."""
    dev = _device(q)
    *ptrs, sl = _span_args(q, k, v, B, s, nh, nkv, hd, lo, hi, slopes, dev)
    T = B * s
    if out is None:
        out = [torch.empty((T, n * hd), dtype=torch.bfloat16, device=q.device) for n in (nh, nkv, nkv)]
    dq, dk, dv = out
    lib = _lib.load()
    scratch = torch.empty(_span_scratch(B, s, nh, nkv, hd), dtype=torch.uint8, device=q.device)
    err = _err(err, q.device)
    _ok(lib.mtk_attn_span_bwd(*ptrs, o.data_ptr(), _rows(o, T, nh * hd, "o", dev),
                              _vec(lse, T * nh, torch.float32, "lse", dev), dout.data_ptr(),
                              _rows(dout, T, nh * hd, "dout", dev), dq.data_ptr(), _rows(dq, T, nh * hd, "dq", dev),
                              dk.data_ptr(), _rows(dk, T, nkv * hd, "dk", dev), dv.data_ptr(),
                              _rows(dv, T, nkv * hd, "dv", dev), scratch.data_ptr(), B, s, nh, nkv, hd,
                              hd ** -0.5 if scale is None else scale, cap, sl, err.data_ptr(), _stream(dev)),
        "attn_span_bwd")
    return dq, dk, dv
