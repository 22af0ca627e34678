"""Cases of the packed-document attention block: rotary positions, query/key norms with the rotation,
and attention over spans (document and prefix masks, capped scores, a distance bias).

`run` computes a case in plain torch, or, where `own` is set, through the framework's kernels.
"""
import math
import random

import torch

own = False

BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
EPS = 1e-5
THETA = 10000.0


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one token at the end of a 131072-token context, 14B GQA heads: a call's latency
        {"name": "rotary_token", "op": "rotary", "T": 1, "heads": 48, "hd": 128, "rot": 128, "inter": False,
         "inverse": False, "n_pos": 131072, "doc": 0},
        # 7B batch of two 4096-token sequences of packed documents, neighbouring columns paired
        {"name": "rotary_7b", "op": "rotary", "T": 8192, "heads": 64, "hd": 128, "rot": 128, "inter": True,
         "inverse": False, "n_pos": 4096, "doc": 700},
        # rotation table of a short context, half of the head rotated
        {"name": "table_4096", "op": "table", "n_pos": 4096, "rot": 64, "scaling": "plain", "factor": 1.0},
        # rotation table of the 131072-token context, extended from 4096 by bands of wavelengths
        {"name": "table_131072", "op": "table", "n_pos": 131072, "rot": 128, "scaling": "bands", "factor": 32.0},
        # 14B forward: 40 query and 8 key heads
        {"name": "qknorm_fwd_14b", "op": "qk_fwd", "T": 4096, "nh": 40, "nkv": 8, "hd": 128, "rot": 128,
         "inter": False, "n_pos": 4096, "doc": 0},
        # 7B backward, packed documents
        {"name": "qknorm_bwd_7b", "op": "qk_bwd", "T": 8192, "nh": 32, "nkv": 32, "hd": 128, "rot": 128,
         "inter": False, "n_pos": 4096, "doc": 700},
        # the tiny decoder's backward, a quarter of the head rotated in neighbouring pairs
        {"name": "qknorm_bwd_tiny", "op": "qk_bwd", "T": 256, "nh": 4, "nkv": 4, "hd": 64, "rot": 16,
         "inter": True, "n_pos": 128, "doc": 0},
        # 7B forward over packed documents with some padding at the end of each sequence
        {"name": "attn_fwd_docs_7b", "op": "attn_fwd", "B": 2, "s": 4096, "nh": 32, "nkv": 32, "hd": 128,
         "doc": 700, "pad": 77, "prefix": 0, "cap": 0.0, "bias": False},
        # one long document whose first quarter is a prefix seen by all of it, capped scores, GQA
        {"name": "attn_fwd_long", "op": "attn_fwd", "B": 1, "s": 16384, "nh": 8, "nkv": 2, "hd": 128,
         "doc": 0, "pad": 0, "prefix": 25, "cap": 30.0, "bias": False},
        # 7B backward over packed documents
        {"name": "attn_bwd_docs_7b", "op": "attn_bwd", "B": 2, "s": 4096, "nh": 32, "nkv": 32, "hd": 128,
         "doc": 700, "pad": 77, "prefix": 0, "cap": 0.0, "bias": False},
        # 14B GQA backward, causal, capped scores
        {"name": "attn_bwd_cap_14b", "op": "attn_bwd", "B": 1, "s": 4096, "nh": 40, "nkv": 8, "hd": 128,
         "doc": 0, "pad": 0, "prefix": 0, "cap": 50.0, "bias": False},
        # small ragged backward: short documents with prefixes, a distance bias, 64-wide heads, one key head
        {"name": "attn_bwd_ragged", "op": "attn_bwd", "B": 2, "s": 333, "nh": 4, "nkv": 1, "hd": 64,
         "doc": 90, "pad": 21, "prefix": 40, "cap": 0.0, "bias": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "table", "qk_fwd", "qk_bwd", "attn_fwd", "attn_bwd", "attn_fwd", "attn_bwd"])
    if op == "table":
        return {"op": op, "n_pos": _log_int(rng, 100, 131072), "rot": rng.choice([8, 16, 32, 64, 96, 128]),
                "scaling": rng.choice(["plain", "linear", "base", "bands"]), "factor": rng.choice([2.0, 8.0, 32.0])}
    hd = rng.choice([64, 128])
    inter = rng.random() < 0.5
    if op == "rotary":
        heads = rng.choice([2, 5, 8, 24, 32, 48, 64])
        T = _log_int(rng, 1, 8192 * 64 * 128 // (heads * hd))
        n_pos = _log_int(rng, 1, 32768)
        return {"op": op, "T": T, "heads": heads, "hd": hd, "rot": rng.choice([hd // 4, hd // 2, hd]), "inter": inter,
                "inverse": rng.random() < 0.5, "n_pos": n_pos, "doc": rng.choice([0, 0, 300])}
    nh, nkv = rng.choice([(4, 4), (4, 1), (8, 2), (16, 16), (32, 32), (40, 8), (32, 8)])
    if op in ("qk_fwd", "qk_bwd"):
        T = _log_int(rng, 1, 8192 * 64 * 128 // ((nh + nkv) * hd))
        return {"op": op, "T": T, "nh": nh, "nkv": nkv, "hd": hd, "rot": rng.choice([hd // 4, hd // 2, hd]),
                "inter": inter, "n_pos": _log_int(rng, 1, 32768), "doc": rng.choice([0, 0, 300])}
    B = rng.choice([1, 1, 2, 4])
    s = _log_int(rng, 1, 4096)
    cap = rng.choice([0.0, 0.0, 30.0, 50.0])
    c = {"op": op, "B": B, "s": s, "nh": nh if B * nh <= 64 else 16, "nkv": nkv if B * nh <= 64 else 16, "hd": hd,
         "doc": rng.choice([0, 0, 50, 400, 1500]), "pad": rng.choice([0, 0, s // 9]),
         "prefix": rng.choice([0, 0, 30, 100]), "cap": cap, "bias": rng.random() < 0.3}
    while work(c)["flops"] > 4.2e11:
        s = s * 4 // 5
        c.update(s=s, pad=s // 9 if c["pad"] else 0)
    return c


# ---------------------------------------------------------------------------- documents
def _lengths(n, doc, salt):
    """Document lengths that fill n rows: one of n rows where doc is 0, else about doc rows each."""
    if n <= 0:
        return []
    if not doc:
        return [n]
    r, out, left = random.Random(1000003 * n + 101 * doc + salt), [], n
    while left > 0:
        k = min(left, max(1, int(r.expovariate(1.0 / doc))))
        out.append(k)
        left -= k
    return out


def _documents(case, seed):
    """Per sequence, the documents' (start, length, prefix): lengths of the case, in the seed's order."""
    out = []
    for b in range(case["B"]):
        ls = _lengths(case["s"] - case["pad"], case["doc"], b)
        random.Random(seed * 7919 + b).shuffle(ls)
        at, docs = 0, []
        for k in ls:
            docs.append((at, k, k * case["prefix"] // 100))
            at += k
        out.append(docs)
    return out


def _pairs(case):
    """(query, key) pairs that are seen, over the batch, for one query head."""
    return sum(k * (k + 1) // 2 + p * (p - 1) // 2 if p else k * (k + 1) // 2
               for docs in _documents(case, 0) for _, k, p in docs)


# ---------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "rotary":
        n = case["T"] * case["heads"]
        rows = min(case["T"], case["n_pos"])
        return {"bytes": 4 * n * case["hd"] + 4 * rows * case["rot"] + 4 * case["T"], "flops": 3 * n * case["rot"]}
    if op == "table":
        n = case["n_pos"] * case["rot"] // 2
        return {"bytes": 8 * n, "flops": 10 * n}
    if op in ("qk_fwd", "qk_bwd"):
        n, rows = case["T"] * (case["nh"] + case["nkv"]), min(case["T"], case["n_pos"])
        small = 4 * n + 4 * rows * case["rot"] + 4 * case["T"] + 4 * case["hd"]
        if op == "qk_fwd":
            return {"bytes": 4 * n * case["hd"] + small, "flops": n * (4 * case["hd"] + 3 * case["rot"])}
        return {"bytes": 6 * n * case["hd"] + small + 4 * case["hd"], "flops": n * (9 * case["hd"] + 3 * case["rot"])}
    T, nh, nkv, hd = case["B"] * case["s"], case["nh"], case["nkv"], case["hd"]
    fl = _pairs(case) * nh * hd
    lse = 4 * T * nh
    if op == "attn_fwd":
        return {"bytes": 2 * T * hd * (2 * nh + 2 * nkv) + lse + 8 * T, "flops": 4 * fl}
    return {"bytes": 2 * T * hd * (4 * nh + 4 * nkv) + lse + 8 * T, "flops": 10 * fl}


# ---------------------------------------------------------------------------- state
def _positions(T, doc, n_pos, seed):
    """Position of each of T tokens: restarting at each document (a document longer than n_pos starts again)."""
    if not doc:
        return (torch.arange(T, dtype=I32) + (n_pos - 1 if T == 1 else 0)) % n_pos
    ls = _lengths(T, doc, 7)
    random.Random(seed).shuffle(ls)
    return torch.cat([torch.arange(k, dtype=I32) for k in ls]) % n_pos


def _frequencies(rot, theta=THETA, scaling="plain", factor=1.0):
    """Radians a position for each of rot/2 pairs (64 bits)."""
    i = torch.arange(rot // 2, dtype=F64, device="cuda")
    if scaling == "base":
        return (theta * factor ** (rot / (rot - 2))) ** (-2 * i / rot)
    f = theta ** (-2 * i / rot)
    if scaling == "linear":
        return f / factor
    if scaling == "bands":
        w = ((4096 * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return f * (w + (1 - w) / factor)
    return f


def _amplitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "bands" else 1.0


def _table(n_pos, rot):
    a = torch.arange(n_pos, dtype=F64, device="cuda")[:, None] * _frequencies(rot)
    return torch.stack([a.cos(), a.sin()], -1).to(F32)


def prepare(case, seed):
    op = case["op"]
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(BF)

    st = {"case": case, "err": torch.zeros(1, dtype=I32, device="cuda")}
    if op == "table":
        st["theta"] = THETA * random.Random(seed).uniform(1.0, 50.0)  # a table's only input besides its sizes
        return st
    if op == "rotary":
        # columns q | k of a projection that also holds v: the row is longer than what is rotated
        st["x"] = rnd(case["T"], (case["heads"] + 2) * case["hd"])[:, :case["heads"] * case["hd"]]
        st["pos"] = _positions(case["T"], case["doc"], case["n_pos"], seed).cuda()
        st["table"] = _table(case["n_pos"], case["rot"])
        return st
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    if op in ("qk_fwd", "qk_bwd"):
        T = case["T"]
        st["qkv"] = rnd(T, (nh + 2 * nkv) * hd, scale=1.5)
        st["gq"], st["gk"] = ((1 + 0.2 * torch.randn(hd, device="cuda", generator=g)).to(BF) for _ in range(2))
        st["pos"] = _positions(T, case["doc"], case["n_pos"], seed).cuda()
        st["table"] = _table(case["n_pos"], case["rot"])
        if op == "qk_bwd":
            x = st["qkv"][:, :(nh + nkv) * hd].float().view(T, nh + nkv, hd)
            st["rstd"] = (x.square().mean(-1) + EPS).rsqrt()
            st["dy"] = rnd(T, (nh + nkv) * hd, scale=0.1)
        return st
    B, s = case["B"], case["s"]
    T = B * s
    # queries and keys as the norms leave them; larger ones where the cap has something to do
    st["qk"] = rnd(T, (nh + nkv) * hd, scale=2.0 if case["cap"] else 1.0)
    st["qkv"] = rnd(T, (nh + 2 * nkv) * hd)
    lo, hi = torch.zeros(T, dtype=I32), torch.zeros(T, dtype=I32)
    for b, docs in enumerate(_documents(case, seed)):
        for at, k, p in docs:
            rows = slice(b * s + at, b * s + at + k)
            lo[rows] = at
            hi[rows] = at + torch.clamp(torch.arange(1, k + 1, dtype=I32), min=p)
    st["lo"], st["hi"] = lo.cuda(), hi.cuda()
    st["slopes"] = 2.0 ** (-8.0 * torch.arange(1, nh + 1, device="cuda", dtype=F32) / nh) if case["bias"] else None
    st["scale"] = 1.0 / math.sqrt(hd)
    if op == "attn_bwd":
        st["o"], st["lse"] = _plain_attn_fwd(st)
        st["dout"] = rnd(T, nh * hd, scale=0.1)
    return st


# ---------------------------------------------------------------------------- plain forms
def _rotate(x, table, pos, rot, inter, inverse=False):
    """x [T, heads, hd] in 32 bits, the first rot columns of each head rotated."""
    cs = table[pos.long()][:, None]
    c, s = cs[..., 0], -cs[..., 1] if inverse else cs[..., 1]
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :rot // 2], r[..., rot // 2:])
    na, nb = a * c - b * s, b * c + a * s
    new = torch.stack([na, nb], -1).flatten(-2) if inter else torch.cat([na, nb], -1)
    return torch.cat([new, x[..., rot:]], -1)


def _plain_rotary(st):
    c = st["case"]
    x = st["x"].float().reshape(c["T"], c["heads"], c["hd"])
    return _rotate(x, st["table"], st["pos"], c["rot"], c["inter"], c["inverse"]).flatten(1).to(BF)


def _plain_table(st):
    c = st["case"]
    f = _frequencies(c["rot"], st["theta"], c["scaling"], c["factor"])
    a = torch.arange(c["n_pos"], dtype=F64, device="cuda")[:, None] * f
    return (_amplitude(c) * torch.stack([a.cos(), a.sin()], -1)).to(F32)


def _plain_qk_fwd(st):
    c = st["case"]
    T, nh, nkv, hd = c["T"], c["nh"], c["nkv"], c["hd"]
    x = st["qkv"][:, :(nh + nkv) * hd].float().reshape(T, nh + nkv, hd)
    r = (x.square().mean(-1) + EPS).rsqrt()
    g = torch.cat([st["gq"].float().expand(nh, hd), st["gk"].float().expand(nkv, hd)])
    y = _rotate(x * r[..., None] * g, st["table"], st["pos"], c["rot"], c["inter"])
    return y.flatten(1).to(BF), r


def _plain_qk_bwd(st):
    c = st["case"]
    T, nh, nkv, hd = c["T"], c["nh"], c["nkv"], c["hd"]
    x = st["qkv"][:, :(nh + nkv) * hd].float().reshape(T, nh + nkv, hd)
    r = st["rstd"][..., None]
    g = torch.cat([st["gq"].float().expand(nh, hd), st["gk"].float().expand(nkv, hd)])
    u = _rotate(st["dy"].float().view(T, nh + nkv, hd), st["table"], st["pos"], c["rot"], c["inter"], inverse=True)
    xh = x * r
    ug = u * g
    dx = r * (ug - xh * (ug * xh).mean(-1, keepdim=True))
    dg = (u * xh).sum(0)
    return dx.flatten(1).to(BF), dg[:nh].sum(0).to(BF), dg[nh:].sum(0).to(BF)


def _heads(x, B, s, n, hd, groups=1):
    """[B*s, n*hd] as 32-bit [B, n/groups, groups, s, hd]."""
    return x.float().reshape(B, s, n // groups, groups, hd).permute(0, 2, 3, 1, 4)


def _scores(st):
    """Scores in 32 bits with what is not seen at -inf, and the cap's derivative."""
    c = st["case"]
    B, s, nh, nkv, hd = c["B"], c["s"], c["nh"], c["nkv"], c["hd"]
    q = _heads(st["qk"][:, :nh * hd], B, s, nh, hd, nh // nkv)
    k = _heads(st["qk"][:, nh * hd:], B, s, nkv, hd)
    z = (q @ k.transpose(-1, -2)) * st["scale"]
    slope = None
    if c["cap"]:
        t = torch.tanh(z / c["cap"])
        z, slope = c["cap"] * t, 1 - t * t
    j = torch.arange(s, device="cuda", dtype=I32)
    if c["bias"]:
        z = z - st["slopes"].view(nkv, nh // nkv, 1, 1) * (j[:, None] - j).abs().float()
    lo, hi = (st[n].view(B, 1, 1, s, 1) for n in ("lo", "hi"))
    return q, k, z.masked_fill((j < lo) | (j >= hi), -math.inf), slope


def _plain_attn_fwd(st):
    c = st["case"]
    B, s, nh, nkv, hd = c["B"], c["s"], c["nh"], c["nkv"], c["hd"]
    _, _, z, _ = _scores(st)
    v = _heads(st["qkv"][:, (nh + nkv) * hd:], B, s, nkv, hd)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(z - m)
    l = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m + torch.log(l)) / math.log(2.0)
    return o.permute(0, 3, 1, 2, 4).reshape(B * s, nh * hd).to(BF), lse.reshape(B, nh, s)


def _plain_attn_bwd(st):
    c = st["case"]
    B, s, nh, nkv, hd = c["B"], c["s"], c["nh"], c["nkv"], c["hd"]
    G = nh // nkv
    q, k, z, slope = _scores(st)
    v = _heads(st["qkv"][:, (nh + nkv) * hd:], B, s, nkv, hd)
    do, o = _heads(st["dout"], B, s, nh, hd, G), _heads(st["o"], B, s, nh, hd, G)
    lse = st["lse"].view(B, nkv, G, s, 1) * math.log(2.0)
    p = torch.exp(z - torch.where(lse == -math.inf, torch.zeros_like(lse), lse))
    dv = (p.transpose(-1, -2) @ do).sum(2)
    ds = p * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
    if slope is not None:
        ds = ds * slope
    dq = (ds @ k) * st["scale"]
    dk = (ds.transpose(-1, -2) @ q).sum(2) * st["scale"]
    return (dq.permute(0, 3, 1, 2, 4).reshape(B * s, nh * hd).to(BF),
            dk.transpose(1, 2).reshape(B * s, nkv * hd).to(BF), dv.transpose(1, 2).reshape(B * s, nkv * hd).to(BF))


PLAIN = {"rotary": _plain_rotary, "table": _plain_table, "qk_fwd": _plain_qk_fwd, "qk_bwd": _plain_qk_bwd,
         "attn_fwd": _plain_attn_fwd, "attn_bwd": _plain_attn_bwd}


# ---------------------------------------------------------------------------- the framework's calls
def _own(st):
    from host_memory_streamed_stream_gb300 import kernels as K

    c = st["case"]
    op, err = c["op"], st["err"]
    if op == "table":
        f = K.rotary_inv_freq(c["rot"], theta=st["theta"], scaling=c["scaling"], factor=c["factor"],
                              original_positions=4096, low=1.0, high=32.0)
        return K.rotary_table(f, c["n_pos"], amplitude=_amplitude(c))
    if op == "rotary":
        return K.rotary(st["x"], c["heads"], c["hd"], st["table"], positions=st["pos"], interleaved=c["inter"],
                        inverse=c["inverse"], err=err)
    nh, nkv, hd = c["nh"], c["nkv"], c["hd"]
    if op == "qk_fwd":
        return K.qk_norm_rope(st["qkv"], st["gq"], st["gk"], nh, nkv, hd, st["table"], positions=st["pos"],
                              interleaved=c["inter"], eps=EPS, err=err)
    if op == "qk_bwd":
        return K.qk_norm_rope_bwd(st["dy"], st["qkv"], st["gq"], st["gk"], st["rstd"], nh, nkv, hd, st["table"],
                                  positions=st["pos"], interleaved=c["inter"], err=err)
    q, k, v = st["qk"][:, :nh * hd], st["qk"][:, nh * hd:], st["qkv"][:, (nh + nkv) * hd:]
    kw = dict(lo=st["lo"], hi=st["hi"], scale=st["scale"], cap=c["cap"], slopes=st["slopes"], err=err)
    if op == "attn_fwd":
        return K.attn_span_fwd(q, k, v, c["B"], c["s"], nh, nkv, hd, **kw)
    return K.attn_span_bwd(q, k, v, st["o"], st["lse"], st["dout"], c["B"], c["s"], nh, nkv, hd, **kw)


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- 64 bits
def _turn(x, table, pos, rot, inter, sign):
    """The first rot columns of each head as complex numbers times the table's (64 bits)."""
    w = torch.complex(table[..., 0].double(), sign * table[..., 1].double())[pos.long()].unsqueeze(1)
    head, rest = x[..., :rot].unflatten(-1, (-1, 2) if inter else (2, -1)), x[..., rot:]
    z = w * (torch.complex(head[..., 0], head[..., 1]) if inter else torch.complex(head[..., 0, :], head[..., 1, :]))
    return torch.cat([torch.stack([z.real, z.imag], -1 if inter else -2).flatten(-2), rest], -1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "table":
        r, n = case["rot"], case["n_pos"]
        base = st["theta"] * (case["factor"] ** (r / (r - 2)) if case["scaling"] == "base" else 1.0)
        f = torch.exp(torch.arange(0, r, 2, dtype=F64) * (-math.log(base) / r))
        if case["scaling"] == "linear":
            f = f / case["factor"]
        elif case["scaling"] == "bands":
            turns = 4096 * f / (2 * math.pi)
            keep = ((turns - 1.0) / 31.0).clamp(0, 1)
            f = keep * f + (1 - keep) * f / case["factor"]
        angle = torch.outer(torch.arange(n, dtype=F64), f).cuda()
        return torch.view_as_real(torch.polar(torch.full_like(angle, _amplitude(case)), angle))
    if op == "rotary":
        x = st["x"].double().reshape(case["T"], case["heads"], case["hd"])
        return _turn(x, st["table"], st["pos"], case["rot"], case["inter"], -1 if case["inverse"] else 1).flatten(1)
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    if op in ("qk_fwd", "qk_bwd"):
        T, H = case["T"], nh + nkv
        x = st["qkv"].double().reshape(T, nh + 2 * nkv, hd)[:, :H]
        r = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / hd + EPS)
        n = x * r
        g = torch.stack([st["gq"].double()] * nh + [st["gk"].double()] * nkv)
        if op == "qk_fwd":
            return _turn(n * g, st["table"], st["pos"], case["rot"], case["inter"], 1).flatten(1), r[..., 0]
        u = _turn(st["dy"].double().reshape(T, H, hd), st["table"], st["pos"], case["rot"], case["inter"], -1)
        dn = u * g
        # the derivative of x r(x): r (1 - n n^T / hd) (the mean with eps in it, as r has)
        dx = r * dn - r * n * (dn * n).sum(-1, keepdim=True) / hd
        dg = torch.einsum("thd,thd->hd", u, n)
        return dx.flatten(1), dg[:nh].sum(0), dg[nh:].sum(0)
    B, s = case["B"], case["s"]
    G = nh // nkv
    back = op == "attn_bwd"
    q = st["qk"][:, :nh * hd].reshape(B, s, nh, hd)
    k = st["qk"][:, nh * hd:].reshape(B, s, nkv, hd)
    v = st["qkv"].reshape(B, s, nh + 2 * nkv, hd)[:, :, nh + nkv:]
    j = torch.arange(s, device="cuda")
    o = torch.zeros(B, s, nh, hd, dtype=F64, device="cuda")
    lse = torch.zeros(B, nh, s, dtype=F64, device="cuda")
    dq, dk, dv = torch.zeros_like(o), *(torch.zeros(B, s, nkv, hd, dtype=F64, device="cuda") for _ in range(2))
    far = (j[:, None] - j[None]).abs().double() if case["bias"] else None
    for b in range(B):
        lo, hi = st["lo"][b * s:(b + 1) * s].long(), st["hi"][b * s:(b + 1) * s].long()
        seen = (j[None] >= lo[:, None]) & (j[None] < hi[:, None])
        some = seen.any(1)
        for h in range(nh):
            a, c, e = q[b, :, h].double(), k[b, :, h // G].double(), v[b, :, h // G].double()
            z = a @ c.T * st["scale"]
            if case["cap"]:
                z = torch.tanh(z / case["cap"])
                cut = 1 - z * z if back else None
                z = z * case["cap"]
            if case["bias"]:
                z = z - float(st["slopes"][h]) * far
            z = torch.where(seen, z, torch.full((), -math.inf, dtype=F64, device="cuda"))
            top = torch.logsumexp(z, 1)
            lse[b, h] = top / math.log(2.0)
            p = torch.exp(z - torch.where(some, top, torch.zeros_like(top))[:, None])
            o[b, :, h] = p @ e
            if back:
                d = st["dout"].reshape(B, s, nh, hd)[b, :, h].double()
                dv[b, :, h // G] += p.T @ d
                ds = p * (d @ e.T - (d * o[b, :, h]).sum(1, keepdim=True))
                if case["cap"]:
                    ds = ds * cut
                dq[b, :, h] = ds @ c * st["scale"]
                dk[b, :, h // G] += ds.T @ a * st["scale"]
    if back:
        return dq.reshape(B * s, -1), dk.reshape(B * s, -1), dv.reshape(B * s, -1)
    return o.reshape(B * s, -1), lse
