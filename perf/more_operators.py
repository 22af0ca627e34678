"""Cases of the ends of a fine-tuning step: the embedding with its gradient by sorted tokens, layer norm, and the
losses on a policy's logits (clipped policy loss with a KL term, preference loss over pairs of sequences).

`run` computes a case in plain torch, or, where `own` is set, through the framework's kernels.
"""
import math
import random

import torch

own = False

BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
TYPES = {"f32": F32, "bf16": BF}
EPS = 1e-5


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # the tiny decoder's batch, odd vocabulary whose last columns are padding: a call's latency
        {"name": "policy_tiny", "op": "policy", "T": 256, "V": 1021, "type": "bf16", "banned": 5, "masked": 40,
         "seq": 50, "hi": 0.2, "kl": 0.04, "scale": 1.0, "weighted": True},
        # 7B batch of sampled answers with their prompts, logits as the LM head's GEMM leaves them, temperature 0.7
        {"name": "policy_7b", "op": "policy", "T": 8192, "V": 32000, "type": "f32", "banned": 0, "masked": 25,
         "seq": 700, "hi": 0.28, "kl": 0.04, "scale": 1 / 0.7, "weighted": True},
        # two short pairs, no reference model, mean log-probabilities
        {"name": "pref_small", "op": "pref", "pairs": 2, "seq": 70, "V": 1021, "type": "f32", "masked": 30,
         "tail": 9, "kind": "sigmoid", "ref": False, "average": True, "smoothing": 0.0, "margin": 0.5, "beta": 2.0},
        # 14B vocabulary, pairs of answers to the same prompts, bf16 logits
        {"name": "pref_14b", "op": "pref", "pairs": 4, "seq": 500, "V": 152064, "type": "bf16", "masked": 25,
         "tail": 100, "kind": "sigmoid", "ref": True, "average": False, "smoothing": 0.1, "margin": 0.0,
         "beta": 0.1},
        # one row of the 14B width: a call's latency
        {"name": "ln_fwd_row", "op": "ln_fwd", "T": 1, "h": 5120, "type": "bf16", "bias": True, "pad": 0},
        # 7B batch, fp32 residual stream
        {"name": "ln_fwd_7b", "op": "ln_fwd", "T": 8192, "h": 4096, "type": "f32", "bias": True, "pad": 0},
        # odd width, rows inside a wider bf16 buffer, no bias
        {"name": "ln_bwd_ragged", "op": "ln_bwd", "T": 333, "h": 1160, "type": "bf16", "dy": "bf16", "res": False,
         "bias": False, "pad": 24},
        # 7B batch, fp32 residual stream and gradient
        {"name": "ln_bwd_7b", "op": "ln_bwd", "T": 8192, "h": 4096, "type": "f32", "dy": "f32", "res": True,
         "bias": True, "pad": 0},
        # the tiny decoder's batch: a call's latency
        {"name": "embed_fwd_tiny", "op": "embed_fwd", "T": 256, "h": 256, "V": 1024, "type": "bf16", "masked": 10},
        # 14B batch, fp32 residual stream
        {"name": "embed_fwd_14b", "op": "embed_fwd", "T": 4096, "h": 5120, "V": 152064, "type": "f32", "masked": 0},
        # 7B batch with a tenth of padding
        {"name": "embed_bwd_7b", "op": "embed_bwd", "T": 8192, "h": 4096, "V": 32000, "type": "f32", "masked": 10},
        # one 131072-token sequence, 7B width, bf16 gradient
        {"name": "embed_bwd_long", "op": "embed_bwd", "T": 131072, "h": 4096, "V": 32000, "type": "bf16",
         "masked": 0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["policy", "policy", "pref", "pref", "ln_fwd", "ln_bwd", "embed_fwd", "embed_bwd"])
    kind = rng.choice(["f32", "bf16"])
    if op in ("policy", "pref"):
        V = _log_int(rng, 64, 152064)
        rows = min(8192, 8192 * 32000 // V)
        c = {"op": op, "V": V, "type": kind, "masked": rng.choice([0, 25, 60])}
        if op == "policy":
            c.update(T=_log_int(rng, 1, rows), banned=rng.choice([0, 0, 7]), seq=_log_int(rng, 10, 1000),
                     hi=rng.choice([0.2, 0.28]), kl=rng.choice([0.0, 0.04]), scale=rng.choice([1.0, 1 / 0.7]),
                     weighted=rng.random() < 0.7)
            return c
        pairs = _log_int(rng, 1, 32)
        loss = rng.choice(["sigmoid", "sigmoid", "hinge", "square"])
        c.update(pairs=pairs, seq=_log_int(rng, 1, max(1, min(2000, rows // (3 * pairs)))),
                 tail=rng.choice([0, 0, 31]), kind=loss, ref=rng.random() < 0.7, average=rng.random() < 0.3,
                 smoothing=rng.choice([0.0, 0.1]), margin=rng.choice([0.0, 0.3]), beta=rng.choice([0.1, 0.5]))
        return c
    if op in ("ln_fwd", "ln_bwd"):
        h = 8 * _log_int(rng, 4, 2048)
        c = {"op": op, "T": _log_int(rng, 1, 8192 * 4096 // h), "h": h, "type": kind, "bias": rng.random() < 0.7,
             "pad": rng.choice([0, 0, 16])}
        if op == "ln_bwd":
            c.update(dy=rng.choice(["f32", "bf16"]), res=rng.random() < 0.5)
        return c
    h = 8 * _log_int(rng, 8, 1024)
    V = _log_int(rng, 100, min(152064, (1 << 30) // h))
    return {"op": op, "T": _log_int(rng, 1, min(131072, (1 << 28) // h)), "h": h, "V": V, "type": kind,
            "masked": rng.choice([0, 10, 50])}


# ---------------------------------------------------------------------------- sequences and tokens
def _lengths(n, mean, salt):
    """Lengths that fill n rows, about `mean` each."""
    r, out, left = random.Random(1000003 * n + 101 * mean + salt), [], n
    while left > 0:
        k = min(left, max(1, int(r.uniform(0.4, 1.6) * mean)))
        out.append(k)
        left -= k
    return out


def _sequences(case):
    """(lengths, of which prompt) of the case's sequences; rows behind the last one are padding."""
    if case["op"] == "policy":
        ls = _lengths(case["T"], case["seq"], 0)
    else:
        r = random.Random(case["pairs"] * 7919 + case["seq"])
        ls = [max(1, int(r.uniform(0.5, 1.5) * case["seq"])) for _ in range(2 * case["pairs"])]
    return ls, [k * case["masked"] // 100 for k in ls]


def _rows(case):
    """(rows, trained rows)"""
    ls, prompt = _sequences(case)
    return sum(ls) + case.get("tail", 0), sum(ls) - sum(prompt)


def _frequency(V):
    """Share of each token id, most frequent first."""
    p = 1.0 / (torch.arange(V, dtype=F64) + 2.7)
    return p / p.sum()


def _tokens(case, g):
    T, V = case["T"], case["V"]
    cdf = torch.cumsum(_frequency(V), 0).cuda()
    rank = torch.searchsorted(cdf, torch.rand(T, device="cuda", generator=g, dtype=F64)).clamp(max=V - 1)
    ids = torch.randperm(V, device="cuda", generator=g)[rank].to(I32)
    ids[T - T * case["masked"] // 100:] = -1
    return ids


# ---------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("policy", "pref"):
        T, n = _rows(case)
        esz = 4 if case["type"] == "f32" else 2
        small = 6 if op == "policy" else 5
        return {"bytes": n * case["V"] * esz + 2 * T * case["V"] + 4 * small * T, "flops": 8 * n * case["V"]}
    T, h = case["T"], case["h"]
    esz = 4 if case["type"] == "f32" else 2
    if op == "ln_fwd":
        return {"bytes": T * h * (esz + 2) + 8 * T + 4 * h, "flops": 8 * T * h}
    if op == "ln_bwd":
        per = esz + (4 if case["dy"] == "f32" else 2) + esz + (2 if esz == 4 else 0) + (esz if case["res"] else 0)
        return {"bytes": T * h * per + 8 * T + 6 * h, "flops": 14 * T * h}
    V, n = case["V"], case["T"] - case["T"] * case["masked"] // 100
    if op == "embed_fwd":
        distinct = float((1 - (1 - _frequency(V)) ** n).sum())
        return {"bytes": int(distinct) * h * 2 + T * h * esz + 4 * T, "flops": n * h}
    return {"bytes": n * h * esz + 2 * V * h + 4 * T, "flops": n * h}


# ---------------------------------------------------------------------------- state
def _logits(case, labels, g):
    """Logits of a model that has some idea of the label, in rows a multiple of 64 columns apart."""
    T, V = labels.numel(), case["V"]
    buf = torch.zeros(T, (V + 63) // 64 * 64, dtype=TYPES[case["type"]], device="cuda")
    z = buf[:, :V]
    for a in range(0, T, 1024):
        n = min(1024, T - a)
        part = 2.0 * torch.randn(n, V, device="cuda", generator=g)
        up = 4.0 + 8.0 * torch.rand(n, 1, device="cuda", generator=g)
        part.scatter_add_(1, labels[a:a + n].long().clamp(min=0)[:, None], up)
        z[a:a + n] = part
    if case.get("banned"):
        z[:, V - case["banned"]:] = -math.inf
    return z


def prepare(case, seed):
    op = case["op"]
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, scale=1.0, dtype=BF):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)

    st = {"case": case, "err": torch.zeros(1, dtype=I32, device="cuda")}
    if op in ("policy", "pref"):
        ls, prompt = _sequences(case)
        order = list(range(len(ls)))
        random.Random(seed).shuffle(order)
        ls, prompt = [ls[i] for i in order], [prompt[i] for i in order]
        T = _rows(case)[0]
        labels = torch.randint(0, case["V"] - case.get("banned", 0), (T,), device="cuda", generator=g, dtype=I32)
        where, at = torch.zeros(T, dtype=torch.bool), 0
        for k, p in zip(ls, prompt):
            where[at + p:at + k] = True
            at += k
        labels[~where.cuda()] = -1
        st["labels"] = labels
        st["logits"] = _logits(case, labels, g)
        logp = _logp(case, st["logits"], labels)[0]
        st["ref"] = (logp + 0.3 * torch.randn(T, device="cuda", generator=g)).float()
        if op == "pref":
            st["bounds"] = torch.tensor([0] + ls, dtype=I32).cumsum(0).to(I32).cuda()
            st["ref"] = st["ref"] if case["ref"] else None
            return st
        if not case["kl"]:
            st["ref"] = None
        old = (logp + 0.15 * torch.randn(T, device="cuda", generator=g)).float()
        # no ratio within rounding of the clip's borders, where the gradient jumps
        ratio = (logp - old.double()).exp()
        near = torch.minimum((ratio - 0.8).abs(), (ratio - 1 - case["hi"]).abs()) < 1e-4
        st["old"] = torch.where(near, old + 1e-3, old)
        adv = torch.randn(len(ls), device="cuda", generator=g)
        st["adv"] = torch.repeat_interleave(adv, torch.tensor(ls, device="cuda"))
        # every sequence counts the same, whatever its length
        each = torch.tensor([1.0 / (max(1, k - p) * len(ls)) for k, p in zip(ls, prompt)], device="cuda")
        st["weights"] = torch.repeat_interleave(each, torch.tensor(ls, device="cuda")) if case["weighted"] else None
        return st
    T, h, kind = case["T"], case["h"], TYPES[case["type"]]
    if op in ("ln_fwd", "ln_bwd"):
        # a residual stream with a mean and a few large channels
        big = 1 + 15 * (torch.rand(h, device="cuda", generator=g) < 0.01).float()
        x = torch.randn(T, h + case["pad"], device="cuda", generator=g)[:, :h]
        buf = torch.zeros(T, h + case["pad"], dtype=kind, device="cuda")
        buf[:, :h] = (0.3 + 1.5 * x) * big
        st["x"] = buf[:, :h]
        st["gamma"] = (1 + 0.2 * torch.randn(h, device="cuda", generator=g)).to(BF)
        st["beta"] = rnd(h, scale=0.2) if case["bias"] else None
        if op == "ln_bwd":
            _, st["mean"], st["rstd"] = _plain_ln_fwd(st)
            st["dy"] = rnd(T, h, scale=0.1, dtype=TYPES[case["dy"]])
            st["dres"] = rnd(T, h, scale=0.1, dtype=kind) if case["res"] else None
        return st
    st["tok"] = _tokens(case, g)
    st["scale"] = math.sqrt(h)
    if op == "embed_fwd":
        st["E"] = torch.empty(case["V"], h, dtype=BF, device="cuda")
        for a in range(0, case["V"], 16384):
            n = min(16384, case["V"] - a)
            st["E"][a:a + n] = rnd(n, h, scale=0.02)
    else:
        st["dx"] = rnd(T, h, scale=0.1, dtype=kind)
    return st


# ---------------------------------------------------------------------------- plain forms
def _logp(case, logits, labels):
    """Log-probability of each label, the rows' log of the sum (64 bits), and exp(z - max) with its sum."""
    z = logits.float() * case.get("scale", 1.0)
    m = z.amax(1, keepdim=True)
    zl = z.gather(1, labels.long().clamp(min=0)[:, None])
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True, dtype=F64)
    lse = m.double() + torch.log(total)
    return torch.where(labels >= 0, (zl - lse)[:, 0], 0.0), lse[:, 0], e, total.float()


def _grad_logits(case, labels, e, total, dlogp):
    """dlogp (onehot - softmax) in bf16."""
    k = dlogp.float()[:, None] * case.get("scale", 1.0)
    d = e.mul_(-k / total)
    d.scatter_add_(1, labels.long().clamp(min=0)[:, None], k)
    return torch.where((labels >= 0)[:, None], d, 0.0).to(BF)


def _plain_policy(st):
    c, labels = st["case"], st["labels"]
    logp, _, e, total = _logp(c, st["logits"], labels)
    ratio = torch.exp(logp - st["old"])
    adv = st["adv"].double()
    plain, cut = ratio * adv, ratio.clamp(1 - 0.2, 1 + c["hi"]) * adv
    loss = -torch.minimum(plain, cut)
    d = torch.where(plain <= cut, -plain, 0.0)
    if c["kl"]:
        far = st["ref"] - logp
        loss = loss + c["kl"] * (torch.exp(far) - far - 1)
        d = d + c["kl"] * (1 - torch.exp(far))
    w = st["weights"] if c["weighted"] else 1.0 / labels.numel()
    loss = torch.where(labels >= 0, w * loss, 0.0)
    return loss.sum(0, keepdim=True).float(), loss.float(), logp.float(), _grad_logits(c, labels, e, total, w * d)


def _segment(bounds, T):
    """Sequence of each row (the number of sequences behind the last one)."""
    return torch.searchsorted(bounds[1:].contiguous(), torch.arange(T, device="cuda", dtype=I32), right=True)


def _plain_pref(st):
    c, labels = st["case"], st["labels"]
    T, n = labels.numel(), 2 * c["pairs"]
    logp, lse, e, total = _logp(c, st["logits"], labels)
    logp = logp.float()
    seg = _segment(st["bounds"], T)
    trained = (labels >= 0) & (seg < n)
    term = torch.where(trained, logp.double() - (st["ref"] if c["ref"] else 0.0), 0.0)
    s = torch.zeros(n + 1, dtype=F64, device="cuda").index_add_(0, seg, term)[:n]
    count = torch.zeros(n + 1, dtype=F64, device="cuda").index_add_(0, seg, trained.double())[:n].clamp(min=1)
    if c["average"]:
        s = s / count
    h = c["beta"] * (s[0::2] - s[1::2]) - c["margin"]
    if c["kind"] == "sigmoid":
        loss = (1 - c["smoothing"]) * torch.log1p(torch.exp(-h)) + c["smoothing"] * torch.log1p(torch.exp(h))
        d = -(1 - c["smoothing"]) / (1 + torch.exp(h)) + c["smoothing"] / (1 + torch.exp(-h))
    elif c["kind"] == "hinge":
        loss, d = (1 - h).clamp(min=0), -(h < 1).double()
    else:
        loss, d = ((h - 0.5) / c["beta"]) ** 2, 2 * (h - 0.5) / c["beta"] ** 2
    d = c["beta"] * d / c["pairs"]
    ds = torch.stack([d, -d], 1).flatten()
    if c["average"]:
        ds = ds / count
    dlogp = torch.where(trained, torch.cat([ds, ds[:1]])[seg], 0.0)
    return (loss.mean(0, keepdim=True).float(), (c["beta"] * s).float(), logp,
            torch.where(labels >= 0, lse, 0.0).float(), dlogp.float(), _grad_logits(c, labels, e, total, dlogp))


def _plain_ln_fwd(st):
    x = st["x"].float()
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = (xc.square().mean(1, keepdim=True) + EPS).rsqrt()
    y = xc * rstd * st["gamma"].float()
    if st["beta"] is not None:
        y = y + st["beta"].float()
    return y.to(BF), mean[:, 0], rstd[:, 0]


def _plain_ln_bwd(st):
    c = st["case"]
    r = st["rstd"][:, None]
    n = (st["x"].float() - st["mean"][:, None]) * r
    dy = st["dy"].float()
    u = dy * st["gamma"].float()
    dx = r * (u - u.mean(1, keepdim=True) - n * (u * n).mean(1, keepdim=True))
    if c["res"]:
        dx = dx + st["dres"].float()
    return (dx.to(st["x"].dtype), dx.to(BF) if c["type"] == "f32" else None, (dy * n).sum(0).to(BF),
            dy.sum(0).to(BF) if c["bias"] else None)


def _plain_embed_fwd(st):
    tok = st["tok"]
    x = st["E"][tok.long().clamp(min=0)].float() * st["scale"]
    return torch.where((tok >= 0)[:, None], x, 0.0).to(TYPES[st["case"]["type"]])


def _plain_embed_bwd(st):
    V, tok = st["case"]["V"], st["tok"]
    acc = torch.zeros(V + 1, st["dx"].shape[1], dtype=F32, device="cuda")
    acc.index_add_(0, torch.where(tok >= 0, tok, V).long(), st["dx"].float())
    return (acc[:V] * st["scale"]).to(BF)


PLAIN = {"policy": _plain_policy, "pref": _plain_pref, "ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd,
         "embed_fwd": _plain_embed_fwd, "embed_bwd": _plain_embed_bwd}


# ---------------------------------------------------------------------------- the framework's calls
def _own(st):
    from host_memory_streamed_stream_gb300 import kernels as K

    c, err = st["case"], st["err"]
    op = c["op"]
    if op == "policy":
        return K.policy_loss(st["logits"], st["labels"], st["old"], st["adv"], ref_logp=st["ref"],
                             weights=st["weights"], clip_low=0.2, clip_high=c["hi"], kl=c["kl"], scale=c["scale"],
                             err=err)
    if op == "pref":
        logp, lse = K.token_logprobs(st["logits"], st["labels"], err=err)
        loss, rewards, dlogp = K.preference_loss(logp, st["bounds"], labels=st["labels"], ref_logp=st["ref"],
                                                 kind=c["kind"], beta=c["beta"], margin=c["margin"],
                                                 smoothing=c["smoothing"], average=c["average"])
        return loss, rewards, logp, lse, dlogp, K.token_logprobs_bwd(st["logits"], st["labels"], lse, dlogp)
    if op == "ln_fwd":
        return K.layernorm_fwd(st["x"], st["gamma"], st["beta"], eps=EPS)
    if op == "ln_bwd":
        return K.layernorm_bwd(st["dy"], st["x"], st["gamma"], st["mean"], st["rstd"], dres=st["dres"],
                               bias=c["bias"])
    if op == "embed_fwd":
        return K.embed_lookup(st["tok"], st["E"], scale=st["scale"], dtype=TYPES[c["type"]], err=err)
    return K.embed_lookup_bwd(st["tok"], st["dx"], c["V"], scale=st["scale"], err=err)


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- 64 bits
def _by_rows(st, scale):
    """logsumexp of every row and the label's logit minus it."""
    lse = torch.cat([torch.logsumexp(z.double() * scale, 1) for z in st["logits"].split(512)])
    at = torch.arange(lse.numel(), device="cuda")
    return lse, st["logits"][at, st["labels"].long()].double() * scale - lse


def _weighted_softmax(st, scale, lse, k):
    """k (onehot - softmax) for every row, a masked one's gradient being 0. (float32 holds a bf16's 64-bit value to 2^-24.)"""
    labels = st["labels"].long()
    out = torch.zeros(st["logits"].shape, dtype=F32, device="cuda")
    for a in range(0, labels.numel(), 512):
        rows = slice(a, a + 512)
        p = torch.exp(st["logits"][rows].double() * scale - lse[rows, None])
        hot = torch.zeros_like(p)
        hot[torch.arange(p.shape[0], device="cuda"), labels[rows]] = 1.0
        out[rows] = torch.where(labels[rows, None] < 0, torch.zeros_like(p), (hot - p) * k[rows, None]).float()
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "policy":
        a = case["scale"]
        lse, lp = _by_rows(st, a)
        seen = st["labels"] >= 0
        adv, old = st["adv"].double(), st["old"].double()
        r = torch.exp(lp - old)
        up = adv >= 0  # where the clip holds: above for a gain, below for a loss
        held = torch.where(up, r > 1 + case["hi"], r < 1 - 0.2)
        bound = torch.where(up, torch.full_like(r, 1 + case["hi"]), torch.full_like(r, 1 - 0.2))
        loss = -adv * torch.where(held, bound, r)
        k = torch.where(held, torch.zeros_like(r), -adv * r)
        if case["kl"]:
            q = torch.exp(st["ref"].double() - lp)
            loss = loss + case["kl"] * (q - torch.log(q) - 1)
            k = k + case["kl"] * (1 - q)
        w = st["weights"].double() if case["weighted"] else torch.full_like(r, 1.0 / r.numel())
        zero = torch.zeros_like(r)
        loss, k, lp = (torch.where(seen, v, zero) for v in (w * loss, w * k, lp))
        return loss.sum().reshape(1), loss, lp, _weighted_softmax(st, a, lse, a * k)
    if op == "pref":
        lse, lp = _by_rows(st, 1.0)
        seen = st["labels"] >= 0
        zero = torch.zeros_like(lp)
        lp, top = torch.where(seen, lp, zero), torch.where(seen, lse, zero)
        ends, n, beta = st["bounds"].tolist(), case["pairs"], case["beta"]
        score, share = [], []
        for j in range(2 * n):
            rows = slice(ends[j], ends[j + 1])
            use = seen[rows].nonzero()[:, 0]
            v = lp[rows][use] - (st["ref"][rows][use].double() if case["ref"] else 0.0)
            share.append(1.0 / max(1, use.numel()) if case["average"] else 1.0)
            score.append(float(v.sum()) * share[-1])
        d, loss = zero.clone(), 0.0
        for i in range(n):
            m = beta * (score[2 * i] - score[2 * i + 1]) - case["margin"]
            if case["kind"] == "sigmoid":
                up = 1 / (1 + math.exp(-m))
                e = case["smoothing"]
                loss += -(1 - e) * math.log(up) - e * math.log1p(-up)
                slope = up - (1 - e)
            elif case["kind"] == "hinge":
                loss += max(0.0, 1 - m)
                slope = -1.0 if m < 1 else 0.0
            else:
                loss += (m / beta - 0.5 / beta) ** 2
                slope = (2 * m - 1) / beta ** 2
            for j, sign in ((2 * i, 1.0), (2 * i + 1, -1.0)):
                d[ends[j]:ends[j + 1]] = sign * slope * beta / n * share[j]
        d = torch.where(seen, d, zero)
        return (torch.tensor([loss / n], dtype=F64), torch.tensor(score, dtype=F64) * beta, lp, top, d,
                _weighted_softmax(st, 1.0, lse, d))
    if op == "ln_fwd":
        x = st["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        y = (x - mean) / torch.sqrt(var + EPS) * st["gamma"].double()
        if st["beta"] is not None:
            y += st["beta"].double()
        return y, mean[:, 0], 1 / torch.sqrt(var[:, 0] + EPS)
    if op == "ln_bwd":
        dy, r, h = st["dy"].double(), st["rstd"].double()[:, None], case["h"]
        n = (st["x"].double() - st["mean"].double()[:, None]) * r
        u = dy * st["gamma"].double()
        # u less its parts along the constant row and along n, as the mean and the size are held
        dx = r * (u - u.sum(1, keepdim=True) / h - n * ((n * u).sum(1, keepdim=True) / h))
        if st["dres"] is not None:
            dx += st["dres"].double()
        return (dx, dx if case["type"] == "f32" else None, torch.einsum("th,th->h", dy, n),
                torch.einsum("th->h", dy) if case["bias"] else None)
    tok = st["tok"].long()
    if op == "embed_fwd":
        x = torch.zeros(tok.numel(), case["h"], dtype=F64, device="cuda")
        at = (tok >= 0).nonzero()[:, 0]
        x[at] = st["E"].index_select(0, tok[at]).double() * st["scale"]
        return x
    # runs of equal tokens, by columns
    order = torch.argsort(tok, stable=True)
    order = order[tok[order] >= 0]
    ids, counts = torch.unique_consecutive(tok[order], return_counts=True)
    out = torch.zeros(case["V"], case["h"], dtype=F64, device="cuda")
    for a in range(0, case["h"], 256):
        cols = slice(a, a + 256)
        run = torch.segment_reduce(st["dx"][order, cols].double(), "sum", lengths=counts, axis=0)
        out[ids, cols] = run * st["scale"]
    return out
