"""Measured cases of the token-encoder operators: rotary positions, packed
attention with its gradient, and the clipping of gradients by their global
norm.

They are the operators that make the token embeddings which MaxSim scores,
and that train them: the rotation and the attention run once a layer on
CSR-packed documents (the layout of ``maxsim_score_varlen``), and the clipping
once a step on the gradients of the whole encoder.

``run`` computes an operator either in its plain form (elementary torch
operations in fp32, rounded once at the end) or, where ``own`` is true, through
the framework's entry points. ``exact`` gives the same outputs from the
definitions in fp64.
"""
import math
import statistics

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one search query on its way through a layer: 32 tokens, 12 heads of
        # 64; q and k heads are rotated together in the fused projection
        _rotary("rotary_query", docs=1, max_len=32, heads=24, of=36, dim=64, rot=64, dtype="bf16"),
        # a batch of document pages of 1024 tokens, grouped heads of 128
        _rotary("rotary_pages", docs=96, max_len=1024, heads=20, of=24, dim=128, rot=128, dtype="bf16"),
        # the gradient's rotation for one long text: positions far beyond the
        # trained length (ramped frequencies), neighbouring dimensions paired,
        # only the first half of each head rotated
        _rotary("rotary_long_gradient", docs=1, max_len=131071, heads=10, of=10, dim=128, rot=64, dtype="fp16",
                pairs="interleaved", scaling="yarn", factor=16.0, original=8192, inverse=True),
        # one query padded with mask tokens: all 32 rows are encoded, 11 are attended to
        _attention("attention_query", docs=1, max_len=32, heads=12, kv_heads=12, dim=64, dtype="bf16", hidden="query"),
        # an indexing batch of passages, packed: round(lognormal(ln 70, 0.5)) tokens
        _attention("attention_passages", docs=2500, max_len=256, lengths="lognormal", heads=12, kv_heads=12, dim=64,
                   dtype="bf16"),
        # an indexing batch of pages of 1024 tokens, whose first part (the
        # image's patches) is seen by all tokens; grouped heads of 128
        _attention("attention_pages", docs=48, max_len=1024, heads=16, kv_heads=4, dim=128, dtype="bf16", mask="prefix"),
        # one long text with an odd number of tokens, each token seeing those before it
        _attention("attention_long", docs=1, max_len=16411, heads=8, kv_heads=2, dim=128, dtype="bf16", mask="causal"),
        # a training step on pages: capped scores, forward and backward
        _attention("attention_train_pages", docs=24, max_len=1024, heads=16, kv_heads=16, dim=128, dtype="bf16",
                   cap=30.0, train=True),
        # a training step on ragged texts, some of them empty or with hidden
        # keys, with a bias that grows with the distance
        _attention("attention_train_ragged", docs=160, max_len=512, lengths="uniform", heads=12, kv_heads=12, dim=64,
                   dtype="fp16", slopes=True, hidden="some", train=True),
        # the gradients of a projection head: a few small tensors
        _clip("clip_head", tensors=10, largest=98304, dtype="fp32", max_norm=1.0),
        # the gradients of a whole encoder of 12 layers: matrices and vectors
        _clip("clip_encoder", tensors=196, largest=1966080, dtype="bf16", max_norm=1.0),
        # the gradients of a batch of document pages and queries, which need no clipping
        _clip("clip_embeddings", tensors=2, largest=2000 * 1024 * 128, dtype="fp32", max_norm=1e6),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rotary", "attention", "attention", "attention", "clip"])
    if op == "rotary":
        dim = rng.choice([32, 48, 64, 96, 128])
        heads = rng.randint(1, 24)
        long = rng.random() < 0.5
        docs = 1 if long else spread(1, 300)
        return _rotary(None, docs=docs, max_len=spread(1, 131072) if long else spread(1, 1024),
                       lengths="fixed" if long else rng.choice(["fixed", "lognormal", "uniform"]),
                       heads=heads, of=heads + rng.randint(0, 8), dim=dim,
                       rot=rng.choice([dim, dim // 2]), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                       pairs=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                       factor=rng.choice([2.0, 8.0, 16.0]), original=8192, inverse=rng.random() < 0.3)
    if op == "clip":
        tensors = spread(1, 60)
        return _clip(None, tensors=tensors, largest=spread(16, 4000000), odd=rng.randint(0, 1) == 1,
                     dtype=rng.choice(["bf16", "fp16", "fp32"]), max_norm=rng.choice([0.5, 1.0, 1e6]))
    train = rng.random() < 0.5
    kv = rng.choice([1, 2, 4, 8, 12])
    heads = kv * rng.choice([1, 1, 2, 4] if kv < 8 else [1, 2])
    dim = rng.choice([32, 64, 64, 72, 96, 128, 128])
    # a text of one token has no gradient but its values': training starts at two dozen
    max_len = spread(24, 4096) if train else spread(1, 16384)
    most = 2.5e10 if train else 6.0e10  # pairs of a row and a key times heads and dimensions: below the largest listed ones
    top = max(1, min(3000, int(most / (max_len * max_len * heads * max(dim, 64)))))
    return _attention(None, docs=spread(1, top), max_len=max_len, lengths=rng.choice(["fixed", "lognormal", "uniform"]),
                      heads=heads, kv_heads=kv, dim=dim, dtype=rng.choice(["bf16", "fp16"]),
                      mask=rng.choice(["full", "full", "causal", "prefix"]), cap=rng.choice([0.0, 0.0, 30.0]),
                      slopes=rng.random() < 0.3, hidden=rng.choice(["none", "none", "some"]), train=train)


def _named(name, case):
    return dict(case, name=name) if name else case


def _rotary(name, docs, max_len, heads, of, dim, rot, dtype, lengths="fixed", pairs="half", scaling="none", factor=1.0,
            original=0, inverse=False):
    return _named(name, {"op": "rotary", "docs": docs, "max_len": max_len, "lengths": lengths, "heads": heads,
                         "of": of, "dim": dim, "rot": rot, "dtype": dtype, "pairs": pairs, "scaling": scaling,
                         "factor": factor if scaling != "none" else 1.0, "original": original if scaling == "yarn" else 0,
                         "inverse": inverse})


def _attention(name, docs, max_len, heads, kv_heads, dim, dtype, lengths="fixed", mask="full", cap=0.0, slopes=False,
               hidden="none", train=False):
    return _named(name, {"op": "attention", "docs": docs, "max_len": max_len, "lengths": lengths, "heads": heads,
                         "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "mask": mask, "cap": cap, "slopes": slopes,
                         "hidden": hidden, "train": train})


def _clip(name, tensors, largest, dtype, max_norm, odd=False):
    return _named(name, {"op": "clip", "tensors": tensors, "largest": largest, "dtype": dtype, "max_norm": max_norm,
                         "odd": odd})


# --------------------------------------------------------- lengths and sizes

def _lengths(case):
    """Document lengths at the quantiles of their distribution, so that every
    seed has the same ones, in another order."""
    n, top = case["docs"], case["max_len"]
    u = [(i + 0.5) / n for i in range(n)]
    if case["lengths"] == "lognormal":
        z = statistics.NormalDist()
        mid = top * 70.0 / 256.0
        return [min(top, max(1, round(mid * math.exp(0.5 * z.inv_cdf(x))))) for x in u]
    if case["lengths"] == "uniform":
        return [max(int(x * (top + 1)), 1 if n == 1 else 0) for x in u]
    return [top] * n


def _seen(case):
    """(length, keys that are not hidden, prefix) of each document."""
    got = []
    for i, n in enumerate(_lengths(case)):
        keys = n
        if case["hidden"] == "query":
            keys = (n + 2) // 3
        elif case["hidden"] == "some":
            keys = (0 if i % 8 == 5 else n // 2 if i % 8 == 2 else n)
        got.append((n, keys, min(keys, n // 3)))
    return got


def _pairs(case):
    """Pairs of a row and a key that it sees, over all documents, for one head."""
    total = 0
    for n, k, p in _seen(case):
        if case["mask"] == "full":
            total += n * k
        else:
            p = p if case["mask"] == "prefix" else 0
            total += p * p + (k * (k + 1) - p * (p + 1)) // 2 + (n - k) * k
    return total


def _clip_sizes(case):
    """Gradient sizes: every layer-like group has matrices and short vectors."""
    n, top = case["tensors"], case["largest"]
    if n == 2:
        return [top, max(1, top // 125)]
    sizes = []
    for i in range(n):
        m = (top, top // 4, 768, top // 4, 768, top // 4, 768, top)[i % 8]
        sizes.append(max(1, min(m, top)) | (1 if case["odd"] else 0))
    return sizes


def work(case):
    if case["op"] == "rotary":
        t = sum(_lengths(case))
        e = _BYTES[case["dtype"]]
        return {"bytes": 2.0 * t * case["heads"] * case["dim"] * e, "flops": 3.0 * t * case["heads"] * case["rot"]}
    if case["op"] == "clip":
        n = sum(_clip_sizes(case))
        return {"bytes": 2.0 * n * _BYTES[case["dtype"]], "flops": 3.0 * n}
    t, d, h, g, e = sum(_lengths(case)), case["dim"], case["heads"], case["kv_heads"], _BYTES[case["dtype"]]
    forward = t * d * (2 * h + 2 * g) * e
    products = 2
    if case["train"]:  # dO in, dq, dk and dv out, the rows' statistics out
        forward += t * d * (2 * h + 2 * g) * e + 4 * t * h
        products += 5
    return {"bytes": float(forward), "flops": 2.0 * products * _pairs(case) * h * d}


# ----------------------------------------------------------------- the inputs

def _gen(seed, device=DEV):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _offsets(lengths):
    off = torch.zeros(len(lengths) + 1, dtype=torch.int64)
    off[1:] = torch.cumsum(torch.tensor(lengths, dtype=torch.int64), 0)
    return off.to(DEV)


def _frequencies(case):
    """Turns a position of each pair, in units of 2^-64, and the amplitude: the
    table that a program makes once for its encoder."""
    r, base, s = case["rot"], 10000.0, case["factor"]
    if case["scaling"] == "ntk":
        base *= s ** (r / (r - 2.0))
    i = torch.arange(r // 2, dtype=torch.float64)
    theta = torch.exp(-(2.0 * i / r) * math.log(base))
    amplitude = 1.0
    if case["scaling"] == "linear":
        theta = theta / s
    elif case["scaling"] == "yarn":
        def place(turns):
            return r * math.log(case["original"] / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        lo, hi = max(0, math.floor(place(32.0))), min(r - 1, math.ceil(place(1.0)))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        theta = theta * (1.0 - ramp) + theta / s * ramp
        amplitude = 0.1 * math.log(s) + 1.0
    return (theta * (2.0 ** 64 / (2.0 * math.pi))).to(torch.int64).to(DEV), amplitude


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "clip":
        sizes = _clip_sizes(case)
        n = sum(sizes)
        dt = _DT[case["dtype"]]
        s["flat"] = torch.empty(n, dtype=dt, device=DEV)
        s["flat_out"] = torch.empty(n, dtype=dt, device=DEV)
        for a in range(0, n, 1 << 26):
            b = min(n, a + (1 << 26))
            s["flat"][a:b] = (torch.randn(b - a, generator=g, device=DEV) * 0.02).to(dt)
        s["grads"] = list(torch.split(s["flat"], sizes))
        s["outs"] = list(torch.split(s["flat_out"], sizes))
        return s
    order = torch.randperm(case["docs"], generator=_gen(seed, "cpu")).tolist()
    if case["op"] == "rotary":
        lengths = _lengths(case)
        s["offsets"] = _offsets([lengths[i] for i in order])
        whole = torch.randn((sum(lengths), case["of"], case["dim"]), generator=g, device=DEV).to(_DT[case["dtype"]])
        s["x"] = whole[:, :case["heads"]]
        s["freq"], s["amplitude"] = _frequencies(case)
        return s
    seen = [_seen(case)[i] for i in order] if case["docs"] > 1 else _seen(case)
    h, kv, d, dt = case["heads"], case["kv_heads"], case["dim"], _DT[case["dtype"]]
    s["offsets"] = _offsets([n for n, _, _ in seen])
    s["longest"] = max(n for n, _, _ in seen)
    t = sum(n for n, _, _ in seen)
    whole = torch.randn((t, h + 2 * kv, d), generator=g, device=DEV)
    if case["cap"]:
        whole[:, :h] *= 4.0  # scores that reach into the cap
    whole = whole.to(dt)
    s["q"], s["k"], s["v"] = whole[:, :h], whole[:, h:h + kv], whole[:, h + kv:]
    s["key_len"] = s["prefix_len"] = s["slopes_t"] = None
    if case["hidden"] != "none":
        s["key_len"] = torch.tensor([k for _, k, _ in seen], dtype=torch.int32, device=DEV)
    if case["mask"] == "prefix":
        s["prefix_len"] = torch.tensor([p for _, _, p in seen], dtype=torch.int32, device=DEV)
    if case["slopes"]:
        s["slopes_t"] = torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], dtype=torch.float32, device=DEV)
    if case["train"]:
        s["dO"] = (torch.randn((t, h, d), generator=g, device=DEV) * 0.1).to(dt)
    return s


# -------------------------------------------------------------- one operator

def run(state):
    if state["op"] == "rotary":
        return _own_rotary(state) if own else _plain_rotary(state)
    if state["op"] == "clip":
        return _own_clip(state) if own else _plain_clip(state)
    return _own_attention(state) if own else _plain_attention(state)


def _own_rotary(s):
    import maxsim_scoring_02_gb300 as m
    return m.maxsim_rotary(s["x"], s["freq"], offsets=s["offsets"], interleaved=s["pairs"] == "interleaved",
                           amplitude=s["amplitude"], inverse=s["inverse"])


def _own_clip(s):
    import maxsim_scoring_02_gb300 as m
    norm = m.maxsim_clip_grad_norm(s["grads"], s["max_norm"], out=s["outs"])
    return norm, s["flat_out"]


def _own_attention(s):
    import maxsim_scoring_02_gb300 as m
    how = dict(key_len=s["key_len"], mask=s["mask"], prefix_len=s["prefix_len"], cap=s["cap"], slopes=s["slopes_t"])
    if not s["train"]:
        return m.maxsim_attention(s["q"], s["k"], s["v"], s["offsets"], **how)
    out, lse = m.maxsim_attention(s["q"], s["k"], s["v"], s["offsets"], want_lse=True, **how)
    return (out, lse) + tuple(m.maxsim_attention_backward(s["dO"], s["q"], s["k"], s["v"], out, lse, s["offsets"], **how))


def _places(offsets, t):
    """(document, position within it) of each packed token."""
    at = torch.arange(t, device=offsets.device)
    doc = torch.searchsorted(offsets, at, right=True) - 1
    return doc, at - offsets[doc]


def _plain_rotary(s):
    x, half = s["x"], s["rot"] // 2
    _, pos = _places(s["offsets"], x.shape[0])
    turns = (pos[:, None] * s["freq"][None, :]) >> 32     # wraps at whole turns; 32 bits of the fraction are left
    angle = turns.to(torch.float32) * (2.0 * math.pi / 2.0 ** 32)
    cos, sin = torch.cos(angle)[:, None] * s["amplitude"], torch.sin(angle)[:, None] * s["amplitude"]
    if s["inverse"]:
        sin = -sin
    y = x.to(torch.float32)
    first, second = ((slice(0, s["rot"], 2), slice(1, s["rot"], 2)) if s["pairs"] == "interleaved"
                     else (slice(0, half), slice(half, s["rot"])))
    a, b = y[..., first], y[..., second]
    out = y.clone()
    out[..., first] = a * cos - b * sin
    out[..., second] = b * cos + a * sin
    return out.to(x.dtype)


def _plain_clip(s):
    norm = torch.sqrt(s["flat"].to(torch.float32).square().sum())
    factor = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    s["flat_out"].copy_(s["flat"].to(torch.float32) * factor)
    return norm.reshape(1), s["flat_out"]


def _plain_attention(s):
    """Documents padded to the longest one; hidden places are left out by comparisons."""
    q, off, n = s["q"], s["offsets"], s["longest"]
    t, h, d = q.shape
    kv, docs = s["kv_heads"], off.numel() - 1
    scale = 1.0 / math.sqrt(d)
    pos = torch.arange(n, device=q.device)
    length = off[1:] - off[:-1]
    valid = pos[None, :] < length[:, None]
    rows = (off[:-1, None] + pos[None, :]).clamp(max=t - 1)

    def padded(x):
        return (x[rows].to(torch.float32) * valid[..., None, None]).permute(0, 2, 1, 3)

    def grouped(x):
        return padded(x).reshape(docs, kv, h // kv, n, d)

    keys = length if s["key_len"] is None else s["key_len"].to(torch.int64)
    see = (valid[:, :, None] & (pos[None, None, :] < keys[:, None, None]))[:, None, None]
    if s["mask"] != "full":
        before = pos[None, None, :] <= pos[None, :, None]
        if s["mask"] == "prefix":
            before = before | (pos[None, None, :] < s["prefix_len"][:, None, None])
        see = see & before[:, None, None]
    qf, kf, vf = grouped(q), padded(s["k"])[:, :, None], padded(s["v"])[:, :, None]
    score = torch.matmul(qf, kf.transpose(-1, -2)) * scale
    bent = None
    if s["cap"]:
        bent = torch.tanh(score / s["cap"])
        score = bent * s["cap"]
    if s["slopes_t"] is not None:
        far = (pos[None, :] - pos[:, None]).abs().to(torch.float32)
        score = score - s["slopes_t"].reshape(1, kv, h // kv, 1, 1) * far
    score = torch.where(see, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    lse = top + torch.log(total)
    p = torch.where(total > 0, p / total, 0.0)
    out = torch.matmul(p, vf)
    doc, place = _places(off, t)

    def packed(x):
        return x.reshape(docs, -1, n, x.shape[-1])[doc, :, place]

    if not s["train"]:
        return packed(out).to(q.dtype)
    dO = grouped(s["dO"])
    dv = torch.matmul(p.transpose(-1, -2), dO).sum(2)
    ds = p * (torch.matmul(dO, vf.transpose(-1, -2)) - (dO * out).sum(-1, keepdim=True))
    if bent is not None:
        ds = ds * (1.0 - bent * bent)
    ds = ds * scale
    dq = torch.matmul(ds, kf)
    dk = torch.matmul(ds.transpose(-1, -2), qf).sum(2)
    return (packed(out).to(q.dtype), packed(lse)[..., 0].t().contiguous(),
            packed(dq).to(q.dtype), packed(dk).to(q.dtype), packed(dv).to(q.dtype))


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(s)
    if case["op"] == "clip":
        norm = math.sqrt(math.fsum(float((c.double() ** 2).sum()) for c in torch.split(s["flat"], 1 << 26)))
        factor = min(1.0, case["max_norm"] / (norm + 1e-6))
        return torch.tensor([norm], dtype=torch.float64, device=DEV), s["flat"].double() * factor
    if work(case)["flops"] > 8e12:
        return None
    return _exact_attention(s)


def _exact_rotary(s):
    """Each pair is a complex number, turned by position * theta radians."""
    x, r, f = s["x"].double(), s["rot"], s["factor"]
    base = 10000.0 * (f ** (r / (r - 2.0)) if s["scaling"] == "ntk" else 1.0)
    theta = []
    for i in range(r // 2):
        w = base ** (-2.0 * i / r)
        if s["scaling"] == "linear":
            w /= f
        if s["scaling"] == "yarn":
            lo = max(0, math.floor(r / 2.0 * math.log(s["original"] / (64.0 * math.pi), base)))
            hi = min(r - 1, math.ceil(r / 2.0 * math.log(s["original"] / (2.0 * math.pi), base)))
            part = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            w = w * (1.0 - part) + (w / f) * part
        theta.append(w)
    amplitude = 1.0 + 0.1 * math.log(f) if s["scaling"] == "yarn" else 1.0
    off = s["offsets"]
    pos = torch.cat([torch.arange(n, device=DEV) for n in (off[1:] - off[:-1]).tolist()]).double()
    turn = torch.polar(torch.full((1, 1), amplitude, dtype=torch.float64, device=DEV),
                       pos[:, None] * torch.tensor(theta, dtype=torch.float64, device=DEV))[:, None]
    if s["inverse"]:
        turn = turn.conj()
    y = x.clone()
    if s["pairs"] == "interleaved":
        z = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * turn
        y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * turn
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    return y


def _exact_attention(s):
    """One document after another: softmax over the keys that a row sees."""
    t, h, d = s["q"].shape
    group = h // s["kv_heads"]
    off = s["offsets"].tolist()
    hidden = s["key_len"].tolist() if s["key_len"] is not None else None
    prefix = s["prefix_len"].tolist() if s["prefix_len"] is not None else None
    new = lambda heads: torch.zeros((t, heads, d), dtype=torch.float64, device=DEV)  # noqa: E731
    out, lse = new(h), torch.full((h, t), -math.inf, dtype=torch.float64, device=DEV)
    dq, dk, dv = (new(h), new(s["kv_heads"]), new(s["kv_heads"])) if s["train"] else (None, None, None)
    for b in range(len(off) - 1):
        a, e = off[b], off[b + 1]
        n = e - a
        keys = n if hidden is None else hidden[b]
        if n == 0 or keys == 0:
            continue
        i, j = torch.arange(n, device=DEV)[:, None], torch.arange(keys, device=DEV)[None, :]
        hide = torch.zeros((n, keys), dtype=torch.bool, device=DEV)
        if s["mask"] == "causal":
            hide = j > i
        elif s["mask"] == "prefix":
            hide = (j > i) & (j >= prefix[b])
        for g in range(s["kv_heads"]):
            k, v = s["k"][a:a + keys, g].double(), s["v"][a:a + keys, g].double()
            for hh in range(g * group, (g + 1) * group):
                q = s["q"][a:e, hh].double()
                z = q @ k.T / math.sqrt(d)
                slope = 1.0
                if s["cap"]:
                    c = torch.tanh(z / s["cap"])
                    z, slope = s["cap"] * c, 1.0 - c ** 2
                if s["slopes_t"] is not None:
                    z = z - s["slopes_t"][hh].double() * (i - j).abs()
                z = z.masked_fill(hide, -math.inf)
                l = torch.logsumexp(z, 1)
                p = torch.exp(z - l[:, None])
                o = p @ v
                out[a:e, hh], lse[hh, a:e] = o, l
                if s["train"]:
                    do = s["dO"][a:e, hh].double()
                    dv[a:a + keys, g] += p.T @ do
                    w = p * (do @ v.T - (p * (do @ v.T)).sum(1, keepdim=True)) * slope / math.sqrt(d)
                    dq[a:e, hh] = w @ k
                    dk[a:a + keys, g] += w.T @ q
    return (out, lse, dq, dk, dv) if s["train"] else out
