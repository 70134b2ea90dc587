"""Measured cases of the operators that complete a layer of the token encoder and
its training: root-mean-square norms with the residual's addition and with output
in 8 bits, both directions; dropout whose mask is never stored; and the cross
entropy over a vocabulary whose logits are never kept, with its gradients.

They stand between the attention and the projections of each layer (norm and
dropout, on rows of the hidden state; the last norm's 8-bit rows are embeddings
that are scored), and at the end of the encoder's pretraining on hidden tokens
(cross entropy).

``run`` computes an operator either in its plain form (elementary torch
operations in fp32, rounded once at the end) or, where ``own`` is true, through
the framework's entry points. ``exact`` gives the same outputs from the
definitions in fp64.
"""
import functools
import math

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_LEAST = 1e-30   # rows of smaller values share their scale
_TOP = {"int8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one search query of 32 tokens between two parts of a layer: the
        # residual is added, the sum and its norm come back
        _norm("norm_query", rows=32, dim=768, dtype="bf16", residual=True),
        # a batch of 96 document pages of 1024 tokens through the same
        _norm("norm_pages", rows=96 * 1024, dim=2048, dtype="bf16", residual=True),
        # embeddings of an index: a million short rows, kept in 8 bits
        _norm("norm_embeddings_8bit", rows=1000003, dim=128, dtype="bf16", fmt="e4m3"),
        # hidden states for a product in 8 bits, rows as a slice of a wider buffer
        _norm("norm_hidden_8bit", rows=30011, dim=4096, dtype="bf16", residual=True, fmt="e4m3", pad=64),
        # a training step on 24 pages: dropout, residual and norm, and their gradients
        _norm("norm_train_pages", rows=24 * 1024, dim=2048, dtype="bf16", residual=True, p=0.1, train=True),
        # the same for a small encoder kept in fp32, with an odd width
        _norm("norm_train_odd", rows=4099, dim=771, dtype="fp32", residual=True, p=0.1, train=True),
        # dropout of one short batch's embeddings
        _dropout("dropout_query", rows=32, dim=768, dtype="bf16", p=0.1),
        # the gradient's dropout in fp32, rows of an odd width
        _dropout("dropout_gradient", rows=20011, dim=1001, dtype="fp32", p=0.25),
        # pages: dropout and the residual's addition
        _dropout("dropout_pages", rows=96 * 1024, dim=2048, dtype="bf16", p=0.1, residual=True),
        # the loss of one query's 32 tokens, without gradients
        _loss("loss_query", rows=32, vocab=30011, dim=768, dtype="bf16"),
        # a pretraining step on ragged texts in fp16, some rows without a target
        _loss("loss_train_ragged", rows=1531, vocab=50021, dim=1000, dtype="fp16", train=True, ignored=0.15,
              weighted=True),
        # a pretraining step of a large encoder
        _loss("loss_train_large", rows=8192, vocab=65536, dim=2048, dtype="bf16", train=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm", "norm", "dropout", "loss", "loss"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "loss":
        train = rng.random() < 0.6
        dim = 8 * spread(2, 256)
        rows = spread(1, 8192)
        vocab = spread(2, 65536)
        return _loss(None, rows=rows, vocab=vocab, dim=dim, dtype=rng.choice(["bf16", "fp16"]), train=train,
                     ignored=rng.choice([0.0, 0.15, 0.85]), weighted=rng.random() < 0.5, scale=rng.choice([1.0, 1.0, 0.05]))
    dim = spread(8, 8192)
    if rng.random() < 0.6:
        dim = max(8, dim // 8 * 8)
    rows = spread(1, max(1, min(1000000, int((5e7 if op == "norm" else 2e8) / dim))))
    pad = rng.choice([0, 0, 8, 5])
    residual = rng.random() < 0.6
    if op == "dropout":
        return _dropout(None, rows=rows, dim=dim, dtype=dtype, p=rng.choice([0.05, 0.1, 0.5]), residual=residual, pad=pad)
    train = rng.random() < 0.5
    return _norm(None, rows=rows, dim=dim, dtype=dtype, residual=residual, p=rng.choice([0.0, 0.1]) if train else 0.0,
                 train=train, fmt="none" if train else rng.choice(["none", "e4m3", "int8"]), pad=pad,
                 plain_weight=rng.random() < 0.5)


def _named(name, case):
    return dict(case, name=name) if name else case


def _norm(name, rows, dim, dtype, residual=False, p=0.0, train=False, fmt="none", pad=0, plain_weight=False):
    """plain_weight: the weight has the rows' own type instead of fp32."""
    return _named(name, {"op": "norm", "rows": rows, "dim": dim, "dtype": dtype, "residual": residual, "p": p,
                         "train": train, "fmt": fmt, "pad": pad, "plain_weight": plain_weight})


def _dropout(name, rows, dim, dtype, p, residual=False, pad=0):
    return _named(name, {"op": "dropout", "rows": rows, "dim": dim, "dtype": dtype, "p": p, "residual": residual,
                         "pad": pad})


def _loss(name, rows, vocab, dim, dtype, train=False, ignored=0.0, weighted=False, scale=1.0):
    return _named(name, {"op": "loss", "rows": rows, "vocab": vocab, "dim": dim, "dtype": dtype, "train": train,
                         "ignored": ignored, "weighted": weighted, "scale": scale})


def work(case):
    n, d, e = case["rows"], case["dim"], _BYTES[case["dtype"]]
    if case["op"] == "dropout":
        return {"bytes": float(n * d * e * (3 if case["residual"] else 2)), "flops": 2.0 * n * d}
    if case["op"] == "norm":
        streams = 3.0 if case["residual"] else 1.0          # x; the residual and the sum
        streams += 1.0 / e if case["fmt"] != "none" else 1.0
        if case["train"]:                                   # dy and dsum in, dx out, and the residual's gradient
            streams += 4 if case["p"] else 3
            streams += 0 if case["residual"] else 1         # the sum is kept for the gradient
        return {"bytes": n * d * e * streams + 4.0 * d, "flops": (14.0 if case["train"] else 5.0) * n * d}
    v = case["vocab"]
    tensors = (n * d + v * d) * e
    return {"bytes": float(tensors * (2 if case["train"] else 1) + 16 * n),
            "flops": 2.0 * (3 if case["train"] else 1) * n * v * d}


# ----------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _rows(case, g, spread=1.0):
    """[rows, dim] values, as a slice of a wider buffer where the case has a pad.
    Some columns are ten times as large as the others, as in hidden states."""
    n, d = case["rows"], case["dim"]
    t = torch.empty((n, d + case["pad"]), dtype=_DT[case["dtype"]], device=DEV)
    column = torch.where(torch.rand(d + case["pad"], generator=g, device=DEV) < 0.01, 10.0 * spread, spread)
    for a in range(0, n, 1 << 16):
        b = min(n, a + (1 << 16))
        t[a:b] = (torch.randn((b - a, t.shape[1]), generator=g, device=DEV) * column).to(t.dtype)
    return t[:, :d]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "loss":
        n, v, d, dt = case["rows"], case["vocab"], case["dim"], _DT[case["dtype"]]
        s["x"] = torch.randn((n, d), generator=g, device=DEV).to(dt)
        # logits with a spread of 3 about the mean
        s["weight"] = (torch.randn((v, d), generator=g, device=DEV) * (3.0 / (case["scale"] * math.sqrt(d)))).to(dt)
        s["targets"] = torch.randint(0, v, (n,), generator=g, device=DEV)
        if case["ignored"]:
            s["targets"][torch.rand(n, generator=g, device=DEV) < case["ignored"]] = -100
        if case["train"]:
            each = torch.rand(n, generator=g, device=DEV) * 2 if case["weighted"] else torch.ones(n, device=DEV)
            s["dloss"] = each / n
        return s
    s["x"] = _rows(case, g)
    s["res"] = _rows(case, g, 2.0) if case["residual"] else None
    s["rng"] = torch.tensor([1234567 + int(seed), 3], dtype=torch.int64, device=DEV)  # a step's seed, a call's number
    if case["op"] == "norm":
        w = 1.0 + 0.1 * torch.randn(case["dim"], generator=g, device=DEV)
        s["weight"] = w.to(_DT[case["dtype"]]) if case["plain_weight"] else w
        if case["train"]:
            s["dy"], s["dsum"] = _rows(case, g, 0.1), _rows(case, g, 0.1)
    return s


# -------------------------------------------------------------- one operator

def run(state):
    if state["op"] == "norm":
        return _own_norm(state) if own else _plain_norm(state)
    if state["op"] == "dropout":
        return _own_dropout(state) if own else _plain_dropout(state)
    return _own_loss(state) if own else _plain_loss(state)


def _own_dropout(s):
    import maxsim_scoring_02_gb300 as m
    return m.encoder_dropout(s["x"], s["p"], s["rng"], residual=s["res"])


def _own_norm(s):
    import maxsim_scoring_02_gb300 as m
    drop = {"p": s["p"], "rng": s["rng"]} if s["p"] else {}
    if s["fmt"] != "none":
        got = m.encoder_rms_norm(s["x"], s["weight"], residual=s["res"], fmt=s["fmt"], want_sum=s["residual"], **drop)
        return (_values(got[0], got[1]),) + tuple(got[1:])
    if not s["train"]:
        return m.encoder_rms_norm(s["x"], s["weight"], residual=s["res"], want_sum=s["residual"], **drop)
    y, total = m.encoder_rms_norm(s["x"], s["weight"], residual=s["res"], want_sum=True, **drop)
    dx, dres, dw = m.encoder_rms_norm_backward(s["dy"], total, s["weight"], dsum=s["dsum"], **drop)
    return y, total, dx, dres, dw


def _own_loss(s):
    import maxsim_scoring_02_gb300 as m
    loss, lse = m.encoder_cross_entropy(s["x"], s["weight"], s["targets"], scale=s["scale"])
    if not s["train"]:
        return loss, lse
    dx, dw = m.encoder_cross_entropy_backward(s["dloss"], s["x"], s["weight"], s["targets"], lse, scale=s["scale"])
    return loss, lse, dx, dw


def _values(codes, scale):
    """8-bit rows: e4m3 codes are numbers as they are; whole numbers stand for
    their multiples of the row's scale."""
    if codes.dtype == torch.int8:
        return (codes.to(torch.float32) * scale[:, None]).to(torch.bfloat16)
    return codes


# Philox4x32-10 (J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel random numbers:
# as easy as 1, 2, 3", 2011): the key is the seed, the counter (column / 8, row,
# call's number); its four words are eight 16-bit lots for eight columns.
_M0, _M1, _W0, _W1, _LOW = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85, 0xFFFFFFFF


def _round(state, i):
    c0, c1, c2, c3, k0, k1 = state
    a, b = c0 * _M0, c2 * _M1                     # wraps at 2^64; the words are cut out of that
    return ((((b >> 32) & _LOW) ^ c1) ^ ((k0 + i * _W0) & _LOW), b & _LOW,
            (((a >> 32) & _LOW) ^ c3) ^ ((k1 + i * _W1) & _LOW), a & _LOW, k0, k1)


def _kept(rows, dim, p, rng):
    """Which elements stay, and the factor of those that do."""
    limit = round(p * 65536)
    seed, call = rng[0], rng[1]
    c0 = torch.arange((dim + 7) // 8, device=DEV).expand(rows, -1)
    c1 = torch.arange(rows, device=DEV)[:, None].expand_as(c0)
    words = functools.reduce(_round, range(10), (c0, c1, call & _LOW, (call >> 32) & _LOW, seed & _LOW,
                                                 (seed >> 32) & _LOW))[:4]
    lots = torch.stack([w >> shift & 0xFFFF for w in words for shift in (0, 16)], -1)
    return lots.reshape(rows, -1)[:, :dim] >= limit, 65536.0 / (65536 - limit)


def _dropped(x, p, rng):
    if not p:
        return x.to(torch.float32)
    keep, factor = _kept(x.shape[0], x.shape[1], p, rng)
    return torch.where(keep, x.to(torch.float32) * factor, 0.0)


def _plain_dropout(s):
    y = _dropped(s["x"], s["p"], s["rng"])
    if s["res"] is not None:
        y = y + s["res"].to(torch.float32)
    return y.to(s["x"].dtype)


def _plain_norm(s):
    dt, eps = s["x"].dtype, 1e-6
    total = _dropped(s["x"], s["p"], s["rng"])
    if s["res"] is not None:
        total = total + s["res"].to(torch.float32)
    total = total.to(dt)                     # the norm is that of the sum as it is kept
    h, w = total.to(torch.float32), s["weight"].to(torch.float32)
    rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + eps)
    y = h * rstd * w
    if s["fmt"] != "none":
        scale = y.abs().amax(1).clamp_min(_LEAST) / _TOP[s["fmt"]]
        codes = y / scale[:, None]
        codes = torch.round(codes).to(torch.int8) if s["fmt"] == "int8" else codes.to(torch.float8_e4m3fn)
        return (_values(codes, scale), scale) + ((total,) if s["residual"] else ())
    if not s["train"]:
        return (y.to(dt), total) if s["residual"] else y.to(dt)
    dy = s["dy"].to(torch.float32)
    g = dy * w
    back = (g - h * ((g * h).mean(1, keepdim=True) * rstd.square())) * rstd + s["dsum"].to(torch.float32)
    dw = (dy * h * rstd).sum(0)
    return y.to(dt), total, _dropped(back, s["p"], s["rng"]).to(dt), back.to(dt), dw.to(s["weight"].dtype)


def _plain_loss(s):
    x, w, t = s["x"].to(torch.float32), s["weight"].to(torch.float32), s["targets"]
    live = t >= 0
    at = t.clamp_min(0)[:, None]
    z = torch.matmul(x, w.t()) * s["scale"]
    top = z.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    loss = torch.where(live, (lse - z.gather(1, at))[:, 0], 0.0)
    if not s["train"]:
        return loss, lse[:, 0]
    part = torch.where(live, s["dloss"], 0.0)[:, None] * s["scale"]
    dz = torch.exp(z - lse) * part
    dz.scatter_add_(1, at, -part)
    return loss, lse[:, 0], torch.matmul(dz, w).to(s["x"].dtype), torch.matmul(dz.t(), x).to(s["x"].dtype)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dropout":
        return _exact_sum(s)
    if case["op"] == "norm":
        return _exact_norm(s)
    if work(case)["flops"] > 1.2e13:
        return None
    return _exact_loss(s)


def _exact_keep(s, a, b):
    """The rows a .. b of the mask, the generator's products made of 16-bit parts."""
    def wide(m, c):  # (high, low) words of the 64-bit product of two 32-bit numbers
        m1, m0, c1, c0 = m >> 16, m & 65535, c >> 16, c & 65535
        mid = m1 * c0 + (m0 * c0 >> 16)
        mid2 = m0 * c1 + (mid & 65535)
        return m1 * c1 + (mid >> 16) + (mid2 >> 16), ((mid2 & 65535) << 16) + (m0 * c0 & 65535)

    seed, call = (int(v) % 2 ** 64 for v in s["rng"].tolist())
    groups = -(-s["dim"] // 8)
    number = torch.arange(a * groups, b * groups, device=DEV)
    ctr = [number % groups, number // groups, torch.full_like(number, call % 2 ** 32),
           torch.full_like(number, call // 2 ** 32)]
    key = [seed % 2 ** 32, seed // 2 ** 32]
    for _ in range(10):
        h0, l0 = wide(0xD2511F53, ctr[0])
        h1, l1 = wide(0xCD9E8D57, ctr[2])
        ctr = [h1 ^ ctr[1] ^ key[0], l1, h0 ^ ctr[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    lots = torch.empty((number.numel(), 8), dtype=torch.int32, device=DEV)
    for i in range(4):
        lots[:, 2 * i] = (ctr[i] % 65536).to(torch.int32)
        lots[:, 2 * i + 1] = (ctr[i] // 65536).to(torch.int32)
    return lots.view(b - a, groups * 8)[:, :s["dim"]] >= round(s["p"] * 65536)


def _chunks(s):
    step = max(1, (1 << 24) // s["dim"])
    return [(a, min(s["rows"], a + step)) for a in range(0, s["rows"], step)]


def _exact_drop(s, v, a, b):
    if not s["p"]:
        return v
    return v.masked_fill(~_exact_keep(s, a, b), 0.0) / (1.0 - round(s["p"] * 65536) / 65536)


def _exact_sum(s):
    parts = []
    for a, b in _chunks(s):
        v = _exact_drop(s, s["x"][a:b].double(), a, b)
        parts.append(v if s["res"] is None else v + s["res"][a:b].double())
    return torch.cat(parts)


def _exact_norm(s):
    total, w, dt = _exact_sum(s), s["weight"].double(), s["x"].dtype
    outs, dw = [], torch.zeros(s["dim"], dtype=torch.float64, device=DEV)
    for a, b in _chunks(s):
        h = total[a:b].to(dt).double()       # as it is kept
        r = 1.0 / torch.sqrt((h * h).sum(1, keepdim=True) / s["dim"] + 1e-6)
        unit = h * r
        y = unit * w
        if s["fmt"] != "none":
            step = torch.clamp(y.abs().max(1).values, min=_LEAST) / _TOP[s["fmt"]]
            if s["fmt"] == "int8":
                outs.append((torch.round(y / step[:, None]) * step[:, None], step))
            else:
                outs.append((y / step[:, None], step))   # the numbers that the codes round
        elif s["train"]:
            dy = s["dy"][a:b].double()
            dw += (dy * unit).sum(0)
            du = dy * w
            back = r * (du - unit * (unit * du).sum(1, keepdim=True) / s["dim"]) + s["dsum"][a:b].double()
            outs.append((y, _exact_drop(s, back, a, b), back))
        else:
            outs.append((y,))
    got = [torch.cat(part) for part in zip(*outs)]
    if s["train"]:
        return got[0], total, got[1], got[2], dw
    return tuple(got) + ((total,) if s["residual"] else ()) if len(got) > 1 or s["residual"] else got[0]


def _exact_loss(s):
    """Some rows at a time: the softmax of all their logits."""
    n, c = s["rows"], s["scale"]
    x, w = s["x"].double(), s["weight"].double()
    loss, lse = torch.zeros(n, dtype=torch.float64, device=DEV), torch.empty(n, dtype=torch.float64, device=DEV)
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    for a in range(0, n, 2048):
        b = min(n, a + 2048)
        z = torch.log_softmax(x[a:b] @ w.T * c, 1)
        first = x[a:b] @ w[0] * c
        lse[a:b] = first - z[:, 0]
        rows = torch.nonzero(s["targets"][a:b] >= 0)[:, 0]
        places = s["targets"][a:b][rows]
        loss[a + rows] = -z[rows, places]
        if s["train"]:
            u = torch.zeros_like(z)
            u[rows] = z[rows].exp()
            u[rows, places] -= 1.0
            u *= (s["dloss"][a:b].double() * c)[:, None]
            dx[a:b] = u @ w
            dw += u.T @ x[a:b]
    return (loss, lse, dx, dw) if s["train"] else (loss, lse)
