"""Plain fp64 forms of the operators on rows of hidden states and of the cross
entropy, with bounds on how far a result may be off.

u: half a step of the type (bf16 2^-8, fp16 2^-11, fp32 2^-24 of the value), and
2^-25 for fp16 numbers below its smallest normal one.

Sums of a row's squares: a thread adds at most 32 squares, a warp joins in 5 steps, a
block in at most 32, so the sum is within 70 * 2^-24 = 4.2e-6 of itself, its root
within half of that; the few roundings around it stay below 2^-21. ROW = 2^-18
(3.8e-6) covers both.

Products on the tensor cores: a sum of n products in fp32 is off by at most
n * 2^-23 of the sum of their sizes.
"""
import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
ROW = 2.0 ** -18


def philox_words(c, k):
    """Philox4x32-10 in Python's whole numbers: four counter words, two key words."""
    c, k = list(c), list(k)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def lots(rows, d, seed, call, first=0):
    """[rows, d] 16-bit lots of the rows from `first` on."""
    m32 = np.uint64(0xFFFFFFFF)
    groups = (d + 7) // 8
    c0 = np.broadcast_to(np.arange(groups, dtype=np.uint64), (rows, groups)).copy()
    c1 = np.broadcast_to(np.arange(first, first + rows, dtype=np.uint64)[:, None], (rows, groups)).copy()
    c2, c3 = (np.full_like(c0, (call >> s) & 0xFFFFFFFF) for s in (0, 32))
    k0, k1 = (np.uint64((seed >> s) & 0xFFFFFFFF) for s in (0, 32))
    for i in range(10):
        a, b = c0 * np.uint64(0xD2511F53), c2 * np.uint64(0xCD9E8D57)
        c0, c1, c2, c3 = (b >> np.uint64(32)) ^ c1 ^ k0, b & m32, (a >> np.uint64(32)) ^ c3 ^ k1, a & m32
        k0, k1 = (k0 + np.uint64(0x9E3779B9)) & m32, (k1 + np.uint64(0xBB67AE85)) & m32
    words = np.stack([c0, c1, c2, c3], -1)
    both = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], -1)
    return torch.from_numpy(both.reshape(rows, groups * 8)[:, :d].astype(np.int32))


def kept(rows, d, p, rng, device):
    """The mask, and what kept elements are multiplied by."""
    limit = round(p * 65536)
    seed, call = (int(v) & (2 ** 64 - 1) for v in rng.tolist())
    return (lots(rows, d, seed, call) >= limit).to(device), 65536.0 / (65536 - limit)


def dropout(x, p, rng, residual=None):
    """(value, bound): a kept element's factor is rounded to fp32, the sum rounded once."""
    keep, f = kept(*x.shape, p, rng, x.device)
    part = torch.where(keep, x.double() * f, 0.0)
    y = part if residual is None else part + residual.double()
    tol = U[x.dtype] * y.abs() + TINY[x.dtype] + 2.0 ** -23 * (part.abs() + y.abs())
    return y, tol


def norm(h, weight, eps):
    h = h.double()
    rstd = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h * rstd * (1.0 if weight is None else weight.double()), rstd


def norm_backward(dy, h, weight, eps, dsum=None):
    """(dresidual, its bound before rounding to the type, dweight, the sum of its terms' sizes)."""
    h64, dy64 = h.double(), dy.double()
    rstd = norm(h, None, eps)[1]
    g = dy64 * (1.0 if weight is None else weight.double())
    c = (g * h64).mean(1, keepdim=True) * rstd ** 2
    size = rstd * (g.abs() + h64.abs() * (g * h64).abs().mean(1, keepdim=True) * rstd ** 2)
    back = rstd * (g - h64 * c)
    if dsum is not None:
        back = back + dsum.double()
        size = size + dsum.double().abs()
    term = dy64 * h64 * rstd
    return back, 2 * ROW * size, term.sum(0), term.abs().sum(0)


def cross_entropy(x, w, targets, scale=1.0, dloss=None):
    """Dict of fp64 loss, lse (and dx, dw with dloss), each with its bound under
    "loss_tol" and so on.

    A logit is off by D = d 2^-23 scale sum|x||w|, at most; so are lse and the
    target's logit, on top of 2^-17 for exponentials, sums and logarithm, and of
    the rounding of numbers of lse's size (2^-22 of it). A weight exp(z - lse) is
    then off by twice that, relatively. dz is rounded to the type (u; in fp16 its
    smallest step is 2^-25 in units of 2^-14 of the largest dloss), sums of n
    products by n 2^-23, results once more (u)."""
    u, tiny = U[x.dtype], TINY[x.dtype]
    T, d = x.shape
    X, W = x.double(), w.double()
    r = {k: torch.empty(T, dtype=torch.float64, device=x.device) for k in ("loss", "loss_tol", "lse", "lse_tol")}
    if dloss is not None:
        for k, like in (("dx", X), ("dw", W)):
            r[k], r[k + "_tol"] = torch.zeros_like(like), torch.zeros_like(like)
    step = max(1, (1 << 26) // w.shape[0])
    live_all = (targets >= 0) & (targets < w.shape[0])
    top = 0.0
    if dloss is not None:
        top = dloss[live_all].double().abs().max().item() if bool(live_all.any()) else 0.0
    for a in range(0, T, step):
        b = min(T, a + step)
        z = X[a:b] @ W.T * scale
        off = (X[a:b].abs() @ W.abs().T).amax(1) * scale * d * 2.0 ** -23
        lse = torch.logsumexp(z, 1)
        live, t = live_all[a:b], targets[a:b].clamp(0, w.shape[0] - 1)[:, None]
        r["lse"][a:b] = lse
        r["lse_tol"][a:b] = off + 2.0 ** -17 + 2.0 ** -22 * lse.abs()
        r["loss"][a:b] = torch.where(live, lse - z.gather(1, t)[:, 0], 0.0)
        r["loss_tol"][a:b] = 2 * off + 2.0 ** -17 + 2.0 ** -22 * (lse.abs() + z.gather(1, t)[:, 0].abs())
        if dloss is None:
            continue
        part = torch.where(live, dloss[a:b].double(), 0.0)[:, None] * scale
        p = torch.exp(z - lse[:, None])
        dz = p * part
        dz.scatter_add_(1, t, -part)
        E = u * dz.abs() + p * part.abs() * (2 * r["lse_tol"][a:b, None] + 2.0 ** -18)
        E += tiny * 2.0 ** -13 * top * scale * (part != 0)
        fp = 2.0 ** -23 * dz.abs()
        r["dx"][a:b] = dz @ W
        r["dx_tol"][a:b] = (E + w.shape[0] * fp) @ W.abs()
        r["dw"] += dz.T @ X[a:b]
        r["dw_tol"] += (E + T * fp).T @ X[a:b].abs()
    if dloss is not None:
        for k in ("dx", "dw"):
            r[k + "_tol"] += u * r[k].abs() + tiny
    return r


def within(got, want, tol, name=""):
    """Elementwise within the bound; 1e-30 lets exact zeros be zeros."""
    got = got.double()
    assert got.shape == want.shape, name
    assert torch.isfinite(got).all(), name
    over = ((got - want).abs() - tol - 1e-30).max().item() if got.numel() else 0.0
    assert over <= 0, f"{name}: {over:.3e} over the bound"
