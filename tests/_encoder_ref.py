"""Plain fp64 forms of the token-encoder operators, with bounds on how far a
result may be off.

Unit roundoffs: u = 2^-8 (bf16), 2^-11 (fp16), 2^-24 (fp32). Attention, for
inputs N(0,1) and d <= 128: a score's fp32 sum of d products is off by at most
scale * d * 2^-23 * sum|q||k| <= 1.4e-4, which moves a weight and its row's
denominator by as much, so weights are within FP = 4e-4 of themselves before
they are rounded (u), and a result is rounded once more (u):
  |out - ref| <= (2u + FP) * sum_j p |v|
  dV: (2u + FP) * sum_i p |dO|
  dS: E = u |dS| + u p scale sum|dO||out| + FP p scale (sum|dO||v| + sum|dO||out|)
      (its rounding; delta made from the rounded out; the fp32 sums)
  dQ: u |dQ| + E @ |K|, dK: u |dK| + E^T @ |Q|
fp16 numbers below 2^-14 lie 2^-24 apart, so every rounding to fp16 (of a
weight, of dS, of a result) may be off by TINY = 2^-25 instead.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
FP = 4e-4
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


def scores(q, k, scale, cap, slope, n_rows):
    """Scores before masking, and the cap's derivative; q [n, d], k [m, d]."""
    z = q @ k.T * scale
    bend = torch.ones_like(z)
    if cap > 0:
        t = torch.tanh(z / cap)
        z, bend = cap * t, 1 - t * t
    i = torch.arange(q.shape[0], device=q.device)[:, None]
    j = torch.arange(k.shape[0], device=q.device)[None, :]
    return z - slope * (i - j).abs().double(), bend, i, j


def attention(q, k, v, lengths, key_len=None, mask="full", prefix_len=None, scale=None, cap=0.0, slopes=None, dO=None,
              bounds=True):
    """Dict of fp64 out, lse (and dq, dk, dv with dO), each with its bound under
    "out_tol" and so on. Keys from key_len on are cut off, not multiplied by 0."""
    u, tiny = U[q.dtype], TINY[q.dtype]
    T, H, d = q.shape
    G = k.shape[1]
    dev = q.device
    scale = 1 / math.sqrt(d) if scale is None else scale
    new = lambda h: torch.zeros((T, h, d), dtype=torch.float64, device=dev)  # noqa: E731
    r = {"out": new(H), "out_tol": new(H), "lse": torch.full((H, T), -math.inf, dtype=torch.float64, device=dev)}
    if dO is not None:
        for n, h in (("dq", H), ("dk", G), ("dv", G)):
            r[n], r[n + "_tol"] = new(h), new(h)
    a = 0
    for b, n in enumerate(lengths):
        m = n if key_len is None else min(n, int(key_len[b]))
        if n and m:
            for h in range(H):
                g = h // (H // G)
                Q, K, V = q[a:a + n, h].double(), k[a:a + m, g].double(), v[a:a + m, g].double()
                z, bend, i, j = scores(Q, K, scale, cap, 0.0 if slopes is None else slopes[h].double(), n)
                if mask != "full":
                    seen = j <= i
                    if mask == "prefix":
                        seen = seen | (j < int(prefix_len[b]))
                    z = torch.where(seen, z, -math.inf)
                lse = torch.logsumexp(z, 1)
                p = torch.exp(z - lse[:, None])
                o = p @ V
                r["out"][a:a + n, h], r["lse"][h, a:a + n] = o, lse
                r["out_tol"][a:a + n, h] = (2 * u + FP) * (p @ V.abs()) + tiny * (1 + V.abs().sum(0))
                if dO is not None:
                    D = dO[a:a + n, h].double()
                    dP, delta = D @ V.T, (D * o).sum(1, keepdim=True)
                    dS = p * (dP - delta) * bend * scale
                    r["dq"][a:a + n, h] += dS @ K
                    r["dk"][a:a + m, g] += dS.T @ Q
                    r["dv"][a:a + m, g] += p.T @ D
                    around = (D.abs() * o.abs()).sum(1, keepdim=True)
                    E = u * dS.abs() + p * scale * (u * around + FP * (D.abs() @ V.abs().T + around)) + tiny * (p > 0)
                    r["dq_tol"][a:a + n, h] += E @ K.abs()
                    r["dk_tol"][a:a + m, g] += E.T @ Q.abs()
                    r["dv_tol"][a:a + m, g] += (2 * u + FP) * (p.T @ D.abs()) + tiny * (1 + D.abs().sum(0))
        a += n
    if dO is not None:
        for n in ("dq", "dk"):
            r[n + "_tol"] += u * r[n].abs() + tiny
    return r


def check(got, ref, name):
    """Elementwise within the bound; 1e-30 lets exact zeros be zeros."""
    x, y, tol = got.double(), ref[name], ref[name + "_tol"]
    assert torch.isfinite(x).all(), name
    over = ((x - y).abs() - tol - 1e-30).max() if x.numel() else torch.tensor(0.0)
    assert over <= 0, f"{name}: {over.item():.3e} over the bound"


def rotary_angles(positions, rot_dim, base=10000.0, scaling="none", factor=1.0, original_length=0):
    """[T, rot_dim/2] fp64 angles and the amplitude, from the definitions."""
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    theta = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    amplitude = 1.0
    if scaling == "linear":
        theta = [t / factor for t in theta]
    if scaling == "yarn":
        amplitude = 0.1 * math.log(factor) + 1
        # pair i turns original_length * theta_i / 2 pi times; i as a real number where that is 32 and 1
        where = lambda turns: rot_dim / 2 * math.log(original_length / (2 * math.pi * turns), base)  # noqa: E731
        lo, hi = max(0, math.floor(where(32))), min(rot_dim - 1, math.ceil(where(1)))
        ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3))) for i in range(rot_dim // 2)]
        theta = [t * (1 - c) + t / factor * c for t, c in zip(theta, ramp)]
    return positions.double()[:, None] * torch.tensor(theta, dtype=torch.float64, device=positions.device), amplitude


def rotary(x, angles, amplitude, rot_dim, interleaved=False, inverse=False):
    y = x.double().clone()
    c, s = torch.cos(angles)[:, None] * amplitude, torch.sin(angles)[:, None] * amplitude
    if inverse:
        s = -s
    a, b = (slice(0, rot_dim, 2), slice(1, rot_dim, 2)) if interleaved else \
        (slice(0, rot_dim // 2), slice(rot_dim // 2, rot_dim))
    x1, x2 = x[..., a].double(), x[..., b].double()
    y[..., a], y[..., b] = x1 * c - x2 * s, x2 * c + x1 * s
    return y
