"""Pretrains a one-layer token encoder on hidden tokens on a GPU, every operator but
the matrix products of its projections, and the embedding table's lookup with its
gradient, from this library. The layer has no feed-forward part.

Texts of random lengths, packed, in which some tokens are replaced by a mask token;
the loss is the cross entropy of the hidden tokens over the whole vocabulary. The
layer is pre-normed:

    e = dropout(table[tokens])            embeddings
    y = norm(e);  q, k, v = y W_qkv;  a = attention(rotary(q), rotary(k), v)
    h = e + dropout(a W_out);  z = norm(h)
    loss = cross entropy(z W_head^T, hidden tokens)

Dropout's masks are made again in the backward pass from the step's seed; the
logits of the vocabulary are never kept. The last norm can also give its rows in
8 bits, as embeddings that maxsim_score_i8 takes.

    python examples/pretrain_encoder.py [--steps 30]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import maxsim_scoring_02_gb300 as m  # noqa: E402


class Encoder:
    """Weights in fp32, used in bf16; `names` are those of the trained ones."""

    names = ("table", "norm_in", "w_qkv", "w_out", "norm_out", "head")

    def __init__(self, vocab, width, heads, dim, seed, p=0.1, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.dim, self.p = heads, dim, p

        def weight(*shape, scale):
            return torch.randn(shape, generator=g, device=device) * scale

        self.table = weight(vocab, width, scale=1.0)
        self.w_qkv = weight(width, 3 * heads * dim, scale=width ** -0.5)
        self.w_out = weight(heads * dim, width, scale=(heads * dim) ** -0.5)
        self.head = weight(vocab, width, scale=width ** -0.5)
        self.norm_in, self.norm_out = torch.ones(width, device=device), torch.ones(width, device=device)
        self.freq, self.amplitude = m.maxsim_rotary_frequencies(dim, device=device)

    def hidden(self, tokens, offsets, seed):
        """The sum h [T, width] that the last norm takes, and what backward needs."""
        h, t = self.heads, tokens.shape[0]
        rng = [torch.stack([seed, torch.full_like(seed, i)]) for i in range(2)]   # a number for each dropout
        e = m.encoder_dropout(self.table.bfloat16()[tokens], self.p, rng[0])
        y = m.encoder_rms_norm(e, self.norm_in)
        qkv = (y @ self.w_qkv.bfloat16()).view(t, 3 * h, self.dim)
        qk = qkv[:, :2 * h]
        m.maxsim_rotary(qk, self.freq, offsets=offsets, amplitude=self.amplitude, out=qk)
        q, k, v = qkv[:, :h], qkv[:, h:2 * h], qkv[:, 2 * h:]
        a, lse = m.maxsim_attention(q, k, v, offsets, want_lse=True)
        o = a.view(t, -1) @ self.w_out.bfloat16()
        return o, (tokens, offsets, rng, e, y, q, k, v, a, lse)

    def embeddings(self, tokens, offsets, seed):
        """Rows in 8 bits and their scales, of unit length: documents or queries of maxsim_score_i8."""
        o, saved = self.hidden(tokens, offsets, seed)
        unit = torch.full_like(self.norm_out, self.norm_out.shape[0] ** -0.5)
        return m.encoder_rms_norm(o, unit, residual=saved[3], p=self.p, rng=saved[2][1], fmt="int8")

    def loss(self, tokens, targets, offsets, seed, backward=True):
        """The mean loss of the hidden tokens (targets >= 0), and the gradients of
        `names` in their order."""
        o, (tokens, offsets, rng, e, y, q, k, v, a, lse) = self.hidden(tokens, offsets, seed)
        h, t, p = self.heads, tokens.shape[0], self.p
        z, total = m.encoder_rms_norm(o, self.norm_out, residual=e, p=p, rng=rng[1], want_sum=True)
        head = self.head.bfloat16()
        each, denominators = m.encoder_cross_entropy(z, head, targets)
        count = (targets >= 0).sum().clamp_min(1)
        loss = each.sum() / count
        if not backward:
            return loss, None
        dloss = (1.0 / count).expand(t).float().contiguous()
        dz, d_head = m.encoder_cross_entropy_backward(dloss, z, head, targets, denominators)
        do, de, d_norm_out = m.encoder_rms_norm_backward(dz, total, self.norm_out, p=p, rng=rng[1])
        da = (do @ self.w_out.bfloat16().t()).view(t, h, self.dim)
        d_qkv = torch.empty((t, 3 * h, self.dim), dtype=torch.bfloat16, device=z.device)
        m.maxsim_attention_backward(da, q, k, v, a, lse, offsets, dq=d_qkv[:, :h], dk=d_qkv[:, h:2 * h], dv=d_qkv[:, 2 * h:])
        d_qk = d_qkv[:, :2 * h]
        m.maxsim_rotary(d_qk, self.freq, offsets=offsets, amplitude=self.amplitude, inverse=True, out=d_qk)
        dy = d_qkv.view(t, -1) @ self.w_qkv.bfloat16().t()
        # the embeddings' gradient: through the first norm, and past it
        de, _, d_norm_in = m.encoder_rms_norm_backward(dy, e, self.norm_in, dsum=de)
        de = m.encoder_dropout(de, p, rng[0], out=de)
        d_table = torch.zeros_like(self.table).index_add_(0, tokens, de.float())
        return loss, (d_table, d_norm_in, (y.t() @ d_qkv.view(t, -1)).float(), (a.view(t, -1).t() @ do).float(), d_norm_out,
                      d_head.float())


def batch(n, longest, vocab, seed, device="cuda"):
    """n packed texts in which each token follows from the one before it (and
    the text's own step), an eighth of them hidden behind token 0."""
    g = torch.Generator().manual_seed(seed)
    lengths = torch.randint(1, longest + 1, (n,), generator=g)
    texts = [(int(a) + torch.arange(k) * int(b)) % (vocab - 1) + 1
             for k, a, b in zip(lengths.tolist(), torch.randint(0, vocab, (n,), generator=g), torch.randint(1, 9, (n,), generator=g))]
    tokens = torch.cat(texts)
    hide = torch.rand(tokens.shape[0], generator=g) < 0.125
    offsets = torch.zeros(n + 1, dtype=torch.int64)
    offsets[1:] = torch.cumsum(lengths, 0)
    return (torch.where(hide, 0, tokens).to(device), torch.where(hide, tokens, -100).to(device), offsets.to(device))


def step(encoder, data, seed, lr, max_norm=1.0):
    """One training step; returns the loss and the gradient's norm."""
    loss, grads = encoder.loss(*data, seed)
    norm = m.maxsim_clip_grad_norm(list(grads), max_norm)
    for name, g in zip(encoder.names, grads):
        getattr(encoder, name).sub_(lr * g)
    return loss, norm


def train(steps=30, n=64, longest=96, vocab=5000, width=256, heads=4, dim=64, lr=0.5, seed=0):
    """The losses of `steps` steps, each on a new batch."""
    m.load_library()
    encoder = Encoder(vocab, width, heads, dim, seed)
    number = torch.zeros((), dtype=torch.int64, device="cuda")
    losses = []
    for i in range(steps):
        loss, norm = step(encoder, batch(n, longest, vocab, seed=1000 + i), number, lr)
        number += 1                       # on the device, so that a captured step draws anew
        losses.append(loss.item())
        if i % 5 == 0 or i == steps - 1:
            print(f"step {i:3d}  loss {losses[-1]:.4f}  gradient norm {norm.item():.4f}  (uniform {math.log(vocab):.4f})")
    status, _ = m.maxsim_device_status()
    assert status == 0
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=30)
    train(ap.parse_args().steps)
