"""Trains a one-layer token encoder with MaxSim on a GPU, every operator but the
matrix products from this library.

A layer of rotary positions and attention turns random token features of queries
and documents into embeddings; MaxSim scores all pairs; the loss is the cross
entropy of each query's own document among the batch. The gradient goes back
through the saved argmax, the attention and the rotation, is clipped by its
global norm, and a step of plain gradient descent follows.

    python examples/train_encoder.py [--steps 30]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import maxsim_scoring_02_gb300 as m  # noqa: E402


class Encoder:
    """x [T, width] -> embeddings [T, 128], T packed tokens of `offsets`."""

    def __init__(self, width, heads, dim, seed, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.dim = heads, dim

        def weight(n_in, n_out):
            return torch.randn((n_in, n_out), generator=g, device=device) / math.sqrt(n_in)

        # kept in fp32, used in bf16
        self.w_qkv, self.w_out = weight(width, 3 * heads * dim), weight(heads * dim, 128)
        self.freq, self.amplitude = m.maxsim_rotary_frequencies(dim, device=device)

    def forward(self, x, offsets, key_len):
        """Returns the embeddings and what backward needs. q and k heads lie side by
        side in the projection's output and are rotated together, in place."""
        h, t = self.heads, x.shape[0]
        qkv = (x @ self.w_qkv.bfloat16()).view(t, 3 * h, self.dim)
        qk = qkv[:, :2 * h]
        m.maxsim_rotary(qk, self.freq, offsets=offsets, amplitude=self.amplitude, out=qk)
        q, k, v = qkv[:, :h], qkv[:, h:2 * h], qkv[:, 2 * h:]
        out, lse = m.maxsim_attention(q, k, v, offsets, key_len=key_len, want_lse=True)
        y = (out.view(t, -1) @ self.w_out.bfloat16()).float()
        scale = y.norm(dim=1, keepdim=True).clamp_min(1e-6)
        return (y / scale).bfloat16(), (x, q, k, v, out, lse, y / scale, scale, offsets, key_len)

    def backward(self, d_embedding, saved):
        """Gradients of (w_qkv, w_out) for the embeddings' gradient [T, 128] fp32."""
        x, q, k, v, out, lse, unit, scale, offsets, key_len = saved
        h, t = self.heads, x.shape[0]
        dy = ((d_embedding - unit * (unit * d_embedding).sum(1, keepdim=True)) / scale).bfloat16()
        d_out = (dy @ self.w_out.bfloat16().t()).view(t, h, self.dim)
        d_qkv = torch.empty((t, 3 * h, self.dim), dtype=torch.bfloat16, device=x.device)
        m.maxsim_attention_backward(d_out, q, k, v, out, lse, offsets, key_len=key_len, dq=d_qkv[:, :h],
                                    dk=d_qkv[:, h:2 * h], dv=d_qkv[:, 2 * h:])
        d_qk = d_qkv[:, :2 * h]
        m.maxsim_rotary(d_qk, self.freq, offsets=offsets, amplitude=self.amplitude, inverse=True, out=d_qk)
        return x.t() @ d_qkv.view(t, -1), out.view(t, -1).t() @ dy


def batch(n, nq, nd, width, seed, device="cuda"):
    """Queries of nq rows, some of them mask tokens that are encoded but not
    attended to, and padded documents that hold their query's features among others."""
    g = torch.Generator(device=device).manual_seed(seed)
    d = torch.randn((n, nd, width), generator=g, device=device)
    q = d[:, :nq] + 0.5 * torch.randn((n, nq, width), generator=g, device=device)
    q_len = torch.randint(nq // 2, nq + 1, (n,), generator=g, device=device, dtype=torch.int32)
    d_len = torch.randint(nd // 2, nd + 1, (n,), generator=g, device=device, dtype=torch.int32)
    return q.bfloat16(), q_len, d.bfloat16(), d_len


def step(encoder, data, lr, max_norm=1.0, temperature=4.0):
    """One training step; returns the loss and the gradient's norm."""
    q, q_len, d, d_len = data
    n, nq, width = q.shape
    nd = d.shape[1]
    q_off = torch.arange(n + 1, device=q.device) * nq      # padded rows are packed rows, too
    d_off = torch.arange(n + 1, device=q.device) * nd
    Q, q_saved = encoder.forward(q.view(-1, width), q_off, q_len)
    D, d_saved = encoder.forward(d.view(-1, width), d_off, d_len)
    Q, D = Q.view(n, nq, 128), D.view(n, nd, 128)
    scores, argmax = m.maxsim_score(Q, D, d_len, want_argmax=True)
    p = torch.softmax(scores / temperature, dim=1)
    loss = -torch.log(p.diagonal()).mean()
    d_scores = (p - torch.eye(n, device=q.device)) / (n * temperature)
    dQ, dD = m.maxsim_backward(Q, D, argmax, d_scores, doc_len=d_len)
    grads = [a + b for a, b in zip(encoder.backward(dQ.view(-1, 128), q_saved), encoder.backward(dD.view(-1, 128), d_saved))]
    norm = m.maxsim_clip_grad_norm(grads, max_norm)
    for w, g in zip((encoder.w_qkv, encoder.w_out), grads):
        w.sub_(lr * g)
    return loss, norm


def train(steps=30, n=64, nq=32, nd=200, width=256, heads=4, dim=64, lr=8.0, seed=0):
    """The losses of `steps` steps, each on a new batch."""
    m.load_library()
    encoder = Encoder(width, heads, dim, seed)
    losses = []
    for i in range(steps):
        loss, norm = step(encoder, batch(n, nq, nd, width, seed=1000 + i), lr)
        losses.append(loss.item())
        if i % 5 == 0 or i == steps - 1:
            print(f"step {i:3d}  loss {losses[-1]:.4f}  gradient norm {norm.item():.4f}")
    status, _ = m.maxsim_device_status()
    assert status == 0
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=30)
    train(ap.parse_args().steps)
