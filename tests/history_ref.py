"""Plain 64-bit references of the behaviour-history operators (CPU, from the
definitions; they share no code with the library)."""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24  # unit roundoff of fp32
U16 = 2.0 ** -8   # unit roundoff of bf16 (8 significant bits)
MASK = (1 << 32) - 1


def philox4x32(counter, key, rounds=10):
    """The four output words of one counter, on Python integers."""
    x, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = 0xD2511F53 * x[0], 0xCD9E8D57 * x[2]
        x = [(b >> 32) ^ x[1] ^ k[0], b & MASK, (a >> 32) ^ x[3] ^ k[1], a & MASK]
        k = [(k[0] + 0x9E3779B9) & MASK, (k[1] + 0xBB67AE85) & MASK]
    return x


def keep_mask(n, p, seed, offset):
    """bool [n] and the factor on what is kept."""
    cut = int(p * 65536 + 0.5)
    keep = np.empty((n + 7) // 8 * 8, dtype=bool)
    for g in range((n + 7) // 8):
        c = (offset + g) & ((1 << 64) - 1)
        w = philox4x32([c & MASK, c >> 32, 0, 0], [seed & MASK, (seed >> 32) & MASK])
        for j in range(8):
            keep[8 * g + j] = ((w[j // 2] >> (16 * (j % 2))) & 0xFFFF) >= cut
    return keep[:n], (65536.0 / (65536 - cut) if cut < 65536 else 0.0)


def embed(table, tokens, scale):
    ok = (tokens >= 0) & (tokens < table.shape[0])
    return torch.where(ok[:, None], table.double()[tokens.clamp(0, table.shape[0] - 1)] * scale, 0.0)


def embed_grad(tokens, dout, rows, scale):
    """The gradient, the sum of its terms' magnitudes and each row's count."""
    ok = (tokens >= 0) & (tokens < rows)
    t, g = tokens[ok], dout.double()[ok] * scale
    out = torch.zeros((rows, dout.shape[1]), dtype=torch.float64)
    mag = torch.zeros_like(out)
    out.index_add_(0, t, g)
    mag.index_add_(0, t, g.abs())
    return out, mag, torch.bincount(t, minlength=rows)


def addnorm(x, res, w, eps, keep=None, factor=1.0):
    h = x.double()
    if keep is not None:
        h = torch.where(keep, h * factor, 0.0)
    if res is not None:
        h = h + res.double()
    r = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return h, h * r * w.double(), r[:, 0]


def addnorm_grad(dy, dh, h, w, r, keep=None, factor=1.0):
    dy, h, w, r = dy.double(), h.double(), w.double(), r.double()[:, None]
    g = dy * w
    t = r * g - h * r ** 3 * (g * h).mean(1, keepdim=True)
    if dh is not None:
        t = t + dh.double()
    dx = t if keep is None else torch.where(keep, t * factor, 0.0)
    return dx, t, (dy * h * r).sum(0)


def linattn(q, k, v, offsets, decay, scale, state0=None):
    """o and the last states; q, k, v [rows][H][width]."""
    q, k, v, lam = q.double(), k.double(), v.double(), decay.double()[:, None, None]
    B, H, dk, dv = len(offsets) - 1, q.shape[1], q.shape[2], v.shape[2]
    o = torch.zeros(v.shape, dtype=torch.float64)
    S = torch.zeros((B, H, dk, dv), dtype=torch.float64) if state0 is None else state0.double().clone()
    for b in range(B):
        for t in range(int(offsets[b]), int(offsets[b + 1])):
            S[b] = S[b] * lam + k[t][:, :, None] * v[t][:, None, :]
            o[t] = (q[t][:, :, None] * S[b]).sum(1) * scale
    return o, S


def linattn_grad(q, k, v, do, offsets, decay, scale, state0=None, dstate=None):
    q, k, v, do, lam = q.double(), k.double(), v.double(), do.double(), decay.double()[:, None, None]
    B, H, dk, dv = len(offsets) - 1, q.shape[1], q.shape[2], v.shape[2]
    S = torch.zeros((B, H, dk, dv), dtype=torch.float64) if state0 is None else state0.double().clone()
    W = torch.zeros((B, H, dk, dv), dtype=torch.float64) if dstate is None else dstate.double().clone()
    dq, dkk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b in range(B):
        span = range(int(offsets[b]), int(offsets[b + 1]))
        for t in span:
            S[b] = S[b] * lam + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = (S[b] * do[t][:, None, :]).sum(2) * scale
        for t in reversed(span):
            U = W[b] + scale * q[t][:, :, None] * do[t][:, None, :]
            dkk[t], dvv[t] = (U * v[t][:, None, :]).sum(2), (U * k[t][:, :, None]).sum(1)
            W[b] = U * lam
    return dq, dkk, dvv, W
