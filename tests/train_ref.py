"""Plain 64-bit statement of the router's training operators (CPU, torch and
numpy), for the parity tests: no code of the library, one definition per
function, no cleverness."""
from __future__ import annotations

import numpy as np
import torch

M32 = 0xFFFFFFFF


def philox4x32_10(counter, key):
    """Salmon, Moraes, Dror and Shaw (SC 2011), on Python integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & M32, (a >> 32) ^ c[3] ^ k[1], a & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def random16(index, seed, offset):
    """The 16 random bits of the elements `index` (an array), vectorised over them."""
    i = np.asarray(index, dtype=np.uint64)
    g = i // np.uint64(8)
    low, s32 = np.uint64(M32), np.uint64(32)
    c = [g & low, g >> s32, np.full_like(g, offset & M32), np.full_like(g, offset >> 32 & M32)]
    k = [seed & M32, seed >> 32 & M32]
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> s32) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> s32) ^ c[3] ^ np.uint64(k[1]),
             a & low]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    j = i % np.uint64(8)
    w = np.choose((j // np.uint64(2)).astype(np.int64), c)
    return np.where(j % np.uint64(2) == 1, w >> np.uint64(16), w & np.uint64(0xFFFF)).astype(np.int64)


def keep_and_scale(shape, p, seed, offset, first=0):
    """(which elements stay, what they are multiplied by) for elements first.. of a tensor."""
    n = int(np.prod(shape))
    thr = int(p * 65536 + 0.5)
    keep = random16(np.arange(first, first + n, dtype=np.uint64), seed, offset) >= thr
    return torch.from_numpy(keep.reshape(shape)), (65536 / (65536 - thr) if thr < 65536 else 0.0)


def dropout(x, residual, p, seed, offset):
    keep, scale = keep_and_scale(tuple(x.shape), p, seed, offset)
    y = torch.where(keep, x.double() * scale, torch.zeros((), dtype=torch.float64))
    return y if residual is None else y + residual.double()


def probs(z, router):
    """Router probabilities over all experts; -inf scores get 0, a row of them zeros."""
    if router == "softmax":
        m = z.amax(1, keepdim=True)
        e = torch.exp(z - torch.where(torch.isinf(m), torch.zeros_like(m), m))
        s = e.sum(1, keepdim=True)
        return e / torch.where(s > 0, s, torch.ones_like(s))
    a = torch.sigmoid(z)
    s = a.sum(1, keepdim=True)
    return a / torch.where(s > 0, s, torch.ones_like(s))


def weights(zk, router):
    """The routing weights of the picked scores zk [T][K]."""
    if router == "softmax":
        return torch.softmax(zk, 1)
    a = torch.sigmoid(zk)
    return a / (a.sum(1, keepdim=True) + 1e-6)


def spans(T, cu):
    return [(0, T)] if cu is None else list(zip(cu[:-1], cu[1:]))


def live_tokens(a, b, mask):
    return [t for t in range(a, b) if mask is None or mask[t]]


def balance(z, idx, router, alpha, mask=None, cu=None):
    """(counts, mean_probs, loss): z float64 [T][E], idx [T][K]."""
    (T, E), K = z.shape, idx.shape[1]
    sp = spans(T, cu)
    counts = torch.zeros(len(sp), E, dtype=torch.int64)
    mean = torch.zeros(len(sp), E, dtype=torch.float64)
    loss = torch.zeros((), dtype=torch.float64)
    p = probs(z, router)
    for g, (a, b) in enumerate(sp):
        t = live_tokens(a, b, mask)
        if not t:
            continue
        counts[g] = torch.bincount(idx[t].reshape(-1).long(), minlength=E)
        mean[g] = p[t].mean(0)
        loss = loss + alpha / len(sp) * (counts[g].double() * E / (K * len(t)) * mean[g]).sum()
    return counts, mean, loss


def route_grad(z, idx, router, alpha, d_w=None, counts=None, d_loss=1.0, mask=None, cu=None):
    """The gradient of z by differentiating the formulas of the loss and the weights,
    and the size of the terms that it is the difference of (for the tolerance)."""
    (T, E), K = z.shape, idx.shape[1]
    z = z.double()
    out, size = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    sp = spans(T, cu)
    for g, (a, b) in enumerate(sp):
        t = live_tokens(a, b, mask)
        if not t:
            continue
        if counts is not None:
            p = probs(z[t], router)
            c = counts[g].double()
            n = c.sum() / K
            coef = d_loss * alpha / len(sp) * E * c / (K * n * n) if n > 0 else c * 0
            dot = (p * coef).sum(1, keepdim=True)
            f = p * (torch.sigmoid(-z[t]) if router == "sigmoid" else 1.0)
            out[t] += f * (coef - dot)
            size[t] += f * (coef.abs() + (p * coef.abs()).sum(1, keepdim=True))
        if d_w is not None:
            zk = z[t].gather(1, idx[t].long())
            w = weights(zk, router)
            dw = d_w[t].double()
            f = w * (torch.sigmoid(-zk) if router == "sigmoid" else 1.0)
            out[t] = out[t].scatter_add(1, idx[t].long(), f * (dw - (w * dw).sum(1, keepdim=True)))
            size[t] = size[t].scatter_add(
                1, idx[t].long(), f * (dw.abs() + (w * dw.abs()).sum(1, keepdim=True)))
    return out, size


def combine(y_perm, inv, w, y_shared, residual, p, seed, offset):
    """(y, sum of the terms' magnitudes)."""
    T, K = w.shape
    rows = torch.zeros(T, K, y_perm.shape[1], dtype=torch.float64)
    ok = (inv >= 0) & (inv < T * K)
    rows[ok] = y_perm.double()[inv[ok].long()]
    v = (w.double()[:, :, None] * rows).sum(1)
    size = (w.double()[:, :, None] * rows).abs().sum(1)
    if y_shared is not None:
        v, size = v + y_shared.double(), size + y_shared.double().abs()
    keep, scale = keep_and_scale(tuple(v.shape), p, seed, offset)
    v, size = torch.where(keep, v * scale, v * 0), torch.where(keep, size * scale, size * 0)
    if residual is not None:
        v, size = v + residual.double(), size + residual.double().abs()
    return v, size


def combine_grad(d_y, y_perm, inv, w, p, seed, offset):
    """(dz, d_topk_w, magnitude of its terms, d_y_perm)."""
    T, K = w.shape
    keep, scale = keep_and_scale(tuple(d_y.shape), p, seed, offset)
    dz = torch.where(keep, d_y.double() * scale, torch.zeros((), dtype=torch.float64))
    dw, size = torch.zeros(T, K, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64)
    rows = torch.zeros(T * K, d_y.shape[1], dtype=torch.float64)
    for t in range(T):
        for j in range(K):
            r = int(inv[t, j])
            if 0 <= r < T * K:
                dw[t, j] = (dz[t] * y_perm[r].double()).sum()
                size[t, j] = (dz[t] * y_perm[r].double()).abs().sum()
                rows[r] = w[t, j].double() * dz[t]
    return dz, dw, size, rows
