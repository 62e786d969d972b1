"""The experts' products in 8-bit floating point, plainly and in 64 bits.

Tolerances.  A quantised value is off its value by at most half a step of the
format: 2^-4 (e4m3) or 2^-3 (e5m2) of it, or half the spacing of the format's
subnormals times the scale.  fp32 sums of n products are off by at most
2 n 2^-24 of the sum of the absolute values (every addition rounded, or cut,
by a step of 2^-23 at most); a result is rounded to its type once (check in
_edges).
"""
from __future__ import annotations

import numpy as np
import torch

from tests._edges import HALF, U, np64

B = 128
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
TOP = {E4M3: 448.0, E5M2: 57344.0}
STEP = {E4M3: 2.0 ** -4, E5M2: 2.0 ** -3}          # half a step, relative
LEAST_STEP = {E4M3: 2.0 ** -10, E5M2: 2.0 ** -17}  # half the subnormals' spacing
LEAST = 2.0 ** -100


def blocks(n):
    return -(-n // B)


def quant_rows(x, fmt):
    """x [..., R, C] fp32 on the CPU: q [..., R, C] and s [..., blocks of C, R], the fp32
    operations of the definition, so to the bit."""
    C = x.shape[-1]
    pad = torch.zeros(*x.shape[:-1], blocks(C) * B - C)
    p = torch.cat((x, pad), -1).unflatten(-1, (-1, B))
    amax = p.abs().amax(-1).clamp(min=LEAST)
    top = torch.full_like(amax, TOP[fmt])
    s = torch.where(amax.isfinite(), amax / top, torch.nan)
    q = (p * (top / amax)[..., None]).flatten(-2)[..., :C].to(fmt)
    return q.contiguous(), s.transpose(-1, -2).contiguous()


def quant_tiles(x, fmt):
    R, C = x.shape[-2:]
    p = torch.zeros(*x.shape[:-2], blocks(R) * B, blocks(C) * B)
    p[..., :R, :C] = x
    p = p.unflatten(-1, (-1, B)).unflatten(-3, (-1, B))
    amax = p.abs().amax((-1, -3)).clamp(min=LEAST)
    top = torch.full_like(amax, TOP[fmt])
    s = torch.where(amax.isfinite(), amax / top, torch.nan)
    q = (p * (top / amax)[..., :, None, :, None]).flatten(-2).flatten(-3, -2)[..., :R, :C].to(fmt)
    return q.contiguous(), s.transpose(-1, -2).contiguous()


def values(q, s):
    """What q [..., R, K] with s [..., blocks of K, R or blocks of R] stands for, 64 bits."""
    q, s = np64(q.float()), np.swapaxes(np64(s), -1, -2)
    if s.shape[-2] != q.shape[-2]:
        s = np.repeat(s, B, -2)[..., :q.shape[-2], :]
    return q * np.repeat(s, B, -1)[..., :q.shape[-1]]


def logistic(g):
    return np.exp(-np.logaddexp(0, -g))


def exp_ops(g):
    """Operations' worth of error of sigmoid(g): its exponential is documented to be within
    2 + 1.173 |g| units in the last place, each two of ours, and there are a few more."""
    return 2 * (2 + 1.173 * np.abs(g)) + 6


def swiglu(h):
    """a, and by how much fp32 may be off it."""
    g, u = np.split(h, 2, -1)
    a = g * logistic(g) * u
    return a, exp_ops(g) * U * np.abs(a)


def swiglu_grad(da, h):
    g, u = np.split(h, 2, -1)
    p = logistic(g)
    ops = exp_ops(g) * U
    dg = da * u * p * (1 + g * logistic(-g))
    du = da * g * p
    # 1 - p is off by 2^-24 absolutely, and by what p is
    dgm = np.abs(da * u) * p * (1 + np.abs(g)) * 2 * ops
    return np.concatenate((dg, du), -1), np.concatenate((dgm, np.abs(du) * ops), -1)


def check_quantised(q, s, ref, err, what=""):
    """q [R, C], s [blocks of C, R]: half a step of the format and fp32's err off ref."""
    fmt, v = q.dtype, values(q, s)
    scale = np.repeat(np64(s).T, B, -1)[:, :ref.shape[1]]
    amax = np.maximum(blockmax(np.abs(ref)), LEAST)
    rel = blockmax(err) / amax + 3 * U  # of the scale
    assert np.all(np.abs(np64(s).T * TOP[fmt] - amax) <= rel * amax), what + ": scale"
    tol = err + np.maximum(STEP[fmt] * (np.abs(ref) + err), LEAST_STEP[fmt] * scale)
    tol = tol * (1 + 4 * np.repeat(rel, B, -1)[:, :ref.shape[1]]) + 4 * U * np.abs(ref)
    assert np.all(np.abs(v - ref) <= tol), (what, np.max(np.abs(v - ref) - tol))


def blockmax(a):
    """[R, C] -> [R, blocks of C]"""
    R, C = a.shape
    p = np.zeros((R, blocks(C) * B))
    p[:, :C] = a
    return p.reshape(R, -1, B).max(-1)


def product_ops(K):
    """Of a product over K with a scaled fp32 sum for each 128."""
    return 2 * B + 2 * blocks(K) + 6


def segments(counts, align):
    """offsets of segments of counts rows, each padded to align, and the rows of all."""
    o = np.concatenate(([0], np.cumsum(-(-np.asarray(counts) // align) * align)))
    return torch.tensor(o, dtype=torch.int32)


# ---- the experts' layer for a few tokens ------------------------------------

def requantised(h, err):
    """h [n, F] quantised to e4m3 by blocks of 128, as values, and by how much the same from
    an h off by err may be off: a step where a border is within reach."""
    amax = np.repeat(np.maximum(blockmax(np.abs(h)), LEAST), B, -1)[:, :h.shape[1]]
    rel = np.repeat(blockmax(err), B, -1)[:, :h.shape[1]] / amax + 4 * U
    s = amax / 448.0
    v, d = h / s, err / s + np.abs(h / s) * rel
    rnd = lambda a: torch.from_numpy(np.clip(a, -448, 448)).to(E4M3).double().numpy()  # noqa: E731
    return rnd(v) * s, (np.abs(rnd(v + d) - rnd(v - d)) + np.abs(rnd(v)) * rel) * s


def few(x, ids, w, w1, w2, eight):
    """f [T, C] and by how much fp32 may be off it.  x as it enters the product; w1, w2 as
    they stand; ids -1: dropped."""
    T, C = x.shape
    F = w2.shape[2]
    f, err = np.zeros((T, C)), np.zeros((T, C))
    n1, n2 = (product_ops(C), product_ops(F)) if eight else (2 * C + 4, 2 * F + 4)
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if e < 0:
                continue
            z, zm = w1[e] @ x[t], np.abs(w1[e]) @ np.abs(x[t])
            g, u, gm, um = z[:F], z[F:], zm[:F], zm[F:]
            h = g * logistic(g) * u
            eh = n1 * U * (1.1 * gm * (np.abs(u) + n1 * U * um) + np.abs(g * logistic(g)) * um)
            eh = eh + exp_ops(g) * U * np.abs(h)
            if eight:
                h, eh = (a[0] for a in requantised(h[None], eh[None]))
            else:
                eh = eh + 2.0 ** -16 * np.abs(h)  # two terms of eight bits or more, and their rest
            y, ym = w2[e] @ h, np.abs(w2[e]) @ (np.abs(h) + eh)
            f[t] += w[t, j] * y
            err[t] += abs(w[t, j]) * (np.abs(w2[e]) @ eh + (n2 + 2 * len(ids[t]) + 4) * U * ym)
    return f, err


def check_few(got, f, err):
    g = np64(got)
    tol = err + HALF[got.dtype] * (np.abs(f) + err) + 2.0 ** -25
    assert np.all(np.abs(g - f) <= tol), np.max(np.abs(g - f) - tol)
