"""The operators at the edges of the sub-layers (q/k norm + rotation, router,
sort, dispatch, combine) in plain numpy, 64 bits, from their definitions, each
with the magnitude that its rounding errors scale with.

Tolerances.  A result is rounded to its type once, by at most half a step:
eps/2 |value| (2^-8 for bf16, 2^-11 fp16, 2^-24 fp32), or half the spacing of
the type's subnormals.  Before that it is formed in fp32, each operation off
by at most 2^-24 of its result, so a sum of n products is off by at most
(n + c) 2^-24 of the sum of their absolute values (its magnitude), c counting
the operations before and after the sum.
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U}
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def np64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def check(got, ref, mag, ops, what=""):
    """|got - ref| within half a step of got's type and ops * 2^-24 of mag."""
    dt, g = got.dtype, np64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert np.all(np.isfinite(g)), f"{what}: non-finite values"
    fp32 = ops * U * mag
    tol = fp32 + HALF[dt] * (np.abs(ref) + fp32) + TINY[dt]
    over = np.abs(g - ref) - tol
    assert not over.size or over.max() <= 0, (
        f"{what}: off by {np.abs(g - ref).flat[over.argmax()]:.3e} at "
        f"{np.unravel_index(over.argmax(), over.shape)}, allowed {tol.flat[over.argmax()]:.3e}")


# ---- q/k norm + rotation ---------------------------------------------------

def pairs(R, inter):
    p = np.arange(R // 2)
    return (2 * p, 2 * p + 1) if inter else (p, p + R // 2)


def turn(x, cos, sin, R, inter, sign=1.0):
    """x [T, H, D] with its pairs rotated; cos, sin [T, R/2]."""
    i, j = pairs(R, inter)
    y, c, s = x.copy(), cos[:, None], sign * sin[:, None]
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return y


def turn_mag(m, cos, sin, R, inter):
    """Sum of the absolute terms of a rotation of values of magnitude m."""
    i, j = pairs(R, inter)
    y, c, s = m.copy(), np.abs(cos)[:, None], np.abs(sin)[:, None]
    y[..., i] = m[..., i] * c + m[..., j] * s
    y[..., j] = m[..., j] * c + m[..., i] * s
    return y


def qk_fwd(x, gamma, cos, sin, R, inter, eps):
    """Result and magnitude of one of q, k; cos, sin already by token."""
    D = x.shape[-1]
    den = (x * x).sum(-1, keepdims=True) / D + eps
    rho = np.where(den == 0, 0.0, 1 / np.sqrt(np.where(den == 0, 1, den)))
    a = x * rho * (1.0 if gamma is None else gamma)
    return turn(a, cos, sin, R, inter), turn_mag(np.abs(a), cos, sin, R, inter)


def qk_bwd(dy, x, gamma, cos, sin, R, inter, eps):
    """dx, its magnitude, dgamma and its magnitude."""
    D = x.shape[-1]
    g = 1.0 if gamma is None else gamma
    den = (x * x).sum(-1, keepdims=True) / D + eps
    rho = np.where(den == 0, 0.0, 1 / np.sqrt(np.where(den == 0, 1, den)))
    b, xh = turn(dy, cos, sin, R, inter, -1.0), x * rho
    bm = turn_mag(np.abs(dy), cos, sin, R, inter)
    dx = rho * (b * g - xh * (b * g * xh).sum(-1, keepdims=True) / D)
    gm = bm * np.abs(g)
    dxm = rho * (gm + np.abs(xh) * (gm * np.abs(xh)).sum(-1, keepdims=True) / D)
    return dx, dxm, (b * xh).sum((0, 1)), (bm * np.abs(xh)).sum((0, 1))


def rope_table(P, R, base=10000.0):
    a = np.arange(P)[:, None] * base ** (-np.arange(R // 2) * 2.0 / max(R, 1))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


# ---- router ----------------------------------------------------------------

def logistic(l):
    return np.exp(-np.logaddexp(0, -l))


def top(l, k):
    """The k largest of each row, ties to the lowest index, NaN first."""
    key = np.where(np.isnan(l), np.inf, l)
    first = np.where(np.isnan(l), 0, 1)
    E = l.shape[1]
    return np.stack([np.lexsort((np.arange(E), -key[t], first[t]))[:k]
                     for t in range(l.shape[0])]) if l.shape[0] else np.zeros((0, k), int)


def softmax(v, on):
    v = np.where(on, v, -np.inf)
    m = v.max(-1, keepdims=True)
    p = np.where(np.isneginf(v), 0.0, np.exp(v - np.where(np.isneginf(m), 0, m)))
    s = p.sum(-1, keepdims=True)
    return p / np.where(s == 0, 1, s)


def choice(l, ids):
    """The forward's ids where some may since have been dropped (-1)."""
    ids = np.where(ids < 0, top(l, ids.shape[1]), ids)
    assert all(len(set(row)) == len(row) for row in ids.tolist())
    return ids


def router_scores(l, ids, score, renorm):
    """Weights (scale 1) of the chosen slots; ids -1: dropped after the choice,
    0, but part of the sum that the weights are renormalised by."""
    on = ids >= 0
    lj = np.where(on, np.take_along_axis(l, np.maximum(ids, 0), 1), -np.inf)
    if renorm:
        lj = np.take_along_axis(l, choice(l, ids), 1)
        v = softmax(lj if score == "softmax" else -np.logaddexp(0, -lj), np.ones_like(on))
        return np.where(on, v, 0)
    if score == "softmax":
        p = softmax(l, np.ones_like(l, bool))
        return np.where(on, np.take_along_axis(p, np.maximum(ids, 0), 1), 0)
    return np.where(on, logistic(lj), 0)


def router_bwd(dw, l, ids, score, renorm, scale):
    """dlogits and its magnitude."""
    on, at = ids >= 0, np.maximum(ids, 0)
    a = np.where(on, scale * dw, 0)
    if renorm:  # a dropped slot's expert has its share of the weights' sum
        ids = at = choice(l, ids)
        on = np.ones_like(on)
    v = router_scores(l, ids, score, renorm)
    slope = logistic(-np.take_along_axis(l, at, 1)) if score == "sigmoid" else 1.0
    d, dm = np.zeros_like(l), np.zeros_like(l)
    if renorm or score == "softmax":
        inner, innerm = (a * v).sum(1, keepdims=True), (np.abs(a) * v).sum(1, keepdims=True)
    else:
        inner = innerm = 0.0
    if score == "softmax" and not renorm:
        p = softmax(l, np.ones_like(l, bool))
        d, dm = -p * inner, p * innerm
        inner = innerm = 0.0
    rows = np.broadcast_to(np.arange(l.shape[0])[:, None], ids.shape)
    np.add.at(d, (rows[on], at[on]), (v * slope * (a - inner))[on])
    np.add.at(dm, (rows[on], at[on]), (v * slope * (np.abs(a) + innerm))[on])
    return d, dm


# ---- sort, dispatch, combine -----------------------------------------------

def sort(ids, E, align, R):
    T, k = ids.shape
    flat = ids.reshape(-1)
    counts = np.bincount(flat[flat >= 0], minlength=E)
    offsets = np.concatenate(([0], np.cumsum(-(-counts // align) * align)))
    row_of, slot_of = np.full(T * k, -1), np.full(R, -1)
    for e in range(E):
        at = np.flatnonzero(flat == e)
        row_of[at] = offsets[e] + np.arange(len(at))
    kept = np.flatnonzero(row_of >= 0)
    slot_of[row_of[kept]] = kept
    return counts, offsets, row_of.reshape(T, k), slot_of


def dispatch(x, slot_of, k):
    return np.where((slot_of >= 0)[:, None], x[np.maximum(slot_of, 0) // k], 0)


def gather(ys, row_of):
    return np.where((row_of >= 0)[..., None], ys[np.maximum(row_of, 0)], 0)


def combine(ys, w, row_of):
    g = gather(ys, row_of)
    w = np.ones(row_of.shape) if w is None else w
    return (w[..., None] * g).sum(1), (np.abs(w)[..., None] * np.abs(g)).sum(1)


def combine_bwd(df, ys, w, row_of, slot_of):
    """dys, dw and dw's magnitude."""
    k = row_of.shape[1]
    wf = (np.ones(row_of.shape) if w is None else w).reshape(-1)[np.maximum(slot_of, 0)]
    dys = wf[:, None] * dispatch(df, slot_of, k)
    g = gather(ys, row_of)
    return dys, (g * df[:, None]).sum(-1), (np.abs(g) * np.abs(df[:, None])).sum(-1)
