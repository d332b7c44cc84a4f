"""A cache of few bits, drafted tokens and distillation in plain numpy, and the
error that float32 arithmetic may have against 64 bits."""
from __future__ import annotations

import numpy as np
import torch

from lm_reference import U

TOP = {"e4m3": 448.0, "int8": 127.0, "u4": 15.0}
SMALLEST = 2.0 ** -120
BIG = 2.0 ** 126  # 4 bits: larger magnitudes count as this


# ---- a cache of few bits ----------------------------------------------------------
def e4m3(y: np.ndarray) -> np.ndarray:
    """The nearest e4m3 number, ties to even: steps of an eighth of the power of two
    below, of 2^-9 under 2^-6; y within +-448."""
    y = y.astype(np.float64)
    e = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
    unit = np.exp2(e - 3)
    return np.rint(y / unit) * unit


def quantise(x: np.ndarray, group: int, kind: str):
    """x (n, H, D) float32 to its codes as numbers, scales (n, H, G) and lowest
    values, every step of the definition a float32 operation."""
    x = x.astype(np.float32)
    n, H, D = x.shape
    f = np.float32
    part = f(1) / f(TOP[kind])
    codes = np.zeros((n, H, D))
    G = -(-D // group)
    scales, lows = np.zeros((n, H, G), np.float32), np.zeros((n, H, G), np.float32)
    with np.errstate(all="ignore"):
        for g in range(G):
            v = x[..., g * group:(g + 1) * group].copy()
            fine = np.isfinite(v)
            if kind == "u4":
                v = np.where(fine, np.clip(v, f(-BIG), f(BIG)), v)
                lo = np.where(fine, v, f(np.inf)).min(2)
                hi = np.where(fine, v, f(-np.inf)).max(2)
                some = lo <= hi
                lo = np.where(some, lo, f(0))
                s = np.where(some, (hi - lo) * part, f(0)).astype(np.float32)
                v = v - lo[..., None]
                lows[..., g] = lo
            else:
                s = np.where(fine, np.abs(v), f(0)).max(2) * part
            s = np.where(s < f(SMALLEST), f(0), s)
            inv = np.where(s > 0, f(1) / s, f(0)).astype(np.float32)
            y = (v * inv[..., None]).astype(np.float32)
            y = np.clip(np.where(np.isnan(y), f(0), y), f(0 if kind == "u4" else -TOP[kind]), f(TOP[kind]))
            codes[..., g * group:(g + 1) * group] = e4m3(y) if kind == "e4m3" else np.rint(y)
            scales[..., g] = s
    return codes, scales, lows


def quantise_error(x: np.ndarray, group: int, kind: str):
    """How far a held value may be from x (all finite, scales not tiny): half a step,
    and what the float32 steps to the code and the scale add (4 roundings of
    numbers up to the format's end)."""
    n, H, D = x.shape
    out = np.zeros((n, H, D))
    for a in range(0, D, group):
        v = x[..., a:a + group].astype(np.float64)
        if kind == "u4":
            s = (v.max(2) - v.min(2))[..., None] / 15
            mag = np.abs(v).max(2)[..., None]
            out[..., a:a + group] = s * (0.5 + 5 * 16 * U) + 4 * U * mag
        else:
            s = np.abs(v).max(2)[..., None] / TOP[kind]
            y = np.abs(v) / np.where(s > 0, s, 1)
            step = 0.5 if kind == "int8" else np.maximum(y * 2.0 ** -4, 2.0 ** -10)
            out[..., a:a + group] = s * (step + 5 * U * (y + 1))
    return out


def unpack(codes: torch.Tensor, dim: int) -> np.ndarray:
    """A cache's codes as numbers, (S, H, dim)."""
    if codes.dtype == torch.uint8:
        c = codes.cpu().numpy()
        return np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:2], -1)[..., :dim].astype(np.float64)
    return codes.cpu().float().numpy().astype(np.float64)


def values(codes: np.ndarray, scales: np.ndarray, group: int, four: bool):
    """(S, H, D) values in 64 bits, and the bound of a float32's rounding."""
    per = np.arange(codes.shape[2]) // group
    if four:
        v = codes * scales[..., 0].astype(np.float64)[..., per] + scales[..., 1].astype(np.float64)[..., per]
    else:
        v = codes * scales.astype(np.float64)[..., per]
    return v, U * np.abs(v) + 2.0 ** -150


def read_slots(table, bs, off, n, n_slots, start=None):
    """Each packed token's slot: -1 for zeros, None for rows that are no request's."""
    slots = [None] * n
    for r in range(len(off) - 1):
        for t in range(int(off[r]), int(off[r + 1])):
            p = t - int(off[r]) + (max(int(start[r]), 0) if start is not None else 0)
            b = p // bs
            entry = int(table[r, b]) if b < table.shape[1] else -1
            slot = entry * bs + p % bs
            slots[t] = slot if entry >= 0 and slot < n_slots else -1
    return slots


# ---- drafted tokens ---------------------------------------------------------------
def clean(x: np.ndarray) -> np.ndarray:
    x = x.astype(np.float64)
    return np.where(np.isfinite(x) & (x > 0), x, 0.0)


def verify(p, ids, off, accept, sample, q=None):
    """Request by request from the definition: tokens (-9: no request's row), counts."""
    N, V = p.shape
    tokens, counts = np.full(N, -9, np.int64), []
    for r in range(len(off) - 1):
        lo, hi = int(off[r]), int(off[r + 1])
        if lo == hi:
            counts.append(0)
            continue
        j = lo
        while j < hi - 1:
            x = int(ids[j])
            if not 0 <= x < V:
                break
            qx = 1.0 if q is None else float(clean(q[j, x:x + 1])[0])
            if not float(accept[j]) * qx < float(clean(p[j, x:x + 1])[0]):
                break
            j += 1
        w = clean(p[j])
        if j < hi - 1:
            less = np.zeros(V) if q is None else clean(q[j])
            if q is None and 0 <= int(ids[j]) < V:
                less[int(ids[j])] = 1.0
            rest = np.maximum(w - less, 0.0)
            if rest.sum() > 0:
                w = rest
        run = np.cumsum(w)
        token = -1
        if run[-1] > 0:
            u = float(sample[r])
            past = np.flatnonzero((run > max(u, 0.0) * run[-1]) & (w > 0)) if u < 1 else np.zeros(0)
            token = int(past[0]) if past.size else int(np.flatnonzero(w > 0)[-1])
        tokens[lo:hi] = -1
        tokens[lo:j] = ids[lo:j]
        tokens[j] = token
        counts.append(j - lo + (token >= 0))
    return tokens, np.array(counts)


# ---- distillation -----------------------------------------------------------------
def _softmax(x):
    m = x.max()
    e = np.exp(x - m)
    return m, e, e.sum()


def distill(z, ids, t, T, dloss=None):
    """Row by row in 64 bits: losses, their bound, and with dloss the gradient and
    its bound (both before the last rounding).

    A float32 exponent (x - max) * (log2 e / T) is off by at most 4 U of its size
    (difference, constant, product, and the exponential's own two roundings
    aside), so a term exp(-d) by 4 U d + 2 U of itself, less than 8 U for all d
    that weigh anything: d exp(-d) < 0.37 bounds what far terms add to a sum of at
    least 1.  A sum of n terms in runs and trees adds at most (longest run + 20) U,
    and each new maximum in a run rescales it, 8 U more."""
    N, V = z.shape
    loss, ltol = np.zeros(N), np.zeros(N)
    grad, gtol = np.zeros_like(z, dtype=np.float64), np.zeros_like(z, dtype=np.float64)
    run = V // 1024 + 8
    with np.errstate(all="ignore"):
        for n in range(N):
            on = [k for k in range(ids.shape[1]) if 0 <= ids[n, k] < V and t[n, k] != -np.inf]
            if not on or np.all(z[n] == -np.inf):
                continue
            y, at, x = z[n] / T, ids[n, on], t[n, on] / T
            zm, ze, zs = _softmax(y)
            tm, te, ts = _softmax(x)
            te[te < 2.0 ** -126] = 0.0  # (which float32 does not hold)
            q, P = ze / zs, te / ts
            sum_z = (9 * run + 40) * U
            sum_t = (9 * 8 + 40) * U
            diff = np.where(P > 0, (x - tm) - (y[at] - zm), 0.0)
            loss[n] = T * T * (np.sum(np.where(P > 0, P * diff, 0.0)) + np.log(zs) - np.log(ts))
            each = P * np.abs(diff) * (4 * U * np.abs(x - tm) + 4 * U + sum_t)
            ltol[n] = T * T * (np.sum(np.where(P > 0, each, 0.0)) + sum_z + sum_t)
            if not np.isfinite(loss[n]):
                ltol[n] = 0.0
            if dloss is None:
                continue
            g = q.copy()
            bound = q * (4 * U * np.minimum(np.abs(y - zm), 200) + 6 * U + sum_z)
            np.add.at(g, at, -P)
            np.add.at(bound, at, P * (4 * U * np.minimum(np.abs(x - tm), 200) + (6 + ids.shape[1]) * U + sum_t))
            c = float(dloss[n]) * T
            grad[n] = c * g
            # (one rounding of the factor, of the difference and of the product)
            gtol[n] = abs(c) * (bound + 3 * U * np.abs(g)) + 2.0 ** -126 * (1 + abs(c))
    return (loss, ltol) if dloss is None else (loss, ltol, grad, gtol)
