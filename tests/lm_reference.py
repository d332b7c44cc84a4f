"""The operators on token IDs in plain numpy, 64 bits, and the error that
float32 arithmetic with one rounding on the way out may have against them."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24  # half a step of float32, relative


def half_step(dtype: torch.dtype) -> float:
    return torch.finfo(dtype).eps / 2


def smallest(dtype: torch.dtype) -> float:
    """Half a step among the subnormals."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def embed(weight, ids, scale, pad_id=-1):
    V = weight.shape[0]
    ok = (ids >= 0) & (ids < V) & (ids != pad_id)
    return np.where(ok[:, None], weight[np.where(ok, ids, 0)] * scale, 0.0)


def embed_grad(grad, ids, n_rows, scale, pad_id=-1):
    """The gradient, and a bound of its float32 error before the last
    rounding: n terms added in any order are off by at most (n - 1) U times
    the sum of their magnitudes, and the scale adds one rounding."""
    out = np.zeros((n_rows, grad.shape[1]))
    mag = np.zeros_like(out)
    ok = (ids >= 0) & (ids < n_rows) & (ids != pad_id)
    np.add.at(out, ids[ok], grad[ok])
    np.add.at(mag, ids[ok], np.abs(grad[ok]))
    n = np.bincount(ids[ok], minlength=n_rows)[:, None]
    return out * scale, (n + 2) * U * mag * abs(scale)


def process_logits(x, prompts=None, made=None, rep=None, freq=None, pres=None, bias=None,
                   masks=None, mask_row=None):
    """Row by row from the definition.  prompts, made: a list of IDs per row;
    bias: a dict per row.  Returns the logits and the bound of their error
    before the last rounding: every step's rounding is at most U of a value no
    larger than the sum of the magnitudes in it."""
    out, tol = x.copy(), np.zeros_like(x)
    V = x.shape[1]
    for b in range(x.shape[0]):
        y, t = out[b], tol[b]
        c = np.zeros(V)
        if made is not None:
            c = np.bincount([v for v in made[b] if 0 <= v < V], minlength=V).astype(float)
        seen = c > 0
        if prompts is not None:
            seen = seen.copy()
            seen[[v for v in prompts[b] if 0 <= v < V]] = True
        r = 1.0 if rep is None else float(rep[b])
        f = 0.0 if freq is None else float(freq[b])
        p = 0.0 if pres is None else float(pres[b])
        y[seen] = np.where(y[seen] > 0, y[seen] / r, y[seen] * r)
        mag = np.abs(y)
        y[c > 0] -= (f * c + p)[c > 0]
        mag += np.abs(f) * c + np.abs(p)
        for v, w in (bias[b] if bias is not None else {}).items():
            y[v] += w
            mag[v] += abs(w)
        t[:] = 4 * U * mag
        if mask_row is not None and mask_row[b] >= 0:
            word = masks[mask_row[b]].astype(np.uint32)
            v = np.arange(V)
            y[((word[v >> 5] >> (v & 31).astype(np.uint32)) & 1) == 0] = -np.inf
    return out, tol


def block_tables(off, cached, free, table, bs):
    """table (a new one), slots, positions, lengths, used; no free block: -1."""
    table = table.copy()
    slots, positions, lengths, taken = [], [], [], 0
    for r in range(len(cached)):
        new = int(off[r + 1] - off[r])
        have, want = -(-int(cached[r]) // bs), -(-(int(cached[r]) + new) // bs)
        for j in range(have, want):
            if j < table.shape[1]:
                table[r, j] = free[taken + j - have] if taken + j - have < len(free) else -1
        for pos in range(int(cached[r]), int(cached[r]) + new):
            blk = int(table[r, pos // bs]) if pos // bs < table.shape[1] else -1
            slots.append(blk * bs + pos % bs if blk >= 0 else -1)
            positions.append(pos)
        taken += want - have
        lengths.append(int(cached[r]) + new)
    return (table, np.array(slots, np.int64), np.array(positions, np.int32),
            np.array(lengths, np.int32), taken)


def check(got: torch.Tensor, want: np.ndarray, tol: np.ndarray | float, what: str = "") -> None:
    """|got - want| <= tol + half a step of got's type (of a value up to
    |want| + tol); infinities and NaN in the same places."""
    g = f64(got)
    assert g.shape == want.shape, (g.shape, want.shape)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(g), np.isnan(want)), what
    assert np.array_equal(g[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    lim = tol + half_step(got.dtype) * (np.abs(want) + tol) + smallest(got.dtype)
    with np.errstate(invalid="ignore"):
        off = np.where(fine, np.abs(g - want) - lim, -1.0)
    worst = int(np.argmax(off)) if off.size else 0
    assert not off.size or off.flat[worst] <= 0, \
        f"{what}: {g.flat[worst]} for {want.flat[worst]}, {off.flat[worst]:.3g} past the bound"
