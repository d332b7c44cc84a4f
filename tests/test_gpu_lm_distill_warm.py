"""Distillation at temperatures where the loss is small beside T^2: losses and gradients
within a bound of their own size, against the definition in long double (64 bits of
mantissa), down to students that are their teachers."""
import numpy as np
import pytest
import torch

import lm_draft_reference as ref
from lm_reference import U, check, f64
from byte_level_bpe_pretokenize_amd import _lib, lm

from gpu_util import device
from test_gpu_lm import BF16, F16, F32, dev, gen, randn, status
from test_gpu_lm_distill import rows

pytestmark = pytest.mark.gpu

L = np.longdouble
EXACT = 2.0 ** -63  # half a step of a long double
SUM = 2.0 ** -53


def warm(z, ids, t, T, dloss):
    """Row by row: losses, their bound, the gradient, its bound (before the last
    rounding), and which rows the bounds of the listed tokens' differences hold for.

    With a = (z - largest z) / T, b the same of the list, d = b - a, x = mean d - d
    (by P): float32 terms exp(-s) are off by (4 s + 4) U of themselves, products of
    them by as much, sums in 64 bits by 2 SUM for each doubling of their length (20).
    Where the listed tokens hold more than 3 / 4,
      loss / T^2 = log(1 + A) + log(1 + B),  A = sum P (exp(x) - 1 - x),  B = rest / listed
    A's terms are not negative: each is off by (4 |b| + 4) U, their weights' sum by 8 U,
    and by |d| and x in 64 bits, (|b| + |a|) SUM (1 + |x|) |x|, twice.  B is off by the
    rest's terms' errors and by the listed ones' 8 U of itself, and by 40 SUM where the
    sums' difference is nothing.  q - P = P (exp(x - loss / T^2) - 1) then, off by P's
    error, the exponent's, and one factor's and one product's rounding.  The exponent is
    -d - log(sum P exp(-d)) - log(1 + B), so errors u_k of the P_k (which add up to
    nothing, as the P do to 1) change it by sum u_k exp(-d_k) / sum P exp(-d), at most
    sum P |exp(x) - 1| (4 |b| + 12) U to first order: all of a row's entries by the same
    relative to q, which is more than P's own error where q is near P.  Otherwise the
    bounds are those of sums in 32 bits (lm_draft_reference.py)."""
    N, V = z.shape
    loss, ltol, grad, gtol = ref.distill(z, ids, t, T, dloss)
    near = np.zeros(N, bool)
    for n in range(N):
        on = np.array([k for k in range(ids.shape[1]) if 0 <= ids[n, k] < V and t[n, k] != -np.inf], int)
        if not on.size or np.all(z[n] == -np.inf):
            continue
        at = ids[n, on]
        a = (z[n].astype(L) - z[n].max()) / L(T)
        b = (t[n, on].astype(L) - t[n, on].max()) / L(T)
        with np.errstate(all="ignore"):
            ea, eb = np.exp(a), np.exp(b)
        keep = eb >= 2.0 ** -126
        at, b, eb = at[keep], b[keep], eb[keep]
        held = ea[at].sum()
        if not held > 0.75 * ea.sum() or not np.all(np.isfinite(ea[at])) or np.any(ea[at] == 0):
            continue
        near[n] = True
        P, q = eb / eb.sum(), ea / ea.sum()
        d = b - a[at]
        mean = (P * d).sum()
        x = mean - d
        loss[n] = float(L(T) ** 2 * (P * (d - np.log(eb.sum()) + np.log(ea.sum()))).sum())
        # (log1p and expm1 of long doubles for the bound's parts alone)
        phi = np.expm1(x) - x
        A = (P * phi).sum()
        out = np.ones(V, bool)
        out[at] = False
        rest = (ea[out] * (4 * np.abs(np.where(ea[out] > 0, a[out], 0)) + 4)).sum() * U / held
        B = max(float(abs(ea.sum() / held - 1)), 0.0)
        off = (P * phi * (4 * np.abs(b) + 12) * U).sum() + rest + B * 8 * U + 40 * SUM
        off += 2 * (P * (np.abs(b) + np.abs(a[at]) + np.abs(mean)) * np.abs(np.expm1(x))).sum() * SUM
        off += float(A) * 40 * SUM
        ltol[n] = float(T * T * (off + 8 * EXACT * (1 + np.abs(d).max() + np.log(V))))
        g = q.copy()
        np.add.at(g, at, -P)
        c = float(dloss[n]) * T
        grad[n] = (c * g).astype(np.float64)
        bound = q * (4 * np.where(q > 0, np.abs(a), 0) + 8 + 40) * U
        lost = (np.abs(P * np.expm1(x - loss[n] / T ** 2)) * (4 * np.abs(b) + 16) * U +
                q[at] * (off + (P * np.abs(np.expm1(x)) * (4 * np.abs(b) + 12)).sum() * U + 4 * (np.abs(b) + np.abs(a[at]) + np.abs(mean)) * SUM))
        bound[at] = 0
        np.add.at(bound, at, lost)
        twice = np.bincount(at, minlength=V) > 1
        np.add.at(bound, at[twice[at]], (P * (4 * np.abs(b) + 16) * U)[twice[at]])
        gtol[n] = (abs(c) * (bound + 3 * U * np.abs(g))).astype(np.float64) + 2.0 ** -126 * (1 + abs(c))
    return loss, ltol, grad, gtol, near


def check_warm(z, ids, t, T, gt=None, seed=0, all_near=True, bits=0, gradient=True):
    st = status()
    dl = torch.randn(z.shape[0], device=device(), generator=gen(seed))
    losses, stats = lm.distill(z, dev(ids), t, T, status=st)
    loss, ltol, grad, gtol, near = warm(f64(z), ids, f64(t), float(np.float32(T)), f64(dl))
    assert not all_near or near.all()
    check(losses, loss, ltol, "loss")
    got = lm.distill_grad(z, dev(ids), t, stats, dl, T, out_dtype=gt, status=st)
    if gradient:
        check(got, grad, gtol, "grad")
    assert int(st.item()) == bits
    over = z.clone() if got.dtype is z.dtype else None
    again = lm.distill_grad(z if over is None else over, dev(ids), t, stats, dl, T, out=over, out_dtype=gt, status=st)
    assert torch.equal(again, got)
    return losses, got


def all_listed(N, V, noise, dtype, tdtype, seed):
    """Students near their teachers, which list all tokens, in any order."""
    z = randn((N, V), F32, seed) * 2
    ids = np.stack([np.random.default_rng(seed + n).permutation(V) for n in range(N)]).astype(np.int32)
    t = torch.gather(z + noise * randn((N, V), F32, seed + 1), 1, dev(ids).long()).to(tdtype)
    return z.to(dtype), ids, t


WARM = [4.001, 8.0, 32.0, 256.0, 4096.0, 2.0 ** 20]


@pytest.mark.parametrize("T", WARM)
@pytest.mark.parametrize("V", [2, 50, 1000, 1024])
def test_a_student_near_its_teacher(V, T):
    losses, grad = check_warm(*all_listed(20, V, 0.1, F32, F32, V), T, F32)
    # (what it must not depend on: the loss goes to half the differences' variance)
    assert bool((losses > 0).all()) and bool((losses < 0.05).all())


@pytest.mark.parametrize("T", WARM)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_a_student_that_is_its_teacher(dtype, T):
    """Nothing is left, but for what 64 bits lose: the largest logits are subtracted
    from both sides before they are compared."""
    z, ids, t = all_listed(20, 777, 0.0, dtype, dtype, 5)
    t = torch.gather(z, 1, dev(ids).long())
    losses, grad = check_warm(z, ids, t, T)
    assert bool((losses.abs() <= T * T * 2.0 ** -48).all())
    assert bool((grad.float().abs() <= T * 2.0 ** -44).all())


@pytest.mark.parametrize("T", WARM)
@pytest.mark.parametrize("dtype,gt", [(BF16, BF16), (F16, F32), (F32, BF16)])
def test_other_types(dtype, gt, T):
    check_warm(*all_listed(20, 600, 0.3, dtype, F32, 9), T, gt)


@pytest.mark.parametrize("shift", [300.0, -4096.0])
def test_logits_shifted_by_a_constant(shift):
    z, ids, t = all_listed(10, 500, 0.0, F32, F32, 3)
    z = (z * 64).round() / 64  # (the shift is exact)
    t = torch.gather(z, 1, dev(ids).long()) + shift
    losses, _ = check_warm(z, ids, t, 1000.0)
    assert bool((losses.abs() <= 1e6 * 2.0 ** -48).all())


@pytest.mark.parametrize("T", [8.0, 100.0, 4096.0])
@pytest.mark.parametrize("V,K", [(1000, 990), (1000, 700), (1300, 1024), (2048, 1024), (2000, 30)])
def test_a_rest_that_is_not_listed(V, K, T):
    """From little rest to most of the row."""
    z, ids, t = all_listed(15, V, 0.1, F32, F32, V + K)
    check_warm(z, np.ascontiguousarray(ids[:, :K]), t[:, :K].contiguous(), T, F32, all_near=False)


@pytest.mark.parametrize("V", [2049, 9000, 50257])
@pytest.mark.parametrize("T", [4.5, 20.0, 1000.0])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masked_logits_of_large_vocabularies(dtype, T, V):
    """All that a mask lets through is listed, or all but a little.  The gradient there is the
    difference of numbers in 32 bits."""
    z, ids, t = all_listed(12, 900, 0.1, F32, F32, V)
    wide = torch.full((12, V), -float("inf"), device=device())
    place = torch.from_numpy(np.sort(np.random.default_rng(V).choice(V, 900, replace=False))).to(device())
    wide[:, place] = z
    wide[5:, V // 2] = -3.0 * T
    wide[8:, :] = torch.maximum(wide[8:, :], torch.full((), -40.0 * T, device=device()))
    ids = place.cpu().numpy()[ids].astype(np.int32)
    check_warm(wide.to(dtype), ids, t, T, F32, gradient=False, all_near=False)
    losses, stats = lm.distill(wide, dev(ids), t, T)
    dl = torch.ones(12, device=device())
    _, _, grad, gtol = ref.distill(f64(wide), ids, f64(t), float(np.float32(T)), f64(dl))
    check(lm.distill_grad(wide, dev(ids), t, stats, dl, T), grad, gtol, "grad")


@pytest.mark.parametrize("T", [8.0, 300.0])
def test_masks(T):
    """Listed tokens without probability on either side, entries that hold no token,
    rows without anything."""
    z, ids, t = all_listed(14, 600, 0.1, F32, F32, 21)
    inf = float("inf")
    z[1, ids[1, 4]] = -inf               # an infinite loss, a finite gradient
    z[2, ids[2, 7]] = -inf
    t[2, 7] = -inf                       # and none where the teacher gives it nothing
    ids[3, ::2] = -1
    t[4] = -inf
    z[5] = -inf
    t[6, 10:] = -inf
    ids[7] = -1
    t[8, 3] = t[8].max() - 200.0 * T     # (a share that float32 does not hold)
    z[8, ids[8, 3]] = -inf
    z[9, ids[9, 3]] = -300.0 * T         # a share of the student's that it does not hold
    losses, grad = check_warm(z, ids, t, T, F32, all_near=False)
    assert losses[[4, 5, 7]].tolist() == [0, 0, 0] and float(losses[1]) == inf
    assert bool((grad[[4, 5, 7]] == 0).all()) and bool(torch.isfinite(grad).all())
    assert bool(torch.isfinite(losses[[2, 8, 9]]).all())


@pytest.mark.parametrize("T", [8.0, 300.0])
def test_tokens_listed_more_than_once(T):
    z, ids, t = all_listed(10, 400, 0.1, F32, F32, 22)
    ids[1, 3] = ids[1, 0]
    ids[2, 100:104] = ids[2, 9]
    ids[3, ::2] = ids[3, 1::2]           # each of half the tokens twice
    ids[4] = 5
    ids[5, 7:60:2] = ids[5, 6:60:2]      # one of the two, the first or the second, without weight
    t[5, 6:30:2], t[5, 31:60:2] = -float("inf"), -float("inf")
    _, got = check_warm(z, ids, t, T, F32, all_near=False)
    st = lm.distill(z, dev(ids), t, T)[1]
    dl = torch.randn(10, device=device(), generator=gen(0))
    for _ in range(3):
        assert torch.equal(lm.distill_grad(z, dev(ids), t, st, dl, T, out_dtype=F32), got)
    both = np.ascontiguousarray(np.concatenate([ids[:, :200]] * 2, 1))
    check_warm(z[:, :], both, t[:, :200].repeat(1, 2), T, F32, all_near=False)


def test_nan_and_infinity_spread_over_their_row():
    z, ids, t = all_listed(8, 300, 0.1, F32, F32, 10)
    z[1, 3] = float("nan")
    z[2, 200] = float("inf")
    z[3] = float("nan")
    t[4, 2] = float("nan")
    t[5, 9] = float("inf")
    losses, stats = lm.distill(z, dev(ids), t, 16.0)
    grad = lm.distill_grad(z, dev(ids), t, stats, torch.ones(8, device=device()), 16.0)
    assert torch.isnan(losses).tolist() == [False, True, True, True, True, True, False, False]
    assert bool(torch.isnan(grad[1:4]).all()) and bool(torch.isfinite(grad[[0, 6, 7]]).all())
    for n in (4, 5):
        assert bool(torch.isnan(grad[n, dev(ids)[n].long()]).any())


def test_bad_ids():
    z, ids, t = all_listed(6, 500, 0.1, BF16, F32, 11)
    ids[1, 2], ids[2, 0], ids[3, 7], ids[4] = 500, -2, 2 ** 31 - 1, -2 ** 31
    losses, grad = check_warm(z, ids, t, 9.0, all_near=False, bits=_lib.STATUS_BAD_ID)
    assert float(losses[4]) == 0 and bool((grad[4] == 0).all())


@pytest.mark.parametrize("T", [5.0, 20.0, 2.0 ** 20])
def test_short_lists_of_large_vocabularies(T):
    """The usual call: the listed tokens hold little, and sums in 32 bits are near."""
    check_warm(*rows(8, 20001, 40, BF16, F32, 4), T, F32, all_near=False)
    check_warm(*rows(40, 876, 16, BF16, F32, 4), T, F32, all_near=False)


def test_against_differences():
    """The gradient against differences of the loss itself, which 32 bits would not
    resolve: T^2 2^-23 is 0.5 here."""
    T, (z, ids, t) = 2048.0, all_listed(6, 300, 0.3, F32, F32, 16)
    d = torch.randn(z.shape, device=device(), generator=gen(3))
    e = 2.0 ** -7
    up, down = (lm.distill(z + s * e * d, dev(ids), t, T)[0].double() for s in (1, -1))
    leaf = z.clone().requires_grad_()
    lm.distillation(leaf, dev(ids), t, T).sum().backward()
    slope, want = (up - down) / (2 * e), (leaf.grad.double() * d).sum(1)
    # the loss is a parabola up to 1 / T: its differences are off by the losses' roundings, a
    # few U of them, and those of z + s e d, half a step of up to 8 each, by the gradient
    tol = 8 * U * (up.abs() + down.abs()) / (2 * e) + (leaf.grad.double().abs() * 2.0 ** -21).sum(1) / (2 * e)
    assert bool(((slope - want).abs() <= tol + 1e-3 * want.abs() / 1.0).all())


@pytest.mark.parametrize("V,K", [(700, 700), (5000, 600)])
def test_captured_and_replayed_on_another_stream(V, K):
    """Loss and gradient in one graph, replayed with logits that are near the teacher's, far from
    them and near again, between eager calls on two streams at once."""
    T, st, dl = 24.0, status(), torch.ones(9, device=device())
    z, ids, t = torch.zeros(9, V, device=device()), torch.zeros(9, K, dtype=torch.int32, device=device()), \
        torch.zeros(9, K, device=device())
    out = [torch.zeros(9, device=device()), torch.zeros(9, 4, device=device()), torch.zeros(9, V, device=device())]

    def step():
        lm.distill(z, ids, t, T, losses=out[0], stats=out[1], status=st)
        lm.distill_grad(z, ids, t, out[1], dl, T, out=out[2], status=st)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k, noise in enumerate((0.1, 30.0, 0.1, 0.0)):
        z2, ids2, t2 = all_listed(9, K, noise, F32, F32, 60 + k)
        z.fill_(-float("inf") if k % 2 == 0 else -50.0)
        z[:, :K] = z2
        ids.copy_(dev(ids2))
        t.copy_(t2)
        dl.copy_(torch.randn(9, device=device(), generator=gen(k)))
        graph.replay()
        torch.cuda.synchronize()
        loss, ltol, _, _, _ = warm(f64(z), ids2, f64(t), T, f64(dl))
        check(out[0], loss, ltol, "loss")
        streams, got = [torch.cuda.Stream() for _ in range(2)], []
        for _ in range(5):
            for s in streams:
                losses, stats = lm.distill(z, ids, t, T, status=st, stream=s)
                got.append((losses, lm.distill_grad(z, ids, t, stats, dl, T, status=st, stream=s)))
        torch.cuda.synchronize()
        assert all(torch.equal(a, out[0]) and torch.equal(b, out[2]) for a, b in got)
    assert int(st.item()) == 0
