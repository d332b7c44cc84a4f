"""Distillation on the GPU: losses and gradients within the bounds that float32
arithmetic has against 64 bits (lm_draft_reference.py)."""
import numpy as np
import pytest
import torch

import lm_draft_reference as ref
from lm_reference import U, check, f64
from byte_level_bpe_pretokenize_amd import _lib, lm

from gpu_util import device
from test_gpu_lm import BF16, F16, F32, dev, gaps, gen, randn, status, strided

pytestmark = pytest.mark.gpu


def rows(N, V, K, dtype, tdtype, seed, scale=3.0):
    z = (randn((N, V), F32, seed) * scale).to(dtype)
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.choice(V, K, replace=False) for _ in range(N)]).astype(np.int32).reshape(N, K)
    t = (randn((N, K), F32, seed + 1) * scale).to(tdtype)
    return z, ids, t


def check_distill(z, ids, t, T, gt=None, bits=0, seed=0, dloss=None, out=None):
    st = status()
    tids = dev(ids) if isinstance(ids, np.ndarray) else ids
    losses, stats = lm.distill(z, tids, t, T, status=st)
    if dloss is None:
        dloss = torch.randn(z.shape[0], device=device(), generator=gen(seed))
    loss, ltol, grad, gtol = ref.distill(f64(z), tids.cpu().numpy(), f64(t), float(np.float32(T)), f64(dloss))
    check(losses, loss, ltol, "loss")
    got = lm.distill_grad(z, tids, t, stats, dloss, T, out_dtype=gt, out=out, status=st)
    check(got, grad, gtol, "grad")
    assert int(st.item()) == bits
    return losses, stats, got


@pytest.mark.parametrize("dtype,tdtype,gt", [(F32, F32, F32), (BF16, F32, BF16), (F16, F16, F16), (BF16, BF16, F32),
                                             (F32, F16, BF16)])
@pytest.mark.parametrize("N,V,K", [(1, 1, 1), (3, 2, 1), (5, 7, 7), (9, 64, 3), (33, 1000, 20), (17, 4097, 64),
                                   (7, 8192, 1), (6, 16385, 100), (4, 50257, 33), (2, 128256, 64)])
def test_distill(N, V, K, dtype, tdtype, gt):
    check_distill(*rows(N, V, K, dtype, tdtype, V), 1.0, gt)


@pytest.mark.parametrize("T", [0.25, 0.7, 2.0, 8.0])
def test_temperatures(T):
    check_distill(*rows(20, 3001, 40, BF16, F32, 4), T, F32)


@pytest.mark.parametrize("V", [2040, 2047, 2048, 2049, 2060])
def test_both_sides_of_the_variants(V):
    check_distill(*rows(300, V, 9, BF16, F32, 5), 1.5)
    check_distill(*rows(30, V, 200, F32, BF16, 6), 0.8)


@pytest.mark.parametrize("K", [0, 255, 256, 257, 1024])
def test_long_lists(K):
    check_distill(*rows(5, 2000, K, F32, F32, 6), 1.0)
    if K:
        check_distill(*rows(1100, 1100, K, BF16, BF16, 7), 2.0)


def test_far_logits():
    """Large and far apart, in both directions, and constant rows."""
    z, ids, t = rows(12, 5000, 30, F32, F32, 8, scale=40.0)
    z[3] += 1000.0
    z[4] -= 1e6
    z[5] = 17.0
    z[6] = torch.finfo(F32).min
    z[7, :2500], z[7, 2500:] = -1e30, 1e30
    ids[7] = np.arange(2500, 2530)
    t[8] = 3.0
    t[9] = torch.finfo(F32).min
    t[10, 1:] = -1e30
    check_distill(z, ids, t, 1.0)


def test_masks():
    """-infinity in the student's logits and in the teacher's, lowest values, entries
    that hold no token, rows that are left without anything."""
    N, V, K = 24, 3000, 12
    z, ids, t = rows(N, V, K, BF16, F32, 9)
    inf = float("inf")
    z[1, 5:] = -inf                      # five tokens are left
    ids[1] = np.arange(K) % 5
    z[2] = -inf                          # none
    z[3] = torch.finfo(BF16).min
    z[4, ::2] = -inf
    ids[4] = 2 * np.arange(K) + 1        # the listed ones are not masked
    t[5] = -inf                          # a teacher without anything
    t[6, 1:] = -inf                      # with one token
    ids[7] = -1
    ids[8, 3:] = -1
    ids[9, :-1] = -1
    z[10, ids[10, 4]] = -inf             # an infinite loss, a finite gradient
    z[11, ids[11, 4]] = -inf             # and none where the teacher gives it nothing
    t[11, 4] = -inf
    losses, _, grad = check_distill(z, ids, t, 1.3, F32)
    assert losses[[2, 5, 7]].tolist() == [0, 0, 0] and float(losses[10]) == inf
    assert bool((grad[[2, 5, 7]] == 0).all())
    # rows without a loss have zeros whatever comes in
    dl = torch.full((N,), float("nan"), device=device())
    st = lm.distill(z, dev(ids), t, 1.3)[1]
    assert bool((lm.distill_grad(z, dev(ids), t, st, dl, 1.3)[[2, 5, 7]] == 0).all())


def test_a_probability_that_float32_does_not_hold():
    """A listed token 200 below the largest weighs nothing, also where the student's
    logit is -infinity."""
    z, ids, t = rows(4, 3000, 6, F32, F32, 20)
    t[:, 2] = t.amax(1) - 200.0
    z[torch.arange(4, device=device()), dev(ids)[:, 2].long()] = -float("inf")
    losses, _, grad = check_distill(z, ids, t, 1.0)
    assert bool(torch.isfinite(losses).all()) and bool(torch.isfinite(grad).all())


def test_nan_and_infinity_spread_over_their_row():
    z, ids, t = rows(8, 900, 10, F32, F32, 10)
    z[1, 3] = float("nan")
    z[2, 700] = float("inf")
    z[3] = float("nan")
    t[4, 2] = float("nan")
    t[5, 9] = float("inf")
    losses, stats = lm.distill(z, dev(ids), t)
    grad = lm.distill_grad(z, dev(ids), t, stats, torch.ones(8, device=device()))
    assert torch.isnan(losses).tolist() == [False, True, True, True, True, True, False, False]
    assert bool(torch.isnan(grad[1:4]).all()) and bool(torch.isfinite(grad[[0, 6, 7]]).all())
    for n in (4, 5):  # the teacher's: at its tokens
        assert bool(torch.isnan(grad[n, dev(ids)[n].long()]).any())


def test_bad_ids():
    z, ids, t = rows(6, 500, 8, BF16, F32, 11)
    ids[1, 2], ids[2, 0], ids[3, 7], ids[4] = 500, -2, 2 ** 31 - 1, -2 ** 31
    losses, _, grad = check_distill(z, ids, t, 1.0, bits=_lib.STATUS_BAD_ID)
    assert float(losses[4]) == 0 and bool((grad[4] == 0).all())
    with pytest.raises(RuntimeError, match="status 0x4"):
        lm.distill(z, dev(ids), t)


@pytest.mark.parametrize("K", [7, 300])
def test_a_token_listed_more_than_once(K):
    z, ids, t = rows(8, 700, K, F32, F32, 12)
    ids[1, 3] = ids[1, 0]
    ids[2] = 5
    ids[3, ::2] = 600
    ids[4, 1:4] = 699
    a = check_distill(z, ids, t, 1.0)
    b = check_distill(z, ids, t, 1.0)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides(dtype):
    z, ids, t = rows(15, 9001, 21, dtype, dtype, 13)
    wide = strided(dev(ids), 5)
    out = strided(torch.full_like(z, 7.0), 3)
    check_distill(strided(z, 9), wide, strided(t, 2), 1.0, out=out)
    assert bool((gaps(out, 3) == 0).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [50, 8192, 8193, 30001])
def test_in_place(V, dtype):
    """The gradient over the logits themselves, with listed tokens everywhere."""
    z, ids, t = rows(40, V, min(V, 1000), dtype, F32, 14)
    losses, stats, want = check_distill(z, ids, t, 1.0)
    st, dl = status(), torch.randn(40, device=device(), generator=gen(0))
    z = strided(z, 4)
    got = lm.distill_grad(z, dev(ids), t, stats, dl, out=z, status=st)
    assert got is z and torch.equal(z, want) and int(st.item()) == 0
    assert bool((gaps(z, 4) == 0).all())


def test_no_rows():
    z = torch.zeros((0, 50), device=device())
    ids, t = torch.zeros((0, 4), dtype=torch.int32, device=device()), torch.zeros((0, 4), device=device())
    losses, stats = lm.distill(z, ids, t)
    assert losses.shape == (0,) and stats.shape == (0, 4)
    assert lm.distill_grad(z, ids, t, stats, losses).shape == (0, 50)


def test_many_rows():
    """Past 2^21 workgroups, and offsets past 2^31 elements."""
    N, V, K = (1 << 22) - 1, 600, 2
    z = torch.zeros((N, V), dtype=BF16, device=device())
    z[-1, 7] = 5.0
    ids = torch.tensor([[3, 7]], dtype=torch.int32, device=device()).repeat(N, 1)
    t = torch.zeros((N, K), device=device())
    losses, stats = lm.distill(z, ids, t)
    one = np.log(600 / 2)
    assert bool(((losses[:-1].double() - one).abs() <= 80 * U * one).all())
    last = ref.distill(f64(z[-1:]), ids[-1:].cpu().numpy(), f64(t[-1:]), 1.0)
    check(losses[-1:], last[0], last[1])
    g = lm.distill_grad(z, ids, t, stats, torch.ones(N, device=device()), out=z)
    want = torch.full((V,), 1 / V, device=device())
    want[[3, 7]] -= 0.5
    assert bool((g[[0, N // 2, N - 2]].float() - want).abs().max() <= 2.0 ** -8 * 0.5 + 1e-6)


def test_autograd():
    z, ids, t = rows(30, 1200, 16, BF16, F32, 15)
    leaf = z.clone().requires_grad_()
    st = status()
    losses = lm.distillation(leaf, dev(ids), t, 2.0, status=st)
    losses.mean().backward()  # (a broadcast gradient)
    dl = torch.full((30,), 1 / 30, device=device())
    _, _, want = check_distill(z, ids, t, 2.0, dloss=dl)
    assert leaf.grad.dtype == BF16 and torch.equal(leaf.grad, want) and int(st.item()) == 0
    # against plain operations in 64 bits
    x = z.double().requires_grad_()
    lq = torch.log_softmax(x / 2, 1).gather(1, dev(ids).long())
    P = torch.softmax(t.double() / 2, 1)
    (4 * (P * (P.log() - lq)).sum(1)).mean().backward()
    assert bool(((leaf.grad.double() - x.grad).abs() <= 2.0 ** -8 * x.grad.abs() + 1e-7).all())
    with pytest.raises(RuntimeError):
        (g,) = torch.autograd.grad(lm.distillation(leaf, dev(ids), t).sum(), leaf, create_graph=True)
        g.sum().backward()


def test_gradient_against_differences():
    z, ids, t = rows(10, 400, 12, F32, F32, 16)
    leaf = z.clone().requires_grad_()
    d = torch.randn(z.shape, device=device(), generator=gen(3)).double()
    dl = torch.randn(10, device=device(), generator=gen(4))
    (lm.distillation(leaf, dev(ids), t, 1.5) * dl).sum().backward()
    e = 1e-5
    up, down = (ref.distill(f64(z) + s * e * f64(d), ids, f64(t), 1.5)[0] for s in (1, -1))
    slope = float(((up - down) / (2 * e) * f64(dl)).sum())
    mag = float((leaf.grad.double().abs() * d.abs()).sum())
    assert abs(float((leaf.grad.double() * d).sum()) - slope) <= 1e-5 * mag


def test_the_saved_student_counts_as_modified():
    z, ids, t = rows(4, 100, 3, F32, F32, 17)
    leaf = z.clone().requires_grad_()
    y = leaf * 1.0
    loss = lm.distillation(y, dev(ids), t)
    with torch.no_grad():
        lm.distill_grad(y, dev(ids), t, lm.distill(y, dev(ids), t)[1], torch.ones(4, device=device()), out=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.sum().backward()


def test_forward_and_backward_in_a_graph():
    """Captured together (no eager graph of the leaf lives meanwhile), replayed with
    other inputs."""
    z, ids, t = rows(50, 3000, 16, BF16, F32, 18)
    leaf, tids, dl, st = z.clone().requires_grad_(), dev(ids), torch.ones(50, device=device()), status()

    def step():
        losses = lm.distillation(leaf, tids, t, 2.0, status=st)
        return losses, torch.autograd.grad(losses, leaf, dl)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        losses, grad = step()
    losses, grad = losses.detach(), grad
    for k in range(4):
        z2, ids2, t2 = rows(50, 3000, 16, BF16, F32, 30 + k)
        with torch.no_grad():
            leaf.copy_(z2)
        tids.copy_(dev(ids2))
        t.copy_(t2)
        dl.copy_(torch.randn(50, device=device(), generator=gen(k)))
        graph.replay()
        torch.cuda.synchronize()
        want, stats = lm.distill(z2, tids, t2, 2.0)
        assert torch.equal(losses, want) and torch.equal(grad, lm.distill_grad(z2, tids, t2, stats, dl, 2.0)), k
    assert int(st.item()) == 0


def test_another_stream_outlives_its_inputs():
    make = lambda: rows(2000, 4000, 8, BF16, F32, 19)  # noqa: E731
    z, ids, t = make()
    dl, tids = torch.ones(2000, device=device()), dev(ids)
    want = lm.distill(z, tids, t)
    want_g = lm.distill_grad(z, tids, t, want[1], dl)
    side, st = torch.cuda.Stream(), status()
    busy = torch.ones((4096, 4096), device=device())
    copy = z.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(8):
            busy = busy @ busy * 2.0 ** -12
    got = lm.distill(copy, tids, t, status=st, stream=side)
    got_g = lm.distill_grad(copy, tids, t, got[1], dl, status=st, stream=side)
    del copy
    noise = [torch.full_like(z, 9.0) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got_g, want_g) and int(st.item()) == 0
    del noise
