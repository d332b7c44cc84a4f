"""The drafting operators on outputs that are stored past the caches (32 MB and more), on
slabs of logits behind the first, and on tokens of more lanes than a workgroup
takes at once."""
import numpy as np
import pytest
import torch

import lm_draft_reference as ref
from lm_reference import U, check, f64, half_step, smallest
from byte_level_bpe_pretokenize_amd import lm

from gpu_util import device
from test_gpu_lm import BF16, F16, F32, dev, gaps, gen, status, strided
from test_gpu_lm_cache import KINDS, cache_of, check_read, paged
from test_gpu_lm_distill import rows

pytestmark = pytest.mark.gpu

SLAB = 8192  # logits of one workgroup of the gradient
PAST = 32 << 20  # bytes from which outputs go past the caches


def at_the_slabs_ends(ids, V, seed):
    """Each row's list with tokens on both sides of the slabs' ends, some of them
    twice, thrice or in all of the list's second half."""
    rng = np.random.default_rng(seed)
    ends = [v for s in range(0, V + 1, SLAB) for v in (s - 1, s) if 0 <= v < V] + [V - 1]
    N, K = ids.shape
    for n in range(N):
        at = rng.permutation(K)
        ids[n, at[:len(ends)]] = ends
        again = rng.integers(1, 4)
        ids[n, at[len(ends):len(ends) + again * 3]] = np.repeat(rng.choice(ends, 3, replace=False), again)
        if n % 50 == 7:
            ids[n, K // 2:] = ends[n % len(ends)]
    return ids


@pytest.mark.parametrize("N,V,dtype,gt", [(600, 30001, BF16, BF16), (300, 30001, F32, F32), (600, 30000, F16, F16),
                                          (300, 28673, BF16, F32), (2100, 8193, F32, BF16)])
def test_a_gradient_past_the_caches(N, V, dtype, gt):
    """Listed tokens are stored over what the row's vectors stored first."""
    assert N * V * torch.finfo(gt).bits // 8 >= PAST
    z, ids, t = rows(N, V, 60, dtype, F32, V)
    ids = at_the_slabs_ends(ids, V, N)
    dl, st, T = torch.randn(N, device=device(), generator=gen(1)), status(), 1.25
    losses, stats = lm.distill(z, dev(ids), t, T, status=st)
    loss, ltol, grad, gtol = ref.distill(f64(z), ids, f64(t), T, f64(dl))
    check(losses, loss, ltol, "loss")
    got = lm.distill_grad(z, dev(ids), t, stats, dl, T, out_dtype=gt, status=st)
    check(got, grad, gtol, "grad")
    for _ in range(3):
        assert torch.equal(lm.distill_grad(z, dev(ids), t, stats, dl, T, out_dtype=gt, status=st), got)
    if dtype is gt:  # over the logits themselves, whose rows start anywhere
        z = strided(z, 3)
        lm.distill_grad(z, dev(ids), t, stats, dl, T, out=z, status=st)
        assert torch.equal(z, got) and bool((gaps(z, 3) == 0).all())
    assert int(st.item()) == 0


@pytest.mark.parametrize("V", [8193, 20000, 131073])
def test_repeated_tokens_on_all_slabs(V):
    """The same by outputs that the caches keep, and every list in another order."""
    z, ids, t = rows(12, V, 90, BF16, F32, V)
    ids = at_the_slabs_ends(ids, V, 1)
    dl = torch.randn(12, device=device(), generator=gen(2))
    losses, stats = lm.distill(z, dev(ids), t)
    loss, ltol, grad, gtol = ref.distill(f64(z), ids, f64(t), 1.0, f64(dl))
    check(losses, loss, ltol, "loss")
    check(lm.distill_grad(z, dev(ids), t, stats, dl, out_dtype=F32), grad, gtol, "grad")
    back = np.ascontiguousarray(ids[:, ::-1])
    check(lm.distill_grad(z, dev(back), t.flip(1), stats, dl, out_dtype=F32), grad, gtol, "grad")


def held(codes, scales, D, group, four):
    """(S, H, D) values in 64 bits, by torch."""
    if four:
        c = torch.stack((codes & 15, codes >> 4), -1).flatten(2)[..., :D].double()
    else:
        c = codes.float().double()
    s = scales.double().repeat_interleave(group, 2)[:, :, :D]
    return c * s[..., 0] + s[..., 1] if four else c * s


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ot", [BF16, F16, F32])
@pytest.mark.parametrize("H,D,group", [(16, 128, 64), (8, 80, 32), (16, 132, 32), (5, 77, 16)])
def test_a_read_past_the_caches(H, D, group, ot, kind):
    """(Heads of no whole vectors are stored through them at any size.)"""
    rng, bs = np.random.default_rng(3), 16
    n = PAST // (H * D * torch.finfo(ot).bits // 8) + 1001
    lengths = rng.multinomial(n, np.full(7, 1 / 7))
    table, n_slots = paged(lengths, bs, 5)
    c, s = cache_of(n_slots, H, D, kind, group)
    off, st = dev(np.concatenate([[0], np.cumsum(lengths)])), status()
    out = torch.full((n + 5, H, D), 3.0, dtype=ot, device=device())
    lm.cache_read(c, s, group, dev(table), bs, off, n + 5, out=out, status=st)
    p = np.concatenate([np.arange(k) for k in lengths])
    slots = table[np.repeat(np.arange(7), lengths), p // bs].astype(np.int64) * bs + p % bs
    at = dev(slots)
    for a in range(0, n, 8192):
        part = at[a:a + 8192]
        want = held(c[part] if kind == "u4" else c.view(torch.uint8)[part].view(KINDS[kind]), s[part], D, group,
                    kind == "u4")
        got = out[a:min(a + 8192, n)].double()
        # one float32 rounding of the value, and the output's
        tol = U * want.abs() + 2.0 ** -150
        tol = tol + (0 if ot is F32 else half_step(ot) * (want.abs() + tol) + smallest(ot))
        assert bool(((got - want).abs() <= tol).all()), a
    assert bool((out[n:] == 3.0).all()) and int(st.item()) == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ot", [BF16, F32])
@pytest.mark.parametrize("H,D,group", [(64, 256, 128), (64, 250, 32), (1024, 33, 16), (40, 1024, 512), (3, 1023, 256)])
def test_tokens_of_more_lanes_than_a_workgroup_takes_at_once(H, D, group, ot, kind):
    lengths, bs = [3, 0, 14, 1], 4
    table, n_slots = paged(lengths, bs)
    c, s = cache_of(n_slots, H, D, kind, group)
    off = 1 + np.concatenate([[0], np.cumsum(lengths)])
    check_read(c, s, group, table, bs, off, int(off[-1]) + 2, D, kind, ot)
