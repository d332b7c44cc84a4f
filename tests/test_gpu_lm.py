"""The operators on token IDs on the GPU, against plain implementations in 64
bits (lm_reference.py) with the bounds that float32 arithmetic and one rounding
on the way out give."""
import numpy as np
import pytest
import torch

import lm_reference as ref
from byte_level_bpe_pretokenize_amd import BPEError, _lib, lm

from gpu_util import device

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    return torch.Generator(device=device()).manual_seed(seed)


def randn(shape, dtype, seed):
    return torch.randn(shape, device=device(), generator=gen(seed)).to(dtype)


def strided(t, extra):
    """The same matrix with rows `extra` elements further apart, off alignment."""
    n, m = t.shape
    big = torch.zeros(n * (m + extra) + 1, dtype=t.dtype, device=t.device)[1:]
    view = big.view(n, m + extra)[:, :m]
    view.copy_(t)
    return view


def gaps(view, extra):
    """What lies between the rows of a matrix that strided() made."""
    n, m = view.shape
    return view._base.view(-1)[1:].view(n, m + extra)[:, m:]


def ids_of(n, vocab, seed, kind="zipf"):
    rng = np.random.default_rng(seed)
    if kind == "one":
        ids = np.full(n, vocab // 2)
    elif kind == "distinct":
        ids = rng.permutation(max(n, vocab))[:n] % vocab
    else:
        ids = np.minimum(rng.zipf(1.3, n) - 1, vocab - 1)
    return ids.astype(np.int32)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(device())
    return t if dtype is None else t.to(dtype)


def status():
    return torch.zeros(1, dtype=torch.int32, device=device())


# ---- embed --------------------------------------------------------------------
@pytest.mark.parametrize("wt,ot", [(BF16, BF16), (F32, BF16), (F32, F32), (F16, F16), (BF16, F32),
                                   (F16, BF16), (F32, F16)])
@pytest.mark.parametrize("n,V,D", [(1, 1, 1), (2, 5, 3), (65, 768, 7), (64, 300, 8), (33, 300, 9),
                                   (1000, 50, 64), (130, 1000, 513), (17, 40, 4096), (3, 9, 8191), (3, 2, 1 << 17), (2, 2, (1 << 17) - 1)])
def test_embed(n, V, D, wt, ot):
    w = randn((V, D), wt, 1)
    ids = ids_of(n, V, n)
    st = status()
    got = lm.embed(w, dev(ids), 1.7, out_dtype=ot, status=st)
    scale = float(np.float32(1.7))
    want = ref.embed(ref.f64(w), ids, scale)
    ref.check(got, want, ref.U * np.abs(want), "embed")
    assert int(st.item()) == 0


@pytest.mark.parametrize("wide", [3, 8])
@pytest.mark.parametrize("D", [5, 24, 1001])
def test_embed_strides_pad_bad_ids(D, wide):
    V, n = 50, 77
    w = strided(randn((V, D), BF16, 2), wide)
    ids = ids_of(n, V, 3)
    ids[::5] = 49
    ids[7], ids[8], ids[9] = -1, V, 2**31 - 1
    ids[10] = -2**31
    out = strided(torch.full((n, D), 7.0, dtype=BF16, device=device()), wide)
    st = status()
    got = lm.embed(w, dev(ids), -0.5, pad_id=49, out=out, status=st)
    assert got is out and int(st.item()) == _lib.STATUS_BAD_ID
    want = ref.embed(ref.f64(w), ids, -0.5, 49)
    ref.check(got, want, 0.0, "embed")
    # nothing between the rows was written
    assert torch.all(gaps(out, wide) == 0)
    with pytest.raises(RuntimeError, match="status 0x4"):
        lm.embed(w, dev(ids), 1.0)


@pytest.mark.parametrize("wt,ot", [(BF16, BF16), (F32, BF16), (F16, F32)])
@pytest.mark.parametrize("n,D", [(33000, 512), (33001, 513), (17001, 1001), (4500, 4104)])
def test_embed_large(n, D, wt, ot):
    V = 300
    w = randn((V, D), wt, 1)
    ids = ids_of(n, V, n)
    ids[::7] = 5
    got = lm.embed(w, dev(ids), 0.3, pad_id=5, out_dtype=ot)
    want = ref.embed(ref.f64(w), ids, float(np.float32(0.3)), 5)
    ref.check(got, want, ref.U * np.abs(want), "embed")


@pytest.mark.parametrize("V,D,ot,extra", [(700, 1001, BF16, 3), (40, 4096, F16, 0), (9000, 2056, BF16, 0)])
def test_embed_by_sorted_ids(V, D, ot, extra):
    n = (512 << 20) // (2 * D) + 77
    assert lm.embed_workspace_bytes(n, V, D, F32, ot) > 0
    w = strided(randn((V, D), F32, 1), extra)
    ids = ids_of(n, V, 2)
    ids[::11] = V - 1
    ids[5], ids[n - 1], ids[n // 2] = -1, V, -2**31
    t, st = dev(ids), status()
    got = lm.embed(w, t, 1.3, pad_id=V - 1, out_dtype=ot, status=st)
    assert int(st.item()) == _lib.STATUS_BAD_ID
    # the same bits as in pieces, which go by the IDs' own order
    for a in range(0, n, 50000):
        assert lm.embed_workspace_bytes(min(50000, n - a), V, D, F32, ot) == 0
        assert torch.equal(got[a:a + 50000], lm.embed(w, t[a:a + 50000], 1.3, pad_id=V - 1, out_dtype=ot,
                                                      status=st))
    some = np.unique(np.concatenate([np.arange(70), np.arange(n - 70, n), [n // 2],
                                     np.random.default_rng(3).integers(0, n, 500)]))
    want = ref.embed(ref.f64(w), ids[some], float(np.float32(1.3)), V - 1)
    ref.check(got[dev(some)], want, ref.U * np.abs(want))
    # a workspace of the caller's
    space = torch.empty(lm.embed_workspace_bytes(n, V, D, F32, ot), dtype=torch.uint8, device=device())
    assert torch.equal(got, lm.embed(w, t, 1.3, pad_id=V - 1, out_dtype=ot, workspace=space, status=st))


def test_embed_pad_outside_the_table():
    w = randn((10, 16), F32, 4)
    ids = np.array([3, 999, 9], np.int32)
    got = lm.embed(w, dev(ids), pad_id=999)
    ref.check(got, ref.embed(ref.f64(w), ids, 1.0, 999), 0.0)


def test_embed_nan_and_infinity_stay_in_their_rows():
    w = randn((4, 40), BF16, 5)
    w[1], w[2] = float("nan"), float("inf")
    got = lm.embed(w, dev(np.array([0, 3, 1, 2, 3], np.int32)), 2.0, pad_id=3).float().cpu()
    assert torch.isfinite(got[0]).all() and torch.all(got[1] == 0) and torch.all(got[4] == 0)
    assert torch.isnan(got[2]).all() and torch.all(got[3] == float("inf"))


def test_embed_shapes():
    w = randn((9, 12), F32, 6)
    ids = dev(np.arange(6, dtype=np.int32).reshape(2, 3))
    assert lm.embed(w, ids).shape == (2, 3, 12)
    assert torch.equal(lm.embed(w, ids), w[ids.long()])
    assert lm.embed(w, ids[:0]).shape == (0, 3, 12)


def test_embed_past_32_bits():
    # rows whose offsets pass 2^31 and 2^32 elements
    V, D = 1_100_000, 4096
    w = torch.empty((V, D), dtype=BF16, device=device())
    ids = np.array([0, 524_287, 524_288, 1_048_576, V - 1], np.int32)
    for i in ids:
        w[int(i)] = randn((D,), BF16, int(i))
    got = lm.embed(w, dev(ids), 3.0)
    ref.check(got, ref.f64(w[dev(ids).long()]) * 3.0, 0.0)


# ---- embed_grad -----------------------------------------------------------------
@pytest.mark.parametrize("gt,ot", [(BF16, F32), (BF16, BF16), (F32, F32), (F16, F32), (F16, F16)])
@pytest.mark.parametrize("n,V,D", [(1, 1, 1), (2, 5, 3), (8, 600, 8), (63, 3, 9), (65, 511, 7),
                                   (1000, 512, 64), (4097, 768, 513), (300, 40, 4096),
                                   (9000, 300000, 24), (5000, 2, 40)])
def test_embed_grad(n, V, D, gt, ot):
    g = randn((n, D), gt, n)
    ids = ids_of(n, V, n)
    st = status()
    got = lm.embed_grad(g, dev(ids), V, 0.75, out_dtype=ot, status=st)
    want, tol = ref.embed_grad(ref.f64(g), ids, V, 0.75)
    ref.check(got, want, tol, "embed_grad")
    assert int(st.item()) == 0 and got.dtype == ot


@pytest.mark.parametrize("kind", ["one", "distinct", "zipf"])
@pytest.mark.parametrize("n", [1, 9, 64, 2047, 2048, 2049, 4096, 4097, 20000, 70001])
def test_embed_grad_lengths(n, kind):
    V, D = 1500, 72
    g = randn((n, D), BF16, n)
    ids = ids_of(n, V, n + 1, kind)
    got = lm.embed_grad(g, dev(ids), V)
    want, tol = ref.embed_grad(ref.f64(g), ids, V, 1.0)
    ref.check(got, want, tol, kind)
    assert torch.equal(got, lm.embed_grad(g, dev(ids), V))  # the same bits again


@pytest.mark.parametrize("n,V,kind", [(524_289, 1000, "zipf"), (600_001, 300_000, "distinct"),
                                      (1_700_003, 77, "zipf"), (1_100_000, 40, "one")])
def test_embed_grad_many_ids(n, V, kind):
    D = 16
    g = randn((n, D), F32, n)
    ids = ids_of(n, V, n, kind)
    ids[::17] = V - 1
    got = lm.embed_grad(g, dev(ids), V, pad_id=V - 1)
    want, tol = ref.embed_grad(ref.f64(g), ids, V, 1.0, V - 1)
    ref.check(got, want, tol, kind)
    # whole numbers, so that every sum is exact: no position left out or twice
    g = torch.randint(-8, 9, (n, D), device=device(), generator=gen(n)).float()
    want, _ = ref.embed_grad(ref.f64(g), ids, V, 1.0, V - 1)
    assert np.array_equal(ref.f64(lm.embed_grad(g, dev(ids), V, pad_id=V - 1)), want)


@pytest.mark.parametrize("n", [100, 3001])
@pytest.mark.parametrize("D", [5, 513, 2056])
@pytest.mark.parametrize("ot", [F32, BF16])
def test_embed_grad_accumulates(D, ot, n):
    V = 200
    g = strided(randn((n, D), BF16, 1), 3)
    ids = ids_of(n, V, 2)
    ids[ids == 7] = 8  # a row without tokens
    first = randn((V, D), ot, 3)
    out = strided(first, 5)
    lm.embed_grad(g, dev(ids), V, -1.5, out=out, accumulate=True)
    want, tol = ref.embed_grad(ref.f64(g), ids, V, -1.5)
    base = ref.f64(first)
    ref.check(out, base + want, tol + ref.U * (np.abs(base) + np.abs(want)))
    assert torch.equal(out[7], first[7])
    assert torch.all(gaps(out, 5) == 0)


@pytest.mark.parametrize("n", [1999, 5000])
def test_embed_grad_pad_and_bad_ids(n):
    V, D = 100, 16
    g = randn((n, D), F32, 1)
    ids = ids_of(n, V, 2)
    ids[::3] = 99
    ids[1], ids[2], ids[n - 1] = -1, V, -2**31
    g[0] = float("nan")  # a pad position
    st = status()
    got = lm.embed_grad(g, dev(ids), V, pad_id=99, status=st)
    want, tol = ref.embed_grad(ref.f64(g), ids, V, 1.0, 99)
    ref.check(got, want, tol)
    assert int(st.item()) == _lib.STATUS_BAD_ID and torch.all(got[99] == 0)
    # every position a pad: zeros
    assert torch.all(lm.embed_grad(g, torch.full((n,), 99, dtype=torch.int32, device=device()), V,
                                   pad_id=99) == 0)


def test_embed_grad_of_nothing():
    ids = torch.zeros(0, dtype=torch.int32, device=device())
    got = lm.embed_grad(torch.zeros((0, 24), device=device()), ids, 50)
    assert got.shape == (50, 24) and torch.all(got == 0)
    out = torch.ones((50, 24), device=device())
    lm.embed_grad(torch.zeros((0, 24), device=device()), ids, 50, out=out, accumulate=True)
    assert torch.all(out == 1)


def test_embed_grad_past_32_bits():
    # gradient rows, and rows of the result, past 2^32 elements
    n, D = 1_060_000, 4096
    g = torch.zeros((n, D), dtype=BF16, device=device())
    ids = torch.randint(0, 1000, (n,), dtype=torch.int32, device=device(), generator=gen(1))
    V = 1_055_000
    at = torch.tensor([5, 524_300, 1_050_000, n - 1], device=device())
    ids[at] = torch.tensor([V - 1, 1_050_001, V - 1, 600_000], dtype=torch.int32, device=device())
    for i in at.tolist():
        g[i] = randn((D,), BF16, i)
    got = lm.embed_grad(g, ids, V, out_dtype=BF16)
    x = ref.f64(g[at])
    ref.check(got[V - 1], x[0] + x[2], 2 * ref.U * (np.abs(x[0]) + np.abs(x[2])))
    ref.check(got[1_050_001], x[1], 0.0)
    ref.check(got[600_000], x[3], 0.0)
    assert float(got[V - 2].abs().max()) == 0 and float(got[3].abs().max()) == 0


def test_embed_grad_infinity_stays_in_its_row():
    ids = dev(np.array([1, 2, 1, 3], np.int32))
    g = torch.ones((4, 16), device=device())
    g[1] = float("inf")
    got = lm.embed_grad(g, ids, 5).cpu()
    assert got[:, 0].tolist() == [0, 2, float("inf"), 1, 0]


# ---- autograd ---------------------------------------------------------------------
def test_embedding_gradient():
    V, D, scale = 60, 40, 3.0
    ids = dev(ids_of(200, V, 1).reshape(4, 50))
    w = randn((V, D), F32, 2).requires_grad_()
    dy = randn((4, 50, D), F32, 3)
    out = lm.embedding(w, ids, scale, pad_id=5)
    out.backward(dy)
    want, tol = ref.embed_grad(ref.f64(dy.view(200, D)), ids.flatten().cpu().numpy(), V, scale, 5)
    ref.check(w.grad, want, tol)
    # against differences: embed is linear in w, so the step can be large
    d = randn((V, D), F32, 4)
    with torch.no_grad():
        diff = (lm.embedding(w + d, ids, scale, pad_id=5).double()
                - lm.embedding(w - d, ids, scale, pad_id=5).double()) / 2
    lhs, rhs = (diff * dy).sum(), (w.grad.double() * d).sum()
    # the sums w + d and w - d and the products round to float32
    mag = (dy.abs() * scale * (w.detach().abs().max() + d.abs().max())).sum()
    assert abs(float(lhs - rhs)) <= 8 * ref.U * float(mag)


def test_embedding_gradient_in_bfloat16():
    w = randn((30, 24), BF16, 1).requires_grad_()
    ids = dev(ids_of(100, 30, 2))
    st = status()
    out = lm.embedding(w, ids, 2.0, out_dtype=F32, status=st)
    dy = randn((100, 24), F32, 3)
    out.backward(dy)
    want, tol = ref.embed_grad(ref.f64(dy), ids.cpu().numpy(), 30, 2.0)
    ref.check(w.grad, want, tol)
    assert w.grad.dtype == BF16 and int(st.item()) == 0


def test_embedding_has_no_second_derivative():
    w = randn((30, 24), F32, 1).requires_grad_()
    dy = randn((10, 24), F32, 2).requires_grad_()
    (g,) = torch.autograd.grad(lm.embedding(w, dev(ids_of(10, 30, 3))), w, dy, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


# ---- logits -------------------------------------------------------------------------
def logits_case(B, V, lt, seed, prompt=40, made=12, bias=5, masks=3, stride=0):
    rng = np.random.default_rng(seed)
    x = randn((B, V), F32, seed).mul_(3).to(lt)
    prompts = [ids_of(rng.integers(0, prompt + 1), V, seed + 10 + b).tolist() for b in range(B)]
    gen_ids = np.minimum(rng.zipf(1.4, (B, made)) - 1, V - 1).astype(np.int32)
    lens = rng.integers(0, made + 1, B).astype(np.int32)
    biases = [{int(v): float(np.float32(rng.uniform(-5, 5)))
               for v in sorted(rng.choice(V, rng.integers(0, min(bias, V) + 1), replace=False))}
              for _ in range(B)]
    words = (V + 31) // 32
    mk = rng.integers(0, 2**32, (masks, words), dtype=np.uint64).astype(np.uint32)
    mk[0] = 0  # a mask that leaves nothing
    mrow = rng.integers(-1, masks, B).astype(np.int32)
    par = {k: rng.uniform(lo, hi, B).astype(np.float32)
           for k, lo, hi in (("repetition", 0.7, 1.6), ("frequency", -0.5, 1.0), ("presence", -0.5, 1.0))}
    off = np.concatenate([[0], np.cumsum([len(p) for p in prompts])]).astype(np.int64)
    boff = np.concatenate([[0], np.cumsum([len(p) for p in biases])]).astype(np.int64)
    args = dict(
        prompt_ids=dev(np.array(sum(prompts, []), np.int32)), prompt_off=dev(off),
        out_ids=dev(gen_ids), out_len=dev(lens), bias_off=dev(boff),
        bias_ids=dev(np.array([v for b in biases for v in b], np.int32)),
        bias_values=dev(np.array([w for b in biases for w in b.values()], np.float32)),
        mask=dev(mk.view(np.int32)), mask_row=dev(mrow), **{k: dev(v) for k, v in par.items()})
    want, tol = ref.process_logits(
        ref.f64(x), prompts, [g[:n].tolist() for g, n in zip(gen_ids, lens)], par["repetition"],
        par["frequency"], par["presence"], biases, mk, mrow)
    return x, args, want, tol


@pytest.mark.parametrize("lt,ot", [(BF16, F32), (BF16, BF16), (F32, F32), (F16, F32), (F16, F16)])
@pytest.mark.parametrize("B,V", [(1, 1), (2, 3), (3, 33), (5, 768), (2, 4095), (2, 4096), (9, 4097),
                                 (3, 32256), (2, 50001)])
def test_logits(B, V, lt, ot):
    x, args, want, tol = logits_case(B, V, lt, B + V)
    st = status()
    got = lm.process_logits(x, out_dtype=ot, status=st, **args)
    ref.check(got, want, tol, "logits")
    assert int(st.item()) == 0


@pytest.mark.parametrize("V", [100, 9001])
def test_logits_in_place_and_strided(V):
    x, args, want, tol = logits_case(6, V, BF16, V)
    y = strided(x, 3)
    args["out_ids"] = strided(args["out_ids"], 5)
    args["mask"] = strided(args["mask"], 2)
    got = lm.process_logits(y, out=y, **args)
    assert got is y
    ref.check(got, want, tol)
    assert torch.all(gaps(y, 3) == 0)


def test_logits_long_history():
    for lt, V in ((F32, 20000), (BF16, 8192), (BF16, 24577)):
        x, args, want, tol = logits_case(3, V, lt, 5, prompt=30000, made=5000, bias=300)
        ref.check(lm.process_logits(x, **args), want, tol)


@pytest.mark.parametrize("bias", [512, 513, 900, 4000])
def test_logits_many_biases(bias):
    x, args, want, tol = logits_case(4, 9000, F32, bias, bias=bias)
    ref.check(lm.process_logits(x, **args), want, tol)
    # and every one of the row's first IDs biased
    n = min(bias, 9000)
    off = torch.arange(5, device=device()) * n
    ids = torch.arange(n, dtype=torch.int32, device=device()).repeat(4)
    val = randn((4 * n,), F32, bias)
    got = lm.process_logits(x, bias_off=off, bias_ids=ids, bias_values=val)
    want = x.clone()
    want[:, :n] += val.view(4, n)
    assert torch.equal(got, want)


@pytest.mark.parametrize("keep", [(), ("prompt_ids", "prompt_off", "repetition"),
                                  ("out_ids", "out_len", "frequency"), ("out_ids", "out_len", "presence"),
                                  ("bias_off", "bias_ids", "bias_values"), ("mask", "mask_row")])
def test_logits_groups_left_out(keep):
    V = 5000
    x, args, _, _ = logits_case(4, V, F32, 8)
    use = {k: v for k, v in args.items() if k in keep}
    got = lm.process_logits(x, **use)
    h = {k: v.cpu().numpy() for k, v in args.items()}
    cut = lambda ids, off: [ids[off[b]:off[b + 1]].tolist() for b in range(4)]  # noqa: E731
    want, tol = ref.process_logits(
        ref.f64(x), cut(h["prompt_ids"], h["prompt_off"]) if "prompt_ids" in keep else None,
        [h["out_ids"][b, :h["out_len"][b]].tolist() for b in range(4)] if "out_ids" in keep else None,
        h["repetition"] if "repetition" in keep else None, h["frequency"] if "frequency" in keep else None,
        h["presence"] if "presence" in keep else None,
        [dict(zip(i, v)) for i, v in zip(cut(h["bias_ids"], h["bias_off"]), cut(h["bias_values"], h["bias_off"]))]
        if "bias_ids" in keep else None,
        h["mask"].view(np.uint32) if "mask" in keep else None, h["mask_row"] if "mask" in keep else None)
    ref.check(got, want, tol)
    if not keep:
        assert torch.equal(got, x)


def test_logits_infinities_and_nan():
    V = 64
    x = torch.zeros((3, V), device=device())
    x[:, 0], x[:, 1], x[:, 2] = float("inf"), -float("inf"), float("nan")
    x[:, 3] = torch.finfo(F32).min
    hist = dev(np.tile(np.arange(4, dtype=np.int32), (3, 1)))
    mask = torch.tensor([[-1, -1], [0, 0]], dtype=torch.int32, device=device())
    got = lm.process_logits(
        x, out_ids=hist, out_len=dev(np.array([4, 4, 4], np.int32)),
        repetition=torch.full((3,), 2.0, device=device()), presence=torch.ones(3, device=device()),
        mask=mask, mask_row=dev(np.array([0, 1, -1], np.int32))).cpu()
    for b in (0, 2):
        assert got[b, 0] == float("inf") and got[b, 1] == -float("inf") and torch.isnan(got[b, 2])
        assert got[b, 3] == -float("inf") and torch.all(got[b, 4:] == 0)
    assert torch.all(got[1] == -float("inf"))  # a row that the mask empties, NaN and all


def test_logits_status_bits():
    V = 9000
    x, args, _, _ = logits_case(3, V, F32, 11, masks=2)

    def bits(**kw):
        st = status()
        got = lm.process_logits(x, status=st, **{**args, **kw})
        assert got.shape == x.shape
        return int(st.item())

    def with_(t, at, v):
        t = t.clone()
        t[at] = v
        return t

    assert bits() == 0
    big = args["prompt_ids"].numel() + 1
    assert bits(prompt_off=with_(args["prompt_off"], 3, big)) == _lib.STATUS_BAD_ID_OFFSETS
    assert bits(prompt_off=with_(args["prompt_off"], 0, -1)) == _lib.STATUS_BAD_ID_OFFSETS
    assert bits(bias_off=with_(args["bias_off"], 1, 10**12)) == _lib.STATUS_BAD_ID_OFFSETS
    assert bits(out_len=with_(args["out_len"], 1, 13)) == _lib.STATUS_BAD_LENGTH
    assert bits(out_len=with_(args["out_len"], 1, -1)) == _lib.STATUS_BAD_LENGTH
    assert bits(mask_row=with_(args["mask_row"], 1, 2)) == _lib.STATUS_BAD_MASK_ROW
    assert bits(mask_row=with_(args["mask_row"], 1, -2)) == _lib.STATUS_BAD_MASK_ROW
    off, ids, val = (dev(np.array(a, t)) for a, t in (([0, 2, 2, 2], np.int64), ([8, 8], np.int32),
                                                      ([1, 2], np.float32)))
    assert bits(bias_off=off, bias_ids=ids, bias_values=val) == _lib.STATUS_BAD_BIAS
    for v in (-1, V, 2**31 - 1, -2**31):
        st = status()
        hist = dev(np.array([[4, v], [4, 4], [v, 4]], np.int32))
        got = lm.process_logits(x, out_ids=hist, out_len=dev(np.array([2, 2, 2], np.int32)),
                                frequency=args["frequency"], status=st)
        want, tol = ref.process_logits(ref.f64(x), made=hist.cpu().tolist(), freq=ref.f64(args["frequency"]))
        ref.check(got, want, tol)
        assert int(st.item()) == _lib.STATUS_BAD_ID


def test_logits_rows_of_nothing():
    x = torch.zeros((0, 50), device=device())
    assert lm.process_logits(x).shape == (0, 50)
    x = torch.ones((2, 40), device=device())
    none = torch.zeros(0, dtype=torch.int32, device=device())
    off = torch.zeros(3, dtype=torch.int64, device=device())
    got = lm.process_logits(x, prompt_ids=none, prompt_off=off, out_ids=none.view(2, 0),
                            out_len=torch.zeros(2, dtype=torch.int32, device=device()), bias_off=off,
                            bias_ids=none, bias_values=none.float(),
                            repetition=torch.full((2,), 9.0, device=device()))
    assert torch.equal(got, x)


def test_logits_past_32_bits():
    # rows whose offsets pass 2^31 elements
    B, V = 40, 60_000_000
    x = torch.zeros((B, V), dtype=BF16, device=device())
    hist = dev(np.full((B, 1), V - 1, np.int32))
    x[:, V - 1] = 4.0
    got = lm.process_logits(x, out=x, out_ids=hist, out_len=torch.ones(B, dtype=torch.int32, device=device()),
                            repetition=torch.full((B,), 2.0, device=device()))
    assert torch.all(got[:, V - 1] == 2.0) and torch.all(got[-1, :V - 1] == 0)


# ---- block tables -----------------------------------------------------------------
def blocks_case(R, bs, seed, most=100, cached=200, empty=0.2, first_block=0):
    rng = np.random.default_rng(seed)
    new = rng.integers(0, most + 1, R) * (rng.random(R) >= empty)
    c = rng.integers(0, cached + 1, R) * (rng.random(R) < 0.7)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
    have, want = -(-c // bs), -(-(c + new) // bs)
    W = int(want.max(initial=0)) + 2
    pool = (rng.permutation(int(have.sum() + (want - have).sum()) + 7) + first_block).astype(np.int32)
    table = np.full((R, W), -1, np.int32)
    at = 0
    for r in range(R):
        table[r, :have[r]] = pool[at:at + have[r]]
        at += have[r]
    return off, c.astype(np.int32), pool[at:].copy(), table


def check_blocks(off, c, free, table, bs, t=None, st=None, want=None):
    t = dev(table) if t is None else t
    s = status() if st is None else st
    slots, pos, lens, used = lm.block_tables(dev(off), int(off[-1]), dev(c), dev(free), t, bs, status=s)
    wt, ws, wp, wl, wu = ref.block_tables(off, c, free, table, bs) if want is None else want
    assert np.array_equal(t.cpu().numpy(), wt)
    assert np.array_equal(slots.cpu().numpy(), ws)
    assert np.array_equal(pos.cpu().numpy(), wp)
    assert np.array_equal(lens.cpu().numpy(), wl)
    assert used.tolist() == [wu]
    return int(s.item())


@pytest.mark.parametrize("bs", [1, 7, 16, 48, 64, 1000])
@pytest.mark.parametrize("R", [1, 2, 63, 300, 2048, 2049, 5000])
def test_blocks(R, bs):
    assert check_blocks(*blocks_case(R, bs, R + bs), bs) == 0


@pytest.mark.parametrize("R,most,cached,empty", [(256, 1, 4000, 0.0), (3, 9000, 0, 0.0), (3000, 3, 5, 0.9),
                                                 (70000, 1, 30, 0.5), (300000, 2, 3, 0.5), (5, 0, 50, 0.0),
                                                 (4000, 0, 50, 0.0)])
def test_blocks_lengths(R, most, cached, empty):
    assert check_blocks(*blocks_case(R, 16, R, most, cached, empty), 16) == 0


def test_blocks_large_numbers():
    # slots past 2^32
    off, c, free, table = blocks_case(40, 16, 3, first_block=2**31 - 9000)
    assert check_blocks(off, c, free, table, 16) == 0
    # positions near 2^31, blocks of 2^20 - 3 tokens, a strided table
    bs = (1 << 20) - 3
    c = np.array([2**31 - 60, 2**30, 0], np.int32)
    off = np.array([0, 50, 120, 125], np.int64)
    have = -(-c.astype(np.int64) // bs)
    table = np.zeros((3, int(have.max()) + 2), np.int32)
    table[:] = np.arange(table.size).reshape(table.shape)
    free = np.array([70000, 70001, 70002], np.int32)
    assert check_blocks(off, c, free, table, bs, t=strided(dev(table), 3)) == 0


@pytest.mark.parametrize("R", [50, 3000])
def test_blocks_run_out(R):
    bs = 16
    off, c, free, table = blocks_case(R, bs, 9)
    free = free[: len(free) // 3]
    assert check_blocks(off, c, free, table, bs) == _lib.STATUS_NO_BLOCKS
    assert check_blocks(off, c, free[:0], table, bs) == _lib.STATUS_NO_BLOCKS
    off, c, free, table = blocks_case(R, bs, 10, most=100, cached=0)
    table = table[:, :3].copy()
    assert check_blocks(off, c, free, table, bs) == _lib.STATUS_TABLE_FULL


@pytest.mark.parametrize("R", [6, 2500])
def test_blocks_bad_lengths_and_offsets(R):
    bs = 16
    off, c, free, table = blocks_case(R, bs, 4, cached=0, empty=0.0)
    bad = c.copy()
    bad[2] = -5
    want = ref.block_tables(off, c, free, table, bs)
    assert check_blocks(off, bad, free, table, bs, want=want) == _lib.STATUS_BAD_LENGTH
    # a length past 2^31 - 1
    long = c.copy()
    long[1] = 2**31 - 2
    st = status()
    slots, pos, lens, _ = lm.block_tables(dev(off), int(off[-1]), dev(long), dev(free), dev(table), bs, status=st)
    assert int(st.item()) & _lib.STATUS_BAD_LENGTH
    assert int(lens[1]) == 2**31 - 1 and int(pos[int(off[1])]) == 2**31 - 2
    assert torch.all(pos[int(off[1]) + 2:int(off[2])] == -1)
    # offsets that are not valid: the bit, and nothing out of bounds (guards around every output)
    T = int(off[-1])
    for at, v in ((0, 3), (R, T - 1), (R, T + 5), (3, -7), (2, 10**15), (R // 2, -10**15), (1, 2**63 - 1), (R - 1, -2**63)):
        o = off.copy()
        o[at] = v
        guard = 64
        slots = torch.full((T + 2 * guard,), -7, dtype=torch.int64, device=device())
        pos = torch.full((T + 2 * guard,), -7, dtype=torch.int32, device=device())
        lens = torch.full((R + 2 * guard,), -7, dtype=torch.int32, device=device())
        tab = torch.full((R + 2, table.shape[1]), -7, dtype=torch.int32, device=device())
        tab[1:-1] = dev(table)
        st = status()
        lm.block_tables(dev(o), T, dev(c), dev(free), tab[1:-1], bs, slots=slots[guard:-guard],
                        positions=pos[guard:-guard], lengths=lens[guard:-guard], status=st)
        assert int(st.item()) & _lib.STATUS_BAD_ID_OFFSETS, (at, v)
        for t in (slots, pos, lens):
            assert torch.all(t[:guard] == -7) and torch.all(t[-guard:] == -7)
        assert torch.all(tab[0] == -7) and torch.all(tab[-1] == -7)


def test_blocks_of_nothing():
    z = lambda n, t: torch.zeros(n, dtype=t, device=device())  # noqa: E731
    slots, pos, lens, used = lm.block_tables(z(1, torch.int64), 0, z(0, torch.int32), z(3, torch.int32),
                                             z((0, 4), torch.int32), 16)
    assert slots.numel() == pos.numel() == lens.numel() == 0 and used.tolist() == [0]
    c = dev(np.array([5, 0], np.int32))
    slots, pos, lens, used = lm.block_tables(z(3, torch.int64), 0, c, z(3, torch.int32),
                                             z((2, 4), torch.int32), 16)
    assert lens.tolist() == [5, 0] and used.tolist() == [0]


def test_blocks_raise_without_a_status():
    off, c, free, table = blocks_case(50, 16, 9)
    with pytest.raises(RuntimeError, match="status 0x20"):
        lm.block_tables(dev(off), int(off[-1]), dev(c), dev(free[:1]), dev(table), 16)


# ---- streams, graphs ----------------------------------------------------------------
def all_four(w, ids, g, x, args, off, c, free, table, T, st, stream=None):
    return (lm.embed(w, ids, 2.0, status=st, stream=stream),
            lm.embed_grad(g, ids, w.shape[0], status=st, stream=stream),
            lm.process_logits(x, status=st, stream=stream, **args),
            *lm.block_tables(off, T, c, free, table, 16, status=st, stream=stream))


def four_inputs():
    V, D, n = 900, 136, 5000
    x, args, _, _ = logits_case(4, 5000, BF16, 1)
    off, c, free, table = blocks_case(2500, 16, 5)
    return (randn((V, D), BF16, 1), dev(ids_of(n, V, 2)), randn((n, D), BF16, 3), x, args, dev(off),
            dev(c), dev(free), dev(table), int(off[-1]))


def test_another_stream():
    inputs = four_inputs()
    want = all_four(*inputs, status())
    side = torch.cuda.Stream()
    st = status()
    torch.cuda.synchronize()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        got = all_four(*inputs, st, stream=side)
        # memory that the calls gave back is not handed out under them
        noise = [torch.full((1 << 20,), 77, dtype=torch.int32, device=device()) for _ in range(8)]
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del noise
    assert int(st.item()) == 0


def test_graph_replays():
    w, ids, g, x, args, off, c, free, table, T = four_inputs()
    st = status()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        all_four(w, ids, g, x, args, off, c, free, table, T, st)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_four(w, ids, g, x, args, off, c, free, table, T, st)
    for k in range(4):
        ids.copy_(dev(ids_of(ids.numel(), w.shape[0], 20 + k, ("zipf", "one", "distinct", "zipf")[k])))
        g.copy_(randn(tuple(g.shape), BF16, 30 + k))
        x.copy_(randn(tuple(x.shape), BF16, 40 + k))
        free.copy_(free.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        entered = table.clone()
        want = all_four(w, ids, g, x, args, off, c, free, table, T, st)
        assert torch.equal(entered, table)
        for a, b in zip(got, want):
            assert torch.equal(a, b), k
    assert int(st.item()) == 0


def test_refusals_on_the_device():
    w = randn((10, 16), F32, 1)
    ids = dev(np.zeros(3, np.int32))
    with pytest.raises(ValueError, match="current device"):
        lm.embed(w, ids.cpu())
    with pytest.raises(TypeError, match="status"):
        lm.embed(w, ids, status=torch.zeros(1, dtype=torch.int64, device=device()))
    with pytest.raises(BPEError):
        lm.embed_grad(randn((3000, 16), F32, 1), torch.zeros(3000, dtype=torch.int32, device=device()),
                      10, workspace=torch.zeros(8, device=device()))
