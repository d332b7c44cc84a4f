"""The operators on token IDs on the GPU at the edges of their kernels' variants:
column slabs with few lanes in use, queues that overflow, wide workgroups, batches
past the caches, inputs that die under a call.  Bounds as in test_gpu_lm.py."""
import numpy as np
import pytest
import torch

import lm_reference as ref
from byte_level_bpe_pretokenize_amd import BPEError, _lib, lm

from gpu_util import device
from test_gpu_lm import (BF16, F16, F32, blocks_case, check_blocks, dev, gaps, gen, ids_of, randn,
                         status, strided)

pytestmark = pytest.mark.gpu


# ---- embed by sorted IDs -------------------------------------------------------
@pytest.mark.parametrize("D", [8, 9, 513, 520, 1015])
def test_embed_by_sorted_ids_few_lanes(D):
    """The last slab of 512 columns has 1, 2 or most lanes in use; the positions
    that the wave stores to are held by all 64."""
    n, V, ot = (512 << 20) // (2 * D) + 77, 700, BF16
    assert lm.embed_workspace_bytes(n, V, D, F32, ot) > 0
    w = randn((V, D), F32, D)
    ids = (torch.rand(n, device=device(), generator=gen(D)) ** 3 * V).to(torch.int32)
    out = strided(torch.full((n, D), 7.0, dtype=ot, device=device()), 3)
    st = status()
    lm.embed(w, ids, 0.5, out=out, status=st)
    assert int(st.item()) == 0
    # a power of two: the plain product rounds the same
    step = 1 << 20
    for a in range(0, n, step):
        want = (w * 0.5).to(ot)[ids[a:a + step].long()]
        assert torch.equal(out[a:a + step], want), (D, a)
    assert torch.all(gaps(out, 3) == 0)


def test_embed_of_the_most_rows():
    """More than 2^33 pieces of four elements (an output of 71 GB), and workgroups
    past 2^22."""
    n, D, V = 953_000_001, 37, 1000
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB")
    w = randn((V, D), BF16, 1)
    ids = torch.arange(n, dtype=torch.int32, device=device()) % V
    st = status()
    got = lm.embed(w, ids, 0.5, status=st)
    want = (w.float() * 0.5).to(BF16)
    whole = n // V
    for a in range(0, whole, 20000):
        b = min(whole, a + 20000)
        assert bool((got[a * V:b * V].view(b - a, V, D) == want).all()), a
    assert torch.equal(got[whole * V:], want[:n - whole * V]) and int(st.item()) == 0


# ---- the gradient by sorted IDs, float32 to half precision ------------------------
@pytest.mark.parametrize("ot", [BF16, F16])
@pytest.mark.parametrize("n,V,D", [(2049, 90, 7), (3001, 1500, 72), (6144, 300, 513), (6145, 300, 520),
                                   (40000, 2000, 1001)])
def test_embed_grad_narrows(n, V, D, ot):
    g = randn((n, D), F32, n)
    ids = ids_of(n, V, n)
    ids[5], ids[n - 1] = -1, V
    st = status()
    got = lm.embed_grad(g, dev(ids), V, 0.3, out_dtype=ot, status=st)
    want, tol = ref.embed_grad(ref.f64(g), ids, V, float(np.float32(0.3)))
    ref.check(got, want, tol, "embed_grad")
    first = randn((V, D), ot, 9)
    out = first.clone()
    lm.embed_grad(g, dev(ids), V, 0.3, out=out, accumulate=True, status=st)
    base = ref.f64(first)
    ref.check(out, base + want, tol + ref.U * (np.abs(base) + np.abs(want)), "accumulate")


@pytest.mark.parametrize("n", [2049, 5000, 9000])
def test_embedding_of_a_bfloat16_table_to_float32(n):
    w = randn((70, 264), BF16, 1).requires_grad_()
    ids = ids_of(n, 70, 2)
    dy = randn((n, 264), F32, 3)
    st = status()
    lm.embedding(w, dev(ids), 2.0, out_dtype=F32, status=st).backward(dy)
    want, tol = ref.embed_grad(ref.f64(dy), ids, 70, 2.0)
    assert w.grad.dtype == BF16 and int(st.item()) == 0
    ref.check(w.grad, want, tol)


def test_embed_grad_of_the_most_ids():
    """2^30 IDs (a gradient of 17 GB): whole numbers whose sums are exact."""
    n, V, D, rows = 1 << 30, 1 << 16, 8, 1 << 14
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    ids = torch.arange(V, dtype=torch.int32, device=device()).repeat(rows)
    # position t = (j, v): (v + j) % 5 - 1, and the column
    j = torch.arange(rows, device=device(), dtype=torch.int32)[:, None]
    v = torch.arange(V, device=device(), dtype=torch.int32)
    g = torch.empty((n, D), dtype=BF16, device=device())
    want = torch.zeros((V, D), device=device())
    for a in range(0, rows, 1024):
        x = ((v + j[a:a + 1024]) % 5 - 1).to(BF16)[:, :, None] * torch.arange(1, D + 1, device=device()).to(BF16)
        g.view(rows, V, D)[a:a + 1024] = x
        want += x.float().sum(0)
    st = status()
    got = lm.embed_grad(g, ids, V, status=st)
    assert torch.equal(got, want) and int(st.item()) == 0


# ---- logits: queues that overflow, wide workgroups with a queue ----------------------
def check_logits(V, lists, lt, ot, seed):
    """lists: for each row its prompt, its generated IDs and how many biases."""
    rng = np.random.default_rng(seed)
    B = len(lists)
    x = randn((B, V), lt, seed).mul_(3)
    prompts, made = [np.asarray(r[0]) for r in lists], [np.asarray(r[1]) for r in lists]
    out_ids = np.zeros((B, max(len(m) for m in made)), np.int32)
    for b, m in enumerate(made):
        out_ids[b, :len(m)] = m
    biases = [{int(v): float(np.float32(rng.uniform(-5, 5)))
               for v in np.sort(rng.choice(V, r[2], replace=False))} for r in lists]
    par = {k: rng.uniform(lo, hi, B).astype(np.float32)
           for k, lo, hi in (("repetition", 0.7, 1.6), ("frequency", -0.5, 1.0), ("presence", -0.5, 1.0))}
    mask = rng.integers(0, 2**32, (2, (V + 31) // 32), dtype=np.uint64).astype(np.uint32)
    row = np.arange(B, dtype=np.int32) % 3 - 1
    cat = lambda a, t: dev(np.concatenate(a).astype(t))  # noqa: E731
    off = lambda a: dev(np.concatenate([[0], np.cumsum([len(p) for p in a])]).astype(np.int64))  # noqa: E731
    st = status()
    got = lm.process_logits(
        x, prompt_ids=cat(prompts, np.int32), prompt_off=off(prompts), out_ids=dev(out_ids),
        out_len=dev(np.array([len(m) for m in made], np.int32)), bias_off=off(biases),
        bias_ids=cat([np.array(list(b), np.int64) for b in biases], np.int32),
        bias_values=cat([np.array(list(b.values())) for b in biases], np.float32),
        mask=dev(mask.view(np.int32)), mask_row=dev(row), out_dtype=ot, status=st,
        **{k: dev(v) for k, v in par.items()})
    want, tol = ref.process_logits(ref.f64(x), [p.tolist() for p in prompts], [m.tolist() for m in made],
                                   par["repetition"], par["frequency"], par["presence"], biases, mask, row)
    ref.check(got, want, tol, "logits")
    assert int(st.item()) == 0


def distinct(lo, hi, n, seed):
    return np.random.default_rng(seed).permutation(np.arange(lo, hi))[:n]


@pytest.mark.parametrize("lt,ot", [(F32, F32), (BF16, F32), (F16, F16)])
def test_logits_queue_overflows(lt, ot):
    """256 threads: lists that fit one step, with more distinct tokens in a slab
    than its queue has places (512); exactly 512; one more."""
    V = 9000
    check_logits(V, [(distinct(0, 4096, 1000, 1), distinct(0, 4096, 1000, 2), 200),
                     (distinct(4096, 8192, 1024, 3), [], 0),
                     (distinct(0, 4096, 512, 4), [], 0),
                     (distinct(0, 4096, 513, 5), distinct(8192, V, 600, 6), 256),
                     ([], distinct(4000, 4700, 700, 7), 3)], lt, ot, 8)


@pytest.mark.parametrize("lt,ot", [(F32, F32), (BF16, F32), (BF16, BF16)])
def test_logits_wide_workgroups(lt, ot):
    """1,024 threads, which the batch's average prompt chooses, on rows of every
    kind: short lists (a queue), more distinct tokens in a slab than its queue
    has places (1,024), up to 1,024 biases with a queue and more without."""
    V = 17000
    rng = np.random.default_rng(1)
    check_logits(V, [(rng.integers(0, V, 60000), [], 0),
                     (rng.integers(0, V, 5), rng.integers(0, V, 9), 4),
                     ([], [], 0),
                     (distinct(0, 8192, 3000, 2), distinct(0, 8192, 3000, 3), 10),
                     (distinct(0, 8192, 1024, 4), [], 0),
                     (distinct(8192, 16384, 1025, 5), distinct(16384, V, 600, 6), 5),
                     (rng.integers(0, V, 40), rng.integers(0, V, 50), 513),
                     (rng.integers(0, V, 40), [], 600),
                     ([], rng.integers(0, V, 4096), 1000),
                     (rng.integers(0, V, 4096), [], 1024),
                     (rng.integers(0, V, 7), [3, 3, 3], 1025),
                     (rng.integers(0, V, 4097), rng.integers(0, V, 4100), 700)], lt, ot, 9)


@pytest.mark.parametrize("lt,ot", [(F32, F32), (BF16, F32), (F32, BF16)])
def test_logits_wide_workgroups_past_the_caches(lt, ot):
    V = 2_000_003
    rng = np.random.default_rng(2)
    check_logits(V, [(rng.integers(0, V, 50000), rng.integers(0, V, 700), 30)] +
                 [(rng.integers(0, V, 20), rng.integers(0, V, 5000), 600)] * 8, lt, ot, 10)


@pytest.mark.parametrize("B", [(1 << 23) + 5, (1 << 24) - 1])
def test_logits_of_very_many_rows(B):
    """Up to the launch with the most workgroups: 2^24 - 1."""
    V = 3
    x = torch.randn((B, V), device=device(), generator=gen(1))
    made = torch.randint(0, V, (B, 1), dtype=torch.int32, device=device(), generator=gen(2))
    st = status()
    got = lm.process_logits(x, out_ids=made, out_len=torch.ones(B, dtype=torch.int32, device=device()),
                            presence=torch.full((B,), 0.5, device=device()), status=st)
    want = x - 0.5 * (torch.arange(V, device=device()) == made)
    assert torch.equal(got, want) and int(st.item()) == 0
    more = torch.zeros(((1 << 24), V), device=device())
    with pytest.raises(BPEError):
        lm.process_logits(more)


# ---- block tables past the caches ----------------------------------------------------
@pytest.mark.parametrize("R,most,bs", [(2048, 4000, 48), (30, 300_000, 16), (5000, 1600, 16), (2049, 4000, 1)])
def test_blocks_past_the_caches(R, most, bs):
    off, c, free, table = blocks_case(R, bs, R, most=most, cached=500)
    assert off[-1] * 12 >= 32 << 20
    assert check_blocks(off, c, free, table, bs) == 0


@pytest.mark.parametrize("R", [3, 3000])
def test_blocks_table_full_is_about_new_tokens(R):
    """A request of 100 cached tokens in a table of 3 blocks of 16: no bit without
    new tokens, and one with."""
    table = np.zeros((R, 3), np.int32)
    c, new = np.zeros(R, np.int32), np.ones(R, np.int64)
    c[1], new[1] = 100, 0
    off = np.concatenate([[0], np.cumsum(new)])
    free = np.arange(1, R + 1, dtype=np.int32)
    assert check_blocks(off, c, free, table, 16) == 0
    new[1] = 1
    off = np.concatenate([[0], np.cumsum(new)])
    assert check_blocks(off, c, free, table, 16) == _lib.STATUS_TABLE_FULL


# ---- another stream -------------------------------------------------------------------
def test_another_stream_outlives_its_inputs():
    """The inputs' last references go right after the calls, while these still
    wait for earlier work of their stream; what is allocated then is not what
    they read."""
    V, D, n = 900, 136, 5000
    make = lambda k: (randn((V, D), F32, k), dev(ids_of(n, V, k)), randn((n, D), BF16, k),  # noqa: E731
                      randn((8, 5000), F32, k), dev(ids_of(8 * 64, 5000, k).reshape(8, 64)),
                      torch.full((8,), 64, dtype=torch.int32, device=device()),
                      torch.full((8,), 0.5, device=device()))

    def calls(t, st, stream=None):
        return (lm.embed(t[0], t[1], 2.0, status=st, stream=stream),
                lm.embed_grad(t[2], t[1], V, status=st, stream=stream),
                lm.process_logits(t[3], out_ids=t[4], out_len=t[5], frequency=t[6], status=st, stream=stream))

    want = calls(make(1), status())
    busy = torch.ones((4096, 4096), device=device())
    side, st = torch.cuda.Stream(), status()
    for _ in range(3):
        inputs = make(1)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(8):
                busy = busy @ busy * 2.0 ** -12
        got = calls(inputs, st, side)
        del inputs
        noise = [make(2) for _ in range(2)]
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del noise
    assert int(st.item()) == 0
