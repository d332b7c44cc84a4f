"""Verification of drafted tokens on the GPU: tokens and counts equal those of the
definition in 64 bits (lm_draft_reference.py)."""
import numpy as np
import pytest
import torch

import lm_draft_reference as ref
from lm_reference import f64
from byte_level_bpe_pretokenize_amd import BPEError, _lib, lm

from gpu_util import device
from test_gpu_lm import BF16, F16, F32, dev, gen, status, strided

pytestmark = pytest.mark.gpu


def batch(lengths, V, dtype, seed, with_draft=True, near=0.7):
    """Rows of requests with `lengths` drafts: p near q, drafts drawn from q."""
    off = np.concatenate([[0], np.cumsum(np.asarray(lengths) + 1)]).astype(np.int64)
    N = int(off[-1])
    g = gen(seed)
    z = torch.randn((N, V), device=device(), generator=g) * 2
    y = z + near * torch.randn((N, V), device=device(), generator=g)
    y[torch.rand((N, V), device=device(), generator=g) < 0.1] = -torch.inf
    y[:, V // 2] = z[:, V // 2]
    p, q = torch.softmax(y, 1).to(dtype), torch.softmax(z, 1).to(dtype)
    ids = torch.multinomial(q.float(), 1, generator=g).flatten().to(torch.int32) if with_draft \
        else p.argmax(1).to(torch.int32)
    accept = torch.rand(N, device=device(), generator=g)
    sample = torch.rand(len(lengths), device=device(), generator=g)
    return p, q if with_draft else None, ids, off, accept, sample


def check(p, q, ids, off, accept, sample, bits=0):
    st = status()
    tokens = torch.full((p.shape[0],), -9, dtype=torch.int32, device=device())
    got, counts = lm.verify_drafts(p, ids, dev(off) if isinstance(off, np.ndarray) else off, accept, sample, draft=q,
                                   tokens=tokens, status=st)
    assert got is tokens and int(st.item()) == bits
    want, n = ref.verify(f64(p), ids.cpu().numpy(), np.asarray(off), accept.cpu().numpy(), sample.cpu().numpy(),
                         None if q is None else f64(q))
    assert np.array_equal(counts.cpu().numpy(), n), (counts, n)
    assert np.array_equal(got.cpu().numpy(), want)
    return got, counts


@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V", [1, 2, 7, 64, 255, 1000, 4096, 8192, 8193, 16384, 50257, 65536, 65537, 128256])
def test_verify(V, dtype, with_draft):
    lengths = [0, 1, 5, 3, 0, 16, 2] if V < 100000 else [3, 0, 2]
    for seed in range(3 if V < 10000 else 1):
        check(*batch(lengths, V, dtype, V + seed, with_draft))


@pytest.mark.parametrize("near", [0.0, 0.05, 5.0])
def test_verify_near_and_far(near):
    """The same distribution (each draft stands), nearly, and another one."""
    p, q, *rest = batch([8] * 40, 300, F32, 3, near=near)
    _, counts = check(p if near else q.clone(), q, *rest)
    assert near or bool((counts == 9).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("R,V", [(700, 500), (256, 9000), (257, 8193), (300, 12000)])
def test_verify_many(R, V, dtype):
    check(*batch(list(np.random.default_rng(0).integers(0, 9 if V < 1000 else 2, R)), V, dtype, 5))


def test_verify_more_drafts_than_threads():
    p, q, ids, off, accept, sample = batch([3000, 0, 1024, 1025], 20, F32, 7)
    p = q.clone()
    _, counts = check(p, q, ids, off, accept, sample)
    assert counts.tolist() == [3001, 1, 1025, 1026]
    accept[1500] = accept[2500] = 2.0
    accept[3002 + 1023] = 2.0
    accept[3002 + 1025 + 1024] = 2.0
    _, counts = check(p, q, ids, off, accept, sample)
    assert counts.tolist() == [1501, 1, 1024, 1025]


@pytest.mark.parametrize("V", [5, 3000, 20000, 150000])
def test_borders(V):
    """Probabilities of a power of two, whose sums are exact: a share that ends at a
    token's border goes to the next token, and u q = p does not stand."""
    n = 1 << (V.bit_length() - 1)
    p = torch.zeros((2 * n.bit_length() + 3, V), device=device())
    p[:, :n] = 1.0 / n
    N = p.shape[0]
    off = np.arange(N + 1, dtype=np.int64)
    u = torch.tensor([k / n for k in [0, 1, 2, n // 2, n - 1] + [2 ** j for j in range(n.bit_length())]],
                     device=device())[:N]
    sample = torch.zeros(N, device=device())
    sample[:u.numel()] = u.clamp(max=1 - 2 ** -24)
    ids = torch.zeros(N, dtype=torch.int32, device=device())
    got, _ = check(p, None, ids, off, torch.zeros(N, device=device()), sample)
    for t, x in zip(got.tolist(), sample.tolist()):
        assert t == int(x * n)
    q = p.clone()
    two = np.arange(0, N - 1, 2, dtype=np.int64)
    off = np.concatenate([two, [two[-1] + 2]]) if two[-1] + 2 <= N else two
    accept = torch.full((N,), 0.5, device=device())
    q[:, 0] = 2.0 / n
    check(p, q, ids, off, accept, sample[:len(off) - 1].clone())
    _, counts = check(p, q, ids, off, accept - 2 ** -20, sample[:len(off) - 1].clone())
    assert (counts == 2).all()


def test_samples_outside():
    p = torch.tensor([[0.0, 0.25, 0.5, 0.0, 0.25, 0.0]] * 6, device=device())
    sample = torch.tensor([-1.0, 0.0, 1.0, float("nan"), float("inf"), -float("inf")], device=device())
    z = torch.zeros(6, device=device())
    got, _ = check(p, None, torch.zeros(6, dtype=torch.int32, device=device()), np.arange(7), z, sample)
    assert got.tolist() == [1, 1, 4, 4, 4, 1]


def test_accepts_outside():
    p, q, ids, off, accept, sample = batch([6] * 8, 300, F32, 4)
    for x, n in ((-1.0, 7), (float("nan"), 1), (float("inf"), 1), (-float("inf"), 7)):
        accept[:] = x
        q[:, 5] += 1e-6  # (no draft's probability is 0)
        _, counts = check(p, q, ids, off, accept, sample)
        assert counts.tolist() == [n] * 8


@pytest.mark.parametrize("V", [4000, 70000])
def test_what_is_no_probability(V):
    """Negative entries, infinities and NaN count as 0; nothing left of the difference
    goes to the target's row; nothing at all gives no token."""
    p = torch.rand((12, V), device=device(), generator=gen(1))
    q = torch.rand((12, V), device=device(), generator=gen(2))
    for t in (p, q):
        t[:, ::5] = float("nan")
        t[:, 1::7] = float("inf")
        t[:, 2::9] = -1.0
        t[:, 3::11] = -float("inf")
    p[5] = q[5]      # rejected, and nothing is left
    p[6] = 0.0       # rejected: nothing at all
    p[11] = float("nan")
    ids = torch.full((12,), 4, dtype=torch.int32, device=device())
    ids[5] = 3999
    accept = torch.zeros(12, device=device())
    accept[5] = 1.0
    sample = torch.rand(4, device=device(), generator=gen(3))
    off = np.array([0, 3, 7, 9, 12], np.int64)
    check(p, q, ids, off, accept, sample, _lib.STATUS_NO_TOKEN)  # (the last request's row)
    off = np.array([0, 3, 6, 8, 12], np.int64)
    check(p, q, ids, off, accept, sample, _lib.STATUS_NO_TOKEN)
    off = np.array([0, 1, 6, 7, 9], np.int64)
    check(p, q, ids, off, accept, sample, _lib.STATUS_NO_TOKEN)


def test_bad_ids_and_offsets():
    p, q, ids, off, accept, sample = batch([4, 4, 4], 100, F32, 1)
    p = q.clone()
    ids[off[1] - 1] = -5      # a last row's is not looked at
    ids[off[1] + 2] = 100
    ids[off[2] + 1], ids[off[2] + 3] = -1, 2 ** 31 - 1
    check(p, q, ids, off, accept, sample, _lib.STATUS_BAD_ID)
    accept[off[2]] = 2.0      # rejected before the bad one comes to be looked at
    ids[off[1] + 2] = 1
    accept[off[1]] = 2.0
    check(p, q, ids, off, accept, sample)
    check(p, None, ids, off, accept, sample)
    tokens = torch.full((15,), -9, dtype=torch.int32, device=device())
    for bad, fine in (([0, 5, 3, 15], (0,)), ([0, 5, 10, 16], (0, 1)), ([-1, 5, 10, 15], (1, 2)),
                      ([2 ** 62, -2 ** 62, 10, 15], (2,))):
        st = status()
        got, counts = lm.verify_drafts(p, ids, dev(np.array(bad, np.int64)), accept, sample, draft=q, status=st,
                                       tokens=tokens.fill_(-9))
        # (the bad IDs are looked at where the offsets make them drafts)
        assert int(st.item()) & ~_lib.STATUS_BAD_ID == _lib.STATUS_BAD_ID_OFFSETS
        for r in range(3):
            if r not in fine and not 0 <= bad[r] <= bad[r + 1] <= 15:
                assert int(counts[r]) == 0
    with pytest.raises(RuntimeError, match="status 0x10"):
        lm.verify_drafts(p, ids, dev(np.array([0, 5, 10, 16])), accept, sample)


def test_requests_without_rows():
    p, q, ids, off, accept, sample = batch([2, 0, 3], 60, BF16, 1)
    off = np.array([2, 2, 5, 5, 6, 6, 8, 8], np.int64)
    check(p[:9] if p.shape[0] > 9 else p, q, ids, off, accept, torch.rand(7, device=device(), generator=gen(1)))
    got, counts = lm.verify_drafts(p[:0], ids[:0], dev(np.zeros(4, np.int64)), accept[:0], torch.zeros(3, device=device()))
    assert counts.tolist() == [0, 0, 0] and got.numel() == 0
    got, counts = lm.verify_drafts(p, ids, dev(np.zeros(1, np.int64)), accept, sample[:0])
    assert counts.numel() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides(dtype):
    p, q, ids, off, accept, sample = batch([4, 1, 0, 7], 1001, dtype, 2)
    check(strided(p, 3), strided(q, 8), ids, off, accept, sample)
    check(strided(p, 5), None, ids, off, accept, sample)


def test_a_last_row_of_the_draft_is_not_read():
    p, q, ids, off, accept, sample = batch([4, 1, 0, 7], 800, F32, 2)
    want = check(p, q, ids, off, accept, sample)
    q[off[1:] - 1] = float("nan")
    ids[off[1:] - 1] = -77
    got = lm.verify_drafts(p, ids, dev(off), accept, sample, draft=q)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_large_vocabulary():
    V = (1 << 26) - 3
    p = torch.rand((2, V), device=device(), generator=gen(1))
    q = torch.rand((2, V), device=device(), generator=gen(2))
    ids = torch.tensor([V - 1, 0], dtype=torch.int32, device=device())
    for u in (0.0, 0.3, 0.999999):
        got, counts = lm.verify_drafts(p, ids, dev(np.array([0, 2])), torch.full((2,), 1e9, device=device()),
                                       torch.tensor([u], device=device()), draft=q)
        run = torch.cumsum((p[0].double() - q[0].double()).clamp(min=0), 0)
        want = int((run <= float(np.float32(u)) * run[-1]).sum())
        assert counts.tolist() == [1] and got.tolist() == [want, -1]


@pytest.mark.parametrize("V", [900, 70000])
@pytest.mark.parametrize("with_draft", [True, False])
def test_in_place(V, with_draft):
    p, q, ids, off, accept, sample = batch([4, 1, 0, 70, 7] * 3, V, F32 if V < 1000 else BF16, 2, with_draft)
    want = lm.verify_drafts(p, ids, dev(off), accept, sample, draft=q)
    got = lm.verify_drafts(p, ids, dev(off), accept, sample, draft=q, tokens=ids)
    assert got[0] is ids and torch.equal(ids, want[0]) and torch.equal(got[1], want[1])


def test_inference_tensors_are_taken():
    with torch.inference_mode():
        p, q, ids, off, accept, sample = batch([4, 1], 100, F32, 2)
        lm.verify_drafts(p, ids, dev(off), accept, sample, draft=q, tokens=ids)


def test_a_workspace_of_ones_own():
    p, q, ids, off, accept, sample = batch([4, 1, 0, 7], 70000, BF16, 2)
    want = lm.verify_drafts(p, ids, dev(off), accept, sample, draft=q)
    need = lm.verify_drafts_workspace_bytes(4, 70000)
    ws = torch.full((need + 8,), 77, dtype=torch.uint8, device=device())
    got = lm.verify_drafts(p, ids, dev(off), accept, sample, draft=q, workspace=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and bool((ws[need:] == 77).all())
    with pytest.raises(BPEError):
        lm.verify_drafts(p, ids, dev(off), accept, sample, draft=q, workspace=ws[:need - 1])


def test_the_distribution():
    """What comes out first is distributed as the target: 200,000 draws, each
    frequency within five deviations."""
    n, V = 200_000, 8
    g = gen(5)
    p = torch.tensor([0.3, 0.05, 0.0, 0.2, 0.1, 0.25, 0.06, 0.04], device=device())
    q = torch.tensor([0.1, 0.2, 0.1, 0.2, 0.3, 0.02, 0.03, 0.05], device=device())
    ids = torch.multinomial(q, 2 * n, replacement=True, generator=g).to(torch.int32)
    got, _ = lm.verify_drafts(p.expand(2 * n, V).contiguous(), ids, torch.arange(n + 1, device=device()) * 2,
                              torch.rand(2 * n, device=device(), generator=g),
                              torch.rand(n, device=device(), generator=g), draft=q.expand(2 * n, V).contiguous())
    freq = torch.bincount(got.view(n, 2)[:, 0].long(), minlength=V).double() / n
    dev_ = torch.sqrt(p.double() * (1 - p.double()) / n)
    assert bool(((freq - p.double()).abs() <= 5 * dev_ + 1e-7).all())


def test_captured_and_replayed():
    V = 70000  # (a workspace)
    p, q, ids, off, accept, sample = batch([4, 1, 0, 7], V, F32, 2)
    t_off, st = dev(off), status()
    tokens = torch.zeros(p.shape[0], dtype=torch.int32, device=device())
    counts = torch.zeros(4, dtype=torch.int32, device=device())
    step = lambda: lm.verify_drafts(p, ids, t_off, accept, sample, draft=q, tokens=tokens, counts=counts,  # noqa: E731
                                    status=st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        for t, x in zip((p, q, ids), batch([4, 1, 0, 7], V, F32, 10 + k)):
            t.copy_(x)
        accept.uniform_(generator=gen(k))
        sample.uniform_(generator=gen(k + 9))
        tokens.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        want, n = ref.verify(f64(p), ids.cpu().numpy(), off, accept.cpu().numpy(), sample.cpu().numpy(), f64(q))
        assert np.array_equal(tokens.cpu().numpy(), want) and np.array_equal(counts.cpu().numpy(), n)
    assert int(st.item()) == 0


@pytest.mark.parametrize("V", [9000, 70000])
def test_two_streams_at_once(V):
    args = [batch([4, 1, 0, 7], V, F32, k) for k in range(2)]
    offs = [dev(a[3]) for a in args]
    want = [lm.verify_drafts(a[0], a[2], o, a[4], a[5], draft=a[1]) for a, o in zip(args, offs)]
    streams, st = [torch.cuda.Stream() for _ in range(2)], status()
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for k, (a, o, s) in enumerate(zip(args, offs, streams)):
            got[k].append(lm.verify_drafts(a[0], a[2], o, a[4], a[5], draft=a[1], status=st, stream=s))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(x, want[k][0]) and torch.equal(n, want[k][1]) for x, n in got[k])
    assert int(st.item()) == 0


def test_another_stream():
    p, q, ids, off, accept, sample = batch([4, 1, 0, 7], 70000, F32, 2)
    want = lm.verify_drafts(p, ids, dev(off), accept, sample, draft=q)
    side, st = torch.cuda.Stream(), status()
    busy = torch.ones((4096, 4096), device=device())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(8):
            busy = busy @ busy * 2.0 ** -12
    t_off = dev(off)
    torch.cuda.synchronize()
    copies = [t.clone() for t in (p, q)]
    side.wait_stream(torch.cuda.current_stream())
    got = lm.verify_drafts(copies[0], ids, t_off, accept, sample, draft=copies[1], status=st, stream=side)
    del copies
    noise = [torch.full_like(p, 0.5) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and int(st.item()) == 0
    del noise
