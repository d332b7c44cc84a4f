"""A paged cache of few bits on the GPU: codes, scales and status bits equal those of
the definition's float32 steps (lm_draft_reference.py); held values within half a
step; read values within a float32 rounding and the output's."""
import numpy as np
import pytest
import torch

import lm_draft_reference as ref
from lm_reference import check, f64
from byte_level_bpe_pretokenize_amd import _lib, lm

from gpu_util import device
from test_gpu_lm import BF16, F16, F32, dev, gen, randn, status, strided

pytestmark = pytest.mark.gpu

KINDS = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8, "u4": torch.uint8}


def cache_of(n_slots, H, D, kind, group, seed=0):
    """A cache with something in it."""
    c, s, _ = lm.empty_cache(n_slots, H, D, KINDS[kind], group, device=device())
    raw = torch.randint(0, 127, c.shape, dtype=torch.uint8, device=device(), generator=gen(seed + 1))
    if kind == "u4" and D % 2:
        raw[..., -1] &= 15
    c.view(torch.uint8).copy_(raw)
    s.copy_(torch.rand(s.shape, device=device(), generator=gen(seed)) * 0.1)
    return c, s


def tokens_of(n, H, D, dtype, seed, layout="plain"):
    x = randn((n, H, D), dtype, seed)
    x[..., ::7] *= 5
    if layout == "wide":    # the last heads of a wider projection, off alignment
        big = torch.zeros(n * (2 * H + 1) * D + 1, dtype=dtype, device=device())[1:].view(n, 2 * H + 1, D)
        view = big[:, H:2 * H]
    elif layout == "heads":  # head by head
        view = torch.zeros(H, n, D, dtype=dtype, device=device()).transpose(0, 1)
    elif layout == "gaps":   # heads of a wider head
        view = torch.zeros(n, H, D + 3, dtype=dtype, device=device())[..., :D]
    else:
        return x
    return view.copy_(x)


def raw(codes):
    return codes.view(torch.uint8).cpu().numpy()


def check_write(x, slots, c, s, group, kind, D, bits=0, exact_in_64=True):
    """Writes x and compares the whole cache."""
    before_c, before_s = raw(c).copy(), s.cpu().numpy().copy()
    st = status()
    lm.cache_write(x, dev(slots), c, s, group, status=st)
    assert int(st.item()) == bits
    x32 = x.float().cpu().numpy()
    codes, scales, lows = ref.quantise(x32, group, kind)
    ok = (slots >= 0) & (slots < c.shape[0])
    want = ref.unpack(c, D) * 0
    want[slots[ok]] = codes[ok]
    got = ref.unpack(c, D)
    at = np.zeros(c.shape[0], bool)
    at[slots[ok]] = True
    assert np.array_equal(got[at], want[at])
    if kind == "u4" and D % 2:
        assert np.all(raw(c)[at][..., -1] < 16)
    ws = np.stack((scales, lows), -1) if kind == "u4" else scales
    got_s = s.cpu().numpy()
    assert np.array_equal(got_s[slots[ok]], ws[ok])
    # other slots keep what they hold
    assert np.array_equal(raw(c)[~at], before_c[~at]) and np.array_equal(got_s[~at], before_s[~at])
    if exact_in_64:
        v, _ = ref.values(got[slots[ok]], got_s[slots[ok]], group, kind == "u4")
        assert np.all(np.abs(v - x32[ok]) <= ref.quantise_error(x32[ok], group, kind))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("n,H,D,group", [(1, 1, 1, 16), (2, 3, 16, 16), (5, 2, 17, 16), (65, 2, 128, 128),
                                         (33, 8, 80, 32), (7, 10, 77, 64), (40, 16, 128, 64), (3, 1, 1000, 512),
                                         (9, 4, 520, 256), (300, 1, 8, 16), (2, 64, 256, 128), (4, 5, 33, 512)])
def test_write(n, H, D, group, dtype, kind):
    slots = np.random.default_rng(n).permutation(3 * n)[:n].astype(np.int64)
    c, s = cache_of(3 * n, H, D, kind, group)
    check_write(tokens_of(n, H, D, dtype, n), slots, c, s, group, kind, D)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout", ["wide", "heads", "gaps"])
@pytest.mark.parametrize("n,H,D,group", [(19, 6, 64, 32), (1, 4, 24, 32), (70, 1, 33, 16), (5, 3, 1, 16)])
def test_write_strides_and_slots(n, H, D, group, layout, kind):
    slots = np.random.default_rng(n).permutation(200)[:n].astype(np.int64)
    bits = 0
    if n > 4:
        slots[1], slots[2], slots[3], slots[4] = -1, 200, -2, 2 ** 62
        bits = _lib.STATUS_BAD_SLOT
    c, s = cache_of(200, H, D, kind, group)
    check_write(tokens_of(n, H, D, BF16, n, layout), slots, c, s, group, kind, D, bits)


@pytest.mark.parametrize("kind", KINDS)
def test_write_into_a_strided_cache(kind):
    """One layer of a cache that holds several side by side."""
    n, H, D, group = 21, 4, 48, 16
    codes = [cache_of(30, H, D, kind, group, k) for k in range(3)]
    allc = torch.stack([c.view(torch.uint8) for c, _ in codes], 1)
    alls = torch.stack([s for _, s in codes], 1)
    c, s = allc[:, 1].view(KINDS[kind]), alls[:, 1]
    slots = np.random.default_rng(1).permutation(30)[:n].astype(np.int64)
    check_write(tokens_of(n, H, D, F16, 3), slots, c, s, group, kind, D)
    for k in (0, 2):
        assert torch.equal(allc[:, k], codes[k][0].view(torch.uint8)) and torch.equal(alls[:, k], codes[k][1])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_write_what_is_not_finite(dtype, kind):
    n, H, D, group = 24, 2, 50, 16
    x = tokens_of(n, H, D, dtype, 5)
    x[1, 0, 3], x[2, 1, 20], x[3, 0, 49] = float("nan"), float("inf"), -float("inf")
    x[4, 0, :16] = float("nan")
    x[5, 1, 16:32] = float("inf")
    x[6, 1, :16] = 0.0
    x[7, 0, :16] = 0.0
    x[7, 0, 2], x[7, 0, 3], x[7, 0, 4] = float("inf"), float("nan"), -float("inf")
    x[8, 0, :16] = 3.0
    x[9, 1, 48:] = -float("inf")
    slots = np.arange(n, dtype=np.int64)
    c, s = cache_of(n, H, D, kind, group)
    check_write(x, slots, c, s, group, kind, D, _lib.STATUS_NOT_FINITE, False)
    assert bool(torch.isfinite(s).all())
    # and not where the token goes nowhere
    slots[1:10] = -1
    check_write(x, slots, c, s, group, kind, D, 0, False)
    with pytest.raises(RuntimeError, match="status 0x800"):
        lm.cache_write(x, dev(np.arange(n)), c, s, group)


@pytest.mark.parametrize("kind", KINDS)
def test_write_the_ends_of_float32(kind):
    n, H, D, group = 12, 1, 32, 16
    x = tokens_of(n, H, D, F32, 6)
    big = torch.finfo(F32).max
    x[0], x[1] = big, -big
    x[2, 0, ::2], x[2, 0, 1::2] = big, -big
    x[3] *= 2.0 ** 126    # (what passes 2^128 is infinite)
    x[4] *= 2.0 ** -110
    x[5] *= 2.0 ** -117
    x[6] *= 2.0 ** -125   # (subnormals: held as zeros)
    x[7] = torch.finfo(F32).tiny
    x[8, 0, 0] = big
    x[9] = -0.0
    c, s = cache_of(n, H, D, kind, group)
    bits = 0 if bool(torch.isfinite(x).all()) else _lib.STATUS_NOT_FINITE
    check_write(x, np.arange(n), c, s, group, kind, D, bits, False)
    assert bool(torch.isfinite(s).all())


def paged(lengths, bs, seed=0, width=None):
    """Requests' tables over a shuffled pool: (table, slots there)."""
    want = -(-np.asarray(lengths) // bs)
    W = (int(want.max()) if len(want) else 0) + 1 if width is None else width
    pool = np.random.default_rng(seed).permutation(int(want.sum()) + 3)
    table = np.full((len(lengths), W), -1, np.int32)
    k = 0
    for r, w in enumerate(want):
        table[r, :w] = pool[k:k + w]
        k += w
    return table, (int(want.sum()) + 3) * bs


def check_read(c, s, group, table, bs, off, n, D, kind, ot, start=None, layout="plain", bits=0, tab=None):
    H = c.shape[1]
    out = tokens_of(n, H, D, ot, 99, layout)
    first = f64(out)
    st = status()
    got = lm.cache_read(c, s, group, dev(table) if tab is None else tab, bs, dev(np.asarray(off, np.int64)), n,
                        start=None if start is None else dev(start), out=out, status=st)
    assert got is out and int(st.item()) == bits
    v, tol = ref.values(ref.unpack(c, D), s.cpu().numpy(), group, kind == "u4")
    slots = ref.read_slots(table, bs, off, n, c.shape[0], start)
    want, lim = np.zeros((n, H, D)), np.zeros((n, H, D))
    for t, slot in enumerate(slots):
        if slot is None:
            want[t] = first[t]
        elif slot >= 0:
            want[t], lim[t] = v[slot], tol[slot]
    check(out, want, lim, "read")
    rest = [t for t, slot in enumerate(slots) if slot is None]
    assert np.array_equal(f64(out)[rest], first[rest])
    return out


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ot", [BF16, F16, F32])
@pytest.mark.parametrize("lengths,H,D,group,bs", [
    ([1], 1, 1, 16, 16), ([5, 0, 3], 2, 17, 16, 4), ([100, 1, 37], 8, 128, 128, 16), ([64, 65, 63], 3, 77, 64, 7),
    ([0, 0, 200, 0], 10, 80, 32, 48), ([9] * 40, 2, 33, 16, 1), ([33], 1, 1000, 512, 128), ([7, 300], 64, 64, 32, 64)])
def test_read(lengths, H, D, group, bs, ot, kind):
    table, n_slots = paged(lengths, bs)
    c, s = cache_of(n_slots, H, D, kind, group)
    off = np.concatenate([[0], np.cumsum(lengths)])
    check_read(c, s, group, table, bs, off, int(off[-1]), D, kind, ot)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout", ["plain", "wide", "heads", "gaps"])
def test_read_part_of_the_contexts_into_strides(layout, kind):
    """From a position on; rows before the first and behind the last request stay."""
    lengths, bs, H, D = [50, 20, 90, 16], 16, 3, 40
    table, n_slots = paged(lengths, bs)
    c, s = cache_of(n_slots, H, D, kind, 16)
    start = np.array([45, 0, 33, 16], np.int32)
    off = 3 + np.concatenate([[0], np.cumsum(np.array(lengths) - start)])
    check_read(c, s, 16, table, bs, off, int(off[-1]) + 9, D, kind, BF16, start, layout)


@pytest.mark.parametrize("kind", KINDS)
def test_read_bad_pages(kind):
    lengths, bs, H, D = [40, 40, 40], 8, 2, 24
    table, n_slots = paged(lengths, bs, width=5)
    c, s = cache_of(n_slots, H, D, kind, 32)
    off = np.concatenate([[0], np.cumsum(lengths)])
    table[0, 2] = -1
    check_read(c, s, 32, table, bs, off, 120, D, kind, F32)
    table[1, 1] = n_slots // bs
    table[1, 2] = 2 ** 31 - 1
    check_read(c, s, 32, table, bs, off, 120, D, kind, F32, bits=_lib.STATUS_BAD_SLOT)
    start = np.array([0, 0, 39], np.int32)
    check_read(c, s, 32, table, bs, off, 120, D, kind, F32, start, bits=_lib.STATUS_BAD_SLOT | _lib.STATUS_TABLE_FULL)
    start = np.array([-5, 0, 0], np.int32)
    check_read(c, s, 32, table, bs, off, 120, D, kind, F32, start, bits=_lib.STATUS_BAD_SLOT | _lib.STATUS_BAD_LENGTH)
    with pytest.raises(RuntimeError, match="status 0x400"):
        lm.cache_read(c, s, 32, dev(table), bs, dev(off), 120)
    # no table at all
    check_read(c, s, 32, np.zeros((3, 0), np.int32), bs, off, 120, D, kind, F32, bits=_lib.STATUS_TABLE_FULL)


@pytest.mark.parametrize("kind", KINDS)
def test_read_by_a_strided_table_from_a_strided_cache(kind):
    lengths, bs, H, D, group = [50, 20, 90, 16], 16, 3, 40, 16
    table, n_slots = paged(lengths, bs)
    parts = [cache_of(n_slots, H, D, kind, group, k) for k in range(2)]
    c = torch.stack([x.view(torch.uint8) for x, _ in parts], 1)[:, 1].view(KINDS[kind])
    s = torch.stack([x for _, x in parts], 1)[:, 1]
    assert not c.is_contiguous() and not s.is_contiguous()
    off = np.concatenate([[0], np.cumsum(lengths)])
    check_read(c, s, group, table, bs, off, int(off[-1]), D, kind, F16, tab=strided(dev(table), 3))


def test_read_bad_offsets():
    lengths, bs = [40, 40, 40], 8
    table, n_slots = paged(lengths, bs)
    c, s = cache_of(n_slots, 2, 24, "int8", 32)
    for off in ([0, 80, 40, 120], [0, 40, 80, 121], [-1, 40, 80, 120], [2 ** 62, 0, -2 ** 62, 7], [5, 4, 3, 2]):
        st = status()
        lm.cache_read(c, s, 32, dev(table), bs, dev(np.array(off, np.int64)), 120, status=st)
        assert int(st.item()) & _lib.STATUS_BAD_ID_OFFSETS
    st = status()
    start = dev(np.array([2 ** 31 - 20, 0, 0], np.int32))
    got = lm.cache_read(c, s, 32, dev(table), bs, dev(np.array([0, 40, 80, 120])), 120, start=start, status=st)
    assert int(st.item()) == _lib.STATUS_TABLE_FULL | _lib.STATUS_BAD_LENGTH and bool((got[:40] == 0).all())


def test_read_many_requests():
    """More requests than a step of the search, most of them empty."""
    rng = np.random.default_rng(4)
    lengths = rng.integers(0, 40, 5000) * (rng.random(5000) < 0.1)
    table, n_slots = paged(lengths, 16)
    c, s = cache_of(n_slots, 1, 32, "e4m3", 32)
    off = np.concatenate([[0], np.cumsum(lengths)])
    check_read(c, s, 32, table, 16, off, int(off[-1]), 32, "e4m3", BF16)


@pytest.mark.parametrize("kind", KINDS)
def test_far_slots(kind):
    """Codes and scales past 2^32 bytes from the cache's start."""
    H, D, group, bs = 8, 128, 16, 16
    n_slots = (1 << 32) // (H * D // (2 if kind == "u4" else 1)) + 4 * bs
    c, s, _ = lm.empty_cache(n_slots, H, D, KINDS[kind], group, device=device())
    n = 3 * bs
    last = n_slots // bs - 1
    table = np.array([[last, 0, last - 1]], np.int32)
    slots = (table[0, np.arange(n) // bs].astype(np.int64) * bs + np.arange(n) % bs)
    x = tokens_of(n, H, D, BF16, 8)
    st = status()
    lm.cache_write(x, dev(slots), c, s, group, status=st)
    got = lm.cache_read(c, s, group, dev(table), bs, dev(np.array([0, n])), n, out_dtype=F32, status=st)
    x32 = x.float().cpu().numpy()
    tol = ref.quantise_error(x32, group, kind)
    want = x32.astype(np.float64)
    assert int(st.item()) == 0
    assert np.all(np.abs(f64(got) - want) <= tol + 4 * 2.0 ** -24 * (np.abs(want) + tol))


def test_a_head_dimension_of_half_a_byte():
    c, s = cache_of(16, 2, 5, "u4", 16)
    table, off = dev(np.zeros((1, 1), np.int32)), dev(np.array([0, 16]))
    assert lm.cache_read(c, s, 16, table, 16, off, 16).shape == (16, 2, 6)
    got = lm.cache_read(c, s, 16, table, 16, off, 16, dim=5, out_dtype=F32)
    assert torch.equal(got, lm.cache_read(c, s, 16, table, 16, off, 16, out_dtype=F32)[..., :5])


def test_captured_and_replayed():
    """Write and read in one graph, replayed with other tokens and lengths, padded."""
    R, bs, H, D, group = 4, 16, 2, 64, 64
    c, s = cache_of(R * 4 * bs, H, D, "int8", group)
    table = torch.arange(R * 4, dtype=torch.int32, device=device()).view(R, 4)
    x, slots = tokens_of(R, H, D, BF16, 1), torch.zeros(R, dtype=torch.int64, device=device())
    off = torch.zeros(R + 1, dtype=torch.int64, device=device())
    out = torch.zeros(200, H, D, dtype=BF16, device=device())
    st = status()

    def step():
        lm.cache_write(x, slots, c, s, group, status=st)
        lm.cache_read(c, s, group, table, bs, off, 200, out=out, status=st)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        lengths = torch.tensor([10 + k, 1, 40 - k, 3 * k + 1])
        x.copy_(tokens_of(R, H, D, BF16, 50 + k))
        slots.copy_(torch.arange(R) * 4 * bs + lengths - 1)
        off.copy_(torch.cat((torch.zeros(1, dtype=torch.int64), lengths.cumsum(0))))
        out.fill_(7.0)
        want_c, want_s = c.clone(), s.clone()
        graph.replay()
        torch.cuda.synchronize()
        lm.cache_write(x, slots, want_c, want_s, group)
        want = torch.full_like(out, 7.0)
        lm.cache_read(want_c, want_s, group, table, bs, off, 200, out=want)
        assert torch.equal(out, want) and torch.equal(c, want_c) and torch.equal(s, want_s)
        assert bool((out[int(off[-1]):] == 7).all())
    assert int(st.item()) == 0


def test_another_stream_outlives_its_inputs():
    n, H, D, group = 3000, 4, 64, 64
    slots = torch.randperm(n, device=device(), generator=gen(1))
    table = torch.arange(n // 8, dtype=torch.int32, device=device()).view(3, -1)
    off = torch.tensor([0, 1000, 2000, 3000], device=device())
    want_c, want_s = cache_of(n, H, D, "e4m3", group)
    lm.cache_write(tokens_of(n, H, D, BF16, 2), slots, want_c, want_s, group)
    want = lm.cache_read(want_c, want_s, group, table, 8, off, n)
    side, st = torch.cuda.Stream(), status()
    busy = torch.ones((4096, 4096), device=device())
    c, s = cache_of(n, H, D, "e4m3", group)
    x = tokens_of(n, H, D, BF16, 2)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(8):
            busy = busy @ busy * 2.0 ** -12
    lm.cache_write(x, slots, c, s, group, status=st, stream=side)
    got = lm.cache_read(c, s, group, table, 8, off, n, status=st, stream=side)
    del x
    noise = [tokens_of(n, H, D, BF16, 9) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and int(st.item()) == 0
    del noise


def test_scales_of_any_value():
    """What a caller puts into the scales is multiplied as it is."""
    c, s = cache_of(8, 1, 16, "int8", 16)
    c.view(torch.uint8).copy_(torch.arange(128, dtype=torch.uint8, device=device()).view(8, 1, 16) * 2)
    big = torch.finfo(F32).max
    s.copy_(torch.tensor([big / 127, -1.0, float("inf"), float("nan"), 0.0, 2.0 ** -140, big, -big],
                         device=device()).view(8, 1, 1))
    table, off = dev(np.zeros((1, 1), np.int32)), dev(np.array([0, 8]))
    got = lm.cache_read(c, s, 16, table, 8, off, 8, out_dtype=F32)
    want = c.float() * s
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


def test_inference_tensors_are_taken():
    with torch.inference_mode():
        c, s = cache_of(8, 1, 16, "e4m3", 16)
        lm.cache_write(tokens_of(2, 1, 16, F32, 1), dev(np.arange(2)), c, s, 16)


def test_writes_count_as_modified():
    c, s = cache_of(8, 1, 16, "int8", 16)
    v = c._version, s._version
    lm.cache_write(tokens_of(2, 1, 16, F32, 1), dev(np.arange(2)), c, s, 16)
    assert c._version > v[0] and s._version > v[1]
