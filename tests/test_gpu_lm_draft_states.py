"""What the drafting operators leave behind where nothing sensible came in."""
import numpy as np
import pytest
import torch

import lm_draft_reference as ref
from lm_reference import f64
from byte_level_bpe_pretokenize_amd import _lib, lm

from gpu_util import device
from test_gpu_lm import F32, dev, status
from test_gpu_lm_drafts import batch, check
from test_gpu_lm_example import example

pytestmark = pytest.mark.gpu


def test_an_example_without_tokens_ends_by_its_status():
    """Logits that are all NaN leave nothing to draw from: counts are 0, and the last
    token of none is not looked for before the row's first."""
    torch.cuda.set_device(device())
    ex = example()
    model, special, weight = ex.load()
    with pytest.raises(RuntimeError, match="device status"):
        ex.serve_drafts(model, special, torch.full_like(weight, float("nan")), weight, ex.TEXTS, 2)


@pytest.mark.parametrize("V", [40, 9000])
@pytest.mark.parametrize("accept", [-1.0, -2.0 ** -149, -float("inf"), float("inf"), float("nan"), 0.0])
def test_accepts_outside_against_drafts_without_probability(accept, V):
    """A request of one draft for each of q > 0, q = 0 and q that counts as 0, with
    p > 0 and p = 0."""
    nan, inf = float("nan"), float("inf")
    q_at = [0.25, 0.0, -1.0, nan, inf, 0.25, 0.0, -1.0, nan, inf]
    p_at = [0.5] * 5 + [0.0] * 5
    p, q = (torch.full((20, V), 1.0 / V, device=device()) for _ in range(2))
    p[::2, 3], q[::2, 3] = torch.tensor(p_at, device=device()), torch.tensor(q_at, device=device())
    ids = torch.full((20,), 3, dtype=torch.int32, device=device())
    off = np.arange(0, 21, 2)
    _, counts = check(p, q, ids, off, torch.full((20,), accept, device=device()), torch.full((10,), 0.6, device=device()))
    if accept == -inf:
        want = [2, 1, 1, 1, 1, 2, 1, 1, 1, 1]
    elif accept < 0:
        want = [2, 2, 2, 2, 2, 2, 1, 1, 1, 1]
    elif accept == 0:
        want = [2] * 5 + [1] * 5
    else:
        want = [1] * 10
    assert counts.tolist() == want


@pytest.mark.parametrize("V", [100, 70000])
def test_requests_beside_bad_offsets_keep_their_tokens(V):
    """Requests whose offsets are valid and that share no row with another one get
    what they get alone; rows that are no request's are left as they were."""
    p, q, ids, _, accept, sample = batch([4, 4, 4], V, F32, 1)
    for off, fine in (([0, 5, 3, 15], (0,)), ([0, 5, 10, 16], (0, 1)), ([-1, 5, 10, 15], (1, 2)),
                      ([2 ** 62, -2 ** 62, 10, 15], (2,)), ([7, 6, 5, 15], (2,))):
        tokens, st = torch.full((15,), -9, dtype=torch.int32, device=device()), status()
        _, counts = lm.verify_drafts(p, ids, dev(np.array(off, np.int64)), accept, sample, draft=q, tokens=tokens,
                                     status=st)
        assert int(st.item()) == _lib.STATUS_BAD_ID_OFFSETS
        left = np.ones(15, bool)
        for r in range(3):
            lo, hi = off[r], off[r + 1]
            if r not in fine:
                # (3 to 15 is a request by itself, though it has rows of the first one)
                if not 0 <= lo <= hi <= 15:
                    assert int(counts[r]) == 0
                else:
                    left[lo:hi] = False
                continue
            want, n = ref.verify(f64(p), ids.cpu().numpy(), [lo, hi], accept.cpu().numpy(),
                                 sample[r:r + 1].cpu().numpy(), f64(q))
            rows = slice(lo, 3 if off[2] == 3 else hi)  # (the rows that no other request has)
            assert int(counts[r]) == n[0] and np.array_equal(tokens.cpu().numpy()[rows], want[rows])
            left[lo:hi] = False
        assert bool((tokens.cpu()[torch.from_numpy(left)] == -9).all())


def test_a_read_of_no_tokens_looks_at_nothing():
    """No launch, so no status: offsets past the tokens and a negative start."""
    c, s, group = lm.empty_cache(8, 2, 16, torch.int8, device=device())
    table, st = torch.zeros((2, 1), dtype=torch.int32, device=device()), status()
    for off in ([0, 5, 9], [3, 2, 1], [-1, 0, 0]):
        got = lm.cache_read(c, s, group, table, 4, dev(np.array(off, np.int64)), 0,
                            start=dev(np.array([-1, -1], np.int32)), status=st)
        assert got.shape == (0, 2, 16)
    none = lm.cache_read(c, s, group, table[:0], 4, dev(np.array([7], np.int64)), 3, status=st)
    assert none.shape == (3, 2, 16) and int(st.item()) == 0
