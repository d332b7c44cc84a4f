"""What the drafting operators leave behind where nothing sensible came in."""
import numpy as np
import pytest
import torch

from gpu_util import device
from test_gpu_lm_drafts import check
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
