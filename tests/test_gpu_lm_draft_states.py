"""What the drafting operators leave behind where nothing sensible came in."""
import pytest
import torch

from gpu_util import device
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
