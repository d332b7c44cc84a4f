"""The operators on token IDs on the GPU at the edges of their kernels' variants:
column slabs with few lanes in use, queues that overflow, the launches of the
largest batches.  Bounds as in test_gpu_lm.py."""
import pytest
import torch

from byte_level_bpe_pretokenize_amd import lm

from gpu_util import device
from test_gpu_lm import BF16, F32, gaps, gen, randn, status, strided

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
