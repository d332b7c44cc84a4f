"""A cache of few bits, drafted tokens and distillation at the ends of what their
arguments can say, without a GPU: refused before any HIP call."""
import pytest
import torch

from byte_level_bpe_pretokenize_amd import lm
from test_lm_checks import z
from test_lm_draft_checks import leaf, read

I32, I64, I8, F8 = torch.int32, torch.int64, torch.int8, torch.float8_e4m3fn
PAST = 1 << 32  # (what 32 bits hold of it is 0)


@pytest.mark.parametrize("group", [PAST + 16, PAST - 16, 1 << 31, -PAST + 16, PAST ** 2 + 32])
def test_a_group_past_32_bits_is_refused(group):
    """Also where the scales of three layers lie side by side: one per head by such a
    group, three by what 32 bits hold of PAST + 16."""
    codes, scales = z(6, 3, 2, 48, dtype=I8)[:, 1], z(6, 3, 2, 1)[:, 1]
    with pytest.raises(ValueError, match="group: .* out of range"):
        lm.cache_write(z(3, 2, 48), z(3, dtype=I64), codes, scales, group)
    with pytest.raises(ValueError, match="group: .* out of range"):
        lm.cache_read(codes, scales, group, z(1, 2, dtype=I32), 4, z(2, dtype=I64), 3)


@pytest.mark.parametrize("H,D,what", [(1, PAST + 48, "dim"), (PAST + 2, 48, "heads"), (1, 1 << 31, "dim"),
                                      (1 << 31, 16, "heads")])
def test_heads_past_32_bits_are_refused(H, D, what):
    """Tensors of no tokens have any shape."""
    codes, scales = z(0, H, D, dtype=I8), z(0, H, -(-D // 512))
    with pytest.raises(ValueError, match=f"{what}: .* out of range"):
        lm.cache_write(z(0, H, D), z(0, dtype=I64), codes, scales, 512)
    with pytest.raises(ValueError, match=f"{what}: .* out of range"):
        lm.cache_read(codes, scales, 512, z(1, 2, dtype=I32), 4, z(2, dtype=I64), 0)


@pytest.mark.parametrize("call", [
    lambda: lm.distill(z(3, 40), z(3, 5, dtype=I32), z(3, 5), losses=leaf(3) * 1),
    lambda: lm.distill(z(3, 40), z(3, 5, dtype=I32), z(3, 5), stats=leaf(3, 4) * 1),
    lambda: lm.cache_write(z(3, 2, 32), z(3, dtype=I64), leaf(6, 2, 32).to(F8), z(6, 2, 1), 32),
    lambda: read(codes=leaf(6, 2, 32).to(F8)),
])
def test_what_is_filled_or_read_drops_no_gradient(call):
    with pytest.raises(RuntimeError, match="gives no gradient"):
        call()
