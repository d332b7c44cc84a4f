"""The operators on token IDs and autograd: what the calls that give no gradient
refuse (before the device is looked at), and that what they write in place
counts as modified."""
import pytest
import torch

from byte_level_bpe_pretokenize_amd import lm

I32, I64 = torch.int32, torch.int64


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def leaf(*shape):
    return torch.zeros(*shape, requires_grad=True)


CALLS = [
    lambda: lm.embed(leaf(4, 8), z(3, dtype=I32)),
    lambda: lm.embed(z(4, 8), z(3, dtype=I32), out=leaf(3, 8) * 1),
    lambda: lm.embed_grad(leaf(3, 8), z(3, dtype=I32), 4),
    lambda: lm.embed_grad(z(3, 8), z(3, dtype=I32), 4, out=leaf(4, 8) * 1, accumulate=True),
    lambda: lm.process_logits(leaf(2, 40)),
    lambda: lm.process_logits(z(2, 40), repetition=leaf(2)),
    lambda: lm.process_logits(z(2, 40), frequency=leaf(2)),
    lambda: lm.process_logits(z(2, 40), presence=leaf(2)),
    lambda: lm.process_logits(z(2, 40), bias_off=z(3, dtype=I64), bias_ids=z(2, dtype=I32),
                              bias_values=leaf(2)),
    lambda: lm.process_logits(z(2, 40), out=leaf(2, 40) * 1),
]


@pytest.mark.parametrize("call", CALLS)
def test_calls_without_a_gradient_refuse(call):
    with pytest.raises(RuntimeError, match="gives no gradient"):
        call()


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a GPU")
@pytest.mark.parametrize("call", CALLS)
def test_and_do_not_where_none_is_wanted(call):
    with torch.no_grad(), pytest.raises(RuntimeError, match="HIP device"):
        call()


@pytest.mark.gpu
def test_in_place_results_count_as_modified():
    dev = "cuda"
    ids = torch.arange(3, dtype=I32, device=dev)
    x = torch.randn(3, 8, device=dev, requires_grad=True)
    g = torch.randn(3, 8, device=dev)
    writes = [
        lambda y: lm.embed(g, ids, out=y),
        lambda y: lm.embed_grad(g, ids, 3, out=y),
        lambda y: lm.process_logits(y, out=y),
        lambda y: lm.process_logits(y, out=y, stream=torch.cuda.current_stream()),
    ]
    for write in writes:
        y = x.exp()  # kept for its own gradient
        with torch.no_grad():
            write(y)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()


@pytest.mark.gpu
def test_block_tables_counts_as_modified():
    dev = "cuda"
    n = lambda *shape, dtype=I32: torch.zeros(*shape, dtype=dtype, device=dev)  # noqa: E731
    off = torch.tensor([0, 2, 5], device=dev)
    given = dict(slots=n(5, dtype=I64), positions=n(5), lengths=n(2), used=n(1, dtype=I64))
    table, free = n(2, 4), torch.arange(6, dtype=I32, device=dev)
    before = {k: t._version for k, t in given.items()}, table._version, free._version
    lm.block_tables(off, 5, n(2), free, table, 16, **given)
    assert all(t._version > before[0][k] for k, t in given.items())
    assert table._version > before[1] and free._version == before[2]


@pytest.mark.gpu
def test_inference_tensors_are_taken():
    with torch.inference_mode():
        x = torch.zeros(2, 40, device="cuda")
        assert lm.process_logits(x, out=x) is x
