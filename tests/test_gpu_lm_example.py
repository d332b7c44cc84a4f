"""The example that runs the operators on token IDs together, against the same
steps in plain torch operations."""
import importlib.util
import os

import pytest
import torch

from byte_level_bpe_pretokenize_amd import lm

from gpu_util import ROOT, device

pytestmark = pytest.mark.gpu


def example():
    spec = importlib.util.spec_from_file_location("lm_step", os.path.join(ROOT, "examples", "lm_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_serving_steps():
    torch.cuda.set_device(device())
    ex = example()
    model, special, weight = ex.load()
    steps = 9
    texts, made = ex.serve(model, special, weight, ex.TEXTS, steps)
    assert len(texts) == len(ex.TEXTS)
    assert all(c == " " or c.isalpha() and c.isascii() for t in texts for c in t)
    # the same, request by request, without a cache
    ids, off = model.encode_batch_special(*ex.batch(model, ex.TEXTS), bos_id=special["bos"])
    bits = ex.letters_mask(model, weight.shape[0])[0].long()
    v = torch.arange(weight.shape[0], device=model.device)
    allowed = (bits[v // 32] >> (v % 32)) & 1 == 1
    for r in range(len(ex.TEXTS)):
        prompt = ids[off[r]:off[r + 1]].long()
        got = []
        for step in range(steps):
            seq = torch.cat([prompt, torch.tensor(got, dtype=torch.long, device=model.device)])
            x = (weight[seq].double() * weight.shape[1] ** 0.5).mean(0) @ weight.double().t()
            count = torch.bincount(seq[len(prompt):], minlength=len(v)).double()
            seen = torch.bincount(seq, minlength=len(v)) > 0
            x = torch.where(seen, torch.where(x > 0, x / 1.3, x * 1.3), x) - 0.2 * count
            x[special["eos"]] -= 5.0
            x = x.masked_fill(~allowed, -torch.inf)
            best = x.topk(2).values
            assert best[0] - best[1] > 1e-4, "a tie: choose another seed"
            got.append(int(x.argmax()))
        assert made[r].tolist() == got


def test_training_steps():
    ex = example()
    model, special, weight = ex.load()
    losses = ex.train(model, special, weight, ex.TEXTS * 20)
    assert losses[-1] < losses[0] and all(b < a for a, b in zip(losses, losses[1:]))
    # one step's gradient against plain torch operations
    ids, _ = model.encode_batch_special(*ex.batch(model, ex.TEXTS), bos_id=special["bos"])
    w = weight.clone().requires_grad_()
    u = weight.double().requires_grad_()
    (lm.embedding(w, ids) ** 2).sum().backward()
    (u[ids.long()] ** 2).sum().backward()
    assert torch.allclose(w.grad.double(), u.grad, rtol=1e-5, atol=1e-6)


def test_backward_in_a_graph():
    """Forward and backward captured together (no eager graph of the leaf lives
    meanwhile), replayed with other inputs."""
    ex = example()
    model, _, weight = ex.load()
    V, D = weight.shape
    ids = torch.randint(0, V, (4000,), dtype=torch.int32, device=model.device)
    dy = torch.randn(4000, D, device=model.device)
    status = torch.zeros(1, dtype=torch.int32, device=model.device)
    w = weight.clone().requires_grad_()

    def step():
        return torch.autograd.grad(lm.embedding(w, ids, 2.0, status=status), w, dy)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(4):
        ids.copy_(torch.randint(0, V, (4000,), dtype=torch.int32, device=model.device))
        dy.normal_()
        graph.replay()
        torch.cuda.synchronize()
        want = lm.embed_grad(dy, ids, V, 2.0, status=status)
        assert torch.equal(got, want), k
    assert int(status) == 0
