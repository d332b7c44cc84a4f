"""The example's drafting, which runs the cache of few bits, the verification of
drafts and distillation together, against the same steps in 64 bits."""
import numpy as np
import pytest
import torch

import lm_draft_reference as ref
from lm_reference import f64
from byte_level_bpe_pretokenize_amd import lm

from gpu_util import device
from test_gpu_lm_example import example

pytestmark = pytest.mark.gpu


def softmax(x):
    e = np.exp(x - x.max())
    return e / e.sum()


NEAR = 1e-5  # float32 logits may turn a choice this near a border


def may_be(token, w, u):
    """Whether a share of the weights' sum, or one NEAR it, ends at the token."""
    run = np.concatenate([[0], np.cumsum(w)]) / w.sum()
    return w[token] > 0 and run[token] - NEAR <= u <= run[token + 1] + NEAR


@pytest.mark.parametrize("held,kind", [(torch.int8, "int8"), (torch.float8_e4m3fn, "e4m3"), (torch.uint8, "u4")])
def test_serving_with_drafts(held, kind):
    torch.cuda.set_device(device())
    ex = example()
    model, special, weight = ex.load()
    drafter = ex.train_drafter(model, special, weight, ex.TEXTS * 4, steps=4)[0]
    steps, k, heads = 7, 3, 4
    got, numbers = ex.serve_drafts(model, special, weight, drafter, ex.TEXTS, steps, k, heads, held=held)
    ids, off = model.encode_batch_special(*ex.batch(model, ex.TEXTS), bos_id=special["bos"])
    V, D = weight.shape
    bits = ex.letters_mask(model, V)[0].cpu().numpy().astype(np.uint32)
    allowed = (bits[np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)) & 1 == 1
    w, d = f64(weight), f64(drafter)
    # what the cache holds of each token's embedding
    x = lm.embed(weight, torch.arange(V, dtype=torch.int32, device=model.device), D ** 0.5)
    codes, scales, lows = ref.quantise(x.view(V, heads, D // heads).cpu().numpy(), 16, kind)
    s = np.stack((scales, lows), -1) if kind == "u4" else scales
    kept = ref.values(codes, s, 16, kind == "u4")[0].reshape(V, D)
    stood = 0
    for r in range(len(ex.TEXTS)):
        seq = ids[off[r]:off[r + 1]].tolist()
        for (drafts, u, accept, sample), tokens in zip(numbers, got[r]):
            drafts, q, last, m = drafts[r].tolist(), [], seq[-1], len(tokens) - 1
            for i in range(k):
                q.append(np.where(allowed, softmax(np.where(allowed, d[last] @ w.T, -np.inf)), 0.0))
                last = drafts[i]
                assert may_be(last, q[-1], float(u[i, r]))
            assert tokens[:m] == drafts[:m]
            for i in range(m + 1):
                p = softmax(np.where(allowed, kept[seq + drafts[:i]].mean(0) @ w.T, -np.inf))
                if i < k:
                    a, b = float(accept[r, i]) * q[i][drafts[i]], p[drafts[i]]
                    assert a < b * (1 + NEAR) if i < m else a > b * (1 - NEAR)
            assert may_be(tokens[m], np.maximum(p - q[m], 0.0) if m < k else p, float(sample[r]))
            seq += tokens
            stood += m
    assert stood > 0


def test_a_drafters_gradient():
    ex = example()
    model, special, weight = ex.load()
    first, losses = ex.train_drafter(model, special, weight, ex.TEXTS, steps=1, rate=0.5)
    # the same step in 64 bits
    ids, off = model.encode_batch_special(*ex.batch(model, ex.TEXTS), bos_id=special["bos"])
    w = f64(weight)
    V, D = w.shape
    seqs = [ids[off[r]:off[r + 1]].tolist() for r in range(len(ex.TEXTS))]
    z, tops, t = [], [], []
    for seq in seqs:
        for i in range(len(seq)):
            y = (w[seq[:i + 1]] * D ** 0.5).mean(0) @ w.T
            order = np.argsort(-y)
            assert y[order[15]] - y[order[16]] > 1e-5, "a tie: choose another seed"
            z.append(np.zeros(V))
            tops.append(order[:16])
            t.append(y[order[:16]])
    n = len(z)
    loss, _, grad, _ = ref.distill(np.array(z), np.array(tops), np.array(t), 2.0, np.full(n, 1 / n))
    assert abs(losses[0] - loss.mean()) < 1e-5 * loss.mean()
    g = np.zeros((V, D))
    np.add.at(g, [v for seq in seqs for v in seq], grad @ w)
    assert np.abs(f64(first) + 0.5 * V * g).max() < 1e-4 * 0.5 * V * np.abs(g).max()
