"""The operators on token IDs around a toy language model: serving steps and
training steps on text that the library encodes.

    python examples/lm_step.py

Serving: the requests are encoded (a BOS before each), their tokens placed in a
paged cache (lm.block_tables) and embedded (lm.embed); the stand-in for a model
averages what a request has in the cache and multiplies by the embedding table;
the next token comes from the processed logits (lm.process_logits: repetition
and frequency penalties, a bias against EOS, and a mask that lets only tokens
of letters and spaces through), and goes back into the cache.  At the end the
tokens are decoded.

Training: next-token cross entropy of the same stand-in on the encoded text,
with lm.embedding's gradient for the table.
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from byte_level_bpe_pretokenize_amd import Model, lm  # noqa: E402

BLOCK = 16
TEXTS = ["the quick brown fox", "hello hello hello world", "", "a", "numbers 12 and 3456 and words"]


def load(width: int = 64, seed: int = 0):
    """The tiny table's model, its reserved IDs, and an embedding table."""
    model = Model(np.load(os.path.join(ROOT, "assets", "merges_tiny.npy"), allow_pickle=False))
    V = model.vocab_size
    gen = torch.Generator(device=model.device).manual_seed(seed)
    weight = torch.randn(V + 3, width, device=model.device, generator=gen) / width ** 0.5
    return model, {"bos": V, "eos": V + 1, "pad": V + 2}, weight


def batch(model, texts):
    raw = [t.encode() for t in texts]
    data = torch.tensor(list(b"".join(raw)), dtype=torch.uint8, device=model.device)
    off = torch.tensor([0] + list(np.cumsum([len(r) for r in raw])), device=model.device)
    return data, off


def letters_mask(model, n_tokens: int) -> torch.Tensor:
    """(1, ceil(n_tokens / 32)) int32: the tokens made of letters and spaces."""
    V = model.vocab_size
    ids = torch.arange(V, dtype=torch.int32, device=model.device)
    text, off = model.decode_batch(ids, torch.arange(V + 1, device=model.device))
    text, off = bytes(text.cpu().numpy()), off.tolist()
    bits = np.zeros((n_tokens + 31) // 32 * 32, dtype=np.uint64)
    for v in range(V):
        bits[v] = all(c == 0x20 or chr(c).isalpha() and c < 128 for c in text[off[v]:off[v + 1]])
    words = (bits.reshape(-1, 32) << np.arange(32, dtype=np.uint64)).sum(1).astype(np.uint32)
    return torch.from_numpy(words.view(np.int32)[None].copy()).to(model.device)


def serve(model, special, weight, texts, steps: int = 12):
    """The texts continued by `steps` tokens, greedily: (texts, IDs (R, steps))."""
    dev, (V, D), R = model.device, weight.shape, len(texts)
    ids, id_off = model.encode_batch_special(*batch(model, texts), bos_id=special["bos"])
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    # the cache: blocks of BLOCK rows, all of them free
    width = (max((id_off[1:] - id_off[:-1]).tolist()) + steps) // BLOCK + 1
    free = torch.randperm(R * width, device=dev).to(torch.int32)
    cache = torch.zeros(R * width * BLOCK, D, device=dev)
    table = torch.full((R, width), -1, dtype=torch.int32, device=dev)
    lengths = torch.zeros(R, dtype=torch.int32, device=dev)
    one = torch.arange(R + 1, device=dev)  # offsets of one token per request
    made = torch.zeros(R, steps, dtype=torch.int32, device=dev)
    mask, mask_row = letters_mask(model, V), torch.zeros(R, dtype=torch.int32, device=dev)
    full = lambda x, dt=torch.float32: torch.full((R,), x, dtype=dt, device=dev)  # noqa: E731
    new, new_off = ids, id_off
    for step in range(steps):
        slots, positions, lengths, used = lm.block_tables(new_off, new.numel(), lengths, free, table,
                                                          BLOCK, status=status)
        free = free[int(used):]
        cache[slots] = lm.embed(weight, new, D ** 0.5, status=status)
        # the model: the average of a request's rows in the cache
        rows = (table.clamp(min=0).long()[:, :, None] * BLOCK + torch.arange(BLOCK, device=dev)).view(R, -1)
        there = torch.arange(rows.shape[1], device=dev) < lengths[:, None]
        hidden = (cache[rows] * there[:, :, None]).sum(1) / lengths[:, None]
        logits = lm.process_logits(
            hidden @ weight.t(), prompt_ids=ids, prompt_off=id_off, out_ids=made,
            out_len=full(step, torch.int32), repetition=full(1.3), frequency=full(0.2),
            bias_off=one, bias_ids=full(special["eos"], torch.int32), bias_values=full(-5.0),
            mask=mask, mask_row=mask_row, status=status)
        new = logits.argmax(1).to(torch.int32)
        made[:, step] = new
        new_off = one
    if int(status):
        raise RuntimeError(f"device status {int(status):#x}")
    out, off = model.decode_batch(made.view(-1), torch.arange(R + 1, device=dev) * steps)
    out, off = bytes(out.cpu().numpy()), off.tolist()
    return [out[off[r]:off[r + 1]].decode(errors="replace") for r in range(R)], made


def train(model, special, weight, texts, steps: int = 10, rate: float = 0.1):
    """The losses of `steps` steps of gradient descent on the embedding table."""
    ids, id_off = model.encode_batch_special(*batch(model, texts), bos_id=special["bos"],
                                             eos_id=special["eos"])
    status = torch.zeros(1, dtype=torch.int32, device=model.device)
    last = torch.zeros(ids.numel(), dtype=torch.bool, device=model.device)
    last[id_off[1:] - 1] = True  # nothing follows a text's last token
    target = torch.roll(ids, -1).long()
    w = weight.clone().requires_grad_()
    losses = []
    for _ in range(steps):
        x = lm.embedding(w, ids, pad_id=special["pad"], status=status)
        logp = torch.log_softmax(x @ weight.t(), 1)
        loss = -logp.gather(1, target[:, None])[~last].mean()
        (g,) = torch.autograd.grad(loss, w)
        with torch.no_grad():
            w -= rate * weight.shape[0] * g
        losses.append(float(loss.detach()))
    if int(status):
        raise RuntimeError(f"device status {int(status):#x}")
    return losses


if __name__ == "__main__":
    m, sp, table = load()
    for text, more in zip(TEXTS, serve(m, sp, table, TEXTS)[0]):
        print(f"{text!r} -> {more!r}")
    print("losses:", " ".join(f"{x:.3f}" for x in train(m, sp, table, TEXTS * 20)))
