"""The operators on token IDs next to encode and decode, measured: embedding
lookup with scaling (`embed`), its gradient (`embed_grad`), penalties, biases
and grammar masks on logits (`process_logits`), and block tables with slot maps
from request lengths (`block_tables`).

`run` computes each in its plain form (elementary torch operations in 32 bits,
rounded once at the end) or, where `own` is true, through the framework's calls
in `byte_level_bpe_pretokenize_amd.lm`.  `exact` computes them in 64 bits.

Vocabularies are those of this repository's merge tables (256 bytes + 512,
32,000, 50,000, 100,000 or 128,000 merges); request lengths are those of its
serving workload (lognormal(6, 1) bytes clipped to 32-8,192).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
VOCABS = (768, 32256, 50256, 100256, 128256)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 64 requests: one row each, latency
        {"name": "embed decode", "op": "embed", "ids": 64, "vocab": 128256, "width": 4096,
         "weight": "bf16", "out": "bf16", "pad": False},
        # a chunk of ragged prompts, padded in places, on a table whose rows are no multiple of
        # a vector (a factored embedding of odd width)
        {"name": "embed prompts odd width", "op": "embed", "ids": 30011, "vocab": 100256,
         "width": 1001, "weight": "f16", "out": "f16", "pad": True},
        # a training batch (64 sequences of 4,096) through float32 master weights to bfloat16
        {"name": "embed train", "op": "embed", "ids": 262144, "vocab": 32256, "width": 4096,
         "weight": "f32", "out": "bf16", "pad": False},
        # one small sequence on the smallest vocabulary: latency, long sums for few rows
        {"name": "grad tiny", "op": "grad", "ids": 2048, "vocab": 768, "width": 512,
         "grad": "bf16", "out": "f32", "pad": False},
        # the gradient of a training batch, kept in float32
        {"name": "grad train", "op": "grad", "ids": 131072, "vocab": 32256, "width": 4096,
         "grad": "bf16", "out": "f32", "pad": False},
        # a ragged, padded batch on the largest vocabulary: most rows of the gradient stay zero
        {"name": "grad large vocabulary", "op": "grad", "ids": 40009, "vocab": 128256,
         "width": 2048, "grad": "bf16", "out": "bf16", "pad": True},
        # a decode step of few requests
        {"name": "logits few rows", "op": "logits", "rows": 4, "vocab": 50256, "logits": "bf16",
         "out": "f32", "prompt": 700, "made": 100, "bias": 8, "masks": 2},
        # a full decode step of a large batch, the largest vocabulary
        {"name": "logits decode", "op": "logits", "rows": 256, "vocab": 128256, "logits": "bf16",
         "out": "f32", "prompt": 600, "made": 256, "bias": 32, "masks": 8},
        # few requests with long prompts, float32 logits
        {"name": "logits long prompts", "op": "logits", "rows": 24, "vocab": 100256,
         "logits": "f32", "out": "f32", "prompt": 30000, "made": 2000, "bias": 300, "masks": 3},
        # a decode step: one new token each, contexts up to 32,768
        {"name": "blocks decode", "op": "blocks", "requests": 256, "new": 1, "cached": 32768,
         "block": 16},
        # a step that mixes new prompts with running requests, blocks of no power of two
        {"name": "blocks mixed", "op": "blocks", "requests": 1501, "new": 190, "cached": 2000,
         "block": 48},
        # every request of the serving workload at once
        {"name": "blocks serving batch", "op": "blocks", "requests": 65536, "new": 190,
         "cached": 0, "block": 16},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("embed", "grad", "logits", "blocks"))
    if op in ("embed", "grad"):
        width = _log_between(rng, 64, 8192)
        if rng.random() < 0.6:
            width = max(64, width // 64 * 64)
        vocab = rng.choice(VOCABS) if rng.random() < 0.6 else _log_between(rng, 300, 200000)
        vocab = min(vocab, 200_000_000 // width)
        most = (500_000_000 if op == "embed" else 300_000_000) // width
        ids = min(_log_between(rng, 1, 200000), most)
        pair = rng.choice((("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"), ("f16", "f16"))
                          if op == "embed" else
                          (("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f16", "f32")))
        return {"op": op, "ids": ids, "vocab": vocab, "width": width,
                "weight" if op == "embed" else "grad": pair[0], "out": pair[1],
                "pad": rng.random() < 0.5}
    if op == "logits":
        vocab = rng.choice(VOCABS) if rng.random() < 0.6 else _log_between(rng, 300, 150000)
        rows = min(_log_between(rng, 1, 256), 25_000_000 // vocab)
        pair = rng.choice((("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f16", "f32")))
        return {"op": op, "rows": rows, "vocab": vocab, "logits": pair[0], "out": pair[1],
                "prompt": min(_log_between(rng, 1, 20000), 500_000 // rows),
                "made": _log_between(rng, 1, 2000), "bias": rng.choice((0, 1, 8, 32, 300)),
                "masks": rng.choice((0, 1, 3, 8))}
    requests = _log_between(rng, 1, 50000)
    new = 1 if rng.random() < 0.3 else min(_log_between(rng, 2, 2000), max(2, 8_000_000 // requests))
    cached = 0 if rng.random() < 0.4 else min(_log_between(rng, 1, 40000),
                                              max(1, 40_000_000 // requests))
    return {"op": "blocks", "requests": requests, "new": new, "cached": cached,
            "block": rng.choice((16, 32, 64, 128, 48, 1, 7))}


# ---------------------------------------------------------------- inputs
def _zipf_ids(n, vocab, gen):
    """IDs as text gives them: the k-th most frequent one about 1/k as often as the first, the
    order of the IDs by frequency mixed."""
    u = torch.rand(n, device="cuda", dtype=torch.float64, generator=gen)
    rank = (torch.exp(u * math.log(vocab + 1.0)) - 1.0).floor().long().clamp_(0, vocab - 1)
    return torch.randperm(vocab, device="cuda", generator=gen)[rank].to(torch.int32)


def _prepare_embed(case, gen, rng):
    vocab, width, n = case["vocab"], case["width"], case["ids"]
    s = {"case": case, "ids": _zipf_ids(n, vocab, gen), "pad": -1, "scale": math.sqrt(width),
         "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["pad"]:
        # the last ID of the vocabulary fills what ragged sequences leave free
        s["pad"] = vocab - 1
        hole = torch.rand(n, device="cuda", generator=gen) < 0.1
        s["ids"] = torch.where(hole, torch.full_like(s["ids"], vocab - 1), s["ids"])
    if case["op"] == "embed":
        w = torch.empty(vocab, width, device="cuda", dtype=DTYPES[case["weight"]])
        s["weight"] = w.normal_(0.0, 1.0 / math.sqrt(width), generator=gen)
    else:
        dy = torch.empty(n, width, device="cuda", dtype=DTYPES[case["grad"]])
        s["grad"] = dy.normal_(0.0, 1.0, generator=gen)
    return s


def _prepare_logits(case, gen, rng):
    rows, vocab = case["rows"], case["vocab"]
    dev = "cuda"
    logits = torch.empty(rows, vocab, device=dev, dtype=DTYPES[case["logits"]])
    logits.normal_(0.0, 3.0, generator=gen)
    # prompts as encode_batch gives them: packed IDs and offsets
    plen = np.maximum(1, rng.lognormal(math.log(case["prompt"]) - 0.125, 0.5, rows).astype(np.int64))
    poff = np.concatenate([[0], np.cumsum(plen)])
    # what was generated so far, padded to the longest that may be
    made = rng.integers(0, case["made"] + 1, rows).astype(np.int32)
    uniform = lambda lo, hi: torch.from_numpy(rng.uniform(lo, hi, rows).astype(np.float32)).to(dev)  # noqa: E731
    some = torch.from_numpy(rng.random(rows) < 0.3).to(dev)  # requests without the penalties
    one, zero = torch.ones(rows, device=dev), torch.zeros(rows, device=dev)
    s = {"case": case, "logits": logits, "prompt_ids": _zipf_ids(int(poff[-1]), vocab, gen),
         "prompt_off": torch.from_numpy(poff).to(dev),
         "out_ids": _zipf_ids(rows * case["made"], vocab, gen).view(rows, case["made"]),
         "out_len": torch.from_numpy(made).to(dev),
         "repetition": torch.where(some, one, uniform(1.0, 1.5)),
         "frequency": torch.where(some, zero, uniform(0.0, 1.0)),
         "presence": torch.where(some, zero, uniform(0.0, 1.0)),
         "bias_off": None, "bias_ids": None, "bias_values": None, "mask": None, "mask_row": None,
         "status": torch.zeros(1, dtype=torch.int32, device=dev)}
    if case["bias"]:
        per = rng.integers(0, min(case["bias"], vocab) + 1, rows)
        ids = [np.sort(rng.choice(vocab, k, replace=False)) for k in per]
        n = int(per.sum())
        val = rng.uniform(-5.0, 5.0, n)
        val = np.where(rng.random(n) < 0.1, -100.0, val)
        s["bias_off"] = torch.from_numpy(np.concatenate([[0], np.cumsum(per)]).astype(np.int64)).to(dev)
        s["bias_ids"] = torch.from_numpy(np.concatenate(ids).astype(np.int32)).to(dev)
        s["bias_values"] = torch.from_numpy(val.astype(np.float32)).to(dev)
    if case["masks"]:
        # grammar states: the first lets nothing through (a row may end empty), then from few
        # tokens to nearly all; a third of the requests has none
        words = (vocab + 31) // 32
        bits = torch.rand(case["masks"], words, 32, device=dev, generator=gen)
        share = torch.linspace(0.0, 0.95, case["masks"], device=dev)[:, None, None]
        on = (bits < share).long() << torch.arange(32, device=dev)
        s["mask"] = on.sum(-1).to(torch.int32)
        row = rng.integers(0, case["masks"], rows)
        row = np.where(rng.random(rows) < 1 / 3, -1, row)
        s["mask_row"] = torch.from_numpy(row.astype(np.int32)).to(dev)
    return s


def _prepare_blocks(case, gen, rng):
    n, bs = case["requests"], case["block"]
    total, most = n * case["new"], 13 * case["new"]
    if case["new"] == 1:
        new, most = np.ones(n, dtype=np.int64), 1
    else:
        # the serving workload's lengths, scaled to the case's number of tokens, at most 13 times
        # their mean (what is over goes to others); a tenth has one token
        b = np.clip(rng.lognormal(6.0, 1.0, n), 32, 8192) * (rng.random(n) >= 0.1) + 1e-6
        ends = np.floor(np.cumsum(b) / b.sum() * (total - n)).astype(np.int64)
        ends[-1] = total - n
        new = np.minimum(1 + np.diff(ends, prepend=0), most)
        while (over := total - int(new.sum())) > 0:
            at = np.flatnonzero(new < most)[:over]
            new[at] += np.minimum(most - new[at], max(1, over // at.size))
    cached = np.zeros(n, dtype=np.int64)
    if case["cached"]:
        cached = rng.integers(0, case["cached"], n)
    have, want = -(-cached // bs), -(-(cached + new) // bs)
    width = -(-(case["cached"] + most) // bs) + 1  # a request's longest context
    taken, need = int(have.sum()), int((want - have).sum())
    spare = need // 8 + 5
    pool = torch.randperm(taken + need + spare, device="cuda", generator=gen).to(torch.int32)
    have_t = torch.from_numpy(have).cuda()
    at = torch.arange(width, device="cuda")
    first = torch.cumsum(have_t, 0) - have_t
    index = (first[:, None] + at).clamp_(max=taken + need + spare - 1)
    table = torch.where(at < have_t[:, None], pool[index], torch.full((), -1, dtype=torch.int32, device="cuda"))
    off = np.concatenate([[0], np.cumsum(new)])
    return {"case": case, "new_off": torch.from_numpy(off).cuda(), "n_new": int(off[-1]),
            "cached": torch.from_numpy(cached.astype(np.int32)).cuda(),
            "free": pool[taken:].clone(), "table": table, "block": bs,
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    return {"embed": _prepare_embed, "grad": _prepare_embed, "logits": _prepare_logits,
            "blocks": _prepare_blocks}[case["op"]](case, gen, rng)


# ---------------------------------------------------------------- plain forms
def _plain_embed(s):
    x = s["weight"][s["ids"].long()].float() * s["scale"]
    if s["pad"] >= 0:
        x = x * (s["ids"] != s["pad"]).float()[:, None]
    return x.to(DTYPES[s["case"]["out"]])


def _plain_grad(s):
    dy = s["grad"].float()
    if s["pad"] >= 0:
        dy = dy * (s["ids"] != s["pad"]).float()[:, None]
    g = torch.zeros(s["case"]["vocab"], s["case"]["width"], device=dy.device)
    g.index_add_(0, s["ids"].long(), dy)
    return (g * s["scale"]).to(DTYPES[s["case"]["out"]])


def _plain_logits(s):
    x = s["logits"].float()
    rows, vocab = x.shape
    dev = x.device
    row = torch.arange(rows, device=dev)
    # how often each token was generated, and which were seen at all
    out_ids = s["out_ids"].long()
    live = (torch.arange(out_ids.shape[1], device=dev) < s["out_len"][:, None]).float()
    count = torch.zeros(rows, vocab, device=dev).scatter_add_(1, out_ids, live)
    seen = count > 0
    made = seen
    of = torch.repeat_interleave(row, s["prompt_off"].diff(), output_size=s["prompt_ids"].numel())
    seen = seen.index_put((of, s["prompt_ids"].long()), torch.ones((), dtype=torch.bool, device=dev))
    r = s["repetition"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    x = x - (s["frequency"][:, None] * count + s["presence"][:, None] * made.float())
    if s["bias_ids"] is not None:
        of = torch.repeat_interleave(row, s["bias_off"].diff(), output_size=s["bias_ids"].numel())
        x = x.index_put((of, s["bias_ids"].long()), s["bias_values"], accumulate=True)
    if s["mask"] is not None:
        bits = (s["mask"][:, :, None] >> torch.arange(32, device=dev, dtype=torch.int32)) & 1
        allowed = bits.reshape(bits.shape[0], -1)[:, :vocab].bool()
        allowed = allowed[s["mask_row"].clamp(min=0).long()] | (s["mask_row"] < 0)[:, None]
        x = torch.where(allowed, x, torch.full((), -math.inf, device=dev))
    return x.to(DTYPES[s["case"]["out"]])


def _plain_blocks(s):
    bs, table = s["block"], s["table"]
    dev = table.device
    cached, off = s["cached"].long(), s["new_off"]
    new = off.diff()
    have = (cached + bs - 1) // bs
    want = (cached + new + bs - 1) // bs
    need = want - have
    end = torch.cumsum(need, 0)
    at = torch.arange(table.shape[1], device=dev)
    taken = s["free"][(at + (end - need - have)[:, None]).clamp(0, s["free"].numel() - 1)]
    table = torch.where((at >= have[:, None]) & (at < want[:, None]), taken, table)
    of = torch.repeat_interleave(torch.arange(new.numel(), device=dev), new, output_size=s["n_new"])
    pos = torch.arange(s["n_new"], device=dev) - off[of] + cached[of]
    slots = table[of, pos // bs].long() * bs + pos % bs
    return {"table": table, "slots": slots, "positions": pos.to(torch.int32),
            "lengths": (cached + new).to(torch.int32), "used": end[-1:]}


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        from byte_level_bpe_pretokenize_amd import lm
        s = state
        if op == "embed":
            return lm.embed(s["weight"], s["ids"], s["scale"], pad_id=s["pad"],
                            out_dtype=DTYPES[s["case"]["out"]], status=s["status"])
        if op == "grad":
            return lm.embed_grad(s["grad"], s["ids"], s["case"]["vocab"], s["scale"],
                                 pad_id=s["pad"], out_dtype=DTYPES[s["case"]["out"]],
                                 status=s["status"])
        if op == "logits":
            return lm.process_logits(
                s["logits"], prompt_ids=s["prompt_ids"], prompt_off=s["prompt_off"],
                out_ids=s["out_ids"], out_len=s["out_len"], repetition=s["repetition"],
                frequency=s["frequency"], presence=s["presence"], bias_off=s["bias_off"],
                bias_ids=s["bias_ids"], bias_values=s["bias_values"], mask=s["mask"],
                mask_row=s["mask_row"], out_dtype=DTYPES[s["case"]["out"]], status=s["status"])
        slots, positions, lengths, used = lm.block_tables(
            s["new_off"], s["n_new"], s["cached"], s["free"], s["table"], s["block"],
            status=s["status"])
        return {"table": s["table"], "slots": slots, "positions": positions, "lengths": lengths,
                "used": used}
    return {"embed": _plain_embed, "grad": _plain_grad, "logits": _plain_logits,
            "blocks": _plain_blocks}[op](state)


# ---------------------------------------------------------------- floors
def work(case):
    if case["op"] in ("embed", "grad"):
        n, vocab, width = case["ids"], case["vocab"], case["width"]
        if case["op"] == "grad":
            return {"bytes": 4 * n + n * width * SIZE[case["grad"]] + vocab * width * SIZE[case["out"]],
                    "flops": n * width + vocab * width}
        # the rows that n draws of the ID distribution are expected to touch
        k = np.arange(1, vocab + 1, dtype=np.float64)
        p = np.log1p(1.0 / k) / math.log(vocab + 1.0)
        rows = float(np.sum(-np.expm1(n * np.log1p(-p))))
        return {"bytes": int(4 * n + rows * width * SIZE[case["weight"]] + n * width * SIZE[case["out"]]),
                "flops": n * width}
    if case["op"] == "logits":
        cells = case["rows"] * case["vocab"]
        return {"bytes": int(cells * (SIZE[case["logits"]] + SIZE[case["out"]])
                             + 4 * case["rows"] * (case["prompt"] + case["made"] / 2)
                             + 8 * case["rows"] * case["bias"] / 2 + case["masks"] * case["vocab"] / 8),
                "flops": 2 * cells}
    n = case["requests"] * case["new"]
    blocks = case["requests"] * max(1.0 / case["block"], case["new"] / case["block"])
    return {"bytes": int(n * 12 + case["requests"] * 20 + 8 * blocks), "flops": 4 * n}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embed":
        w = s["weight"].double().mul_(s["scale"])
        if s["pad"] >= 0:
            w[s["pad"]] = 0.0
        return torch.index_select(w, 0, s["ids"])
    if case["op"] == "grad":
        # sorted tokens: each row is the difference of two running sums
        ids, order = torch.sort(s["ids"].long())
        edge = torch.searchsorted(ids, torch.arange(case["vocab"] + 1, device="cuda"))
        out = torch.empty(case["vocab"], case["width"], device="cuda", dtype=torch.float64)
        for c in range(0, case["width"], 256):
            part = s["grad"][:, c:c + 256].double()[order]
            total = torch.zeros(part.shape[0] + 1, part.shape[1], device="cuda", dtype=torch.float64)
            torch.cumsum(part, 0, out=total[1:])
            out[:, c:c + 256] = (total[edge[1:]] - total[edge[:-1]]) * s["scale"]
        if s["pad"] >= 0:
            out[s["pad"]] = 0.0
        return out
    if case["op"] == "logits":
        vocab = case["vocab"]
        out = s["logits"].double()
        poff = s["prompt_off"].tolist()
        made = s["out_len"].tolist()
        boff = s["bias_off"].tolist() if s["bias_off"] is not None else None
        mrow = s["mask_row"].tolist() if s["mask_row"] is not None else None
        place = torch.arange(vocab, device="cuda")
        for b in range(case["rows"]):
            x = out[b]
            count = torch.bincount(s["out_ids"][b, :made[b]].long(), minlength=vocab).double()
            prompt = torch.bincount(s["prompt_ids"][poff[b]:poff[b + 1]].long(), minlength=vocab)
            r, f, p = (s[k][b].double() for k in ("repetition", "frequency", "presence"))
            hit = torch.nonzero((prompt > 0) | (count > 0)).flatten()
            v = x[hit]
            x[hit] = torch.clamp(v, min=0) / r + torch.clamp(v, max=0) * r
            x -= f * count
            x[count > 0] -= p
            if boff is not None and boff[b + 1] > boff[b]:
                t = s["bias_ids"][boff[b]:boff[b + 1]].long()
                x[t] += s["bias_values"][boff[b]:boff[b + 1]].double()
            if mrow is not None and mrow[b] >= 0:
                word = s["mask"][mrow[b]].long()[place // 32]
                x[(word >> (place % 32)) % 2 == 0] = -math.inf
        return out
    return None  # whole numbers, the same in any precision
