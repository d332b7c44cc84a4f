"""The operators on token IDs without a GPU: the ABI of include/bpe_lm.h, and
what its host checks and the binding refuse before any HIP call."""
import ctypes as C
import os
import re

import numpy as np
import pytest
import torch

import lm_reference as ref
from byte_level_bpe_pretokenize_amd import _lib, lm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 16  # a pointer that no check follows


def header():
    return open(os.path.join(ROOT, "include", "bpe_lm.h")).read()


def test_header_and_binding_agree():
    text = re.sub(r"/\*.*?\*/", "", header(), flags=re.S)
    assert sorted(set(re.findall(r"\b(bpe_[a-z_]+)\s*\(", text))) == sorted(_lib.LM_SYMBOLS)
    L = _lib.load()
    for name in _lib.LM_SYMBOLS:
        assert hasattr(L, name), name
    fields = re.search(r"typedef struct \{(.*?)\} bpe_logits_args;", text, flags=re.S).group(1)
    names = [n.strip(" *") for line in fields.split(";") for n in line.split(",") if n.strip()]
    assert [n.split()[-1].strip("*") for n in names] == [n for n, _ in _lib.LogitsArgs._fields_]


def test_header_constants():
    for name, value in (("BPE_STATUS_NO_BLOCKS", _lib.STATUS_NO_BLOCKS),
                        ("BPE_STATUS_TABLE_FULL", _lib.STATUS_TABLE_FULL),
                        ("BPE_STATUS_BAD_LENGTH", _lib.STATUS_BAD_LENGTH),
                        ("BPE_STATUS_BAD_MASK_ROW", _lib.STATUS_BAD_MASK_ROW),
                        ("BPE_STATUS_BAD_BIAS", _lib.STATUS_BAD_BIAS),
                        ("BPE_MAX_WIDTH", f"(1 << {_lib.MAX_WIDTH.bit_length() - 1})"),
                        ("BPE_MAX_ROWS", f"((int64_t)1 << {_lib.MAX_ROWS.bit_length() - 1})"),
                        ("BPE_F32", _lib.F32), ("BPE_BF16", _lib.BF16), ("BPE_F16", _lib.F16)):
        assert re.search(rf"#define {name} {re.escape(str(value))}u?\s", header()), name


def embed_rc(weight=P, wt=0, V=100, D=64, ws=64, ids=P, n=5, scale=1.0, pad=-1, out=P, ot=0, os_=64,
             space=None, space_bytes=0, status=P):
    return _lib.load().bpe_embed(weight, wt, V, D, ws, ids, n, scale, pad, out, ot, os_, space,
                                 space_bytes, status, None)


@pytest.mark.parametrize("bad", [
    dict(weight=None), dict(ids=None), dict(out=None), dict(status=None), dict(wt=3), dict(ot=-1),
    dict(V=0), dict(V=_lib.MAX_ROWS + 1), dict(D=0), dict(D=_lib.MAX_WIDTH + 1, ws=1 << 20, os_=1 << 20),
    dict(ws=63), dict(os_=63), dict(n=-1), dict(n=(1 << 30) + 1), dict(pad=-2),
    dict(ws=(1 << 32) + 1), dict(n=1 << 30, D=1 << 17, ws=1 << 17, os_=1 << 17),
])
def test_embed_refuses(bad):
    assert embed_rc(**bad) == _lib.BPE_EINVAL


def test_embed_of_nothing():
    assert embed_rc(n=0, weight=None, ids=None, out=None) == _lib.BPE_OK


def test_embed_workspace():
    assert lm.embed_workspace_bytes(64, 128256, 4096, torch.bfloat16, torch.bfloat16) == 0
    assert lm.embed_workspace_bytes(0, 100, 64, torch.float32, torch.float32) == 0
    assert lm.embed_workspace_bytes(1 << 20, 1 << 20, 4096, torch.float32, torch.bfloat16) == 0
    big = dict(n=262144, V=32256, D=4096, ws=4096, os_=4096, ot=1)
    need = lm.embed_workspace_bytes(262144, 32256, 4096, torch.float32, torch.bfloat16)
    assert 16 * 262144 <= need <= 32 * 262144
    assert embed_rc(**big, space=P, space_bytes=need - 1) == _lib.BPE_EWORKSPACE
    assert embed_rc(**big, space=None, space_bytes=need) == _lib.BPE_EINVAL
    assert embed_rc(**big, space=P + 8, space_bytes=need) == _lib.BPE_EINVAL


def grad_rc(grad=P, gt=1, gs=64, ids=P, n=5000, V=100, D=64, scale=1.0, pad=-1, acc=0, out=P, ot=0,
            os_=64, ws=P, ws_bytes=None, status=P):
    L = _lib.load()
    need = L.bpe_embed_grad_workspace_bytes(n, V, D)
    return L.bpe_embed_grad(grad, gt, gs, ids, n, V, D, scale, pad, acc, out, ot, os_, ws,
                            need if ws_bytes is None else ws_bytes, status, None)


@pytest.mark.parametrize("bad", [
    dict(grad=None), dict(ids=None), dict(out=None), dict(status=None), dict(ws=None), dict(ws=P + 8), dict(gt=7),
    dict(ot=9), dict(V=0), dict(D=0), dict(D=_lib.MAX_WIDTH + 1, gs=1 << 20, os_=1 << 20), dict(gs=63),
    dict(os_=63), dict(n=-1), dict(pad=-2), dict(n=1 << 30, D=1 << 17, gs=1 << 17, os_=1 << 17),
])
def test_embed_grad_refuses(bad):
    assert grad_rc(**bad) == _lib.BPE_EINVAL


def test_embed_grad_workspace():
    L = _lib.load()
    assert grad_rc(ws_bytes=L.bpe_embed_grad_workspace_bytes(5000, 100, 64) - 1) == _lib.BPE_EWORKSPACE
    assert L.bpe_embed_grad_workspace_bytes(0, 100, 64) == 0
    assert L.bpe_embed_grad_workspace_bytes(10, 0, 64) == 0
    assert lm.embed_grad_workspace_bytes(3000, 100, 64) > 3000 * 16 + 100
    # the sorted lists, and at most two rows of float32 per 8 IDs
    n, V, D = 131072, 32256, 4096
    assert L.bpe_embed_grad_workspace_bytes(n, V, D) <= n * D * 4 / 4 + V + 32 * n


def logits_rc(**kw):
    a = dict(logits=P, logits_stride=100, rows=4, vocab=100, out=2 * P, out_stride=100, status=P,
             logits_type=1, out_type=0)
    a.update(kw)
    return _lib.load().bpe_process_logits(C.byref(_lib.LogitsArgs(**a)), None)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(out=None), dict(status=None), dict(rows=-1), dict(vocab=-1),
    dict(vocab=_lib.MAX_ROWS + 1, logits_stride=1 << 28, out_stride=1 << 28), dict(logits_type=3),
    dict(out_type=-1), dict(logits_stride=99), dict(out_stride=99), dict(out=P),
    dict(prompt_ids=P, n_prompt=3), dict(prompt_off=P, n_prompt=3), dict(prompt_off=P, n_prompt=-1),
    dict(made_ids=P, made_width=3, made_stride=3), dict(made_len=P, made_width=3, made_stride=3),
    dict(made_len=P, made_ids=P, made_width=3, made_stride=2),
    dict(made_len=P, made_ids=P, made_width=1 << 21, made_stride=1 << 21),
    dict(bias_ids=P, n_bias=2, bias_values=P), dict(bias_off=P, n_bias=2, bias_ids=P),
    dict(bias_off=P, n_bias=2, bias_values=P), dict(mask=P, n_masks=1, mask_stride=4),
    dict(mask_row=P, n_masks=1, mask_stride=4), dict(mask=P, mask_row=P, n_masks=1, mask_stride=3),
    dict(mask=P, mask_row=P, n_masks=-1, mask_stride=4), dict(rows=1 << 24),
])
def test_logits_refuse(bad):
    assert logits_rc(**bad) == _lib.BPE_EINVAL


def test_logits_of_nothing():
    assert logits_rc(rows=0, logits=None, out=None) == _lib.BPE_OK
    assert logits_rc(vocab=0, logits=None, out=None) == _lib.BPE_OK
    assert _lib.load().bpe_process_logits(None, None) == _lib.BPE_EINVAL


def blocks_rc(off=P, R=3, T=10, cached=P, free=P, n_free=5, table=P, W=4, stride=4, bs=16, slots=P,
              positions=P, lengths=P, used=P, ws=P, ws_bytes=1 << 20, status=P):
    return _lib.load().bpe_block_tables(off, R, T, cached, free, n_free, table, W, stride, bs, slots,
                                        positions, lengths, used, ws, ws_bytes, status, None)


@pytest.mark.parametrize("bad", [
    dict(off=None), dict(cached=None), dict(free=None), dict(table=None), dict(slots=None),
    dict(positions=None), dict(lengths=None), dict(used=None), dict(ws=None, R=5000), dict(ws=P + 4, R=5000), dict(status=None),
    dict(R=-1), dict(T=-1), dict(n_free=-1), dict(W=-1), dict(W=1 << 31, stride=1 << 31),
    dict(stride=3), dict(bs=0), dict(bs=-4), dict(R=0), dict(T=1 << 35), dict(R=(1 << 30) + 1),
])
def test_blocks_refuse(bad):
    assert blocks_rc(**bad) == _lib.BPE_EINVAL


def test_blocks_workspace():
    need = _lib.load().bpe_block_tables_workspace_bytes(5000, 10)
    assert need >= 5000 * 8
    assert blocks_rc(R=5000, ws_bytes=need - 1) == _lib.BPE_EWORKSPACE
    assert _lib.load().bpe_block_tables_workspace_bytes(0, 0) == 0


# ---- the binding: shapes and types are refused before the device is looked at ----
def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


I32, I64 = torch.int32, torch.int64


@pytest.mark.parametrize("error,call", [
    (TypeError, lambda: lm.embed(z(4, 8, dtype=torch.float64), z(3, dtype=I32))),
    (TypeError, lambda: lm.embed(z(4, 8), z(3, dtype=I64))),
    (TypeError, lambda: lm.embed(z(4, 8), z(3, dtype=I32), out_dtype=torch.int32)),
    (ValueError, lambda: lm.embed(z(4, 8, 2), z(3, dtype=I32))),
    (ValueError, lambda: lm.embed(z(8, 4).t(), z(3, dtype=I32))),
    (ValueError, lambda: lm.embed(z(4, 8), z(6, dtype=I32)[::2])),
    (ValueError, lambda: lm.embed(z(4, 8), z(3, dtype=I32), out=z(3, 7))),
    (ValueError, lambda: lm.embed(z(4, 8), z(3, dtype=I32), out=z(2, 8))),
    (ValueError, lambda: lm.embed(z(4, 8), z(3, dtype=I32), out=z(3, 8), out_dtype=torch.float16)),
    (ValueError, lambda: lm.embed(z(1, 8).expand(4, 8), z(3, dtype=I32))),
    (ValueError, lambda: lm.embed(z(4, 8), z(3, dtype=I32), pad_id=1 << 32)),
    (TypeError, lambda: lm.embed_grad(z(3, 8, dtype=I32), z(3, dtype=I32), 4)),
    (ValueError, lambda: lm.embed_grad(z(3, 8), z(4, dtype=I32), 4)),
    (ValueError, lambda: lm.embed_grad(z(2, 2, 8), z(2, 3, dtype=I32), 4)),
    (ValueError, lambda: lm.embed_grad(z(2, 8, 2).transpose(1, 2), z(2, 2, dtype=I32), 4)),
    (ValueError, lambda: lm.embed_grad(z(3, 8), z(3, dtype=I32), 4, accumulate=True)),
    (ValueError, lambda: lm.embed_grad(z(3, 8), z(3, dtype=I32), 4, out=z(5, 8))),
    (ValueError, lambda: lm.embed_grad(z(3, 8), z(3, dtype=I32), 4, workspace=z(4, 4).t())),
    (TypeError, lambda: lm.process_logits(z(2, 40, dtype=I32))),
    (ValueError, lambda: lm.process_logits(z(40))),
    (ValueError, lambda: lm.process_logits(z(2, 40), prompt_ids=z(3, dtype=I32))),
    (ValueError, lambda: lm.process_logits(z(2, 40), prompt_ids=z(3, dtype=I32), prompt_off=z(2, dtype=I64))),
    (TypeError, lambda: lm.process_logits(z(2, 40), prompt_ids=z(3, dtype=I32), prompt_off=z(3, dtype=I32))),
    (ValueError, lambda: lm.process_logits(z(2, 40), out_ids=z(2, 3, dtype=I32))),
    (ValueError, lambda: lm.process_logits(z(2, 40), out_ids=z(1, 3, dtype=I32), out_len=z(2, dtype=I32))),
    (TypeError, lambda: lm.process_logits(z(2, 40), out_ids=z(2, 3, dtype=I64), out_len=z(2, dtype=I32))),
    (ValueError, lambda: lm.process_logits(z(2, 40), repetition=z(3))),
    (TypeError, lambda: lm.process_logits(z(2, 40), presence=z(2, dtype=torch.float64))),
    (ValueError, lambda: lm.process_logits(z(2, 40), bias_ids=z(3, dtype=I32), bias_values=z(3))),
    (ValueError, lambda: lm.process_logits(z(2, 40), bias_off=z(3, dtype=I64), bias_ids=z(3, dtype=I32),
                                           bias_values=z(2))),
    (ValueError, lambda: lm.process_logits(z(2, 40), mask=z(1, 2, dtype=I32))),
    (ValueError, lambda: lm.process_logits(z(2, 40), mask=z(1, 1, dtype=I32), mask_row=z(2, dtype=I32))),
    (TypeError, lambda: lm.process_logits(z(2, 40), mask=z(1, 2), mask_row=z(2, dtype=I32))),
    (ValueError, lambda: lm.process_logits(z(2, 40), out=z(2, 41))),
    (TypeError, lambda: lm.block_tables(z(3, dtype=I32), 4, z(2, dtype=I32), z(5, dtype=I32),
                                        z(2, 3, dtype=I32), 16)),
    (ValueError, lambda: lm.block_tables(z(2, dtype=I64), 4, z(2, dtype=I32), z(5, dtype=I32),
                                         z(2, 3, dtype=I32), 16)),
    (TypeError, lambda: lm.block_tables(z(3, dtype=I64), 4, z(2, dtype=I32), z(5, dtype=I32),
                                        z(2, 3, dtype=I64), 16)),
    (ValueError, lambda: lm.block_tables(z(3, dtype=I64), 4, z(2, dtype=I32), z(5, dtype=I32),
                                         z(1, 3, dtype=I32), 16)),
    (ValueError, lambda: lm.block_tables(z(3, dtype=I64), 4, z(2, dtype=I32), z(5, dtype=I32),
                                         z(2, 3, dtype=I32), 0)),
    (ValueError, lambda: lm.block_tables(z(3, dtype=I64), -1, z(2, dtype=I32), z(5, dtype=I32),
                                         z(2, 3, dtype=I32), 16)),
    (ValueError, lambda: lm.block_tables(z(3, dtype=I64), 4, z(2, dtype=I32), z(5, dtype=I32),
                                         z(2, 3, dtype=I32), 16, slots=z(3, dtype=I64))),
])
def test_binding_refuses(error, call):
    with pytest.raises(error):
        call()


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a GPU")
def test_binding_needs_a_gpu():
    with pytest.raises(RuntimeError, match="HIP device"):
        lm.embed(z(4, 8), z(3, dtype=I32))


# ---- the divisions by multiplication that the kernels use -------------------------
@pytest.mark.parametrize("units", [1, 2, 3, 7, 125, 126, 512, 4095, 16385, 32767, 32768])
def test_division_of_vectors(units):
    """x / units = mulhi(2 x, 2^31 / units + 1) for a workgroup's x < units + 1024,
    up to the widest table's vectors of 4."""
    assert units <= (_lib.MAX_WIDTH + 3) // 4
    magic = (1 << 31) // units + 1
    x = np.arange(units + 1024, dtype=np.uint64)
    assert magic < 1 << 32 and int(x[-1]) * units < 1 << 31
    assert np.array_equal((2 * x * np.uint64(magic)) >> np.uint64(32), x // np.uint64(units))


@pytest.mark.parametrize("bs", [2, 3, 7, 16, 48, 1000, (1 << 20) - 3, (1 << 30) + 1, (1 << 31) - 1])
def test_division_by_the_block_size(bs):
    """x / bs = mulhi(x, 2^(31 + s) / bs + 1) >> (s - 1), 2^s >= bs, for x < 2^31."""
    s = (bs - 1).bit_length()
    magic = (1 << (31 + s)) // bs + 1
    assert magic < 1 << 32
    rng = np.random.default_rng(bs)
    x = np.concatenate([np.arange(5000), (1 << 31) - 1 - np.arange(5000), rng.integers(0, 1 << 31, 20000),
                        np.minimum(bs * rng.integers(0, (1 << 31) // bs + 1, 5000), (1 << 31) - 1),
                        np.clip(bs * rng.integers(0, (1 << 31) // bs + 1, 5000) - 1, 0, (1 << 31) - 1)])
    for v in x.tolist():
        assert (v * magic >> 32) >> (s - 1) == v // bs


# ---- the references against the definitions, by hand ------------------------------
def test_reference_embed_and_grad():
    w = np.arange(12.0).reshape(4, 3)
    ids = np.array([2, 0, 2, 3, 9])
    assert ref.embed(w, ids, 2.0, pad_id=3).tolist() == [[12, 14, 16], [0, 2, 4], [12, 14, 16],
                                                          [0, 0, 0], [0, 0, 0]]
    g, _ = ref.embed_grad(np.ones((5, 3)) * np.arange(1, 6)[:, None], ids, 4, 2.0, pad_id=3)
    assert g.tolist() == [[4, 4, 4], [0, 0, 0], [8, 8, 8], [0, 0, 0]]
    # the gradient against differences of sum(embed * dy)
    rng = np.random.default_rng(0)
    dy, d = rng.normal(size=(5, 3)), rng.normal(size=(4, 3))
    g, _ = ref.embed_grad(dy, ids, 4, 2.0, pad_id=3)
    diff = (ref.embed(w + d, ids, 2.0, 3) - ref.embed(w - d, ids, 2.0, 3)) / 2
    assert abs((diff * dy).sum() - (g * d).sum()) < 1e-12


def test_reference_logits():
    x = np.array([[2.0, -2.0, 4.0, 1.0, 3.0]])
    y, _ = ref.process_logits(x, prompts=[[0, 1]], made=[[2, 2, 7]], rep=[2.0], freq=[0.5], pres=[0.25],
                              bias=[{3: 10.0}], masks=np.array([[0b01111]]), mask_row=[0])
    assert y.tolist() == [[1.0, -4.0, 2.0 - 1.25, 11.0, -np.inf]]


def test_reference_blocks():
    table = np.full((2, 4), -1, np.int32)
    table[0, 0] = 7
    t, slots, pos, lens, used = ref.block_tables([0, 3, 5], [3, 0], [5, 9, 2], table, 4)
    assert t.tolist() == [[7, 5, -1, -1], [9, -1, -1, -1]]
    assert slots.tolist() == [31, 20, 21, 36, 37] and pos.tolist() == [3, 4, 5, 0, 1]
    assert lens.tolist() == [6, 2] and used == 2
