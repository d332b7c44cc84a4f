"""Operators on token IDs at the two ends of a language model, over the C ABI
in include/bpe_lm.h (argument marshalling only).

``embed`` / ``embed_grad`` / ``embedding``: rows of an embedding table by the
IDs that ``Model.encode_batch`` gives, scaled, and the table's gradient.
``process_logits``: penalties for repeated tokens, biases and grammar masks on
the logits of the next token.  ``block_tables``: block tables, slots and
positions of a paged cache from the requests' lengths.  ``cache_write`` /
``cache_read``: a paged cache held in 8 or 4 bits, written by those slots and
read by those tables.  ``verify_drafts``: which drafted tokens stand against the
target's probabilities, and the token drawn after them.  ``distill`` /
``distill_grad`` / ``distillation``: loss on a teacher's top logits, and its
gradient.

Every call takes ``status``, an int32 device tensor of one element that the
caller has cleared: the call ORs _lib.STATUS_* bits into it and does not
synchronize.  Without one the call makes its own, waits for it, and raises
where a bit is set (so a call that is captured into a graph needs one).  Work
goes to ``stream``, or the current stream.

Only ``embedding`` and ``distillation`` take part in autograd.  The other calls
raise where grad mode is on and a matrix or vector given to them requires a
gradient, which they would drop; what they write in place counts as modified.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib
from .api import BPEError

_TYPES = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16, torch.float16: _lib.F16}
# what a cache's codes are kept as: uint8 holds two of 4 bits
_FORMATS = {torch.float8_e4m3fn: _lib.E4M3, torch.int8: _lib.INT8, torch.uint8: _lib.UINT4}


# the current stream's handle by device index; a stream object costs 20 times
# as much, more than all the checks of a call
_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") \
    else lambda dev: torch.cuda.current_stream(dev).cuda_stream


_modified = torch.autograd.graph.increment_version

_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _type(t: torch.dtype, what: str) -> int:
    try:
        return _TYPES[t]
    except KeyError:
        raise TypeError(f"{what}: float32, bfloat16 or float16 expected, got {t}") from None


def _list(t: torch.Tensor, dtype: torch.dtype, n: int, what: str) -> int:
    """The pointer of a contiguous tensor of n entries (n < 0: of any number)."""
    if t.dtype is not dtype or not t.is_contiguous() or (n >= 0 and t.numel() != n):
        if t.dtype is not dtype:
            raise TypeError(f"{what}: {dtype} expected, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{what}: expected a contiguous tensor")
        raise ValueError(f"{what}: {n} entries expected, got {t.numel()}")
    return t.data_ptr()


def _rows(t: torch.Tensor, what: str) -> int:
    """The row stride of a matrix whose rows are consecutive elements."""
    if t.dim() == 2 and t.is_contiguous():
        return t.shape[1]
    if t.dim() != 2:
        raise ValueError(f"{what}: expected a matrix, got {t.dim()} dimensions")
    n, m = t.shape
    if m > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: expected rows of consecutive elements")
    if n > 1:
        s = t.stride(0)
        if s < m:
            raise ValueError(f"{what}: expected rows that do not overlap")
        return s
    return m


def _matrix(t: torch.Tensor, what: str):
    """(rows, columns, row stride) of such a matrix."""
    shape = t.shape
    if len(shape) == 2:
        n, m = shape
        return n, m, m if t.is_contiguous() else _rows(t, what)
    raise ValueError(f"{what}: expected a matrix, got {len(shape)} dimensions")


def _int32(x: int, lo: int, what: str) -> int:
    if not lo <= x < 1 << 31:
        raise ValueError(f"{what}: {x} is out of range")
    return int(x)


def _device(name: str, tensors) -> int:
    """The current device's index; refuses tensors that are elsewhere."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name}: expected tensors on the current device, got one on {t.device}")
    if dev < 0:
        if not torch.cuda.is_available():
            raise RuntimeError("libbpe needs a HIP device; none is visible")
        raise ValueError(f"{name}: expected tensors on the current device, got one on the host")
    if dev != _current_device():
        raise ValueError(f"{name}: expected tensors on the current device, got one on cuda:{dev}")
    return dev


def _status(status: torch.Tensor | None, dev: int) -> torch.Tensor:
    if status is None:
        return torch.zeros(1, dtype=torch.int32, device=dev)
    if status.dtype != torch.int32 or status.numel() != 1:
        raise TypeError("status: int32 tensor of one element expected")
    return status


def _end(name: str, rc: int, own: torch.Tensor | None) -> None:
    """Raises what the call refused or, where it has a status of its own, what
    the device found."""
    if rc != _lib.BPE_OK:
        raise BPEError(rc, name)
    if own is not None:
        st = int(own.item())
        if st:
            raise RuntimeError(f"{name} device status {st:#x}")


def _no_gradient(name: str, instead: str, tensors) -> None:
    """Refuses tensors whose gradient the call would drop."""
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise RuntimeError(f"{name} gives no gradient, and a tensor given to it requires one: "
                               f"{instead}under torch.no_grad(), or with detached tensors")


def _on(stream, call, tensors, *args, **kw):
    """The call with `stream` as the current stream: what it allocates belongs
    to that stream, and the tensors given to it are marked as used there, so
    that no memory freed after the call is handed out while its kernels run."""
    with torch.cuda.stream(stream):
        res = call(*args, **kw)
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    return res


def embed_workspace_bytes(n_ids: int, n_rows: int, width: int, weight_dtype: torch.dtype,
                          out_dtype: torch.dtype) -> int:
    return int(_lib.load().bpe_embed_workspace_bytes(
        n_ids, n_rows, width, _type(weight_dtype, "weight_dtype"), _type(out_dtype, "out_dtype")))


def embed(weight: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, *, pad_id: int = -1,
          out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
          workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
          stream=None) -> torch.Tensor:
    """bpe_embed: ``scale * weight[ids]``, zeros where an ID is ``pad_id``.

    weight (V, D); ids int32, contiguous, any shape; returns ids.shape + (D,)
    of ``out_dtype`` (the weight's by default), or ``out``, a matrix of
    ids.numel() rows, filled.  ``workspace``: a contiguous device tensor of
    embed_workspace_bytes bytes, allocated by the call when left out."""
    if stream is not None:
        return _on(stream, embed, (weight, ids, out, workspace, status), weight, ids, scale,
                   pad_id=pad_id, out=out, out_dtype=out_dtype, workspace=workspace, status=status)
    _no_gradient("embed", "call embedding instead, or embed ", (weight, out))
    pad_id = _int32(pad_id, -1, "pad_id")
    wt = _type(weight.dtype, "weight")
    ws = _rows(weight, "weight")
    ip = _list(ids, torch.int32, -1, "ids")
    n, (V, D) = ids.numel(), weight.shape
    if out is None:
        dt = weight.dtype if out_dtype is None else out_dtype
        ot, os_ = _type(dt, "out_dtype"), D
    else:
        ot, os_ = _type(out.dtype, "out"), _rows(out, "out")
        if tuple(out.shape) != (n, D) or out_dtype not in (None, out.dtype):
            raise ValueError(f"out: ({n}, {D}) of out_dtype expected, got {tuple(out.shape)}")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor")
    dev = _device("embed", (weight, ids, out, workspace, status))
    L = _lib.load()
    st = _status(status, dev)
    res = weight.new_empty((*ids.shape, D), dtype=dt) if out is None else out
    w_ptr, w_bytes = None, 0
    if workspace is not None:
        w_ptr, w_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif n > V:  # (fewer IDs never need one)
        w_bytes = L.bpe_embed_workspace_bytes(n, V, D, wt, ot)
        if w_bytes:
            workspace = torch.empty(w_bytes, dtype=torch.uint8, device=dev)
            w_ptr = workspace.data_ptr()
    rc = L.bpe_embed(weight.data_ptr(), wt, V, D, ws, ip, n, scale, pad_id, res.data_ptr(), ot,
                     os_, w_ptr, w_bytes, st.data_ptr(), _stream(dev))
    if out is not None:
        _modified(out)
    _end("bpe_embed", rc, st if status is None else None)
    return res


def embed_grad_workspace_bytes(n_ids: int, n_rows: int, width: int) -> int:
    return int(_lib.load().bpe_embed_grad_workspace_bytes(n_ids, n_rows, width))


def embed_grad(grad: torch.Tensor, ids: torch.Tensor, n_rows: int, scale: float = 1.0, *,
               pad_id: int = -1, out: torch.Tensor | None = None,
               out_dtype: torch.dtype | None = None, accumulate: bool = False,
               workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """bpe_embed_grad: the gradient of ``embed``'s weight, (n_rows, D).

    grad: the gradient of embed's result, ids.shape + (D,) or (ids.numel(), D);
    returns ``out`` (added to with ``accumulate``) or a new matrix of
    ``out_dtype`` (float32 by default).  ``workspace``: a contiguous device
    tensor of embed_grad_workspace_bytes bytes, allocated by the call when left
    out."""
    if stream is not None:
        return _on(stream, embed_grad, (grad, ids, out, workspace, status), grad, ids, n_rows,
                   scale, pad_id=pad_id, out=out, out_dtype=out_dtype, accumulate=accumulate,
                   workspace=workspace, status=status)
    _no_gradient("embed_grad", "call it ", (grad, out))
    pad_id = _int32(pad_id, -1, "pad_id")
    gt = _type(grad.dtype, "grad")
    ip = _list(ids, torch.int32, -1, "ids")
    n = ids.numel()
    if grad.dim() != 2:
        if grad.shape[:-1] != ids.shape:
            raise ValueError(f"grad: {tuple(ids.shape)} + (width,) expected, got {tuple(grad.shape)}")
        if not grad.is_contiguous():
            raise ValueError("grad: expected a contiguous tensor or a matrix")
        grad = grad.view(n, grad.shape[-1])
    gs, D = _rows(grad, "grad"), grad.shape[1]
    if grad.shape[0] != n:
        raise ValueError(f"grad: {n} rows expected, got {grad.shape[0]}")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        dt = torch.float32 if out_dtype is None else out_dtype
        ot, os_ = _type(dt, "out_dtype"), D
    else:
        ot, os_ = _type(out.dtype, "out"), _rows(out, "out")
        if tuple(out.shape) != (n_rows, D) or out_dtype not in (None, out.dtype):
            raise ValueError(f"out: ({n_rows}, {D}) of out_dtype expected, got {tuple(out.shape)}")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor")
    dev = _device("embed_grad", (grad, ids, out, workspace, status))
    L = _lib.load()
    st = _status(status, dev)
    res = grad.new_empty((n_rows, D), dtype=dt) if out is None else out
    if workspace is None:
        w_bytes = L.bpe_embed_grad_workspace_bytes(n, n_rows, D)
        workspace = torch.empty(w_bytes, dtype=torch.uint8, device=dev) if w_bytes else None
    else:
        w_bytes = workspace.numel() * workspace.element_size()
    rc = L.bpe_embed_grad(grad.data_ptr(), gt, gs, ip, n, n_rows, D, scale, pad_id,
                          1 if accumulate else 0, res.data_ptr(), ot, os_,
                          None if workspace is None else workspace.data_ptr(), w_bytes,
                          st.data_ptr(), _stream(dev))
    if out is not None:
        _modified(out)
    _end("bpe_embed_grad", rc, st if status is None else None)
    return res


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids, scale, pad_id, out_dtype, status):
        ctx.save_for_backward(ids)
        ctx.embed = (weight.shape[0], weight.dtype, scale, pad_id, status)
        return embed(weight, ids, scale, pad_id=pad_id, out_dtype=out_dtype, status=status)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        if not ctx.needs_input_grad[0]:
            return (None,) * 6
        (ids,) = ctx.saved_tensors
        n_rows, dtype, scale, pad_id, status = ctx.embed
        g = embed_grad(grad.contiguous(), ids, n_rows, scale, pad_id=pad_id, out_dtype=dtype,
                       status=status)
        return g, None, None, None, None, None


def embedding(weight: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, *, pad_id: int = -1,
              out_dtype: torch.dtype | None = None,
              status: torch.Tensor | None = None) -> torch.Tensor:
    """``embed`` with ``embed_grad`` as its gradient for autograd (a dense
    gradient of the weight's type), on the current stream."""
    return _Embedding.apply(weight, ids, scale, pad_id, out_dtype, status)


def process_logits(logits: torch.Tensor, *, prompt_ids: torch.Tensor | None = None,
                   prompt_off: torch.Tensor | None = None, out_ids: torch.Tensor | None = None,
                   out_len: torch.Tensor | None = None, repetition: torch.Tensor | None = None,
                   frequency: torch.Tensor | None = None, presence: torch.Tensor | None = None,
                   bias_off: torch.Tensor | None = None, bias_ids: torch.Tensor | None = None,
                   bias_values: torch.Tensor | None = None, mask: torch.Tensor | None = None,
                   mask_row: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   out_dtype: torch.dtype | None = None, status: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """bpe_process_logits: the processed logits, (B, V), of ``out_dtype`` (the
    logits' by default); ``out`` may be ``logits`` itself.

    prompt_ids, prompt_off: each row's prompt, ragged as Model.encode_batch
    gives it (int32, int64 (B + 1)).  out_ids (B, M) int32, out_len (B) int32:
    what each row has generated so far.  repetition, frequency, presence:
    float32 (B).  bias_off int64 (B + 1), bias_ids int32 (increasing within a
    row), bias_values float32.  mask (M, ceil(V / 32)) int32, bit v & 31 of word
    v >> 5 set where token v may come; mask_row (B) int32, -1 for none."""
    if stream is not None:
        kw = dict(prompt_ids=prompt_ids, prompt_off=prompt_off, out_ids=out_ids, out_len=out_len,
                  repetition=repetition, frequency=frequency, presence=presence,
                  bias_off=bias_off, bias_ids=bias_ids, bias_values=bias_values, mask=mask,
                  mask_row=mask_row, out=out, status=status)
        return _on(stream, process_logits, (logits, *kw.values()), logits, out_dtype=out_dtype, **kw)
    _no_gradient("process_logits", "call it ",
                 (logits, repetition, frequency, presence, bias_values, out))
    lt, ls = _type(logits.dtype, "logits"), _rows(logits, "logits")
    B, V = logits.shape

    pp = po = mp = ml = bo = bi = bv = kp = kr = None
    n_prompt = m_width = m_stride = n_bias = k_rows = k_stride = 0
    if prompt_off is not None and prompt_ids is not None:
        n_prompt = prompt_ids.numel()
        pp = _list(prompt_ids, torch.int32, n_prompt, "prompt_ids")
        po = _list(prompt_off, torch.int64, B + 1, "prompt_off")
    elif prompt_off is not None or prompt_ids is not None:
        raise ValueError("prompt_ids and prompt_off come together")
    if out_ids is not None and out_len is not None:
        if out_ids.dtype is not torch.int32:
            raise TypeError(f"out_ids: torch.int32 expected, got {out_ids.dtype}")
        m_stride = _rows(out_ids, "out_ids")
        m_rows, m_width = out_ids.shape
        if m_rows != B:
            raise ValueError(f"out_ids: {B} rows expected, got {m_rows}")
        mp = out_ids.data_ptr()
        ml = _list(out_len, torch.int32, B, "out_len")
    elif out_ids is not None or out_len is not None:
        raise ValueError("out_ids and out_len come together")
    if bias_off is not None and bias_ids is not None and bias_values is not None:
        n_bias = bias_ids.numel()
        bo = _list(bias_off, torch.int64, B + 1, "bias_off")
        bi = _list(bias_ids, torch.int32, n_bias, "bias_ids")
        bv = _list(bias_values, torch.float32, n_bias, "bias_values")
    elif bias_off is not None or bias_ids is not None or bias_values is not None:
        raise ValueError("bias_off, bias_ids and bias_values come together")
    if mask is not None and mask_row is not None:
        if mask.dtype is not torch.int32 and mask.dtype is not torch.uint32:
            raise TypeError(f"mask: torch.int32 expected, got {mask.dtype}")
        k_stride = _rows(mask, "mask")
        k_rows, words = mask.shape
        if words != (V + 31) // 32:
            raise ValueError(f"mask: {(V + 31) // 32} words a row expected, got {words}")
        kp = mask.data_ptr()
        kr = _list(mask_row, torch.int32, B, "mask_row")
    elif mask is not None or mask_row is not None:
        raise ValueError("mask and mask_row come together")
    rp = None if repetition is None else _list(repetition, torch.float32, B, "repetition")
    fp = None if frequency is None else _list(frequency, torch.float32, B, "frequency")
    sp = None if presence is None else _list(presence, torch.float32, B, "presence")
    if out is None:
        dt = logits.dtype if out_dtype is None else out_dtype
        ot, os_ = _type(dt, "out_dtype"), V
    else:
        ot, os_ = _type(out.dtype, "out"), _rows(out, "out")
        if out.shape != logits.shape or out_dtype not in (None, out.dtype):
            raise ValueError(f"out: {tuple(logits.shape)} of out_dtype expected, got {tuple(out.shape)}")
    dev = _device("process_logits", (logits, prompt_ids, prompt_off, out_ids, out_len, repetition,
                  frequency, presence, bias_off, bias_ids, bias_values, mask, mask_row, out, status))
    st = _status(status, dev)
    res = logits.new_empty((B, V), dtype=dt) if out is None else out
    a = _lib.LogitsArgs(logits.data_ptr(), ls, B, V, pp, n_prompt, po, mp, m_width, m_stride, ml,
                        rp, fp, sp, bi, bv, n_bias, bo, kp, k_rows, k_stride, kr, res.data_ptr(), os_, st.data_ptr(), lt, ot)
    rc = _lib.load().bpe_process_logits(C.byref(a), _stream(dev))
    if out is not None:
        _modified(out)
    _end("bpe_process_logits", rc, st if status is None else None)
    return res


def block_tables(new_off: torch.Tensor, n_new: int, cached: torch.Tensor,
                 free_blocks: torch.Tensor, table: torch.Tensor, block_size: int, *,
                 slots: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                 lengths: torch.Tensor | None = None, used: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                 stream=None):
    """bpe_block_tables: enters the blocks that the new tokens need into
    ``table`` (in place) and returns (slots int64 (n_new), positions int32
    (n_new), lengths int32 (R), used int64 (1)), new or the tensors given.

    new_off int64 (R + 1): the new tokens' offsets (Model.encode_batch's
    id_off), n_new of them; cached int32 (R): tokens already in the cache;
    free_blocks int32: the blocks to take, in order; table int32 (R, W)."""
    if stream is not None:
        kw = dict(slots=slots, positions=positions, lengths=lengths, used=used,
                  workspace=workspace, status=status)
        return _on(stream, block_tables, (new_off, cached, free_blocks, table, *kw.values()),
                   new_off, n_new, cached, free_blocks, table, block_size, **kw)
    R = cached.numel()
    op = _list(new_off, torch.int64, R + 1, "new_off")
    cp = _list(cached, torch.int32, R, "cached")
    fp = _list(free_blocks, torch.int32, -1, "free_blocks")
    if table.dtype is not torch.int32:
        raise TypeError(f"table: torch.int32 expected, got {table.dtype}")
    ts = _rows(table, "table")
    t_rows, t_width = table.shape
    if t_rows != R:
        raise ValueError(f"table: {R} rows expected, got {t_rows}")
    if slots is not None:
        _list(slots, torch.int64, n_new, "slots")
    if positions is not None:
        _list(positions, torch.int32, n_new, "positions")
    if lengths is not None:
        _list(lengths, torch.int32, R, "lengths")
    if used is not None:
        _list(used, torch.int64, 1, "used")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor")
    block_size = _int32(block_size, 1, "block_size")
    if n_new < 0:
        raise ValueError(f"n_new: {n_new} is out of range")
    dev = _device("block_tables", (new_off, cached, free_blocks, table, slots, positions, lengths,
                  used, workspace, status))
    L = _lib.load()
    st = _status(status, dev)
    filled = [table]  # the caller's tensors
    if slots is None:
        slots = new_off.new_empty(n_new)
    else:
        filled.append(slots)
    if positions is None:
        positions = cached.new_empty(n_new)
    else:
        filled.append(positions)
    if lengths is None:
        lengths = cached.new_empty(R)
    else:
        filled.append(lengths)
    if used is None:
        used = new_off.new_empty(1)
    else:
        filled.append(used)
    if workspace is None:
        w_bytes = L.bpe_block_tables_workspace_bytes(R, n_new)
        workspace = torch.empty(w_bytes, dtype=torch.uint8, device=dev) if w_bytes else None
    else:
        w_bytes = workspace.numel() * workspace.element_size()
    rc = L.bpe_block_tables(op, R, n_new, cp, fp, free_blocks.numel(), table.data_ptr(),
                            t_width, ts, block_size, slots.data_ptr(), positions.data_ptr(),
                            lengths.data_ptr(), used.data_ptr(),
                            None if workspace is None else workspace.data_ptr(), w_bytes,
                            st.data_ptr(), _stream(dev))
    _modified(filled)
    _end("bpe_block_tables", rc, st if status is None else None)
    return slots, positions, lengths, used


def empty_cache(n_slots: int, heads: int, dim: int, dtype: torch.dtype = torch.float8_e4m3fn,
                group: int | None = None, device="cuda"):
    """A cache of n_slots tokens for cache_write and cache_read, not cleared:
    (codes, scales, group).  dtype: float8_e4m3fn, int8, or uint8 for 4 bits (two
    to a byte).  group: elements per scale, a power of two from 16 to 512 (by
    default the first that holds a head, 512 at most)."""
    if dtype not in _FORMATS:
        raise TypeError(f"dtype: float8_e4m3fn, int8 or uint8 expected, got {dtype}")
    if group is None:
        group = min(512, max(16, 1 << (dim - 1).bit_length()))
    four = dtype == torch.uint8
    G = -(-dim // group)
    codes = torch.empty((n_slots, heads, (dim + 1) // 2 if four else dim), dtype=torch.uint8, device=device)
    scales = torch.empty((n_slots, heads, G, 2) if four else (n_slots, heads, G), device=device)
    return codes.view(dtype), scales, group


def _slots(t: torch.Tensor, row: int, what: str) -> int:
    """The stride of a cache's slots, each of `row` consecutive elements."""
    if t.is_contiguous():
        return row
    if t.numel() and not t[0].is_contiguous():
        raise ValueError(f"{what}: expected slots of consecutive elements")
    if t.shape[0] > 1:
        s = t.stride(0)
        if s < row:
            raise ValueError(f"{what}: expected slots that do not overlap")
        return s
    return row


def _cache(codes: torch.Tensor, scales: torch.Tensor, group: int, heads: int, dim: int):
    """bpe_cache of a cache's tensors."""
    form = _FORMATS.get(codes.dtype)
    if form is None:
        raise TypeError(f"codes: float8_e4m3fn, int8 or uint8 expected, got {codes.dtype}")
    if scales.dtype is not torch.float32:
        raise TypeError(f"scales: torch.float32 expected, got {scales.dtype}")
    # (32 bits each in bpe_cache, which ctypes would fill with what is left of more)
    if not (1 <= group < 1 << 31 and heads < 1 << 31 and dim < 1 << 31):
        _int32(group, 1, "group")
        _int32(heads, 0, "heads")
        _int32(dim, 0, "dim")
    shape, n = scales.shape, codes.shape[0]
    G = (dim + group - 1) // group
    if form == _lib.UINT4:
        width, per, want = (dim + 1) // 2, heads * G * 2, (n, heads, G, 2)
    else:
        width, per, want = dim, heads * G, (n, heads, G)
    if codes.shape != (n, heads, width):
        raise ValueError(f"codes: (slots, {heads}, {width}) expected, got {tuple(codes.shape)}")
    if shape != want:
        raise ValueError(f"scales: {want} expected, got {tuple(shape)}")
    return _lib.Cache(codes.data_ptr(), scales.data_ptr(), n, _slots(codes, heads * width, "codes"),
                      _slots(scales, per, "scales"), heads, dim, group, form)


def _tokens(t: torch.Tensor, what: str):
    """(token stride, head stride) of (n, heads, dim) whose heads are consecutive
    elements; what one token or one head has is not looked at."""
    n, H, D = t.shape
    ts, hs, es = t.stride()
    if es != 1 and D > 1:
        raise ValueError(f"{what}: expected heads of consecutive elements")
    if n > 1 and H > 1:
        fits = ts >= (H - 1) * hs + D and hs >= D or hs >= (n - 1) * ts + D and ts >= D
    else:
        fits = (n <= 1 or ts >= D) and (H <= 1 or hs >= D)
    if not fits:
        raise ValueError(f"{what}: expected heads that do not overlap")
    return ts, hs


def cache_write(x: torch.Tensor, slots: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                group: int, *, status: torch.Tensor | None = None, stream=None) -> None:
    """bpe_cache_write: quantises the tokens ``x`` (n, heads, dim) into ``slots``
    (int64, as block_tables gives them; -1: nowhere) of a cache, in place.

    codes (S, heads, dim) of float8_e4m3fn or int8, or (S, heads, ceil(dim / 2))
    uint8 for 4 bits; scales float32 (S, heads, ceil(dim / group)), with a last
    dimension of 2 for 4 bits (scale, lowest value).  Keys and values side by side
    are one call of twice the heads.  Slots must differ."""
    if stream is not None:
        return _on(stream, cache_write, (x, slots, codes, scales, status), x, slots, codes, scales,
                   group, status=status)
    _no_gradient("cache_write", "call it ", (x, codes, scales))
    xt = _type(x.dtype, "x")
    if x.dim() != 3:
        raise ValueError(f"x: (n, heads, dim) expected, got {x.dim()} dimensions")
    n, H, D = x.shape
    ts, hs = _tokens(x, "x")
    sp = _list(slots, torch.int64, n, "slots")
    c = _cache(codes, scales, group, H, D)
    dev = _device("cache_write", (x, slots, codes, scales, status))
    st = _status(status, dev)
    rc = _lib.load().bpe_cache_write(C.byref(c), x.data_ptr(), xt, n, ts, hs, sp, st.data_ptr(), _stream(dev))
    _modified([codes, scales])
    _end("bpe_cache_write", rc, st if status is None else None)


def cache_read(codes: torch.Tensor, scales: torch.Tensor, group: int, table: torch.Tensor,
               block_size: int, off: torch.Tensor, n: int, *, dim: int | None = None,
               start: torch.Tensor | None = None, out: torch.Tensor | None = None,
               out_dtype: torch.dtype | None = None, status: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """bpe_cache_read: the values of the requests' tokens, packed: (n, heads, dim)
    of ``out_dtype`` (bfloat16 by default), or ``out``, filled.

    codes, scales, group: a cache as cache_write takes it; table int32 (R, W), as
    block_tables keeps it, of blocks of ``block_size``; off int64 (R + 1): the
    requests' places in the packed tokens, n in all; start int32 (R): the position
    of each request's first one (0 by default).  ``dim``: a head's elements
    (needed for an odd head of 4 bits)."""
    if stream is not None:
        kw = dict(start=start, out=out, status=status)
        return _on(stream, cache_read, (codes, scales, table, off, *kw.values()), codes, scales, group,
                   table, block_size, off, n, dim=dim, out_dtype=out_dtype, **kw)
    _no_gradient("cache_read", "call it ", (codes, scales, out))
    if codes.dim() != 3:
        raise ValueError(f"codes: 3 dimensions expected, got {codes.dim()}")
    H = codes.shape[1]
    if dim is None:
        dim = out.shape[2] if out is not None and out.dim() == 3 else \
            codes.shape[2] * (2 if codes.dtype == torch.uint8 else 1)
    c = _cache(codes, scales, group, H, dim)
    if table.dtype is not torch.int32:
        raise TypeError(f"table: torch.int32 expected, got {table.dtype}")
    R, W, tstr = _matrix(table, "table")
    op = _list(off, torch.int64, R + 1, "off")
    fp = None if start is None else _list(start, torch.int32, R, "start")
    block_size = _int32(block_size, 1, "block_size")
    if n < 0:
        raise ValueError(f"n: {n} is out of range")
    if out is None:
        dt = torch.bfloat16 if out_dtype is None else out_dtype
        ot, ts, hs = _type(dt, "out_dtype"), H * dim, dim
    else:
        ot = _type(out.dtype, "out")
        if tuple(out.shape) != (n, H, dim) or out_dtype not in (None, out.dtype):
            raise ValueError(f"out: ({n}, {H}, {dim}) of out_dtype expected, got {tuple(out.shape)}")
        ts, hs = _tokens(out, "out")
    dev = _device("cache_read", (codes, scales, table, off, start, out, status))
    st = _status(status, dev)
    res = scales.new_empty(n, H, dim, dtype=dt) if out is None else out
    rc = _lib.load().bpe_cache_read(C.byref(c), table.data_ptr(), R, W, tstr, block_size, op, fp, n,
                                    res.data_ptr(), ot, ts, hs, st.data_ptr(), _stream(dev))
    if out is not None:
        _modified(out)
    _end("bpe_cache_read", rc, st if status is None else None)
    return res


def verify_drafts_workspace_bytes(n_requests: int, vocab: int) -> int:
    return int(_lib.load().bpe_verify_drafts_workspace_bytes(n_requests, vocab))


def verify_drafts(target: torch.Tensor, draft_ids: torch.Tensor, row_off: torch.Tensor,
                  accept: torch.Tensor, sample: torch.Tensor, *, draft: torch.Tensor | None = None,
                  tokens: torch.Tensor | None = None, counts: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                  stream=None):
    """bpe_verify_drafts: (tokens int32 (N), counts int32 (R)), new or the tensors
    given: each request's drafted tokens that stand and the one drawn after them,
    then -1, in its rows; and how many it got.

    target (N, V): the target's probabilities; row_off int64 (R + 1): the requests'
    rows, one more than their drafts.  draft_ids int32 (N): the token that a row
    verifies (its request's last row: anything); draft (N, V): the probabilities it
    was drawn from, None where the drafts were certain.  accept float32 (N), sample
    float32 (R): uniform in [0, 1).  ``workspace``: a contiguous device tensor of
    verify_drafts_workspace_bytes bytes, allocated by the call when left out."""
    if stream is not None:
        kw = dict(draft=draft, tokens=tokens, counts=counts, workspace=workspace, status=status)
        return _on(stream, verify_drafts, (target, draft_ids, row_off, accept, sample, *kw.values()),
                   target, draft_ids, row_off, accept, sample, **kw)
    _no_gradient("verify_drafts", "call it ", (target, draft, accept, sample))
    pt = _type(target.dtype, "target")
    N, V, ps = _matrix(target, "target")
    R = row_off.numel() - 1
    qp, qs = None, 0
    if draft is not None:
        if draft.dtype is not target.dtype:
            raise TypeError(f"draft: {target.dtype} expected, got {draft.dtype}")
        qn, qv, qs = _matrix(draft, "draft")
        if qn != N or qv != V:
            raise ValueError(f"draft: {tuple(target.shape)} expected, got {tuple(draft.shape)}")
        qp = draft.data_ptr()
    ip = _list(draft_ids, torch.int32, N, "draft_ids")
    op = _list(row_off, torch.int64, -1, "row_off")
    if R < 0:
        raise ValueError("row_off: one entry more than requests expected, got none")
    ap = _list(accept, torch.float32, N, "accept")
    sp = _list(sample, torch.float32, R, "sample")
    if tokens is not None:
        _list(tokens, torch.int32, N, "tokens")
    if counts is not None:
        _list(counts, torch.int32, R, "counts")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor")
    dev = _device("verify_drafts", (target, draft, draft_ids, row_off, accept, sample, tokens, counts,
                  workspace, status))
    L = _lib.load()
    st = _status(status, dev)
    filled = [t for t in (tokens, counts) if t is not None]
    if tokens is None:
        tokens = draft_ids.new_empty(N)
    if counts is None:
        counts = draft_ids.new_empty(R)
    if workspace is None:
        w_bytes = L.bpe_verify_drafts_workspace_bytes(R, V)
        if w_bytes:  # (a float32 tensor of the inputs' device costs less than one of bytes)
            workspace = sample.new_empty((w_bytes + 3) // 4)
    else:
        w_bytes = workspace.numel() * workspace.element_size()
    rc = L.bpe_verify_drafts(target.data_ptr(), pt, N, V, ps, qp, qs, ip, op, R, ap, sp,
                             tokens.data_ptr(), counts.data_ptr(),
                             None if workspace is None else workspace.data_ptr(), w_bytes,
                             st.data_ptr(), _stream(dev))
    if filled:
        _modified(filled)
    _end("bpe_verify_drafts", rc, st if status is None else None)
    return tokens, counts


def _teacher(student, ids, teacher):
    """What a student's and a teacher's rows are passed as."""
    N, V, zs = _matrix(student, "student")
    n, K, is_ = _matrix(ids, "ids")
    tn, tk, ts = _matrix(teacher, "teacher")
    if ids.dtype is not torch.int32:
        raise TypeError(f"ids: torch.int32 expected, got {ids.dtype}")
    if n != N or tn != N or tk != K:
        raise ValueError(f"ids, teacher: {N} rows of the same width expected, got {tuple(ids.shape)} "
                         f"and {tuple(teacher.shape)}")
    return (student.data_ptr(), _type(student.dtype, "student"), N, V, zs, ids.data_ptr(), is_,
            teacher.data_ptr(), _type(teacher.dtype, "teacher"), ts, K)


def distill(student: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor, temperature: float = 1.0,
            *, losses: torch.Tensor | None = None, stats: torch.Tensor | None = None,
            status: torch.Tensor | None = None, stream=None):
    """bpe_distill: (losses float32 (N), stats float32 (N, 4)), new or the tensors
    given: temperature^2 times the divergence of the student's distribution from
    the teacher's over its listed tokens, and what distill_grad needs.

    student (N, V): logits; ids int32 (N, K): the teacher's top tokens, -1 for
    none; teacher (N, K): their logits."""
    if stream is not None:
        kw = dict(losses=losses, stats=stats, status=status)
        return _on(stream, distill, (student, ids, teacher, *kw.values()), student, ids, teacher,
                   temperature, **kw)
    _no_gradient("distill", "call distillation instead, or distill ", (student, teacher, losses, stats))
    a = _teacher(student, ids, teacher)
    N = a[2]
    if losses is not None:
        _list(losses, torch.float32, N, "losses")
    if stats is not None:
        _list(stats, torch.float32, N * 4, "stats")
    dev = _device("distill", (student, ids, teacher, losses, stats, status))
    st = _status(status, dev)
    filled = [t for t in (losses, stats) if t is not None]
    if losses is None:
        losses = student.new_empty(N, dtype=torch.float32)
    if stats is None:
        stats = student.new_empty(N, 4, dtype=torch.float32)
    rc = _lib.load().bpe_distill(*a, temperature, losses.data_ptr(), stats.data_ptr(), st.data_ptr(),
                                 _stream(dev))
    if filled:
        _modified(filled)
    _end("bpe_distill", rc, st if status is None else None)
    return losses, stats


def distill_grad(student: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor, stats: torch.Tensor,
                 dloss: torch.Tensor, temperature: float = 1.0, *, out: torch.Tensor | None = None,
                 out_dtype: torch.dtype | None = None, status: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """bpe_distill_grad: the gradient of ``distill``'s losses, weighted by ``dloss``
    float32 (N), with respect to the student's logits: (N, V) of ``out_dtype`` (the
    student's by default), or ``out``, which may be the student itself, filled.
    stats: what distill gave for the same inputs."""
    if stream is not None:
        kw = dict(out=out, status=status)
        return _on(stream, distill_grad, (student, ids, teacher, stats, dloss, *kw.values()), student,
                   ids, teacher, stats, dloss, temperature, out_dtype=out_dtype, **kw)
    _no_gradient("distill_grad", "call it ", (student, teacher, stats, dloss, out))
    a = _teacher(student, ids, teacher)
    N, V = a[2:4]
    sp = _list(stats, torch.float32, N * 4, "stats")
    dp = _list(dloss, torch.float32, N, "dloss")
    if out is None:
        dt = student.dtype if out_dtype is None else out_dtype
        ot, os_ = _type(dt, "out_dtype"), V
    else:
        ot, os_ = _type(out.dtype, "out"), _rows(out, "out")
        if out.shape != student.shape or out_dtype not in (None, out.dtype):
            raise ValueError(f"out: {tuple(student.shape)} of out_dtype expected, got {tuple(out.shape)}")
    dev = _device("distill_grad", (student, ids, teacher, stats, dloss, out, status))
    st = _status(status, dev)
    res = student.new_empty(N, V, dtype=dt) if out is None else out
    rc = _lib.load().bpe_distill_grad(*a, sp, dp, temperature, res.data_ptr(), ot, os_, st.data_ptr(),
                                      _stream(dev))
    if out is not None:
        _modified(out)
    _end("bpe_distill_grad", rc, st if status is None else None)
    return res


class _Distillation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, student, ids, teacher, temperature, status):
        losses, stats = distill(student, ids, teacher, temperature, status=status)
        ctx.save_for_backward(student, ids, teacher, stats)
        ctx.distill = (temperature, status)
        return losses

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss):
        if not ctx.needs_input_grad[0]:
            return (None,) * 5
        student, ids, teacher, stats = ctx.saved_tensors
        temperature, status = ctx.distill
        g = distill_grad(student, ids, teacher, stats, dloss.contiguous(), temperature, status=status)
        return g, None, None, None, None


def distillation(student: torch.Tensor, ids: torch.Tensor, teacher: torch.Tensor,
                 temperature: float = 1.0, *, status: torch.Tensor | None = None) -> torch.Tensor:
    """``distill``'s losses with ``distill_grad`` as their gradient for autograd, on
    the current stream.  The teacher gets no gradient."""
    if teacher.requires_grad and torch.is_grad_enabled():
        raise RuntimeError("distillation gives no gradient to the teacher, which requires one: detach it")
    return _Distillation.apply(student, ids, teacher, temperature, status)
