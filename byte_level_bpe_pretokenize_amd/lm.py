"""Operators on token IDs at the two ends of a language model, over the C ABI
in include/bpe_lm.h (argument marshalling only).

``embed`` / ``embed_grad`` / ``embedding``: rows of an embedding table by the
IDs that ``Model.encode_batch`` gives, scaled, and the table's gradient.
``process_logits``: penalties for repeated tokens, biases and grammar masks on
the logits of the next token.  ``block_tables``: block tables, slots and
positions of a paged cache from the requests' lengths.

Every call takes ``status``, an int32 device tensor of one element that the
caller has cleared: the call ORs _lib.STATUS_* bits into it and does not
synchronize.  Without one the call makes its own, waits for it, and raises
where a bit is set (so a call that is captured into a graph needs one).  Work
goes to ``stream``, or the current stream.

Only ``embedding`` takes part in autograd.  The other calls raise where grad
mode is on and a matrix or vector given to them requires a gradient, which
they would drop; what they write in place counts as modified.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _lib
from .api import BPEError

_TYPES = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16, torch.float16: _lib.F16}


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
