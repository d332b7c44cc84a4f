"""ctypes declarations for libbpe.so (the C ABI in include/bpe.h)."""
from __future__ import annotations

import ctypes as C
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libbpe.so")

# every symbol include/bpe.h declares
SYMBOLS = (
    "bpe_load_merges", "bpe_parse_merges_text", "bpe_parse_vocab_json", "bpe_train",
    "bpe_free", "bpe_vocab_size", "bpe_max_token_bytes",
    "bpe_encode_workspace_bytes", "bpe_encode_batch", "bpe_encode_batch_noalloc",
    "bpe_encode_special_workspace_bytes", "bpe_encode_batch_special",
    "bpe_decode_workspace_bytes", "bpe_decode_batch", "bpe_decode_batch_special",
    "bpe_stage_timing", "bpe_stage_count", "bpe_stage_name", "bpe_stage_times",
    "bpe_strerror",
)

# every symbol include/bpe_lm.h declares
LM_SYMBOLS = (
    "bpe_embed_workspace_bytes", "bpe_embed", "bpe_embed_grad_workspace_bytes", "bpe_embed_grad", "bpe_process_logits",
    "bpe_block_tables_workspace_bytes", "bpe_block_tables", "bpe_cache_write", "bpe_cache_read",
    "bpe_verify_drafts_workspace_bytes", "bpe_verify_drafts", "bpe_distill", "bpe_distill_grad",
)

BPE_OK, BPE_EINVAL, BPE_EMERGES, BPE_EIDMAP, BPE_EWORKSPACE, BPE_EHIP, BPE_ENOMEM, BPE_ENOTSUP, \
    BPE_EFORMAT, BPE_ESCRATCH = 0, -1, -2, -3, -4, -5, -6, -7, -8, -9
NOALLOC_SCRATCH_BYTES = 128 << 20
STATUS_BAD_DOC_OFFSETS, STATUS_IDS_CAPACITY, STATUS_BAD_ID, STATUS_BYTES_CAPACITY, \
    STATUS_BAD_ID_OFFSETS = 1, 2, 4, 8, 16
STATUS_NO_BLOCKS, STATUS_TABLE_FULL, STATUS_BAD_LENGTH, STATUS_BAD_MASK_ROW, STATUS_BAD_BIAS = \
    32, 64, 128, 256, 512
STATUS_BAD_SLOT, STATUS_NOT_FINITE, STATUS_NO_TOKEN = 1024, 2048, 4096
F32, BF16, F16 = 0, 1, 2
E4M3, INT8, UINT4 = 0, 1, 2
MAX_WIDTH = 1 << 17
MAX_ROWS = 1 << 26
MAX_HEADS = MAX_DIM = MAX_TOP = 1024
OP_ENCODE, OP_DECODE = 0, 1
MAX_MERGES = 1 << 20
MAX_ID = (1 << 24) - 1



class LogitsArgs(C.Structure):
    """bpe_logits_args of include/bpe_lm.h."""
    _fields_ = [
        ("logits", C.c_void_p), ("logits_stride", C.c_int64),
        ("rows", C.c_int64), ("vocab", C.c_int64),
        ("prompt_ids", C.c_void_p), ("n_prompt", C.c_int64), ("prompt_off", C.c_void_p),
        ("made_ids", C.c_void_p), ("made_width", C.c_int64), ("made_stride", C.c_int64),
        ("made_len", C.c_void_p),
        ("repetition", C.c_void_p), ("frequency", C.c_void_p), ("presence", C.c_void_p),
        ("bias_ids", C.c_void_p), ("bias_values", C.c_void_p), ("n_bias", C.c_int64),
        ("bias_off", C.c_void_p),
        ("mask", C.c_void_p), ("n_masks", C.c_int64), ("mask_stride", C.c_int64),
        ("mask_row", C.c_void_p),
        ("out", C.c_void_p), ("out_stride", C.c_int64), ("status", C.c_void_p),
        ("logits_type", C.c_int32), ("out_type", C.c_int32),
    ]


class Cache(C.Structure):
    """bpe_cache of include/bpe_lm.h."""
    _fields_ = [
        ("codes", C.c_void_p), ("scales", C.c_void_p),
        ("n_slots", C.c_int64), ("codes_stride", C.c_int64), ("scales_stride", C.c_int64),
        ("heads", C.c_int32), ("dim", C.c_int32), ("group", C.c_int32), ("format", C.c_int32),
    ]


_lib = None


def load() -> C.CDLL:
    """Load the in-tree libbpe.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m byte_level_bpe_pretokenize_amd.build`")
    L = C.CDLL(LIB_PATH)
    p, i64, i32, sz = C.c_void_p, C.c_int64, C.c_int, C.c_size_t
    L.bpe_load_merges.argtypes = [p, i64, p, p, C.POINTER(p)]
    L.bpe_load_merges.restype = i32
    L.bpe_parse_merges_text.argtypes = [p, i64, p, i64, C.POINTER(C.c_int64)]
    L.bpe_parse_merges_text.restype = i32
    L.bpe_parse_vocab_json.argtypes = [p, i64, p, i64, p]
    L.bpe_parse_vocab_json.restype = i32
    L.bpe_train.argtypes = [p, i64, p, i64, i64, p, p, C.POINTER(C.c_int64), p]
    L.bpe_train.restype = i32
    L.bpe_free.argtypes = [p]
    L.bpe_free.restype = None
    L.bpe_vocab_size.argtypes = [p]
    L.bpe_vocab_size.restype = i64
    L.bpe_max_token_bytes.argtypes = [p]
    L.bpe_max_token_bytes.restype = i64
    L.bpe_encode_workspace_bytes.argtypes = [p, i64, i64]
    L.bpe_encode_workspace_bytes.restype = sz
    L.bpe_encode_batch.argtypes = [p, p, i64, p, i64, p, i64, p, p, sz, p, p]
    L.bpe_encode_batch.restype = i32
    L.bpe_encode_batch_noalloc.argtypes = [p, p, i64, p, i64, p, i64, p, p, p]
    L.bpe_encode_batch_noalloc.restype = i32
    L.bpe_encode_special_workspace_bytes.argtypes = [p, i64, i64]
    L.bpe_encode_special_workspace_bytes.restype = sz
    L.bpe_encode_batch_special.argtypes = [p, p, i64, p, i64, i32, i32, p, i64, p, p, sz, p, p]
    L.bpe_encode_batch_special.restype = i32
    L.bpe_decode_batch_special.argtypes = [p, p, i64, p, i64, i32, i32, p, i64, p, p, sz, p, p]
    L.bpe_decode_batch_special.restype = i32
    L.bpe_decode_workspace_bytes.argtypes = [p, i64, i64]
    L.bpe_decode_workspace_bytes.restype = sz
    L.bpe_decode_batch.argtypes = [p, p, i64, p, i64, p, i64, p, p, sz, p, p]
    L.bpe_decode_batch.restype = i32
    L.bpe_stage_timing.argtypes = [p, i32]
    L.bpe_stage_timing.restype = i32
    L.bpe_stage_count.argtypes = [i32]
    L.bpe_stage_count.restype = i32
    L.bpe_stage_name.argtypes = [i32, i32]
    L.bpe_stage_name.restype = C.c_char_p
    L.bpe_stage_times.argtypes = [p, i32, C.POINTER(C.c_double), i32, C.POINTER(C.c_int64)]
    L.bpe_stage_times.restype = i32
    L.bpe_strerror.argtypes = [i32]
    L.bpe_strerror.restype = C.c_char_p
    f32 = C.c_float
    L.bpe_embed_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
    L.bpe_embed_workspace_bytes.restype = sz
    L.bpe_embed.argtypes = [p, i32, i64, i64, i64, p, i64, f32, i32, p, i32, i64, p, sz, p, p]
    L.bpe_embed.restype = i32
    L.bpe_embed_grad_workspace_bytes.argtypes = [i64, i64, i64]
    L.bpe_embed_grad_workspace_bytes.restype = sz
    L.bpe_embed_grad.argtypes = [p, i32, i64, p, i64, i64, i64, f32, i32, i32, p, i32, i64, p, sz,
                                 p, p]
    L.bpe_embed_grad.restype = i32
    L.bpe_process_logits.argtypes = [C.POINTER(LogitsArgs), p]
    L.bpe_process_logits.restype = i32
    L.bpe_block_tables_workspace_bytes.argtypes = [i64, i64]
    L.bpe_block_tables_workspace_bytes.restype = sz
    L.bpe_block_tables.argtypes = [p, i64, i64, p, p, i64, p, i64, i64, i32, p, p, p, p, p, sz, p, p]
    L.bpe_block_tables.restype = i32
    L.bpe_cache_write.argtypes = [C.POINTER(Cache), p, i32, i64, i64, i64, p, p, p]
    L.bpe_cache_write.restype = i32
    L.bpe_cache_read.argtypes = [C.POINTER(Cache), p, i64, i64, i64, i32, p, p, i64, p, i32, i64, i64, p, p]
    L.bpe_cache_read.restype = i32
    L.bpe_verify_drafts_workspace_bytes.argtypes = [i64, i64]
    L.bpe_verify_drafts_workspace_bytes.restype = sz
    L.bpe_verify_drafts.argtypes = [p, i32, i64, i64, i64, p, i64, p, p, i64, p, p, p, p, p, sz, p, p]
    L.bpe_verify_drafts.restype = i32
    L.bpe_distill.argtypes = [p, i32, i64, i64, i64, p, i64, p, i32, i64, i64, f32, p, p, p, p]
    L.bpe_distill.restype = i32
    L.bpe_distill_grad.argtypes = [p, i32, i64, i64, i64, p, i64, p, i32, i64, i64, p, p, f32, p, i32, i64, p, p]
    L.bpe_distill_grad.restype = i32
    _lib = L
    return L
