/*
 * bpe_lm.h -- operators of libbpe.so on the token IDs that bpe_encode_batch
 * writes and bpe_decode_batch reads: what a language model does with them at
 * its two ends.
 *
 *  - bpe_embed            rows of an embedding table, scaled
 *  - bpe_embed_grad       the table's gradient
 *  - bpe_process_logits   penalties for repeated tokens, biases and grammar
 *                         masks on the logits of the next token
 *  - bpe_block_tables     block tables, slots and positions of a paged cache
 *                         from the requests' lengths
 *
 * Conventions, next to those of bpe.h:
 *  - Every d_* pointer (and every pointer inside bpe_logits_args) is device
 *    memory on the current device.  Nothing is allocated and the host is
 *    never synchronized; every call is kernel launches on `hip_stream` only,
 *    so it can be captured into a graph.
 *  - Host-checkable problems return a negative BPE_E* code and enqueue
 *    nothing.  A count of zero is no problem.
 *  - *d_status (int32, device) receives BPE_STATUS_* bits for what only the
 *    device can see.  These calls do not clear it first: the bits of a chain
 *    of calls add up, so that a step of a model is checked by one read, and no
 *    call spends a launch on clearing.  The caller clears it.  Where a bit is
 *    set the outputs are as stated below, and no access leaves the caller's
 *    buffers.
 *  - Matrices are rows of `width` consecutive elements, `stride` elements
 *    apart (width <= stride <= 2^32).  A pointer need only be aligned to its
 *    element.
 *  - Sums and products are formed in float32 and rounded once, to nearest
 *    even, on the way out.  Results do not depend on scheduling: the same
 *    inputs give the same bits.
 */
#ifndef BPE_LM_H
#define BPE_LM_H

#include "bpe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types of a matrix */
#define BPE_F32 0
#define BPE_BF16 1
#define BPE_F16 2

/* bits of *d_status, next to BPE_STATUS_BAD_ID and BPE_STATUS_BAD_ID_OFFSETS */
#define BPE_STATUS_NO_BLOCKS 32u     /* more blocks needed than free_blocks holds */
#define BPE_STATUS_TABLE_FULL 64u    /* a new token lies past its request's row of the block table */
#define BPE_STATUS_BAD_LENGTH 128u   /* a negative length, or one above its bound */
#define BPE_STATUS_BAD_MASK_ROW 256u /* a mask row below -1 or not below n_masks */
#define BPE_STATUS_BAD_BIAS 512u     /* a row's bias IDs do not increase */

/* limits */
#define BPE_MAX_WIDTH (1 << 17)             /* columns of an embedding table */
#define BPE_MAX_ROWS ((int64_t)1 << 26)     /* rows of an embedding table, columns of logits */
#define BPE_MAX_IDS ((int64_t)1 << 30)      /* IDs per embedding call */

/* Workspace bytes bpe_embed needs: 0, or, for a large output of a table of a
 * wider type whose rows are read several times each, what sorting the IDs
 * takes (always 0 for n_ids <= n_rows). */
size_t bpe_embed_workspace_bytes(int64_t n_ids, int64_t n_rows, int64_t width, int weight_type,
                                 int out_type);

/*
 * out[t] = scale * weight[ids[t]], t in [0, n_ids).
 *  d_weight  [n_rows][width] of weight_type;  d_out  [n_ids][width] of out_type.
 *  pad_id    the ID that stands for no token (its rows of out are zeros), or -1.
 * An ID outside [0, n_rows) that is not pad_id gives a row of zeros and sets
 * BPE_STATUS_BAD_ID.  out must not overlap weight.  d_workspace: device
 * scratch, 16-byte aligned, of workspace_bytes >= bpe_embed_workspace_bytes of
 * the same sizes and types (NULL where that is 0).  The rows of out, in whole
 * 16-byte pieces, take at most 2^34 - 1024 pieces (256 GiB).
 * Returns BPE_OK, BPE_EINVAL, BPE_EWORKSPACE or BPE_EHIP.
 */
int bpe_embed(const void *d_weight, int weight_type, int64_t n_rows, int64_t width,
              int64_t weight_stride, const int32_t *d_ids, int64_t n_ids, float scale,
              int32_t pad_id, void *d_out, int out_type, int64_t out_stride, void *d_workspace,
              size_t workspace_bytes, int32_t *d_status, void *hip_stream);

/* Workspace bytes bpe_embed_grad needs (0 for few IDs and for sizes out of
 * range). */
size_t bpe_embed_grad_workspace_bytes(int64_t n_ids, int64_t n_rows, int64_t width);

/*
 * The gradient of bpe_embed's weight:
 *   out[v] = (accumulate ? out[v] : 0) + scale * sum over ids[t] == v of grad[t].
 *  d_grad    [n_ids][width] of grad_type: the gradient of bpe_embed's out.
 *  d_out     [n_rows][width] of out_type.  Without accumulate every row is
 *            written (zeros for an ID that does not occur); with it, rows of
 *            IDs that do not occur are neither read nor written.
 * Positions whose ID is pad_id add nothing; so do IDs outside [0, n_rows),
 * which set BPE_STATUS_BAD_ID.  Each row's terms are added in float32 in an
 * order that the IDs alone fix.  d_workspace: device scratch, 16-byte aligned,
 * of workspace_bytes >= bpe_embed_grad_workspace_bytes(n_ids, n_rows, width)
 * (NULL where that is 0).  ceil(n_ids / 256) * ceil(width / 512) < 2^24.
 * Returns BPE_OK, BPE_EINVAL, BPE_EWORKSPACE or BPE_EHIP.
 */
int bpe_embed_grad(const void *d_grad, int grad_type, int64_t grad_stride, const int32_t *d_ids,
                   int64_t n_ids, int64_t n_rows, int64_t width, float scale, int32_t pad_id,
                   int accumulate, void *d_out, int out_type, int64_t out_stride,
                   void *d_workspace, size_t workspace_bytes, int32_t *d_status,
                   void *hip_stream);

/*
 * Logits of the next token, one row per request, to processed logits.  For
 * row b and token v, with x = logits[b][v], c the number of times v occurs
 * among the row's generated IDs, and seen = c > 0 or v occurs in its prompt:
 *   seen:  x = x > 0 ? x / repetition[b] : x * repetition[b]
 *   c > 0: x = x - (frequency[b] * c + presence[b])
 *   x = x + the row's bias of v
 *   the row has a mask and v's bit in it is 0: x = -infinity, whatever x was
 * Any group may be left out (NULL): prompt, generated, each penalty (then 1,
 * 0, 0), bias, mask.
 *  logits      [rows][vocab] of logits_type;  out  [rows][vocab] of out_type;
 *              out may be logits itself (same type and stride), else they
 *              must not overlap.
 *  prompt_ids, prompt_off   int32 [n_prompt], int64 [rows + 1]: ragged, as
 *              bpe_encode_batch writes them; offsets that leave [0, n_prompt]
 *              or decrease set BPE_STATUS_BAD_ID_OFFSETS.
 *  made_ids, made_len       int32 [rows][made_width] (made_stride apart) and
 *              int32 [rows]: the first made_len[b] IDs of row b count; a
 *              length outside [0, made_width] sets BPE_STATUS_BAD_LENGTH and
 *              is taken to the nearer end.  made_width < 2^21.
 *  bias_ids, bias_values, bias_off   int32 / float [n_bias], int64 [rows + 1]:
 *              ragged; a row's IDs strictly increase, else BPE_STATUS_BAD_BIAS
 *              (and what bias its tokens get is open).
 *  mask, mask_row   uint32 [n_masks][(vocab + 31) / 32] (mask_stride apart)
 *              and int32 [rows]: bit v & 31 of word v >> 5 of row mask_row[b]
 *              lets v through; -1: no mask.  Another row number outside
 *              [0, n_masks) sets BPE_STATUS_BAD_MASK_ROW and masks nothing.
 * IDs outside [0, vocab) in any list set BPE_STATUS_BAD_ID and count for
 * nothing.  rows * ceil(vocab / 4096) < 2^24.  Returns BPE_OK, BPE_EINVAL or BPE_EHIP.
 */
typedef struct {
  const void *logits;
  int64_t logits_stride;
  int64_t rows, vocab;
  const int32_t *prompt_ids;
  int64_t n_prompt;
  const int64_t *prompt_off;
  const int32_t *made_ids;
  int64_t made_width, made_stride;
  const int32_t *made_len;
  const float *repetition, *frequency, *presence;
  const int32_t *bias_ids;
  const float *bias_values;
  int64_t n_bias;
  const int64_t *bias_off;
  const uint32_t *mask;
  int64_t n_masks, mask_stride;
  const int32_t *mask_row;
  void *out;
  int64_t out_stride;
  int32_t *status;
  int32_t logits_type, out_type;
} bpe_logits_args;

int bpe_process_logits(const bpe_logits_args *args, void *hip_stream);

/* Workspace bytes bpe_block_tables needs (0 for few requests: d_workspace may
 * then be NULL; 8-byte aligned otherwise). */
size_t bpe_block_tables_workspace_bytes(int64_t n_requests, int64_t n_new);

/*
 * Places the new tokens of a batch of requests in a paged cache of blocks of
 * block_size tokens.  Request r has cached[r] tokens in the cache, in the
 * blocks table[r][0 .. have_r), have_r = ceil(cached[r] / block_size), and
 * gets the new tokens [new_off[r], new_off[r + 1]) of the packed batch (the
 * id_off of bpe_encode_batch).  Blocks are taken from free_blocks in order,
 * request by request: with need_r = ceil((cached[r] + new_r) / block_size) -
 * have_r and first_r = need_0 + ... + need_{r-1},
 *   table[r][have_r + j] = free_blocks[first_r + j], 0 <= j < need_r
 *   positions[t] = cached[r] + t - new_off[r]
 *   slots[t] = table[r][positions[t] / block_size] * block_size
 *              + positions[t] % block_size     (int64)
 *   lengths[r] = cached[r] + new_r
 *   used[0] = need_0 + ... + need_{R-1}        (int64)
 * Other entries of the table are not written.  Afterwards the caller drops the
 * first used[0] blocks of free_blocks.
 *  d_table   int32 [n_requests][table_width], table_stride apart, in place.
 *  n_new     the number of new tokens; offsets that are not 0 = new_off[0] <=
 *            ... <= new_off[R] = n_new set BPE_STATUS_BAD_ID_OFFSETS, and the
 *            outputs are not valid.
 * Past the last free block (BPE_STATUS_NO_BLOCKS) table entries and slots are
 * -1; used[0] still counts what is needed.  New tokens past table_width blocks
 * (BPE_STATUS_TABLE_FULL) get slot -1; a request without new tokens is not
 * held against the table's width.  A negative cached length or a length
 * above INT32_MAX sets BPE_STATUS_BAD_LENGTH: the former counts as 0, and
 * tokens past the latter get slot and position -1.  A token in a block whose
 * table entry is negative gets slot -1.
 * n_requests <= 2^30, n_new <= 2^34 - 2048.
 * Returns BPE_OK, BPE_EINVAL, BPE_EWORKSPACE or BPE_EHIP.
 */
int bpe_block_tables(const int64_t *d_new_off, int64_t n_requests, int64_t n_new,
                     const int32_t *d_cached, const int32_t *d_free_blocks, int64_t n_free,
                     int32_t *d_table, int64_t table_width, int64_t table_stride,
                     int32_t block_size, int64_t *d_slots, int32_t *d_positions,
                     int32_t *d_lengths, int64_t *d_used, void *d_workspace,
                     size_t workspace_bytes, int32_t *d_status, void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* BPE_LM_H */
