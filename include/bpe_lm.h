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
 *  - bpe_cache_write,     a paged cache held in 8 or 4 bits: written by those
 *    bpe_cache_read       slots, read back by those tables
 *  - bpe_verify_drafts    which drafted tokens stand against the target's
 *                         probabilities, and the token drawn after them
 *  - bpe_distill,         loss on a teacher's top logits, and its gradient
 *    bpe_distill_grad
 *
 * Conventions, next to those of bpe.h:
 *  - Every d_* pointer (and every pointer inside bpe_logits_args and
 *    bpe_cache) is device memory on the current device.  Nothing is allocated
 *    and the host is never synchronized; every call is kernel launches on
 *    `hip_stream` only, so it can be captured into a graph.
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
 *    inputs give the same bits (but for what is called open below).
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

/* what a cache holds an element in */
#define BPE_E4M3 0 /* 8 bits: sign, 4 of exponent, 3 of mantissa, no infinities (largest 448) */
#define BPE_INT8 1 /* 8 bits: -127 to 127 */
#define BPE_UINT4 2 /* 4 bits: 0 to 15, element 2 i in the lower half of byte i */

/* bits of *d_status, next to BPE_STATUS_BAD_ID and BPE_STATUS_BAD_ID_OFFSETS */
#define BPE_STATUS_NO_BLOCKS 32u     /* more blocks needed than free_blocks holds */
#define BPE_STATUS_TABLE_FULL 64u    /* a new token lies past its request's row of the block table */
#define BPE_STATUS_BAD_LENGTH 128u   /* a negative length, or one above its bound */
#define BPE_STATUS_BAD_MASK_ROW 256u /* a mask row below -1 or not below n_masks */
#define BPE_STATUS_BAD_BIAS 512u     /* a row's bias IDs do not increase */
#define BPE_STATUS_BAD_SLOT 1024u    /* a slot or block past the cache's end, or a slot below -1 */
#define BPE_STATUS_NOT_FINITE 2048u  /* an infinity or NaN among the values to be held */
#define BPE_STATUS_NO_TOKEN 4096u    /* a row to draw from has no positive probability */

/* limits */
#define BPE_MAX_WIDTH (1 << 17)             /* columns of an embedding table */
#define BPE_MAX_ROWS ((int64_t)1 << 26)     /* rows of an embedding table, columns of logits */
#define BPE_MAX_IDS ((int64_t)1 << 30)      /* IDs per embedding call */
#define BPE_MAX_HEADS 1024                  /* heads of a cached token */
#define BPE_MAX_DIM 1024                    /* elements of a head */
#define BPE_MAX_TOP 1024                    /* entries of a teacher's row */

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

/*
 * A paged cache of n_slots tokens, each of `heads` heads of `dim` elements (keys
 * and values side by side are twice the heads).  A head's elements are held in
 * groups of `group` (a power of two from 16 to 512; the last one of a head may
 * be shorter), each with a scale of its own; G = ceil(dim / group).
 *  codes   [n_slots][heads][dim] bytes, or [n_slots][heads][(dim + 1) / 2] of
 *          BPE_UINT4 (the free half of an odd head's last byte is 0); slots
 *          are codes_stride bytes apart.
 *  scales  float [n_slots][heads][G], or [n_slots][heads][G][2] of BPE_UINT4:
 *          the scale and the lowest value; slots are scales_stride floats apart.
 *          An element's value is code * scale (BPE_UINT4: + the lowest value).
 * A pointer need only be aligned to its element.  n_slots <= 2^40, codes_stride
 * <= 2^22, scales_stride <= 2^20.
 */
typedef struct {
  void *codes;
  float *scales;
  int64_t n_slots, codes_stride, scales_stride;
  int32_t heads, dim, group, format;
} bpe_cache;

/*
 * Quantises tokens into their slots.
 *  d_x      [n][heads][dim] of x_type; tokens are token_stride elements apart,
 *           heads head_stride, each at most 2^32: token by token (token_stride
 *           >= (heads - 1) * head_stride + dim) or head by head (head_stride >=
 *           (n - 1) * token_stride + dim).
 *  d_slots  int64 [n]: where each token goes, as bpe_block_tables gives it.  -1:
 *           nowhere.  One outside [-1, n_slots) sets BPE_STATUS_BAD_SLOT and
 *           goes nowhere.  Other slots keep what they hold.  Where two tokens
 *           have the same slot, what it holds afterwards is open.
 * With a the largest magnitude of a group, in float32:
 *   BPE_E4M3   scale = a * (1 / 448)     code = e4m3(x * (1 / scale))
 *   BPE_INT8   scale = a * (1 / 127)     code = round(x * (1 / scale))
 *   BPE_UINT4  scale = (highest - lowest) * (1 / 15)
 *                                        code = round((x - lowest) * (1 / scale))
 * with 1 / 448, 1 / 127, 1 / 15 and 1 / scale rounded to float32, codes rounded
 * to nearest even and kept within the format's range.  A scale below 2^-120 is
 * held as 0, with codes of 0.  Infinities and NaN set BPE_STATUS_NOT_FINITE and
 * do not count for the scale: infinities get the format's ends (codes 127 and
 * -127, 448 and -448, 15 and 0), NaN gets code 0, and a group without a finite
 * element has scale (and lowest value) 0.  BPE_UINT4 takes magnitudes above
 * 2^126 as 2^126, so that a group's width stays finite.
 * n <= 2^30 - 64, n * heads * ceil(dim / group) * group < 2^36.
 * Returns BPE_OK, BPE_EINVAL or BPE_EHIP.
 */
int bpe_cache_write(const bpe_cache *cache, const void *d_x, int x_type, int64_t n,
                    int64_t token_stride, int64_t head_stride, const int64_t *d_slots,
                    int32_t *d_status, void *hip_stream);

/*
 * Reads the requests' tokens back, packed: for t in [off[r], off[r + 1])
 *   out[t] = the values of slot table[r][p / block_size] * block_size + p % block_size,
 *   p = start[r] + t - off[r]
 * formed in float32, with at most one rounding there, and rounded once to
 * out_type.
 *  d_off    int64 [n_requests + 1]: increasing, within [0, n]; offsets that are
 *           not set BPE_STATUS_BAD_ID_OFFSETS, and which tokens are read is
 *           open.  Rows of out outside [off[0], off[n_requests]) are left as
 *           they were.
 *  d_start  int32 [n_requests]: the position of each request's first token to
 *           be read; NULL: 0.  A negative one sets BPE_STATUS_BAD_LENGTH and
 *           counts as 0.
 *  d_table  int32 [n_requests][table_width], table_stride apart, as
 *           bpe_block_tables keeps it.  A token in a block whose entry is
 *           negative is read as zeros; so are tokens past table_width blocks
 *           (BPE_STATUS_TABLE_FULL), past slot n_slots (BPE_STATUS_BAD_SLOT) and
 *           past position INT32_MAX (BPE_STATUS_BAD_LENGTH).
 *  d_out    [n][heads][dim] of out_type, strides as those of d_x.
 * Without tokens or requests (n or n_requests 0) nothing is launched, and what is
 * wrong with the offsets or starts then is not looked for.
 * n <= 2^30 - 64, n * heads * ceil(dim / 8) < 2^33 (float32 of dim a multiple of
 * 4: dim / 4), n_requests <= 2^30.
 * Returns BPE_OK, BPE_EINVAL or BPE_EHIP.
 */
int bpe_cache_read(const bpe_cache *cache, const int32_t *d_table, int64_t n_requests,
                   int64_t table_width, int64_t table_stride, int32_t block_size,
                   const int64_t *d_off, const int32_t *d_start, int64_t n, void *d_out,
                   int out_type, int64_t token_stride, int64_t head_stride, int32_t *d_status,
                   void *hip_stream);

/* Workspace bytes bpe_verify_drafts needs (0 for small vocabularies, for few
 * requests in larger ones, and for sizes out of range). */
size_t bpe_verify_drafts_workspace_bytes(int64_t n_requests, int64_t vocab);

/*
 * Which of a request's drafted tokens stand, and the token that follows them, so
 * that what comes out is distributed as the target alone would draw it.
 * Request r has the rows i in [row_off[r], row_off[r + 1]) of the target's
 * probabilities p; each row but its last verifies the drafted token
 * x_i = draft_ids[i], which was drawn from row i of the draft's probabilities q:
 *   x_i stands if those before it do and accept[i] * q_i[x_i] < p_i[x_i]
 * With j the first row that does not stand (the last row if all drafts do), the
 * next token is drawn from w = max(p_j - q_j, 0) after a draft that does not
 * stand (from p_j if that leaves nothing), from w = p_j at the last row:
 *   the lowest v with w[0] + ... + w[v] > sample[r] * (w[0] + ... + w[V - 1])
 * Comparisons and sums are in 64 bits.  A request of one row has no draft.
 *  tokens   int32 [n_rows]: in a request's rows its drafts that stand, the next
 *           token, then -1.  Rows that are no request's are left as they were.
 *           May be draft_ids itself.
 *  counts   int32 [n_requests]: how many tokens it got (0 without rows).
 *  d_target, d_draft   [n_rows][vocab] of prob_type, rows target_stride and
 *           draft_stride apart.  Rows need not add up to 1.  Negative entries,
 *           infinities and NaN count as 0.  Row j alone is read whole; a
 *           request's last row of d_draft is never read.  d_draft NULL: the
 *           drafts were certain (q is 1 at x_i and 0 elsewhere).
 *  accept, sample      float [n_rows], [n_requests], uniform in [0, 1).  An accept
 *           outside is compared as it is.  Below 0: a token with q > 0 stands
 *           whatever p is, one with q = 0 (what counts as 0 included) if p > 0, or
 *           not at all for -infinity, whose product with 0 is NaN.  NaN: none
 *           stands.  A sample outside takes the nearer end (NaN the upper).
 * A drafted token outside [0, vocab) that comes to be looked at sets
 * BPE_STATUS_BAD_ID and does not stand.  Offsets that decrease or leave
 * [0, n_rows] set BPE_STATUS_BAD_ID_OFFSETS, and their request counts as one
 * without rows.  Where there is nothing to draw from
 * (BPE_STATUS_NO_TOKEN) the next token is -1 and not counted.
 * d_workspace: device scratch, 8-byte aligned, of workspace_bytes >=
 * bpe_verify_drafts_workspace_bytes(n_requests, vocab) (NULL where that is 0).
 * n_rows <= 2^30, vocab <= BPE_MAX_ROWS, n_requests < 2^20, n_requests *
 * min(256, ceil(vocab / 8192)) < 2^24.
 * Returns BPE_OK, BPE_EINVAL, BPE_EWORKSPACE or BPE_EHIP.
 */
int bpe_verify_drafts(const void *d_target, int prob_type, int64_t n_rows, int64_t vocab,
                      int64_t target_stride, const void *d_draft, int64_t draft_stride,
                      const int32_t *d_draft_ids, const int64_t *d_row_off, int64_t n_requests,
                      const float *d_accept, const float *d_sample, int32_t *d_tokens,
                      int32_t *d_counts, void *d_workspace, size_t workspace_bytes,
                      int32_t *d_status, void *hip_stream);

/*
 * The divergence of a student's distribution over the vocabulary from a
 * teacher's over its top tokens.  For row n with the student's logits z, the
 * listed tokens ids[n][k] and the teacher's logits t[n][k], at temperature T:
 *   P_k     = exp(t_k / T) / sum over the listed tokens of exp(t / T)
 *   loss[n] = T^2 * sum_k P_k (log P_k - log softmax(z / T)[ids_k])
 *  d_student  [n_rows][vocab] of student_type;  d_ids  int32 [n_rows][top];
 *  d_teacher  [n_rows][top] of teacher_type.
 *  d_losses   float [n_rows].
 *  d_stats    float [n_rows][4], for bpe_distill_grad: the largest z, the sum of
 *             exp((z - largest) / T), and the same two of the listed t.
 * ID -1 is an entry that holds no token; other IDs outside [0, vocab) set
 * BPE_STATUS_BAD_ID and count as that.  A token that is listed twice counts with
 * both entries.  A row that lists no token above -infinity, or whose logits are
 * all -infinity, has loss 0 and a gradient of zeros.  A term with P_k = 0 is 0,
 * and a P_k below 2^-126 of the largest counts as that; a listed token with another
 * P_k whose z is -infinity makes the loss infinite.
 * The sums are of 32 bits: a loss is off by some 2^-23 T^2 (more in large
 * vocabularies, whose sums are long), which matters where it is itself far below
 * T^2.  At temperatures above 4, where such losses are the rule if the listed tokens
 * are nearly all that the student gives anything to, rows whose listed tokens hold
 * more than 3 / 4 of the student's sum are worked out from the tokens' differences
 * t - z in 64 bits instead, and their losses are off by some 2^-21 of themselves.
 * 2^-20 <= temperature <= 2^20, 0 <= top <= BPE_MAX_TOP, 1 <= vocab <= BPE_MAX_ROWS,
 * n_rows < 2^24.  Returns BPE_OK, BPE_EINVAL or BPE_EHIP.
 */
int bpe_distill(const void *d_student, int student_type, int64_t n_rows, int64_t vocab,
                int64_t student_stride, const int32_t *d_ids, int64_t ids_stride,
                const void *d_teacher, int teacher_type, int64_t teacher_stride, int64_t top,
                float temperature, float *d_losses, float *d_stats, int32_t *d_status,
                void *hip_stream);

/*
 * The gradient of bpe_distill's losses with respect to the student's logits:
 *   grad[n][v] = dloss[n] * T * (softmax(z / T)[v] - sum over ids_k == v of P_k)
 *  d_stats   what bpe_distill gave for the same inputs;  d_dloss  float [n_rows].
 *  d_grad    [n_rows][vocab] of grad_type; may be d_student itself (same type
 *            and stride), else they must not overlap.
 * Rows of loss 0 that bpe_distill names have zeros, whatever dloss is.
 * An entry of a listed token is off by some 2^-22 of dloss T (softmax + P), or, where
 * bpe_distill works a row out from differences and vocab is at most 2,048, of
 * dloss T times the row's typical difference of the two.
 * n_rows * ceil(vocab / 8192) < 2^24.  Returns BPE_OK, BPE_EINVAL or BPE_EHIP.
 */
int bpe_distill_grad(const void *d_student, int student_type, int64_t n_rows, int64_t vocab,
                     int64_t student_stride, const int32_t *d_ids, int64_t ids_stride,
                     const void *d_teacher, int teacher_type, int64_t teacher_stride, int64_t top,
                     const float *d_stats, const float *d_dloss, float temperature, void *d_grad,
                     int grad_type, int64_t grad_stride, int32_t *d_status, void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* BPE_LM_H */
