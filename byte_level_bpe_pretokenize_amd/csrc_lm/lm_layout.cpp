// lm_layout.cpp -- what the host decides for the operators on token IDs from
// the sizes alone: workspace layouts, variants, divisors.  No HIP call.
#include "lm_internal.h"

namespace bpe {

namespace {

int64_t type_bytes(int t) { return t == BPE_F32 ? 4 : 2; }

size_t place(size_t *at, size_t bytes) {
  const size_t p = *at;
  *at += (bytes + 255) / 256 * 256;
  return p;
}

}  // namespace

// Whether the forward is one launch: vectors of 16 bytes of the output (of one
// element in rows of less than 8), kEmbedUnits per workgroup of 256 threads.
// (By sorted IDs a wave has 64 positions and 64 vectors: no more workgroups.)
bool embed_fits(int64_t n_ids, int64_t width, int ot) {
  const int64_t per = width < 8 ? 1 : 16 / type_bytes(ot);
  const int64_t vectors = n_ids * ((width + per - 1) / per);
  return launch_fits((vectors + kEmbedUnits - 1) / kEmbedUnits, 256);
}

// Whether the forward goes by sorted IDs: where many IDs read each row of a
// table whose elements are wider than the output's, so that what the caches
// lose costs more than storing the rows out of order.  262,144 IDs, float32 to
// bfloat16, 32,256 rows of 4,096: 659 us in the order of the IDs, 570 sorted;
// 8,000 rows: 615 and 441; with half the output or 2 IDs per row the two are
// even, and a bfloat16 table is faster in the order of the IDs up to 32 IDs per
// row (437 and 443).
bool by_sorted_ids(int64_t n_ids, int64_t n_rows, int64_t width, int wt, int ot) {
  return width >= 8 && type_bytes(wt) > type_bytes(ot) && n_ids >= 4 * n_rows &&
         n_ids * width * type_bytes(ot) >= 16 * kStreamBytes;
}

GradLayout grad_layout(int64_t n_ids, int64_t n_rows, int64_t width) {
  GradLayout L;
  // the values to sort: the rows, and n_rows for what adds nothing
  int bits = 1;
  while ((n_rows >> bits) != 0) ++bits;
  L.passes = (bits + kDigitBits - 1) / kDigitBits;
  L.bits = (bits + L.passes - 1) / L.passes;
  const int64_t steps = (n_ids + kSortTile - 1) / kSortTile;
  L.sort_steps = (int32_t)((steps + kSortTiles - 1) / kSortTiles);
  L.sort_tiles = L.sort_steps > 0 ? (int32_t)((steps + L.sort_steps - 1) / L.sort_steps) : 0;
  // long tiles for few cut rows, short ones where there would be too few waves
  const int64_t slabs = width < 8 ? 1 : (width + 511) / 512;
  L.tile = kGradTile;
  while (L.tile > 8 && n_ids / L.tile * slabs < 4096) L.tile /= 2;
  L.tiles = (int32_t)((n_ids + L.tile - 1) / L.tile);
  size_t at = 0;
  L.key0 = place(&at, (size_t)n_ids * 4);
  L.key1 = place(&at, (size_t)n_ids * 4);
  L.pos0 = place(&at, (size_t)n_ids * 4);
  L.pos1 = place(&at, (size_t)n_ids * 4);
  L.counts = place(&at, ((size_t)L.sort_tiles << L.bits) * 4);
  L.touched = place(&at, (size_t)n_rows);
  L.part = place(&at, (size_t)L.tiles * 2 * width * 4);
  L.total = at;
  return L;
}

// Whether the sums of a sorted gradient (four tiles and slabs of 512 columns, or
// 16 rows of zeros, per workgroup) and the join of what tile edges cut (one
// tile and slab) are one launch each.
bool grad_fits(int64_t n_ids, int64_t n_rows, int64_t width) {
  const int64_t slabs = width < 8 ? 1 : (width + 511) / 512;
  const int64_t tiles = grad_layout(n_ids, n_rows, width).tiles * slabs;
  return launch_fits((tiles + 3) / 4 + (n_rows + kZeroRows - 1) / kZeroRows, 256) &&
         launch_fits(tiles, 256);
}

// Whether the logits are one launch.
bool logits_fit(const bpe_logits_args &a) {
  return launch_fits((a.vocab + kLogitSlab - 1) / kLogitSlab * a.rows, kLogitThreads);
}

// Whether logits go by workgroups of 1,024 threads and slabs of 8,192 instead of
// 256 and 4,096: where prompts are long on average, since those read a list in
// fewer steps and half as many slabs.  Lists of 30,000 IDs: 24 rows of 100,256
// logits 15.0 us (narrow 18.9), 64 of 128,256 29.5 (34.5), 256 of 128,256 112
// (107); of 600: 24 rows the same, 64 15.9 (13.3), 256 42 (35).  Generated IDs
// do not count: the host has the width of their matrix, which a server makes as
// wide as a generation may ever get, and not how many there are (256 rows with
// room for 8,192 and 128 there: 42 and 35 us; all 8,192 there: 66 and 59).
// Where the wide launch would have too many threads (2^22 rows and more) the
// narrow one, which has fewer, is taken.
bool logits_wide(const bpe_logits_args &a) {
  const int64_t slabs = (a.vocab + kLogitWideSlab - 1) / kLogitWideSlab;
  return a.n_prompt / a.rows > 4096 && launch_fits(slabs * a.rows, kLogitWideThreads);
}

// x / bs = x * magic >> (31 + s) with 2^s >= bs and magic = 2^(31 + s) / bs + 1:
// magic * bs - 2^(31 + s) <= bs, so for x < 2^31 the error stays below 1 / bs.
void block_divisor(int32_t bs, uint32_t *magic, int32_t *shift) {
  int s = 0;
  while (((int64_t)1 << s) < bs) ++s;
  *magic = (uint32_t)(((uint64_t)1 << (31 + s)) / (uint64_t)bs + 1);
  *shift = s - 1;  // of the product's upper half
}

Divisor divisor(int32_t d) {
  Divisor r = {};
  r.d = d;
  if (d > 1) block_divisor(d, &r.magic, &r.shift);
  return r;
}

int32_t cache_groups(const bpe_cache &c) { return (c.dim + c.group - 1) / c.group; }

int32_t cache_row_bytes(const bpe_cache &c) {
  return c.format == BPE_UINT4 ? (c.dim + 1) / 2 : c.dim;
}

bool cache_ok(const bpe_cache &c) {
  if ((c.format != BPE_E4M3 && c.format != BPE_INT8 && c.format != BPE_UINT4) || c.heads < 1 ||
      c.heads > BPE_MAX_HEADS || c.dim < 1 || c.dim > BPE_MAX_DIM || c.group < kCacheMinGroup ||
      c.group > kCacheMaxGroup || (c.group & (c.group - 1)) || c.n_slots < 0 ||
      c.n_slots > (int64_t)1 << 40)
    return false;
  const int64_t most = (int64_t)1 << 32;
  const int64_t scales = (int64_t)c.heads * cache_groups(c) * (c.format == BPE_UINT4 ? 2 : 1);
  // (2^40 slots of 2^22 bytes are addressed in 64 bits)
  return c.codes_stride >= (int64_t)c.heads * cache_row_bytes(c) && c.codes_stride <= most >> 10 &&
         c.scales_stride >= scales && c.scales_stride <= most >> 12 &&
         (c.n_slots == 0 || (c.codes && c.scales));
}

// Strides of tokens and heads: token by token or head by head, without overlap.
bool cache_tokens_ok(const bpe_cache &c, int64_t n, int64_t token_stride, int64_t head_stride) {
  const int64_t most = (int64_t)1 << 32;
  if (n < 0 || n > BPE_MAX_IDS - kCacheTokens) return false;
  const bool many = n > 1, heads = c.heads > 1;
  if ((many && (token_stride < c.dim || token_stride > most)) ||
      (heads && (head_stride < c.dim || head_stride > most)))
    return false;
  return !many || !heads || token_stride >= (c.heads - 1) * head_stride + c.dim ||
         head_stride >= (n - 1) * token_stride + c.dim;
}

// Elements of a read's lane: 16 bytes of output, so that each store of a wave is
// whole lines; but 8 of float32 too, in two stores, in heads of no whole vectors,
// where what comes with each vector costs more than the half lines.  60,000 tokens of
// 16 heads to float32: of 128 in e4m3 91 us with 4 (198 with 8), 64 heads of 77 in int8
// 503 (387).
int32_t cache_read_vec(int32_t dim, int out_type) {
  return out_type == BPE_F32 && dim % 4 == 0 ? 4 : 8;
}

// A token's lanes, and tokens per workgroup: four vectors per thread where
// there are that many.
void cache_shape(CacheArgs *a, bool write, int out_type) {
  a->row_bytes = cache_row_bytes(a->c);
  a->groups = cache_groups(a->c);
  a->group_log2 = 0;
  while (1 << a->group_log2 < a->c.group) ++a->group_log2;
  const int32_t vec = cache_read_vec(a->c.dim, out_type);
  const int32_t per_head = write ? a->groups * (a->c.group / kCacheVec) : (a->c.dim + vec - 1) / vec;
  a->per_head = divisor(per_head);
  a->per_token = divisor(per_head * a->c.heads);
  const int32_t tokens = 4 * kCacheThreads / (per_head * a->c.heads);
  a->tokens = tokens < 1 ? 1 : tokens > kCacheTokens ? kCacheTokens : tokens;
}

// Whether a workgroup per request adds up its row and draws from it, in one launch
// instead of two: while each has a CU of its own, up to where one CU's share of the
// bandwidth costs what the second launch does; for more requests in small
// vocabularies.  float32 with a draft's probabilities, one launch and two, us a
// call from the host (captured in a graph): 4 requests of 50,256 tokens 11.8 and
// 14.7 (11.9 and 8.3), 256 of them 20.5 and 22.7 (21.2 and 23.4), 256 of 32,256
// 15.3 and 17.9 (16.2 and 18.6); 400 of 16,000 16.9 and 16.1, 800 of 8,000 15.2 and
// 16.1, 800 of 16,000 33.5 and 23.9.
bool verify_alone(int64_t n_requests, int64_t vocab) {
  return vocab <= (n_requests <= 256 ? kVerifyAlone : 8192);
}

int32_t verify_regions(int64_t vocab) {
  const int64_t four = (vocab + 4 * kVerifyTile - 1) / (4 * kVerifyTile) * 4;
  return (int32_t)(four < kVerifyMostRegions ? four : kVerifyMostRegions);
}

int32_t verify_tiles(int64_t vocab) {
  const int64_t per = (int64_t)verify_regions(vocab) * kVerifyTile;
  return (int32_t)((vocab + per - 1) / per);
}

// Workgroups of the sums: a wave per four regions.
int64_t verify_workgroups(int64_t n_requests, int64_t vocab) {
  const int64_t per = kVerifyThreads / 16;
  return n_requests * ((verify_regions(vocab) + per - 1) / per);
}

// Whether a cache's tokens are one launch (which the header's bound on lanes is
// stricter than).
bool cache_fits(const CacheArgs &a) {
  return a.n * a.per_token.d < (int64_t)1 << 33 && launch_fits(cache_workgroups(a), kCacheThreads);
}

// Whether the gradient is one launch.
bool distill_grad_fits(int64_t n_rows, int64_t vocab) {
  return launch_fits((vocab + kDistillSlab - 1) / kDistillSlab * n_rows, kDistillThreads);
}

}  // namespace bpe
