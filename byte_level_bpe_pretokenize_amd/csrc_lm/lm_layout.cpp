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

}  // namespace bpe
