// lm_internal.h -- arguments and layouts shared by the host checks (lm_api.cpp),
// the host's layouts (lm_layout.cpp) and the kernels of the operators on token
// IDs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bpe_lm.h"

#if defined(__HIPCC__)
#define BPE_HD __host__ __device__ __forceinline__
#else
#define BPE_HD inline
#endif

namespace bpe {

// Whether that many workgroups of so many threads are one launch (of fewer than
// 2^32 threads).
inline bool launch_fits(int64_t groups, int threads) {
  return groups <= (((int64_t)1 << 32) - 1) / threads;
}

// Outputs of at least this size are stored past the caches (they are larger
// than the L2s together, so nothing of them is there when they are read).
constexpr int64_t kStreamBytes = (int64_t)32 << 20;

// ---- embedding ---------------------------------------------------------------
struct EmbedArgs {
  const void *weight;
  const int32_t *ids;
  void *out;
  int32_t *status;
  int64_t n_rows, n_ids, w_stride, o_stride;
  int32_t width;
  int32_t pad_id;
  float scale;
  uint32_t units;   // vectors per row
  uint32_t magic;   // 2^31 / units + 1: x / units = x * magic >> 31 while x * units < 2^31
  const int32_t *key, *pos;  // the sorted IDs and their positions, or nullptr
  int32_t slabs;             // column groups of 64 vectors
};

// ---- the embedding's gradient ----------------------------------------------
// The IDs are sorted (a stable radix sort of at most kDigitBits bits per pass,
// in at most kSortTiles tiles, whose counts every workgroup reads); the sorted
// list is cut into tiles of `tile` IDs, one wave per tile and 64 vectors of
// columns.
constexpr int kEmbedUnits = 1024;  // vectors per workgroup of the forward
constexpr int kZeroRows = 16;      // rows of the table per workgroup of zeros
constexpr int kGradTile = 256;     // IDs per tile of the sums, at most
constexpr int kDirectWG = 512;
constexpr int kGradDirect = 4 * kDirectWG;  // IDs up to which no sort is made
constexpr int kGradSmall = 6144;            // IDs that one workgroup sorts,
constexpr int64_t kGradSmallRows = 1 << 20; // and rows whose marks it clears
constexpr int kDigitBits = 9;
constexpr int kMaxDigits = 1 << kDigitBits;
constexpr int kSortThreads = 512;
constexpr int kSortTile = 4 * kSortThreads;
constexpr int kSortTiles = 256;

struct GradArgs {
  const void *grad;
  const int32_t *ids;
  void *out;
  int32_t *status;
  int64_t n_rows, n_ids, g_stride, o_stride;
  int32_t width;
  int32_t pad_id;
  float scale;
  int32_t accumulate;
  // workspace
  int32_t *key[2], *pos[2];  // sorted IDs (n_rows: adds nothing) and their positions
  int32_t *counts;           // [sort tiles][digits]
  uint8_t *touched;          // [n_rows] 1: the ID occurs; or nullptr
  float *part;               // [tiles][2][width] sums of rows that a tile's edge cuts
  // launch
  int32_t sort_tiles, sort_steps;    // tiles of kSortTile * sort_steps IDs
  int32_t passes, bits;              // bits of one pass's digit
  int32_t tile;                      // IDs per tile of the sums
  int32_t tiles;
  int32_t slabs;                     // column groups of 64 vectors
  int64_t sum_blocks;
};

struct GradLayout {
  size_t key0, key1, pos0, pos1, counts, touched, part, total;
  int32_t sort_tiles, sort_steps, passes, bits, tile, tiles;
};

bool embed_fits(int64_t n_ids, int64_t width, int ot);
bool by_sorted_ids(int64_t n_ids, int64_t n_rows, int64_t width, int wt, int ot);

// a.key != nullptr: by sorted IDs, after the sort that `sort` describes.
hipError_t launch_embed(const EmbedArgs &a, const GradArgs *sort, int wt, int ot,
                        hipStream_t stream);

GradLayout grad_layout(int64_t n_ids, int64_t n_rows, int64_t width);
bool grad_fits(int64_t n_ids, int64_t n_rows, int64_t width);
hipError_t launch_embed_grad(GradArgs a, int gt, int ot, hipStream_t stream);

// ---- logits ------------------------------------------------------------------
constexpr int kLogitSlab = 4096;         // logits per workgroup,
constexpr int kLogitThreads = 256;       // and threads;
constexpr int kLogitWideSlab = 8192;     // the same of the wide ones
constexpr int kLogitWideThreads = 1024;

// (rows > 0)
bool logits_fit(const bpe_logits_args &a);
bool logits_wide(const bpe_logits_args &a);

hipError_t launch_logits(const bpe_logits_args &a, hipStream_t stream);

// ---- block tables --------------------------------------------------------------
struct BlockArgs {
  const int64_t *off;
  int64_t R, T;
  const int32_t *cached, *free_blocks;
  int64_t n_free;
  int32_t *table;
  int64_t width, stride;
  int32_t bs;
  uint32_t magic;     // x / bs = mulhi(x, magic) >> shift for 0 <= x < 2^31, bs > 1
  int32_t shift;
  int64_t *slots;
  int32_t *positions, *lengths;
  int64_t *used;
  int32_t *status;
  int64_t *first;     // [R] workspace: blocks taken before r within its group
  int64_t *gsum;      // [kBlockGroups] workspace: blocks taken by each group
  int32_t *chunk_req; // [chunks of T] workspace: the request that the chunk begins in
  int32_t group_log2; // requests per group
};

constexpr int kBlockChunk = 2048;     // new tokens per workgroup
constexpr int64_t kBlockMaxNew = ((int64_t)1 << 34) - kBlockChunk;  // (206 GB of outputs)
constexpr int kBlockGroups = 256;     // groups of requests, at most
constexpr int kBlockFused = 2048;     // requests that each workgroup sums by itself
constexpr int kBlockScan = 1024;      // threads of the scan: requests per step

void block_divisor(int32_t bs, uint32_t *magic, int32_t *shift);

hipError_t launch_blocks(const BlockArgs &a, hipStream_t stream);

// ---- a cache of few bits -----------------------------------------------------------
constexpr int kCacheThreads = 256;
constexpr int kCacheVec = 8;       // elements per lane of a write
constexpr int kCacheTokens = 64;   // tokens per workgroup, at most
constexpr int kCacheMinGroup = 16, kCacheMaxGroup = 64 * kCacheVec;  // a wave's lanes at most

// x / d for 0 <= x < 2^31 by a multiplication (block_divisor).
struct Divisor {
  uint32_t magic;
  int32_t shift, d;
};
Divisor divisor(int32_t d);

struct CacheArgs {
  bpe_cache c;
  int32_t row_bytes;      // codes of one head
  int32_t groups;         // of one head
  int32_t group_log2;
  int64_t n;              // tokens
  int64_t t_stride, h_stride;
  int32_t *status;
  // a token's lanes: per head and per token (kCacheVec elements each and whole groups
  // of lanes per group of elements in a write, cache_read_vec elements in a read)
  Divisor per_head, per_token;
  int32_t tokens;         // per workgroup
  // write
  const void *x;
  const int64_t *slots;
  // read
  void *out;
  const int32_t *table, *start;
  const int64_t *off;
  int64_t R, width, stride;
  Divisor bs;
};

int32_t cache_groups(const bpe_cache &c);
int32_t cache_row_bytes(const bpe_cache &c);
bool cache_ok(const bpe_cache &c);
bool cache_tokens_ok(const bpe_cache &c, int64_t n, int64_t token_stride, int64_t head_stride);
int32_t cache_read_vec(int32_t dim, int out_type);
void cache_shape(CacheArgs *a, bool write, int out_type);
bool cache_fits(const CacheArgs &a);  // (shaped)
inline int64_t cache_workgroups(const CacheArgs &a) { return (a.n + a.tokens - 1) / a.tokens; }

// The slot of position p of a request whose blocks are row[0 .. width), or -1
// where it is read as zeros; *status gets why.
BPE_HD int64_t cache_slot(const int32_t *row, int64_t width, int32_t bs, int64_t n_slots,
                          int64_t p, int32_t block, uint32_t *status) {
  if (block >= width) {
    *status |= BPE_STATUS_TABLE_FULL;
    return -1;
  }
  const int32_t entry = row[block];
  if (entry < 0) return -1;
  const int64_t slot = (int64_t)entry * bs + (p - (int64_t)block * bs);
  if (slot >= n_slots) {
    *status |= BPE_STATUS_BAD_SLOT;
    return -1;
  }
  return slot;
}

// The first request in [lo, hi) that ends behind token t, or hi.  In range also
// for offsets that do not increase.  (Growing steps from lo on would take fewer
// loads, but hipcc 7.2 miscompiles their 64-bit minimum: the select that it makes
// for it takes the carry of the sum before it.  tests/test_device_code.py looks for
// that in all that is built.)
BPE_HD int64_t cache_request(const int64_t *off, int64_t lo, int64_t hi, int64_t t) {
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (off[mid + 1] <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

hipError_t launch_cache_write(const CacheArgs &a, int xt, hipStream_t stream);
hipError_t launch_cache_read(const CacheArgs &a, int ot, hipStream_t stream);

// ---- drafted tokens -----------------------------------------------------------------
// A row is added up by regions of `tiles` tiles, four regions a wave.
constexpr int kVerifyTile = 512;
constexpr int kVerifyMostRegions = 4096;
constexpr int kVerifyThreads = 256;
constexpr int64_t kVerifyAlone = 65536;   // tokens that one workgroup adds up and draws from, at most
constexpr int kVerifyAloneThreads = 768;

struct VerifyArgs {
  const void *target, *draft;
  int64_t n_rows, vocab, t_stride, d_stride;
  const int32_t *ids;
  const int64_t *off;
  int64_t R;
  const float *accept, *sample;
  int32_t *tokens, *counts, *status;
  double *sums;   // [R][regions] workspace
  int32_t *rows;  // [R] workspace: the row to draw from
  int32_t regions, tiles;
};

bool verify_alone(int64_t n_requests, int64_t vocab);
int32_t verify_regions(int64_t vocab);  // a multiple of 4
int32_t verify_tiles(int64_t vocab);
int64_t verify_workgroups(int64_t n_requests, int64_t vocab);
hipError_t launch_verify(const VerifyArgs &a, int type, hipStream_t stream);

// ---- distillation -------------------------------------------------------------------
constexpr int kDistillSlab = 8192;    // logits per workgroup of the gradient
constexpr int kDistillThreads = 256;
// Logits up to which one wave takes a row instead of kDistillThreads.  Loss and
// gradient in us, one wave (256 threads): 16,000 rows of 876 bfloat16 logits with
// lists of 16 18 and 18 (40 and 34), 8,000 of 2,048 12 and 14 (24 and 18), 100 of 768
// 4.9 and 4.8 (5.2 and 4.5); behind only for the gradient of float32 rows with long
// lists (16,000 of 876, lists of 200: 45 and 34).
constexpr int kDistillNarrow = 2048;
// Temperature above which rows whose list holds most of the student's sum are worked
// out from the tokens' differences (lm_distill.hip, "warm rows").  Up to it the losses'
// error of some 2^-23 T^2 stays below 2^-18, and kernels do not ask.  At 4 and above,
// loss and gradient of bfloat16 logits in us: 16,000 rows of 876, lists of 16 15.8 and
// 16.4 (16.7 and 18.0), of 200 22.7 and 25.5 (25.8 and 29.4), of all 876, which are such
// rows, 52 and 139 (91 and 213); 8,000 of 2,048, lists of 16 10.4 and 10.6 (12.7 and
// 13.0); 4,096 of 50,257 or 128,256 the same.
constexpr float kDistillWarm = 4.0f;

struct DistillArgs {
  const void *student, *teacher;
  int64_t rows, vocab, s_stride, t_stride;
  const int32_t *ids;
  int64_t i_stride;
  int32_t top, t_type;
  float temperature;
  float *losses, *stats;       // the loss's
  const float *in_stats, *dloss;  // the gradient's
  void *grad;
  int64_t g_stride;
  int32_t *status;
};

bool distill_grad_fits(int64_t n_rows, int64_t vocab);
hipError_t launch_distill(const DistillArgs &a, int st, hipStream_t stream);
hipError_t launch_distill_grad(const DistillArgs &a, int st, int gt, hipStream_t stream);

}  // namespace bpe
