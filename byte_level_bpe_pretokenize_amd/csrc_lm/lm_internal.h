// lm_internal.h -- arguments and layouts shared by the host checks (lm_api.cpp),
// the host's layouts (lm_layout.cpp) and the kernels of the operators on token
// IDs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/bpe_lm.h"

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

}  // namespace bpe
