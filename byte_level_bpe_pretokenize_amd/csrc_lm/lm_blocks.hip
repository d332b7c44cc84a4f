// lm_blocks.hip -- block tables, slots and positions of a paged cache from the
// requests' lengths.
#include "lm_device.h"

namespace bpe {
namespace {

constexpr int BWG = 256;

// x / block size, 0 <= x < 2^31.
__device__ __forceinline__ int32_t block_of(const BlockArgs &a, int32_t x) {
  return (int32_t)(((uint64_t)(uint32_t)x * a.magic) >> a.shift);
}

// Blocks of the first len tokens.
__device__ __forceinline__ int32_t blocks_for(const BlockArgs &a, int32_t len) {
  return len > 0 ? block_of(a, len - 1) + 1 : 0;
}

// Blocks that request r takes.  WRITE: also its length, and into *status what
// is wrong with its offsets and lengths.
template <bool WRITE>
__device__ __forceinline__ int32_t need_of(const BlockArgs &a, int64_t r, uint32_t *status) {
  const int64_t lo = a.off[r], hi = a.off[r + 1];
  const int32_t c = a.cached[r], cached = max(c, 0);
  // (offsets that are not valid still give a count in [0, T])
  const int64_t in = max<int64_t>(min(max<int64_t>(hi, 0), a.T) - min(max<int64_t>(lo, 0), a.T), 0);
  const int64_t full = cached + in;
  const int32_t len = (int32_t)min<int64_t>(full, INT32_MAX);
  if (WRITE) {
    a.lengths[r] = len;
    if (c < 0 || full > INT32_MAX) *status |= BPE_STATUS_BAD_LENGTH;
    if (hi < lo || lo < 0 || hi > a.T || (r == 0 && lo != 0) || (r == a.R - 1 && hi != a.T))
      *status |= BPE_STATUS_BAD_ID_OFFSETS;
  }
  return blocks_for(a, len) - blocks_for(a, cached);
}

// Blocks taken before each request within its group of 2^group_log2 requests,
// and each group's sum: one workgroup per group.
__global__ void __launch_bounds__(kBlockScan) k_block_scan(BlockArgs a) {
  __shared__ int64_t red[kBlockScan / 64];
  const int64_t r0 = (int64_t)blockIdx.x << a.group_log2;
  const int64_t r1 = min(a.R, r0 + (1ll << a.group_log2));
  int64_t carry = 0;
  uint32_t status = 0;
  for (int64_t s = r0; s < r1; s += kBlockScan) {
    const int64_t r = s + threadIdx.x;
    const int64_t need = r < r1 ? need_of<true>(a, r, &status) : 0;
    int64_t total;
    const int64_t ex = block_excl_sum<int64_t, kBlockScan>(need, red, &total);
    if (r < r1) a.first[r] = carry + ex;
    carry += total;
  }
  if (threadIdx.x == 0) a.gsum[blockIdx.x] = carry;
  if (status) atomicOr(a.status, (int32_t)status);
}

struct FillShared {
  int32_t req[kBlockChunk];     // the request that starts at a token, then each token's, less r0
  int64_t red[BWG / 64];
  int32_t wmax[BWG / 64];
  int64_t r0;
};

// The chunk's tokens.  The requests that start in it mark their first token;
// a running maximum gives every token its request.  The token at a block's
// first place in the cache also enters the block into the table: a new block's
// first place always belongs to a new token.
// FUSED (R <= kBlockFused): each workgroup sums the requests' needs itself, one
// launch in all; else `before` holds the groups' running sums.
template <bool FUSED>
__global__ void __launch_bounds__(BWG) k_block_fill(BlockArgs a) {
  __shared__ FillShared s;
  __shared__ int64_t before[FUSED ? kBlockFused : kBlockGroups];
  const int tid = threadIdx.x;
  const int64_t i0 = (int64_t)blockIdx.x * kBlockChunk;
  const int cnt = (int)min<int64_t>(kBlockChunk, a.T - i0);
  uint32_t status = 0;
  int64_t used = 0;
  for (int i = tid; i < kBlockChunk; i += BWG) s.req[i] = 0;
  if (wave_id() == 0 && cnt > 0) {
    const int64_t r = wave_lower_bound(a.off, a.R + 1, i0 + 1) - 1;
    if (lane_id() == 0) s.r0 = min(max<int64_t>(r, 0), a.R - 1);
  }
  if (FUSED) {
    // a thread's requests are consecutive, so that one scan orders them all
    constexpr int PER = kBlockFused / BWG;
    int32_t need[PER];
    int64_t sum = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int64_t r = tid * PER + j;
      need[j] = 0;
      if (r < a.R)
        need[j] = blockIdx.x == 0 ? need_of<true>(a, r, &status) : need_of<false>(a, r, &status);
      sum += need[j];
    }
    int64_t ex = block_excl_sum<int64_t, BWG>(sum, s.red, &used);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      before[tid * PER + j] = ex;
      ex += need[j];
    }
  } else {
    static_assert(kBlockGroups == BWG, "one group per thread");
    const int64_t groups = ((a.R - 1) >> a.group_log2) + 1;
    before[tid] = block_excl_sum<int64_t, BWG>(tid < groups ? a.gsum[tid] : 0, s.red, &used);
  }
  if (blockIdx.x == 0 && tid == 0) {
    *a.used = used;
    if (used > a.n_free) status |= BPE_STATUS_NO_BLOCKS;
  }
  __syncthreads();
  if (cnt > 0) {
    const int64_t r0 = s.r0;
    // requests after r0 that start before the chunk's end
    for (int64_t r = r0 + 1 + tid; r < a.R; r += BWG) {
      const int64_t p = a.off[r] - i0;
      if (p >= cnt) break;
      if (p > 0) atomicMax(&s.req[p], (int32_t)(r - r0));
    }
    __syncthreads();
    constexpr int PER = kBlockChunk / BWG;
    int32_t v[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) v[j] = s.req[tid * PER + j];
#pragma unroll
    for (int j = 1; j < PER; ++j) v[j] = max(v[j], v[j - 1]);
    const int32_t inc = wave_incl_max(v[PER - 1]);
    int32_t left = wave_shift_up1(inc, 0);
    if (lane_id() == 63) s.wmax[wave_id()] = inc;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < BWG / 64; ++w)
      if (w < wave_id()) left = max(left, s.wmax[w]);
#pragma unroll
    for (int j = 0; j < PER; ++j) s.req[tid * PER + j] = max(v[j], left);
    __syncthreads();
    // two tokens per thread and step: slots in 16-byte stores
#pragma unroll
    for (int j = 0; j < kBlockChunk / (2 * BWG); ++j) {
      const int i = (j * BWG + tid) * 2;
      if (i >= cnt) break;
      Vec<int64_t, 2> slot;
      Vec<int32_t, 2> posn;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        slot.v[q] = -1;
        posn.v[q] = -1;
        if (i + q >= cnt) continue;
        const int64_t r = r0 + s.req[i + q];
        const int32_t cached = max(a.cached[r], 0);
        const int64_t pos = cached + (i0 + i + q - a.off[r]);
        if (pos < 0 || pos > INT32_MAX) continue;
        posn.v[q] = (int32_t)pos;
        const int32_t blk = block_of(a, (int32_t)pos);
        const int32_t at = (int32_t)pos - blk * a.bs;
        if (blk >= a.width) {
          status |= BPE_STATUS_TABLE_FULL;
          continue;
        }
        const int32_t have = blocks_for(a, cached);
        int32_t block = -1;
        if (blk < have) {
          block = a.table[r * a.stride + blk];
        } else {
          const int64_t f = (FUSED ? before[r] : before[r >> a.group_log2] + a.first[r]) + blk - have;
          if (f < a.n_free) block = a.free_blocks[f];
          if (at == 0) a.table[r * a.stride + blk] = block;
        }
        if (block >= 0) slot.v[q] = (int64_t)block * a.bs + at;
      }
      if (i + 1 < cnt) {
        store_vec(a.slots + i0 + i, slot);
        store_vec(a.positions + i0 + i, posn);
      } else {
        a.slots[i0 + i] = slot.v[0];
        a.positions[i0 + i] = posn.v[0];
      }
    }
  }
  if (status) atomicOr(a.status, (int32_t)status);
}

// No requests: nothing is taken.
__global__ void k_block_none(int64_t *used) { *used = 0; }

}  // namespace

hipError_t launch_blocks(const BlockArgs &a, hipStream_t stream) {
  if (a.R == 0) {
    hipLaunchKernelGGL(k_block_none, dim3(1), dim3(1), 0, stream, a.used);
    return hipGetLastError();
  }
  const unsigned chunks = a.T > 0 ? (unsigned)((a.T + kBlockChunk - 1) / kBlockChunk) : 1;
  if (a.R <= kBlockFused) {
    hipLaunchKernelGGL(k_block_fill<true>, dim3(chunks), dim3(BWG), 0, stream, a);
  } else {
    const unsigned groups = (unsigned)(((a.R - 1) >> a.group_log2) + 1);
    hipLaunchKernelGGL(k_block_scan, dim3(groups), dim3(kBlockScan), 0, stream, a);
    hipLaunchKernelGGL(k_block_fill<false>, dim3(chunks), dim3(BWG), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace bpe
