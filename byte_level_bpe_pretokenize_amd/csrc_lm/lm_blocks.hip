// lm_blocks.hip -- block tables, slots and positions of a paged cache from the
// requests' lengths.
#include "lm_device.h"

namespace bpe {
namespace {

constexpr int BWG = 256;

// x / block size, 0 <= x < 2^31.
__device__ __forceinline__ int32_t block_of(const BlockArgs &a, int32_t x) {
  return a.bs == 1 ? x : (int32_t)(__umulhi((uint32_t)x, a.magic) >> a.shift);
}

// Blocks of the first len tokens.
__device__ __forceinline__ int32_t blocks_for(const BlockArgs &a, int32_t len) {
  return len > 0 ? block_of(a, len - 1) + 1 : 0;
}

// An offset as a place in the batch, also where it is not valid.
__device__ __forceinline__ int64_t in_batch(const BlockArgs &a, int64_t off) {
  return min(max<int64_t>(off, 0), a.T);
}

// One request: blocks it takes, and what is wrong with its offsets and lengths.
struct Request {
  int64_t lo, hi;   // its new tokens
  int32_t cached;   // tokens in the cache
};

__device__ __forceinline__ Request load_request(const BlockArgs &a, int64_t r) {
  Request q;
  q.lo = a.off[r];
  q.hi = a.off[r + 1];
  q.cached = a.cached[r];
  return q;
}

__device__ __forceinline__ int32_t need_of(const BlockArgs &a, const Request &q, int64_t r,
                                           int32_t *len, uint32_t *status) {
  const int32_t cached = max(q.cached, 0);
  const int64_t full = cached + max<int64_t>(in_batch(a, q.hi) - in_batch(a, q.lo), 0);
  *len = (int32_t)min<int64_t>(full, INT32_MAX);
  if (q.cached < 0 || full > INT32_MAX) *status |= BPE_STATUS_BAD_LENGTH;
  if (q.hi < q.lo || q.lo < 0 || q.hi > a.T || (r == 0 && q.lo != 0) || (r == a.R - 1 && q.hi != a.T))
    *status |= BPE_STATUS_BAD_ID_OFFSETS;
  return blocks_for(a, *len) - blocks_for(a, cached);
}

// Blocks taken before each request within its group of 2^group_log2 requests,
// each group's sum (one workgroup per group), and the request that each chunk
// of tokens begins in.  65,536 requests take 4 to 5 us, a chain of dependent
// loads and two barriers.
__global__ void __launch_bounds__(kBlockScan) k_block_scan(BlockArgs a) {
  __shared__ int64_t red[kBlockScan / 64];
  const int64_t r0 = (int64_t)blockIdx.x << a.group_log2;
  const int64_t r1 = min(a.R, r0 + (1ll << a.group_log2));
  int64_t carry = 0;
  uint32_t status = 0;
  for (int64_t s = r0; s < r1; s += kBlockScan) {
    const int64_t r = s + threadIdx.x;
    int64_t need = 0;
    if (r < r1) {
      const Request q = load_request(a, r);
      int32_t len;
      need = need_of(a, q, r, &len, &status);
      a.lengths[r] = len;
      for (int64_t c = (in_batch(a, q.lo) + kBlockChunk - 1) / kBlockChunk;
           c * kBlockChunk < in_batch(a, q.hi); ++c)
        a.chunk_req[c] = (int32_t)r;
    }
    int64_t total;
    const int64_t ex = block_excl_sum<int64_t, kBlockScan>(need, red, &total);
    if (r < r1) a.first[r] = carry + ex;
    carry += total;
  }
  if (threadIdx.x == 0) a.gsum[blockIdx.x] = carry;
  if (status) atomicOr(a.status, (int32_t)status);
}

constexpr int kNear = 256;  // requests of a chunk whose data is kept in LDS
constexpr int32_t kFar = INT32_MAX;

// Request r0 + k as the pairs of tokens want it: a token's position less its
// place in the chunk, the blocks that were there (kFar: some position is not in
// [0, INT32_MAX)), and the place of its block b in the list of free ones, less b.
struct alignas(16) Near {
  int32_t pos0, have;
  int64_t free0;
};

struct FillShared {
  alignas(16) int32_t req[kBlockChunk];  // the request that starts at a token, then each token's, less r0
  Near near[kNear];
  int64_t red[BWG / 64];
  int32_t wmax[BWG / 64];
  int32_t r0;
  int32_t n_slow;            // pairs of tokens left for the end
  int16_t slow[kBlockChunk / 2];
};

// The chunk's tokens.  The requests that start in it mark their first token;
// a running maximum gives every token its request.  Then two neighbouring
// tokens per thread and step, so that a wave stores whole lines: where they are
// one request's and in new blocks, one read of the request (from LDS), one
// multiply-high for the block and one load of its number and the next one's.
// The pairs that are not (two requests', a block that was partly filled, the
// ends of the table and of the free blocks) are listed and done one token per
// thread afterwards; done in place they cost every wave that path.  They are few
// where requests bring many tokens to an empty cache, all of them in a step of
// one token per request, and in between where blocks are long (65,536 requests
// of 190 tokens: 34 us with blocks of 16 and nothing cached, 40 with up to 1,000
// tokens each, 44 with those in blocks of 128).  The
// token at a block's first place in the cache also enters the block into the
// table: a new block's first place always belongs to a new token.  What bounds
// it is the chain of dependent loads in each workgroup, kept to four (the
// chunk's request, the requests, their groups, the blocks of all tokens), and
// the arithmetic: 31 us for 12.5 M tokens of 65,536 requests after 4 to 5 for
// their sums (157 MB in 34.7 us, 4.5 TB/s; stores alone of those bytes take 22).
// FUSED (R <= kBlockFused): each workgroup sums the requests' needs itself, one
// launch in all.  That is ahead while the workgroups are few: 2,048 requests
// with 20,480 or 198,656 new tokens take 13.0 us (two launches 16.5), with 2.0 M
// tokens 19.1 (17.7), and with 12 M, where 5,860 workgroups sum the same
// requests, 65 (32).  The limit knows the requests alone.
template <bool FUSED, bool STREAM>
__global__ void __launch_bounds__(BWG, FUSED ? 4 : 8) k_block_fill(BlockArgs a) {
  __shared__ FillShared s;
  __shared__ int64_t before[FUSED ? kBlockFused : kBlockGroups];
  const int tid = threadIdx.x;
  const int64_t i0 = (int64_t)blockIdx.x * kBlockChunk;
  const int cnt = (int)min<int64_t>(kBlockChunk, a.T - i0);
  uint32_t status = 0;
  int64_t used = 0;
  for (int i = tid * 4; i < kBlockChunk; i += BWG * 4) lds_store16(&s.req[i], u32x4{});
  if (tid == 0) s.n_slow = 0;
  int64_t r0 = 0;
  if (FUSED) {
    // a thread's requests are consecutive, so that one scan orders them all
    constexpr int PER = kBlockFused / BWG;
    if (tid == 0) s.r0 = 0;
    int32_t need[PER], len[PER];
    int64_t sum = 0;
    int32_t at = -1;
    if (tid * PER < a.R) {
      Request q[PER];
#pragma unroll
      for (int j = 0; j < PER; ++j) q[j] = load_request(a, min<int64_t>(tid * PER + j, a.R - 1));
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int r = tid * PER + j;
        need[j] = 0;
        if (r >= a.R) continue;
        need[j] = need_of(a, q[j], r, &len[j], &status);
        if (blockIdx.x == 0) a.lengths[r] = len[j];
        if (q[j].lo <= i0) at = r;
        sum += need[j];
      }
    }
    if (blockIdx.x != 0) status = 0;  // every workgroup sees the same: one reports
    int64_t ex = block_excl_sum<int64_t, BWG>(sum, s.red, &used);
    if (at >= 0) atomicMax(&s.r0, at);
    if (tid * PER < a.R) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        before[tid * PER + j] = ex;
        ex += need[j];
      }
    }
    __syncthreads();
    r0 = s.r0;
  } else {
    // (the chunk's request is not set where the offsets are not valid)
    if (cnt > 0) r0 = min(max<int64_t>(a.chunk_req[blockIdx.x], 0), a.R - 1);
    if (uniform_wave_id() == 0) {  // the groups' running sums
      static_assert(kBlockGroups == 256, "four groups per lane");
      const int groups = (int)((a.R - 1) >> a.group_log2) + 1;
      int64_t g[4], sum = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) g[j] = tid * 4 + j < groups ? a.gsum[tid * 4 + j] : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) sum += g[j];
      used = wave_incl_sum(sum);
      int64_t ex = used - sum;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        before[tid * 4 + j] = ex;
        ex += g[j];
      }
      used = lane_value(used, 63);
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) {
    *a.used = used;
    if (used > a.n_free) status |= BPE_STATUS_NO_BLOCKS;
  }
  if (cnt > 0) {
    // request r's first token's position less its place in the chunk, and the
    // place of its block b in the list of free ones, less b
    auto place = [&](int64_t r, int64_t lo, int32_t cached, int64_t first, int64_t *pos0,
                     int64_t *free0, int32_t *have) {
      cached = max(cached, 0);
      *pos0 = cached + (i0 - lo);
      *have = blocks_for(a, cached);
      *free0 = (FUSED ? before[r] : before[r >> a.group_log2] + first) - *have;
    };
    // the requests from r0 on that start before the chunk's end
    for (int64_t k = tid;; k += BWG) {
      const int64_t r = min(r0 + k, a.R - 1);
      const int64_t lo = in_batch(a, a.off[r]);
      const int32_t cached = a.cached[r];
      const int64_t first = FUSED ? 0 : a.first[r];
      const int64_t p = r0 + k < a.R ? lo - i0 : cnt;
      if (k < kNear) {
        int64_t pos0, free0;
        int32_t have;
        place(r, lo, cached, first, &pos0, &free0, &have);
        const bool in = pos0 + max<int64_t>(p, 0) >= 0 && pos0 + kBlockChunk < INT32_MAX;
        s.near[k] = Near{(int32_t)pos0, in ? have : kFar, free0};
      }
      if (p > 0 && p < cnt) atomicMax(&s.req[p], (int32_t)k);
      if (!__syncthreads_or(tid == BWG - 1 && p < cnt)) break;  // (they increase)
    }
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
    // Two neighbouring tokens of one request, in one or two new blocks.  All
    // loads of all steps go first (a wait for a load waits for the stores
    // before it as well), unconditional ones, so that they are in flight
    // together.
    constexpr int STEPS = kBlockChunk / (2 * BWG);
    int32_t kk[STEPS], pos[STEPS], blk[STEPS];
    Vec<int32_t, 2> b[STEPS];
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      const int i = (u * BWG + tid) * 2;
      const int2 k = *(const int2 *)&s.req[i];
      const Near q = s.near[min(k.x, kNear - 1)];
      pos[u] = q.pos0 + i;
      blk[u] = block_of(a, pos[u]);
      const int64_t f = q.free0 + blk[u];
      const bool pair = i + 2 <= cnt && k.x == k.y && k.x < kNear && blk[u] >= q.have &&
                        blk[u] + 1 < a.width && f + 1 < a.n_free;
      kk[u] = pair ? k.x : -1;
      b[u] = load_vec<int32_t, 2>(pair ? a.free_blocks + f : (const int32_t *)a.off);
      if (!pair && i < cnt) s.slow[atomicAdd(&s.n_slow, 1)] = (int16_t)i;
    }
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      if (kk[u] < 0) continue;
      const int i = (u * BWG + tid) * 2;
      const int32_t at = pos[u] - blk[u] * a.bs;
      const bool two = at + 1 == a.bs;
      if (at == 0 || two) {  // a block's first token enters it
        int32_t *entry = a.table + (r0 + kk[u]) * a.stride + blk[u];
        if (at == 0) entry[0] = b[u].v[0];
        if (two) entry[1] = b[u].v[1];
      }
      const int64_t s0 = (int64_t)b[u].v[0] * a.bs + at, s1 = (int64_t)b[u].v[1] * a.bs;
      const bool ok0 = b[u].v[0] >= 0, ok1 = b[u].v[1] >= 0;
      Vec<int64_t, 2> slot;
      Vec<int32_t, 2> posn;
      slot.v[0] = ok0 ? s0 : -1;
      slot.v[1] = two ? (ok1 ? s1 : -1) : ok0 ? s0 + 1 : -1;
      posn.v[0] = pos[u];
      posn.v[1] = pos[u] + 1;
      store_vec<int64_t, 2, STREAM>(a.slots + i0 + i, slot);
      store_vec(a.positions + i0 + i, posn);
    }
    __syncthreads();
    // the other tokens one by one, side by side
    for (int j = tid; j < s.n_slow * 2; j += BWG) {
      const int i = s.slow[j >> 1] + (j & 1);
      if (i >= cnt) continue;
      const int64_t r = r0 + s.req[i];
      int64_t at64, free0, slot = -1;
      int32_t have, position = -1;
      place(r, in_batch(a, a.off[r]), a.cached[r], FUSED ? 0 : a.first[r], &at64, &free0, &have);
      at64 += i;
      if (at64 >= 0 && at64 <= INT32_MAX) {
        position = (int32_t)at64;
        const int32_t bk = block_of(a, position), at = position - bk * a.bs;
        if (bk >= a.width) {
          status |= BPE_STATUS_TABLE_FULL;
        } else {
          int32_t *entry = a.table + r * a.stride + bk;
          int32_t block = -1;
          if (bk < have) block = *entry;
          else if (free0 + bk < a.n_free) block = a.free_blocks[free0 + bk];
          if (bk >= have && at == 0) *entry = block;
          if (block >= 0) slot = (int64_t)block * a.bs + at;
        }
      }
      a.slots[i0 + i] = slot;
      a.positions[i0 + i] = position;
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
  const bool big = a.T * 12 >= kStreamBytes;
  if (a.R <= kBlockFused) {
    if (big) hipLaunchKernelGGL((k_block_fill<true, true>), dim3(chunks), dim3(BWG), 0, stream, a);
    else hipLaunchKernelGGL((k_block_fill<true, false>), dim3(chunks), dim3(BWG), 0, stream, a);
  } else {
    const unsigned groups = (unsigned)(((a.R - 1) >> a.group_log2) + 1);
    hipLaunchKernelGGL(k_block_scan, dim3(groups), dim3(kBlockScan), 0, stream, a);
    if (big) hipLaunchKernelGGL((k_block_fill<false, true>), dim3(chunks), dim3(BWG), 0, stream, a);
    else hipLaunchKernelGGL((k_block_fill<false, false>), dim3(chunks), dim3(BWG), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace bpe
