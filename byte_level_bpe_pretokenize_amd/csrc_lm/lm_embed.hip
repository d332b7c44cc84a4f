// lm_embed.hip -- rows of an embedding table by token ID, scaled, and the
// table's gradient.
#include "lm_device.h"

namespace bpe {
namespace {

// ---- forward -----------------------------------------------------------------
// out[t] = scale * weight[ids[t]].  The output, n_ids * units vectors of E
// elements, is cut flat over the grid, so no lane idles whatever the width; a
// thread's row and column come from one multiply-high.  The last vector of a
// row whose width is no multiple of E starts at width - E and writes a few
// elements a second time with the same values.  U vectors per thread: their
// ID loads, then their row loads, are in flight together.
template <typename TI, typename TO, int E, int U>
__global__ void __launch_bounds__(256) k_embed(EmbedArgs a) {
  const int tid = threadIdx.x;
  const int64_t base = (int64_t)blockIdx.x * (256 * U);
  const int64_t t0 = base / a.units;
  const uint32_t u0 = (uint32_t)(base - t0 * a.units);
  int32_t id[U];
  int64_t t[U];
  int32_t col[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const uint32_t x = u0 + k * 256 + tid;
    const uint32_t q = __umulhi(2 * x, a.magic);
    t[k] = t0 + q;
    col[k] = min((int)((x - q * a.units) * E), a.width - E);
    id[k] = a.ids[min(t[k], a.n_ids - 1)];
  }
  Vec<TI, E> w[U];
  bool ok[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    ok[k] = id[k] >= 0 && id[k] < a.n_rows && id[k] != a.pad_id;
    w[k] = load_vec<TI, E>((const TI *)a.weight + (ok[k] ? id[k] : 0) * a.w_stride + col[k]);
  }
  bool bad = false;
#pragma unroll
  for (int k = 0; k < U; ++k) {
    if (t[k] >= a.n_ids) continue;
    bad |= !ok[k] && (id[k] < 0 || id[k] != a.pad_id);
    Vec<TO, E> r;
#pragma unroll
    for (int e = 0; e < E; ++e) r.v[e] = from_f32<TO>(ok[k] ? (float)w[k].v[e] * a.scale : 0.f);
    store_vec<TO, E>((TO *)a.out + t[k] * a.o_stride + col[k], r);
  }
  if (bad) atomicOr(a.status, (int32_t)BPE_STATUS_BAD_ID);
}

// ---- gradient: sort ------------------------------------------------------------
// The key of a position: its ID, or n_rows for one that adds nothing (the pad
// ID, an ID outside the table), which sorts behind every row.
__device__ __forceinline__ int32_t grad_key(const GradArgs &a, int32_t id, bool *bad) {
  if (id >= 0 && id == a.pad_id) return (int32_t)a.n_rows;
  if (id >= 0 && id < a.n_rows) return id;
  *bad = true;
  return (int32_t)a.n_rows;
}

// Digit counts of one tile.  The first pass also clears the row marks (its
// workgroups' share each).
__global__ void __launch_bounds__(kSortThreads) k_grad_count(GradArgs a, int pass) {
  __shared__ int32_t cnt[kMaxDigits];
  const int tid = threadIdx.x, digits = 1 << a.bits;
  const int64_t i0 = (int64_t)blockIdx.x * kSortTile;
  for (int d = tid; d < digits; d += kSortThreads) cnt[d] = 0;
  if (pass == 0)
    for (int64_t v = (int64_t)blockIdx.x * kSortThreads + tid; v < a.n_rows;
         v += (int64_t)gridDim.x * kSortThreads)
      a.touched[v] = 0;
  __syncthreads();
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kSortTile / kSortThreads; ++j) {
    const int64_t i = i0 + j * kSortThreads + tid;
    if (i < a.n_ids) {
      const int32_t k = pass == 0 ? grad_key(a, a.ids[i], &bad) : a.key[(pass + 1) & 1][i];
      atomicAdd(&cnt[(k >> (pass * a.bits)) & (digits - 1)], 1);
    }
  }
  if (bad) atomicOr(a.status, (int32_t)BPE_STATUS_BAD_ID);
  __syncthreads();
  for (int d = tid; d < digits; d += kSortThreads) a.counts[(int64_t)blockIdx.x * digits + d] = cnt[d];
}

// One pass's scatter of one tile.  A key's place: the keys of smaller digits
// (the column sums of `counts`, scanned), the keys of its digit in earlier
// tiles, in earlier waves of the tile and before it in its wave.  Each wave
// takes 256 consecutive keys, 64 at a time; the lanes with equal digits find
// each other by a ballot per digit bit.
__global__ void __launch_bounds__(kSortThreads) k_grad_scatter(GradArgs a, int pass) {
  constexpr int NW = kSortThreads / 64;
  constexpr int PER = kSortTile / kSortThreads;
  __shared__ int32_t base[NW][kMaxDigits];
  __shared__ int32_t red[NW];
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_id();
  const int digits = 1 << a.bits, shift = pass * a.bits;
  const bool last = pass == a.passes - 1;
  const int64_t i0 = (int64_t)blockIdx.x * kSortTile + wv * (64 * PER);
  for (int d = tid; d < NW * kMaxDigits; d += kSortThreads) (&base[0][0])[d] = 0;
  int32_t key[PER], pos[PER];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int64_t i = i0 + j * 64 + lane;
    key[j] = -1;
    pos[j] = (int32_t)i;
    if (i < a.n_ids) {
      if (pass == 0) {
        key[j] = grad_key(a, a.ids[i], &bad);
      } else {
        key[j] = a.key[(pass + 1) & 1][i];
        pos[j] = a.pos[(pass + 1) & 1][i];
      }
    }
  }
  // thread d < digits: the digit's keys in all tiles and in the earlier ones
  int32_t all = 0, before = 0;
  if (tid < digits)
    for (int s = 0; s < a.sort_tiles; ++s) {
      const int32_t c = a.counts[(int64_t)s * digits + tid];
      all += c;
      if (s < (int)blockIdx.x) before += c;
    }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (key[j] >= 0) atomicAdd(&base[wv][(key[j] >> shift) & (digits - 1)], 1);
  int32_t total;
  const int32_t ex = block_excl_sum<int32_t, kSortThreads>(all, red, &total);
  if (tid < digits) {
    int32_t run = ex + before;
    for (int w = 0; w < NW; ++w) {
      const int32_t c = base[w][tid];
      base[w][tid] = run;
      run += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const bool live = key[j] >= 0;
    const int d = (key[j] >> shift) & (digits - 1);
    uint64_t same = __ballot(live);
    for (int b = 0; b < a.bits; ++b) {
      const bool bit = (d >> b) & 1;
      const uint64_t m = __ballot(bit);
      same &= bit ? m : ~m;
    }
    if (live) {
      const int leader = __ffsll((unsigned long long)same) - 1;
      const int rank = __popcll(same & ((1ull << lane) - 1));
      int32_t at = 0;
      if (lane == leader) at = atomicAdd(&base[wv][d], __popcll(same));
      at = __shfl(at, leader, 64) + rank;
      a.key[pass & 1][at] = key[j];
      a.pos[pass & 1][at] = pos[j];
      if (last && key[j] < a.n_rows) a.touched[key[j]] = 1;
    }
  }
}

// ---- gradient: sums --------------------------------------------------------------
// Elements of a lane's vector before `skip` belong to its left neighbour (the
// last vector of a row whose width is no multiple of E): loaded, not stored.
template <typename TO, int E>
__device__ __forceinline__ void grad_store(const GradArgs &a, int64_t row, int col, int skip,
                                           const float (&acc)[E]) {
  TO *p = (TO *)a.out + row * a.o_stride + col;
  if (skip == 0) {
    Vec<TO, E> r;
    if (a.accumulate) {
      r = load_vec<TO, E>(p);
#pragma unroll
      for (int e = 0; e < E; ++e) r.v[e] = from_f32<TO>((float)r.v[e] + acc[e] * a.scale);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) r.v[e] = from_f32<TO>(acc[e] * a.scale);
    }
    store_vec<TO, E>(p, r);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e >= skip) p[e] = from_f32<TO>((a.accumulate ? (float)p[e] : 0.f) + acc[e] * a.scale);
  }
}

// A lane's column in slab s: its vector's start, and how many of its elements
// belong to its left neighbour; false past the row's end.
template <int E>
__device__ __forceinline__ bool grad_col(const GradArgs &a, int s, int *col, int *skip) {
  const int c = (s * 64 + lane_id()) * E;
  if (c >= a.width) return false;
  *col = min(c, a.width - E);
  *skip = c - *col;
  return true;
}

constexpr int kRowsAhead = 8;   // gradient rows in flight per wave

// Workgroups below sum_blocks: one wave per tile of the sorted list and slab of
// 64 vectors of columns, adding up the rows of each ID in the order of the
// list.  A row whose positions all lie in the tile is finished here; of one
// that a tile's edge cuts, the tile's share goes to `part` (slot 0: the row
// began in an earlier tile; slot 1: it begins here and goes on).  The other
// workgroups write zeros to the rows that no ID names.
template <typename TG, typename TO, int E>
__global__ void __launch_bounds__(256) k_grad_sum(GradArgs a) {
  const int lane = lane_id(), wv = uniform_wave_id();
  if (blockIdx.x >= a.sum_blocks) {
    const int64_t r0 = (int64_t)(blockIdx.x - a.sum_blocks) * kZeroRows;
    for (int r = 0; r < kZeroRows && r0 + r < a.n_rows; ++r) {
      if (a.n_ids > 0 && a.touched[r0 + r]) continue;
      TO *p = (TO *)a.out + (r0 + r) * a.o_stride;
      Vec<TO, E> z;
#pragma unroll
      for (int e = 0; e < E; ++e) z.v[e] = from_f32<TO>(0.f);
      for (int c = threadIdx.x * E; c < a.width; c += 256 * E)
        store_vec<TO, E>(p + min(c, a.width - E), z);
    }
    return;
  }
  const int64_t w = (int64_t)blockIdx.x * 4 + wv;
  const int tile = (int)(w / a.slabs), slab = (int)(w - (int64_t)tile * a.slabs);
  if (tile >= a.tiles) return;
  int col = 0, skip = 0;
  const bool mine = grad_col<E>(a, slab, &col, &skip);
  const int fin = (a.passes - 1) & 1;
  const int64_t i0 = (int64_t)tile * a.tile;
  const int n = (int)min<int64_t>(a.tile, a.n_ids - i0);
  // lane l holds the l-th key and position of the tile
  const int32_t none = (int32_t)a.n_rows;
  const int32_t k = lane < n ? a.key[fin][i0 + lane] : none;
  const int32_t p = lane < n ? a.pos[fin][i0 + lane] : 0;
  const int32_t prev = i0 > 0 ? a.key[fin][i0 - 1] : -1;
  const int32_t next = i0 + n < a.n_ids ? a.key[fin][i0 + n] : -1;
  const int m = __popcll(__ballot(k < none));  // rows that add something come first
  if (m == 0) return;
  const TG *g = (const TG *)a.grad + col;
  float acc[E] = {};
  int32_t cur = lane_value(k, 0);
  bool from_left = cur == prev;
  float *part = a.part + (int64_t)tile * 2 * a.width + col;
  auto flush = [&](bool to_right) {
    if (!mine) return;
    if (from_left || to_right) {
      float *q = part + (from_left ? 0 : a.width);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e >= skip) q[e] = acc[e];
    } else {
      grad_store<TO, E>(a, cur, col, skip, acc);
    }
  };
  for (int b = 0; b < m; b += kRowsAhead) {
    // (lanes past the row's end load its first vector: every lane stays
    // active around the lane reads)
    Vec<TG, E> x[kRowsAhead];
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j)
      x[j] = load_vec<TG, E>(g + (int64_t)lane_value(p, min(b + j, m - 1)) * a.g_stride);
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
      if (b + j >= m) break;
      const int32_t kk = lane_value(k, b + j);
      if (kk != cur) {
        flush(false);
        from_left = false;
        cur = kk;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += (float)x[j].v[e];
    }
  }
  flush(m == n && next == cur);
}

// Rows that tile edges cut: one workgroup per tile and slab; it has work when a
// row begins in its tile and goes on in the next.  Its four waves add up the
// tiles' shares, every fourth each, and join theirs in order.
template <typename TO, int E>
__global__ void __launch_bounds__(256) k_grad_join(GradArgs a) {
  __shared__ float sh[4][64][E];
  const int lane = lane_id(), wv = wave_id();
  const int tile = (int)(blockIdx.x / a.slabs), slab = (int)(blockIdx.x - (unsigned)tile * a.slabs);
  const int fin = (a.passes - 1) & 1;
  const int32_t *key = a.key[fin];
  const int64_t i0 = (int64_t)tile * a.tile, i1 = i0 + a.tile;
  if (i1 >= a.n_ids) return;
  const int32_t cur = key[i1 - 1];
  if (cur >= a.n_rows || key[i1] != cur) return;
  if (key[i0] == cur && i0 > 0 && key[i0 - 1] == cur) return;  // it began earlier
  // the tiles that begin inside the row: tile + 1 .. tile + run
  int run = 0;
  for (int j = tile + 1;; j += 64) {
    const int64_t i = (int64_t)(j + lane) * a.tile;
    const int c = __popcll(__ballot(i < a.n_ids && key[min(i, a.n_ids - 1)] == cur));
    run += c;
    if (c < 64) break;
  }
  int col = 0, skip = 0;
  const bool mine = grad_col<E>(a, slab, &col, &skip);
  float acc[E] = {};
  if (mine) {
    const float *p = a.part + (int64_t)tile * 2 * a.width + col;
    if (wv == 0) {
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = p[a.width + e];
    }
#pragma unroll 4
    for (int j = 1 + wv; j <= run; j += 4) {
      const Vec<float, E> x = load_vec<float, E>(p + (int64_t)j * 2 * a.width);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += x.v[e];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sh[wv][lane][e] = acc[e];
  }
  __syncthreads();
  if (wv == 0 && mine) {
#pragma unroll
    for (int w = 1; w < 4; ++w)
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += sh[w][lane][e];
    grad_store<TO, E>(a, cur, col, skip, acc);
  }
}

template <typename TI, typename TO, int E>
hipError_t embed_as(EmbedArgs a, hipStream_t stream) {
  constexpr int U = kEmbedUnits / 256;
  a.units = (uint32_t)((a.width + E - 1) / E);
  a.magic = (1u << 31) / a.units + 1;
  const int64_t total = a.n_ids * a.units;
  hipLaunchKernelGGL((k_embed<TI, TO, E, U>), dim3((unsigned)((total + 256 * U - 1) / (256 * U))),
                     dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <typename TI, typename TO>
hipError_t embed_of(const EmbedArgs &a, hipStream_t stream) {
  return a.width >= 8 ? embed_as<TI, TO, 8>(a, stream) : embed_as<TI, TO, 1>(a, stream);
}

template <typename TI>
hipError_t embed_from(const EmbedArgs &a, int ot, hipStream_t stream) {
  if (ot == BPE_F32) return embed_of<TI, float>(a, stream);
  if (ot == BPE_BF16) return embed_of<TI, bf16_t>(a, stream);
  return embed_of<TI, f16_t>(a, stream);
}

template <typename TG, typename TO, int E>
hipError_t grad_as(GradArgs a, hipStream_t stream) {
  a.slabs = (a.width + 64 * E - 1) / (64 * E);
  for (int pass = 0; a.n_ids > 0 && pass < a.passes; ++pass) {
    hipLaunchKernelGGL(k_grad_count, dim3(a.sort_tiles), dim3(kSortThreads), 0, stream, a, pass);
    hipLaunchKernelGGL(k_grad_scatter, dim3(a.sort_tiles), dim3(kSortThreads), 0, stream, a, pass);
  }
  a.sum_blocks = a.n_ids > 0 ? ((int64_t)a.tiles * a.slabs + 3) / 4 : 0;
  const int64_t zero = a.accumulate ? 0 : (a.n_rows + kZeroRows - 1) / kZeroRows;
  if (a.sum_blocks + zero > 0)
    hipLaunchKernelGGL((k_grad_sum<TG, TO, E>), dim3((unsigned)(a.sum_blocks + zero)), dim3(256), 0,
                       stream, a);
  if (a.n_ids > a.tile)
    hipLaunchKernelGGL((k_grad_join<TO, E>), dim3((unsigned)((int64_t)a.tiles * a.slabs)),
                       dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <typename TG, typename TO>
hipError_t grad_of(const GradArgs &a, hipStream_t stream) {
  return a.width >= 8 ? grad_as<TG, TO, 8>(a, stream) : grad_as<TG, TO, 1>(a, stream);
}

template <typename TG>
hipError_t grad_from(const GradArgs &a, int ot, hipStream_t stream) {
  if (ot == BPE_F32) return grad_of<TG, float>(a, stream);
  if (ot == BPE_BF16) return grad_of<TG, bf16_t>(a, stream);
  return grad_of<TG, f16_t>(a, stream);
}

}  // namespace

hipError_t launch_embed(const EmbedArgs &a, int wt, int ot, hipStream_t stream) {
  if (wt == BPE_F32) return embed_from<float>(a, ot, stream);
  if (wt == BPE_BF16) return embed_from<bf16_t>(a, ot, stream);
  return embed_from<f16_t>(a, ot, stream);
}

hipError_t launch_embed_grad(GradArgs a, int gt, int ot, hipStream_t stream) {
  if (gt == BPE_F32) return grad_from<float>(a, ot, stream);
  if (gt == BPE_BF16) return grad_from<bf16_t>(a, ot, stream);
  return grad_from<f16_t>(a, ot, stream);
}

}  // namespace bpe
