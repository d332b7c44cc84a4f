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
// ID loads, then their row loads, are in flight together.  E is 16 bytes of the
// output, so that a wave's stores are whole lines.  BIG: the output is stored
// past the caches (bfloat16 rows of 4,096 of a table of 32,256, 262,144 IDs:
// 552 us without, 472 with; 32,768 IDs: 75 and 62; 65,536 of a float32 table to
// bfloat16: 177 and 167).
// Bound by memory: the 2.41 GB of the largest of these (each row of the table
// read once) move at 5.1 TB/s.  Rows that fell out of the L2s and are read
// again come on top of them; where the table's elements are wider than the
// output's those cost most, and large batches of such go by sorted IDs
// (k_embed_runs) instead: 659 us here for the same IDs of a float32 table.
// Column slabs, one per XCD or one after another, keep more of these rows in
// the caches but store shorter runs: 648 to 788 us.
// 64 IDs take 3.2 us.
template <typename TI, typename TO, int E, int U, bool BIG>
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
    TO *p = (TO *)a.out + t[k] * a.o_stride + col[k];
    store_vec<TO, E, BIG>(p, r);
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

// Digit counts of one tile (131,072 IDs: 4.7 us a pass, and 8.8 us the scatter;
// both wait on a few dependent loads).  The first pass also clears the row marks (its
// workgroups' share each).
__global__ void __launch_bounds__(kSortThreads) k_grad_count(GradArgs a, int pass) {
  __shared__ int32_t cnt[kMaxDigits];
  const int tid = threadIdx.x, digits = 1 << a.bits;
  const int64_t i0 = (int64_t)blockIdx.x * kSortTile * a.sort_steps;
  for (int d = tid; d < digits; d += kSortThreads) cnt[d] = 0;
  if (pass == 0 && a.touched)
    for (int64_t v = (int64_t)blockIdx.x * kSortThreads + tid; v < a.n_rows;
         v += (int64_t)gridDim.x * kSortThreads)
      a.touched[v] = 0;
  __syncthreads();
  bool bad = false;
  for (int s = 0; s < a.sort_steps; ++s) {
#pragma unroll
    for (int j = 0; j < kSortTile / kSortThreads; ++j) {
      const int64_t i = i0 + (int64_t)s * kSortTile + j * kSortThreads + tid;
      if (i < a.n_ids) {
        const int32_t k = pass == 0 ? grad_key(a, a.ids[i], &bad) : a.key[(pass + 1) & 1][i];
        atomicAdd(&cnt[(k >> (pass * a.bits)) & (digits - 1)], 1);
      }
    }
  }
  if (bad) atomicOr(a.status, (int32_t)BPE_STATUS_BAD_ID);
  __syncthreads();
  for (int d = tid; d < digits; d += kSortThreads) a.counts[(int64_t)blockIdx.x * digits + d] = cnt[d];
}

// The place of each lane's key (negative: none) among those of its digit:
// next[digit] is the wave's next one.  The lanes with equal digits find each
// other by a ballot per digit bit.  Called by whole waves.
__device__ __forceinline__ bool place_key(int32_t key, int shift, int bits, int32_t *next,
                                          int32_t *at) {
  const bool live = key >= 0;
  const int d = (key >> shift) & ((1 << bits) - 1);
  uint64_t same = __ballot(live);
  for (int b = 0; b < bits; ++b) {
    const bool bit = (d >> b) & 1;
    const uint64_t m = __ballot(bit);
    same &= bit ? m : ~m;
  }
  if (!live) return false;
  const int leader = __ffsll((unsigned long long)same) - 1;
  int32_t first = 0;
  if (lane_id() == leader) first = atomicAdd(&next[d], __popcll(same));
  *at = __shfl(first, leader, 64) + __popcll(same & ((1ull << lane_id()) - 1));
  return true;
}

// One pass's scatter of one tile.  A key's place: the keys of smaller digits
// (the column sums of `counts`, scanned), the keys of its digit in earlier
// tiles, in earlier waves of the tile and before it in its wave.  Each wave
// takes sort_steps times 256 consecutive keys, 64 at a time; with more than one
// step it reads them twice, to count and to place.
__global__ void __launch_bounds__(kSortThreads) k_grad_scatter(GradArgs a, int pass) {
  constexpr int NW = kSortThreads / 64;
  constexpr int PER = kSortTile / kSortThreads;
  __shared__ int32_t base[NW][kMaxDigits];
  __shared__ int32_t red[NW];
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_id();
  const int digits = 1 << a.bits, shift = pass * a.bits;
  const bool last = pass == a.passes - 1;
  const int64_t i0 = ((int64_t)blockIdx.x * kSortTile + wv * (64 * PER)) * a.sort_steps;
  for (int d = tid; d < NW * kMaxDigits; d += kSortThreads) (&base[0][0])[d] = 0;
  int32_t key[PER], pos[PER];
  bool bad = false;
  auto load = [&](int s) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int64_t i = i0 + s * (64 * PER) + j * 64 + lane;
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
  };
  load(0);
  // thread d < digits: the digit's keys in all tiles and in the earlier ones
  int32_t all = 0, before = 0;
  if (tid < digits)
#pragma unroll 16
    for (int s = 0; s < a.sort_tiles; ++s) {
      const int32_t c = a.counts[(int64_t)s * digits + tid];
      all += c;
      if (s < (int)blockIdx.x) before += c;
    }
  __syncthreads();
  for (int s = 0;;) {
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (key[j] >= 0) atomicAdd(&base[wv][(key[j] >> shift) & (digits - 1)], 1);
    if (++s == a.sort_steps) break;
    load(s);
  }
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
  for (int s = 0; s < a.sort_steps; ++s) {
    if (a.sort_steps > 1) load(s);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      int32_t at;
      if (!place_key(key[j], shift, a.bits, base[wv], &at)) continue;
      a.key[pass & 1][at] = key[j];
      a.pos[pass & 1][at] = pos[j];
      if (last && a.touched && key[j] < a.n_rows) a.touched[key[j]] = 1;
    }
  }
}

// The whole sort of up to kGradSmall IDs by one workgroup, the list between
// the passes in LDS: one launch instead of two per pass (3,000 IDs of 768
// rows of 256: 26 us with those, 21 with this; 8,192 IDs: 31 and 31).
__global__ void __launch_bounds__(kGradSmall / 8) k_grad_sort(GradArgs a) {
  constexpr int NT = kGradSmall / 8, NW = NT / 64, PER = 8;
  __shared__ int32_t base[NW][kMaxDigits];
  __shared__ int32_t keys[kGradSmall];
  __shared__ uint16_t places[kGradSmall];
  __shared__ int32_t red[NW];
  const int tid = threadIdx.x, lane = lane_id(), wv = wave_id();
  const int n = (int)a.n_ids, digits = 1 << a.bits, fin = (a.passes - 1) & 1;
  int32_t key[PER], pos[PER];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    pos[j] = wv * (64 * PER) + j * 64 + lane;
    key[j] = pos[j] < n ? a.ids[pos[j]] : -1;
  }
  // (the marks' region is whole 16-byte groups)
  for (int64_t v = (int64_t)tid * 16; v < a.n_rows; v += NT * 16) *(u32x4 *)(a.touched + v) = u32x4{};
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (pos[j] < n) key[j] = grad_key(a, key[j], &bad);
  if (bad) atomicOr(a.status, (int32_t)BPE_STATUS_BAD_ID);
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    for (int d = tid; d < NW * kMaxDigits; d += NT) (&base[0][0])[d] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (key[j] >= 0) atomicAdd(&base[wv][(key[j] >> shift) & (digits - 1)], 1);
    __syncthreads();
    int32_t all = 0, total;
    if (tid < digits)
      for (int w = 0; w < NW; ++w) all += base[w][tid];
    int32_t run = block_excl_sum<int32_t, NT>(all, red, &total);
    if (tid < digits)
      for (int w = 0; w < NW; ++w) {
        const int32_t c = base[w][tid];
        base[w][tid] = run;
        run += c;
      }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      int32_t at;
      if (!place_key(key[j], shift, a.bits, base[wv], &at)) continue;
      if (pass < a.passes - 1) {
        keys[at] = key[j];
        places[at] = (uint16_t)pos[j];
      } else {
        a.key[fin][at] = key[j];
        a.pos[fin][at] = pos[j];
        if (key[j] < a.n_rows) a.touched[key[j]] = 1;
      }
    }
    if (pass == a.passes - 1) break;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = wv * (64 * PER) + j * 64 + lane;
      key[j] = i < n ? keys[i] : -1;
      pos[j] = i < n ? places[i] : 0;
    }
  }
}

// ---- forward, by sorted IDs ------------------------------------------------------
// The same rows in the order of their IDs: one wave per 64 positions of the
// sorted list and 64 vectors of columns loads a row of the table once and
// stores it to all of its positions.  kRunAhead positions' rows are loaded
// before the last ones are stored.  Bound by the stores, whose rows lie in no
// order: the 262,144 IDs of above take 540 us after 30 for the sort (1, 4, 8 or
// 16 waves per workgroup, stored past the caches or not: the same).
constexpr int kRunAhead = 4;

template <typename TI, typename TO, int E>
__global__ void __launch_bounds__(256) k_embed_runs(EmbedArgs a) {
  const int lane = lane_id();
  const int64_t w = (int64_t)blockIdx.x * 4 + uniform_wave_id();
  const int64_t tile = w / a.slabs;
  const int slab = (int)(w - tile * a.slabs);
  const int64_t i0 = tile * 64;
  if (i0 >= a.n_ids) return;
  const int n = (int)min<int64_t>(64, a.n_ids - i0);
  const int c = (slab * 64 + lane) * E, col = min(c, a.width - E);
  const bool mine = c < a.width;
  const int32_t key = a.key[i0 + min(lane, n - 1)], pos = a.pos[i0 + min(lane, n - 1)];
  const int32_t none = (int32_t)a.n_rows;
  Vec<TI, E> x[2][kRunAhead];
  Vec<TO, E> r;
  int32_t cur = -1;
  // (each row's first position loads it; every lane stays active around the
  // lane reads)
  auto fetch = [&](Vec<TI, E> (&y)[kRunAhead], int at) {
#pragma unroll
    for (int j = 0; j < kRunAhead; ++j) {
      const int i = min(at + j, n - 1);
      const int32_t k = lane_value(key, i);
      if (k != none && (i == 0 || k != lane_value(key, i - 1)))
        y[j] = load_vec<TI, E>((const TI *)a.weight + k * a.w_stride + col);
    }
  };
  auto put = [&](Vec<TI, E> (&y)[kRunAhead], int at) {
#pragma unroll
    for (int j = 0; j < kRunAhead; ++j) {
      if (at + j >= n) break;
      const int32_t k = lane_value(key, at + j);
      if (k != cur) {
        cur = k;
#pragma unroll
        for (int e = 0; e < E; ++e)
          r.v[e] = from_f32<TO>(k != none ? (float)y[j].v[e] * a.scale : 0.f);
      }
      const int64_t t = lane_value(pos, at + j);
      if (mine) store_vec<TO, E, true>((TO *)a.out + t * a.o_stride + col, r);
    }
  };
  fetch(x[0], 0);
  for (int b = 0; b < n; b += 2 * kRunAhead) {
    if (b + kRunAhead < n) fetch(x[1], b + kRunAhead);
    put(x[0], b);
    if (b + 2 * kRunAhead < n) fetch(x[0], b + 2 * kRunAhead);
    if (b + kRunAhead < n) put(x[1], b + kRunAhead);
  }
}

// ---- gradient: sums --------------------------------------------------------------
// A lane has 8 columns of a slab of 512: one vector of E = 8 elements, or,
// where either side is float32, two of E = 4 (256 columns apart), so that a
// wave's accesses are whole lines.  Columns of a lane's vector g: its start,
// and how many of its elements belong to its left neighbour (the last vector
// of a row whose width is no multiple of E); false past the row's end.
template <int E>
__device__ __forceinline__ bool grad_col(const GradArgs &a, int vec, int *col, int *skip) {
  const int c = (vec * 64 + lane_id()) * E;
  *col = 0;
  *skip = 0;
  if (c >= a.width) return false;
  *col = min(c, a.width - E);
  *skip = c - *col;
  return true;
}

// Elements before `skip` belong to the left neighbour: loaded, not stored.
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
    store_vec<TO, E, true>(p, r);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e >= skip) p[e] = from_f32<TO>((a.accumulate ? (float)p[e] : 0.f) + acc[e] * a.scale);
  }
}

constexpr int kRowsAhead = 8;  // gradient rows in flight per wave

// Workgroups below sum_blocks: one wave per tile of the sorted list and slab of
// 64 * G vectors of columns, adding up the rows of each ID in the order of the
// list.  A row whose positions all lie in the tile is finished here; of one
// that a tile's edge cuts, the tile's share goes to `part` (slot 0: the row
// began in an earlier tile; slot 1: it begins here and goes on).  The other
// workgroups write zeros to the rows that no ID names.
// The next kRowsAhead rows are loaded before the last ones are worked on: a
// wait for a load waits for every earlier store too, and these are earlier
// than the stores.
// Bound by memory: 131,072 bfloat16 rows of 4,096 into 32,256 float32 rows,
// 1.60 GB, take 329 us, 4.9 TB/s (without the loads ahead 361, with one vector
// of 8 elements per lane 377).
template <typename TG, typename TO, int E, int G>
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
        store_vec<TO, E, true>(p + min(c, a.width - E), z);
    }
    return;
  }
  const int64_t w = (int64_t)blockIdx.x * 4 + wv;
  const int tile = (int)(w / a.slabs), slab = (int)(w - (int64_t)tile * a.slabs);
  if (tile >= a.tiles) return;
  int col[G], skip[G];
  bool mine[G];
#pragma unroll
  for (int g = 0; g < G; ++g) mine[g] = grad_col<E>(a, slab * G + g, &col[g], &skip[g]);
  const int fin = (a.passes - 1) & 1;
  const int64_t i0 = (int64_t)tile * a.tile;
  const int n = (int)min<int64_t>(a.tile, a.n_ids - i0);
  const int32_t none = (int32_t)a.n_rows;
  const int32_t *key = a.key[fin] + i0, *place = a.pos[fin] + i0;
  const int32_t prev = i0 > 0 ? key[-1] : -1;
  const int32_t next = i0 + n < a.n_ids ? key[n] : -1;
  float acc[G][E] = {};
  int32_t cur = key[0];
  if (cur >= none) return;
  bool from_left = cur == prev;
  auto flush = [&](bool to_right) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (!mine[g]) continue;
      if (from_left || to_right) {
        // (a vector that starts inside its left neighbour writes the shared
        // elements a second time with the same values)
        Vec<float, E> r;
#pragma unroll
        for (int e = 0; e < E; ++e) r.v[e] = acc[g][e];
        store_vec<float, E>(
            a.part + ((int64_t)tile * 2 + (from_left ? 0 : 1)) * a.width + col[g], r);
      } else {
        grad_store<TO, E>(a, cur, col[g], skip[g], acc[g]);
      }
    }
  };
  // lane l holds the key and position l of the list's next 64; positions past
  // the last that adds something are not there (they come last)
  int32_t k = lane < n ? key[lane] : none, p = lane < n ? place[lane] : 0;
  Vec<TG, E> x[2][kRowsAhead][G];
  // (lanes past the row's end load its first vector: every lane stays active
  // around the lane reads)
  auto fetch = [&](Vec<TG, E> (&y)[kRowsAhead][G], int at, int m) {
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
      const TG *row = (const TG *)a.grad + (int64_t)lane_value(p, min(at + j, m - 1)) * a.g_stride;
#pragma unroll
      for (int g = 0; g < G; ++g) y[j][g] = load_vec<TG, E, true>(row + col[g]);
    }
  };
  auto add = [&](Vec<TG, E> (&y)[kRowsAhead][G], int32_t keys, int at, int m) {
#pragma unroll
    for (int j = 0; j < kRowsAhead; ++j) {
      if (at + j >= m) break;
      const int32_t kk = lane_value(keys, at + j);
      if (kk != cur) {
        flush(false);
        from_left = false;
        cur = kk;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int e = 0; e < E; ++e) acc[g][e] = 0.f;
      }
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[g][e] += (float)y[j][g].v[e];
    }
  };
  int m = __popcll(__ballot(k < none));
  fetch(x[0], 0, m);
  for (int s = 0;;) {
    // the 64 after these, whose loads end before they are needed
    const int t = s + 64 + lane;
    const int32_t k1 = t < n ? key[t] : none, p1 = t < n ? place[t] : 0;
    const int32_t k0 = k;
    const int m0 = m;
    static_assert(64 % (2 * kRowsAhead) == 0, "two buffers in turn");
    for (int b = 0; b < m0; b += 2 * kRowsAhead) {
      if (b + kRowsAhead < m0) fetch(x[1], b + kRowsAhead, m0);
      add(x[0], k0, b, m0);
      if (b + 2 * kRowsAhead < m0) {
        fetch(x[0], b + 2 * kRowsAhead, m0);
      } else if (m0 == 64) {
        k = k1;
        p = p1;
        m = __popcll(__ballot(k < none));
        if (m > 0) fetch(x[0], 0, m);
      }
      if (b + kRowsAhead < m0) add(x[1], k0, b + kRowsAhead, m0);
    }
    s += 64;
    if (m0 < 64 || s >= n || m == 0) break;
  }
  // (a tile that ends in positions that add nothing: next is `none`, not cur)
  flush(next == cur);
}

// Few IDs (n_ids <= kGradDirect): no sort.  One workgroup per position and two
// slabs; it has work when its position is the first of its ID.  It lists the
// ID's positions in order and adds up their rows: up to kRowsAhead rows by one
// wave per slab, more by all eight waves, every eighth row each, joined in
// order.  The other workgroups mark which of their rows occur and write zeros
// to the rest.  One launch instead of three or four, which is what such a call
// costs: 2,048 IDs of 768 rows of 512 take 10 us, most of it the chain of
// dependent loads (the IDs, the rows of the most frequent ID), and 20 by sorted
// IDs.  Every workgroup reads all IDs again, so the work grows with their square
// and with the width.  The limit kGradDirect fits narrow tables, and is past the
// even point of wide ones; in us, this and the sort, bfloat16 rows:
//                   1,024 IDs     2,048 IDs     4,096 IDs
//   768 x 512          9   19       11   20       21   22
//   768 x 4,096       17   21       30   24       71   31
//   768 x 8,192       29   24       56   29      138   37
//   32,256 x 512      12   29       16   30       29   32
//   32,256 x 4,096    64   68       80   70      126   76
//   32,256 x 8,192   126  119      157  123      244  133
constexpr int kDirectSlabs = 2;
constexpr int kDirectZero = 32;  // rows of the table per workgroup of zeros

template <typename TG, typename TO, int E, int G>
__global__ void __launch_bounds__(kDirectWG) k_grad_direct(GradArgs a) {
  constexpr int NW = kDirectWG / 64, PER = kGradDirect / kDirectWG;
  __shared__ float sh[NW][64][G * E];
  __shared__ int16_t list[kGradDirect];
  __shared__ int32_t red[NW];
  __shared__ int32_t touched[kDirectZero];
  const int tid = threadIdx.x, lane = lane_id(), wv = uniform_wave_id();
  const int n = (int)a.n_ids;
  int32_t id[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) id[j] = a.ids[min(tid * PER + j, n - 1)];
  if (blockIdx.x >= a.sum_blocks) {
    const int64_t r0 = (int64_t)(blockIdx.x - a.sum_blocks) * kDirectZero;
    if (tid < kDirectZero) touched[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (id[j] >= r0 && id[j] < r0 + kDirectZero && id[j] != a.pad_id) touched[id[j] - r0] = 1;
    __syncthreads();
    for (int r = wv; r < kDirectZero && r0 + r < a.n_rows; r += NW) {
      if (touched[r]) continue;
      TO *p = (TO *)a.out + (r0 + r) * a.o_stride;
      Vec<TO, E> z;
#pragma unroll
      for (int e = 0; e < E; ++e) z.v[e] = from_f32<TO>(0.f);
      for (int c = lane * E; c < a.width; c += 64 * E) store_vec<TO, E>(p + min(c, a.width - E), z);
    }
    return;
  }
  const int groups = (a.slabs + kDirectSlabs - 1) / kDirectSlabs;
  const int t = (int)(blockIdx.x / (unsigned)groups);
  const int s0 = (int)(blockIdx.x - (unsigned)(t * groups)) * kDirectSlabs;
  const int s1 = min(s0 + kDirectSlabs, a.slabs);
  bool bad = false;
  const int32_t cur = grad_key(a, a.ids[t], &bad);
  if (bad && s0 == 0 && tid == 0) atomicOr(a.status, (int32_t)BPE_STATUS_BAD_ID);
  if (cur >= a.n_rows) return;
  int32_t mine = 0;
  bool earlier = false;
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (tid * PER + j < n && id[j] == cur) {
      ++mine;
      earlier |= tid * PER + j < t;
    }
  if (__syncthreads_or(earlier)) return;
  int32_t cnt;
  int32_t at = block_excl_sum<int32_t, kDirectWG>(mine, red, &cnt);
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (tid * PER + j < n && id[j] == cur) list[at++] = (int16_t)(tid * PER + j);
  __syncthreads();
  const bool all = cnt > kRowsAhead;  // every wave on every slab
  const int step = all ? NW : 1;
  for (int s = all ? s0 : s0 + wv; s < s1; s += all ? 1 : NW) {
    int col[G], skip[G];
    bool in[G];
#pragma unroll
    for (int g = 0; g < G; ++g) in[g] = grad_col<E>(a, s * G + g, &col[g], &skip[g]);
    float acc[G][E] = {};
    for (int b = all ? wv : 0; b < cnt; b += step * kRowsAhead) {
      Vec<TG, E> x[kRowsAhead][G];
#pragma unroll
      for (int j = 0; j < kRowsAhead; ++j) {
        const TG *row = (const TG *)a.grad + (int64_t)list[min(b + j * step, cnt - 1)] * a.g_stride;
#pragma unroll
        for (int g = 0; g < G; ++g) x[j][g] = load_vec<TG, E>(row + col[g]);
      }
#pragma unroll
      for (int j = 0; j < kRowsAhead; ++j)
        if (b + j * step < cnt) {
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[g][e] += (float)x[j][g].v[e];
        }
    }
    if (all) {
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int e = 0; e < E; ++e) sh[wv][lane][g * E + e] = acc[g][e];
      __syncthreads();
      if (wv == 0) {
#pragma unroll
        for (int w = 1; w < NW; ++w)
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[g][e] += sh[w][lane][g * E + e];
      }
      __syncthreads();
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
      if (in[g] && (!all || wv == 0)) grad_store<TO, E>(a, cur, col[g], skip[g], acc[g]);
  }
}

// Rows that tile edges cut: one workgroup per tile and slab; it has work when a
// row begins in its tile and goes on in the next.  Its four waves add up the
// tiles' shares, every fourth each, and join theirs in order (7 us for 512
// tiles of 4,096 columns).
template <typename TO, int E, int G>
__global__ void __launch_bounds__(256) k_grad_join(GradArgs a) {
  __shared__ float sh[4][64][G * E];
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
  int col[G], skip[G];
  bool mine[G];
#pragma unroll
  for (int g = 0; g < G; ++g) mine[g] = grad_col<E>(a, slab * G + g, &col[g], &skip[g]);
  // (lanes past the row's end add up its first vector and store nothing)
  float acc[G][E] = {};
  const float *p = a.part + (int64_t)tile * 2 * a.width;
  if (wv == 0) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const Vec<float, E> x = load_vec<float, E>(p + a.width + col[g]);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[g][e] = x.v[e];
    }
  }
#pragma unroll 4
  for (int j = 1 + wv; j <= run; j += 4) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const Vec<float, E> x = load_vec<float, E>(p + (int64_t)j * 2 * a.width + col[g]);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[g][e] += x.v[e];
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int e = 0; e < E; ++e) sh[wv][lane][g * E + e] = acc[g][e];
  __syncthreads();
  if (wv == 0) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
      for (int w = 1; w < 4; ++w)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[g][e] += sh[w][lane][g * E + e];
      if (mine[g]) grad_store<TO, E>(a, cur, col[g], skip[g], acc[g]);
    }
  }
}

template <typename TI, typename TO, int E, bool BIG>
hipError_t embed_as(EmbedArgs a, hipStream_t stream) {
  constexpr int U = kEmbedUnits / 256;
  a.units = (uint32_t)((a.width + E - 1) / E);
  a.magic = (1u << 31) / a.units + 1;
  const int64_t groups = (a.n_ids * a.units + kEmbedUnits - 1) / kEmbedUnits;
  hipLaunchKernelGGL((k_embed<TI, TO, E, U, BIG>), dim3((unsigned)groups), dim3(256), 0,
                     stream, a);
  return hipGetLastError();
}

void launch_sort(const GradArgs &a, hipStream_t stream) {
  for (int pass = 0; pass < a.passes; ++pass) {
    hipLaunchKernelGGL(k_grad_count, dim3(a.sort_tiles), dim3(kSortThreads), 0, stream, a, pass);
    hipLaunchKernelGGL(k_grad_scatter, dim3(a.sort_tiles), dim3(kSortThreads), 0, stream, a, pass);
  }
}

template <typename TI, typename TO>
hipError_t embed_of(EmbedArgs a, hipStream_t stream) {
  if (a.width < 8) return embed_as<TI, TO, 1, false>(a, stream);
  const bool big = a.n_ids * a.width * (int64_t)sizeof(TO) >= kStreamBytes;
  constexpr int E = 16 / sizeof(TO);
  if (a.key) {
    a.slabs = (a.width + 64 * E - 1) / (64 * E);
    const int64_t waves = (a.n_ids + 63) / 64 * a.slabs;
    hipLaunchKernelGGL((k_embed_runs<TI, TO, E>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0,
                       stream, a);
    return hipGetLastError();
  }
  return big ? embed_as<TI, TO, E, true>(a, stream) : embed_as<TI, TO, E, false>(a, stream);
}

template <typename TI>
hipError_t embed_from(const EmbedArgs &a, int ot, hipStream_t stream) {
  if (ot == BPE_F32) return embed_of<TI, float>(a, stream);
  if (ot == BPE_BF16) return embed_of<TI, bf16_t>(a, stream);
  return embed_of<TI, f16_t>(a, stream);
}

template <typename TG, typename TO, int E, int G>
hipError_t grad_as(GradArgs a, hipStream_t stream) {
  a.slabs = (a.width + 64 * G * E - 1) / (64 * G * E);
  if (a.n_ids > 0 && a.n_ids <= kGradDirect) {
    a.sum_blocks = a.n_ids * ((a.slabs + kDirectSlabs - 1) / kDirectSlabs);
    const int64_t zero = a.accumulate ? 0 : (a.n_rows + kDirectZero - 1) / kDirectZero;
    hipLaunchKernelGGL((k_grad_direct<TG, TO, E, G>), dim3((unsigned)(a.sum_blocks + zero)),
                       dim3(kDirectWG), 0, stream, a);
    return hipGetLastError();
  }
  const bool small = a.n_ids <= kGradSmall && a.n_rows <= kGradSmallRows;
  if (a.n_ids > 0 && small)
    hipLaunchKernelGGL(k_grad_sort, dim3(1), dim3(kGradSmall / 8), 0, stream, a);
  if (a.n_ids > 0 && !small) launch_sort(a, stream);
  a.sum_blocks = a.n_ids > 0 ? ((int64_t)a.tiles * a.slabs + 3) / 4 : 0;
  const int64_t zero = a.accumulate ? 0 : (a.n_rows + kZeroRows - 1) / kZeroRows;
  if (a.sum_blocks + zero > 0)
    hipLaunchKernelGGL((k_grad_sum<TG, TO, E, G>), dim3((unsigned)(a.sum_blocks + zero)), dim3(256),
                       0, stream, a);
  if (a.n_ids > a.tile)
    hipLaunchKernelGGL((k_grad_join<TO, E, G>), dim3((unsigned)((int64_t)a.tiles * a.slabs)),
                       dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <typename TG, typename TO>
hipError_t grad_of(const GradArgs &a, hipStream_t stream) {
  if (a.width < 8) return grad_as<TG, TO, 1, 1>(a, stream);
  if constexpr (sizeof(TG) == 4 || sizeof(TO) == 4) return grad_as<TG, TO, 4, 2>(a, stream);
  else return grad_as<TG, TO, 8, 1>(a, stream);
}

template <typename TG>
hipError_t grad_from(const GradArgs &a, int ot, hipStream_t stream) {
  if (ot == BPE_F32) return grad_of<TG, float>(a, stream);
  if (ot == BPE_BF16) return grad_of<TG, bf16_t>(a, stream);
  return grad_of<TG, f16_t>(a, stream);
}

}  // namespace

hipError_t launch_embed(const EmbedArgs &a, const GradArgs *sort, int wt, int ot,
                        hipStream_t stream) {
  if (sort) launch_sort(*sort, stream);
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
