// lm_verify.hip -- drafted tokens against the target's probabilities, and the
// token drawn after those that stand.
#include "lm_device.h"

namespace bpe {
namespace {

constexpr int TILE = kVerifyTile;  // tokens: 8 per lane of a wave
static_assert(TILE == 64 * 8, "8 per lane");

// The sum over the lanes below and this one, every lane active: six DPP moves and
// adds (prefixes of rows of 16 lanes, then of rows and halves).
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_f64(double v) {
  return __longlong_as_double(dpp64<CTRL, ROW_MASK>(__double_as_longlong(v)));
}
__device__ __forceinline__ double wave_scan(double v) {
  v += dpp_f64<0x111, 0xF>(v);
  v += dpp_f64<0x112, 0xF>(v);
  v += dpp_f64<0x114, 0xF>(v);
  v += dpp_f64<0x118, 0xF>(v);
  v += dpp_f64<0x142, 0xA>(v);
  v += dpp_f64<0x143, 0xC>(v);
  return v;
}
// Lane l's value in every lane (l the same in every lane).
__device__ __forceinline__ double lane_f64(double v, int l) {
  return __longlong_as_double(lane_value((int64_t)__double_as_longlong(v), l));
}

// A probability; what is none (all but positive normal and subnormal numbers, one
// comparison by class) counts as 0.
__device__ __forceinline__ float probability(float x) {
  return __builtin_amdgcn_classf(x, 0x180) ? x : 0.f;
}

// A request's rows; none where its offsets are not valid.
struct Rows {
  int64_t lo, hi;
  bool bad;
};
__device__ __forceinline__ Rows load_rows(const VerifyArgs &a, int64_t r) {
  Rows q = {a.off[r], a.off[r + 1], false};
  if (q.lo < 0 || q.hi < q.lo || q.hi > a.n_rows) {
    q.bad = true;
    q.hi = q.lo;
  }
  return q;
}

// The first row whose draft does not stand, less lo; the last row if all do.  Each
// wave by itself, a lane per row.
template <typename T, bool DRAFT>
__device__ __forceinline__ int first_rejected(const VerifyArgs &a, const Rows &rows) {
  const int n_drafts = (int)(rows.hi - rows.lo - 1);
  for (int s = 0; s < n_drafts; s += 64) {
    const int i = s + lane_id();
    bool stands = i < n_drafts;
    if (stands) {
      const int64_t row = rows.lo + i;
      const int32_t x = a.ids[row];
      const float u = a.accept[row];
      stands = x >= 0 && x < a.vocab;
      if (stands) {
        const float p = probability((float)((const T *)a.target)[row * a.t_stride + x]);
        const float q = DRAFT ? probability((float)((const T *)a.draft)[row * a.d_stride + x]) : 1.f;
        stands = (double)u * (double)q < (double)p;  // (exact)
      }
    }
    const uint64_t not_ = ~__ballot(stands);
    if (not_) return s + __ffsll((unsigned long long)not_) - 1;
  }
  return n_drafts;
}

// The row to draw from.
template <typename T, bool DRAFT>
struct Row {
  static constexpr int E = 16 / sizeof(T), N = 8 / E;  // vectors of 8 tokens
  const T *p, *q;
  int V;
  int32_t drafted;

  __device__ __forceinline__ Row(const VerifyArgs &a, int64_t row, bool rejected) {
    p = (const T *)a.target + row * a.t_stride;
    q = DRAFT ? (const T *)a.draft + row * a.d_stride : nullptr;
    V = (int)a.vocab;
    drafted = !DRAFT && rejected ? a.ids[row] : -1;
  }

  // 8 tokens' probabilities, as they lie in memory.
  struct Eight {
    Vec<T, E> x[N], y[N];
  };
  // Those from v on: unconditional loads, so that many are in flight together; past
  // the row's last 8 tokens those.  (V >= 8)
  template <bool LESS>
  __device__ __forceinline__ void load(int64_t v, Eight *r) const {
    const int at = (int)min<int64_t>(v, V - 8);
#pragma unroll
    for (int i = 0; i < N; ++i) r->x[i] = load_vec<T, E>(p + at + i * E);
    if (DRAFT && LESS) {
#pragma unroll
      for (int i = 0; i < N; ++i) r->y[i] = load_vec<T, E>(q + at + i * E);
    }
  }
  template <bool LESS>
  __device__ __forceinline__ double weight(float x, float y, int64_t v) const {
    float w = probability(x);
    if (!LESS) return w;
    // (the larger one, less the other: the difference or 0 with one operation in
    // 64 bits, which cost more)
    if (DRAFT) return (double)fmaxf(w, probability(y)) - (double)probability(y);
    return v == drafted ? (double)fmaxf(w, 1.f) - 1.0 : (double)w;
  }
  // Their weights; zeros past the row's end.
  template <bool LESS>
  __device__ __forceinline__ void weights(int64_t v, const Eight &r, double *w) const {
    if (v + 8 <= V) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = weight<LESS>((float)r.x[i / E].v[i % E], DRAFT && LESS ? (float)r.y[i / E].v[i % E] : 0.f, v + i);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = v + i < V ? weight<LESS>((float)p[v + i], DRAFT && LESS ? (float)q[v + i] : 0.f, v + i) : 0.0;
    }
  }
};

// The sums of the four regions from g on, a wave's, in every lane.
template <typename T, bool DRAFT, bool LESS>
__device__ __forceinline__ void four_sums(const VerifyArgs &a, const Row<T, DRAFT> &row, int g, double *sum) {
  const int lane = lane_id();
  const int64_t region = (int64_t)a.tiles * TILE, v0 = g * region + lane * 8;
  double s[4] = {};
  for (int t = 0; t < a.tiles; ++t) {
    typename Row<T, DRAFT>::Eight x[4];
    if (row.V >= 8) {
#pragma unroll
      for (int k = 0; k < 4; ++k) row.template load<LESS>(v0 + k * region + t * TILE, &x[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      double w[8];
      row.template weights<LESS>(v0 + k * region + t * TILE, x[k], w);
      s[k] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) sum[k] = lane_f64(wave_scan(s[k]), 63);
}
template <typename T, bool DRAFT>
__device__ __forceinline__ void four_sums(const VerifyArgs &a, const Row<T, DRAFT> &row, int g, bool less,
                                          double *sum) {
  if (less) four_sums<T, DRAFT, true>(a, row, g, sum);
  else four_sums<T, DRAFT, false>(a, row, g, sum);
}

// The first of the values that a lane holds (n of them from index i0 on, by get)
// whose running sum, over the lanes and then over each lane's values, passes
// `share`; -1 if none does.  *before: the sum of those before it.  *last: the last
// index with a positive value.  All in every lane.
template <typename F>
__device__ __forceinline__ int64_t first_past(F get, int n, int64_t i0, double share, double *before,
                                              int64_t *last) {
  double mine = 0.0;
  for (int i = 0; i < n; ++i) mine += get(i);
  const double inc = wave_scan(mine);
  double run = *before + (inc - mine), at = 0.0;
  int hit = -1, top = -1;
  for (int i = 0; i < n; ++i) {
    const double w = get(i), next = run + w;
    if (w > 0.0) {
      if (next > share && hit < 0) {
        hit = i;
        at = run;
      }
      top = i;
    }
    run = next;
  }
  const uint64_t hits = __ballot(hit >= 0), some = __ballot(top >= 0);
  if (some) {
    const int l = 63 - __clzll((long long)some);
    *last = lane_value(i0 + top, l);
  }
  if (!hits) {
    *before += lane_f64(inc, 63);
    return -1;
  }
  const int l = __ffsll((unsigned long long)hits) - 1;
  *before = lane_f64(at, l);
  return lane_value(i0 + hit, l);
}

// The token drawn from a row whose regions' sums are there, or -1: a wave's work.
// The region in which the running sum passes the sampled share of the total, read
// again (from L2), and the token in it.  Which sums decide is fixed by the sizes
// alone.  A region's sum and its scan add in different orders; where that leaves
// no token past the share in the region, its last one of positive weight is it.
template <typename T, bool DRAFT, typename F>
__device__ __forceinline__ int32_t draw(const VerifyArgs &a, const Row<T, DRAFT> &row, bool less, float u, F sum) {
  const int lane = lane_id(), per = (a.regions + 63) / 64;
  // a lane's regions are consecutive; those of up to 131,072 tokens are loaded
  // together and kept
  constexpr int KEPT = 4;
  double kept[KEPT];
#pragma unroll
  for (int i = 0; i < KEPT; ++i) {
    const int g = lane * per + i;
    kept[i] = i < per && g < a.regions ? sum(g) : 0.0;
  }
  auto mine = [&](int i) { return lane * per + i < a.regions ? sum(lane * per + i) : 0.0; };
  double total = 0.0;
  if (per <= KEPT) {
#pragma unroll
    for (int i = 0; i < KEPT; ++i) total += kept[i];
  } else {
    for (int i = 0; i < per; ++i) total += mine(i);
  }
  total = lane_f64(wave_scan(total), 63);
  if (!(total > 0.0)) return -1;
  // (past the upper end, NaN included, the last token of positive weight)
  const double share = u < 1.f ? fmax((double)u, 0.0) * total : total;
  double before = 0.0;
  int64_t g_last = 0, last = -1;
  int64_t g = per <= KEPT ? first_past([&](int i) { return kept[i]; }, KEPT, lane * per, share, &before, &g_last)
                          : first_past(mine, per, lane * per, share, &before, &g_last);
  if (g < 0) {
    g = g_last;
    before = -INFINITY;  // its last token of positive weight
  }
  const int64_t begin = g * ((int64_t)a.tiles * TILE);
  for (int t = 0; t < a.tiles; ++t) {
    const int64_t v = begin + t * TILE + lane * 8;
    typename Row<T, DRAFT>::Eight x;
    double w[8];
    if (less) {
      if (row.V >= 8) row.template load<true>(v, &x);
      row.template weights<true>(v, x, w);
    } else {
      if (row.V >= 8) row.template load<false>(v, &x);
      row.template weights<false>(v, x, w);
    }
    const int64_t hit = first_past([&](int i) { return w[i]; }, 8, v, share,
                                   &before, &last);
    if (hit >= 0) return (int32_t)hit;
  }
  return (int32_t)last;
}

// The sums of the rows to draw from by regions, four a wave, so that few requests
// fill the GPU too.  Each wave looks at the request's drafts itself: a lane each, no
// barrier.  192 requests of 128,256 float32 tokens, four drafts at most, read 131 MB
// in 26 us, 5.0 TB/s, bound by memory.  (A workgroup per request alone took 44 us
// for them, bound by what one CU has in flight.)
template <typename T, bool DRAFT>
__global__ void __launch_bounds__(kVerifyThreads) k_verify_sums(VerifyArgs a) {
  constexpr int W = kVerifyThreads / 64;
  const uint32_t per = (uint32_t)((a.regions / 4 + W - 1) / W);  // workgroups a request
  const uint32_t r = blockIdx.x / per;
  const int g = (int)((blockIdx.x - r * per) * W + uniform_wave_id()) * 4;
  const Rows rows = load_rows(a, r);
  if (rows.lo == rows.hi || g >= a.regions) return;
  const int j = first_rejected<T, DRAFT>(a, rows);
  const bool rejected = rows.lo + j < rows.hi - 1;
  const Row<T, DRAFT> row(a, rows.lo + j, rejected);
  double sum[4];
  four_sums(a, row, g, rejected, sum);
  const int lane = lane_id();
  if (lane < 4)
    a.sums[(int64_t)r * a.regions + g + lane] = lane < 2 ? (lane == 0 ? sum[0] : sum[1]) : lane == 2 ? sum[2] : sum[3];
  if (g == 0 && lane == 0) a.rows[r] = j;
}

// The next tokens.  ALONE: a workgroup per request, whose waves add up the regions
// and whose first one draws; else a wave per request, after k_verify_sums.  A chain
// of dependent accesses: 4.1 us after the sums; alone 6.6 us for up to 16,384 tokens
// and 11.5 for 50,256 (4 requests; two launches of 4.4 and 4.1).  The drawing is one
// wave's, by DPP scans without barriers: a workgroup's scans took twice as long.
template <typename T, bool DRAFT, bool ALONE>
__global__ void __launch_bounds__(ALONE ? kVerifyAloneThreads : 64) k_verify_draw(VerifyArgs a) {
  __shared__ double sums[ALONE ? kVerifyAlone / TILE : 1];
  const int lane = lane_id(), wave = uniform_wave_id();
  const int64_t r = blockIdx.x;
  const Rows rows = load_rows(a, r);
  uint32_t status = rows.bad ? BPE_STATUS_BAD_ID_OFFSETS : 0;
  if (rows.lo == rows.hi) {
    if (threadIdx.x == 0) {
      a.counts[r] = 0;
      if (status) atomicOr(a.status, (int32_t)status);
    }
    return;
  }
  const int n = (int)(rows.hi - rows.lo);
  const float u = a.sample[r];
  const int j = ALONE ? first_rejected<T, DRAFT>(a, rows) : __builtin_amdgcn_readfirstlane(a.rows[r]);
  const bool rejected = j < n - 1;
  const Row<T, DRAFT> row(a, rows.lo + j, rejected);
  int32_t token;
  if (ALONE) {
    for (int again = 0;; ++again) {
      for (int g = wave * 4; g < a.regions; g += (int)blockDim.x / 16) {
        double sum[4];
        four_sums(a, row, g, rejected && !again, sum);
        if (lane == 0) {
#pragma unroll
          for (int k = 0; k < 4; ++k) sums[g + k] = sum[k];
        }
      }
      __syncthreads();
      token = draw(a, row, rejected && !again, u, [&](int g) { return sums[g]; });
      // nothing is left of the difference: the target's own row
      if (token >= 0 || !rejected || again) break;
      __syncthreads();
    }
    if (wave != 0) return;
  } else {
    double *sums = a.sums + r * a.regions;
    token = draw(a, row, rejected, u, [&](int g) { return sums[g]; });
    if (token < 0 && rejected) {
      for (int g = 0; g < a.regions; g += 4) {
        double sum[4];
        four_sums(a, row, g, false, sum);
        if (lane == 0) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            __hip_atomic_store(&sums[g + k], sum[k], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
      }
      __threadfence();
      token = draw(a, row, false, u, [&](int g) {
        return __hip_atomic_load(&sums[g], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      });
    }
  }
  if (token < 0) status |= BPE_STATUS_NO_TOKEN;
  for (int i = lane; i < n; i += 64) {
    const int32_t x = a.ids[rows.lo + i];
    if (i == j && rejected && (x < 0 || x >= a.vocab)) status |= BPE_STATUS_BAD_ID;
    a.tokens[rows.lo + i] = i < j ? x : i == j ? token : -1;
  }
  if (lane == 0) a.counts[r] = j + (token >= 0);
  if (status) atomicOr(a.status, (int32_t)status);
}

template <typename T, bool DRAFT>
hipError_t verify_launch(const VerifyArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)a.R);
  if (verify_alone(a.R, a.vocab)) {
    // (a wave per four regions)
    const int threads = a.regions * 16 < kVerifyAloneThreads ? a.regions * 16 : kVerifyAloneThreads;
    hipLaunchKernelGGL((k_verify_draw<T, DRAFT, true>), grid, dim3(threads), 0, stream, a);
  } else {
    hipLaunchKernelGGL((k_verify_sums<T, DRAFT>), dim3((unsigned)verify_workgroups(a.R, a.vocab)),
                       dim3(kVerifyThreads), 0, stream, a);
    hipLaunchKernelGGL((k_verify_draw<T, DRAFT, false>), grid, dim3(64), 0, stream, a);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t verify_as(const VerifyArgs &a, hipStream_t stream) {
  return a.draft ? verify_launch<T, true>(a, stream) : verify_launch<T, false>(a, stream);
}

}  // namespace

hipError_t launch_verify(const VerifyArgs &a, int type, hipStream_t stream) {
  if (type == BPE_F32) return verify_as<float>(a, stream);
  if (type == BPE_BF16) return verify_as<bf16_t>(a, stream);
  return verify_as<f16_t>(a, stream);
}

}  // namespace bpe
