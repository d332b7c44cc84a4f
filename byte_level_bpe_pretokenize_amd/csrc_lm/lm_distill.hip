// lm_distill.hip -- the divergence of a student's distribution from a teacher's
// over its top tokens, and its gradient.
#include <float.h>

#include "lm_device.h"

namespace bpe {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// A running maximum and the sum of exp((x - maximum) / T) below it, k = log2(e) /
// T.  It starts at the lowest finite value: a -infinity adds 0 to that, and a row
// of lowest values is still a distribution.  A NaN or +infinity makes the sum NaN.
struct Soft {
  float m, s;
};
constexpr Soft kNothing = {-FLT_MAX, 0.f};

__device__ __forceinline__ float power(float x, float k) { return __builtin_amdgcn_exp2f(x * k); }

// The largest of the wave's values and their sum, in every lane (every lane
// active): six DPP moves each, as in wave_incl_sum.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float moved(float old, float x) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(x), CTRL, ROW_MASK, 0xF, false));
}
__device__ __forceinline__ float lane63(float x) {
  return __int_as_float(lane_value(__float_as_int(x), 63));
}
__device__ __forceinline__ float wave_largest(float x) {
  x = fmaxf(x, moved<0x111, 0xF>(x, x));
  x = fmaxf(x, moved<0x112, 0xF>(x, x));
  x = fmaxf(x, moved<0x114, 0xF>(x, x));
  x = fmaxf(x, moved<0x118, 0xF>(x, x));
  x = fmaxf(x, moved<0x142, 0xA>(x, x));
  x = fmaxf(x, moved<0x143, 0xC>(x, x));
  return lane63(x);
}
__device__ __forceinline__ float wave_total(float x) {
  x += moved<0x111, 0xF>(0.f, x);
  x += moved<0x112, 0xF>(0.f, x);
  x += moved<0x114, 0xF>(0.f, x);
  x += moved<0x118, 0xF>(0.f, x);
  x += moved<0x142, 0xA>(0.f, x);
  x += moved<0x143, 0xC>(0.f, x);
  return lane63(x);
}
__device__ __forceinline__ Soft wave_soft(Soft x, float k) {
  const float m = wave_largest(x.m);
  return Soft{m, wave_total(x.s * power(x.m - m, k))};
}

// Elements of p[0 .. n) before its first 16-byte boundary.  Rows of odd width start
// anywhere: 4,096 rows of 50,257 bfloat16 logits take 75 us with vectors from the
// boundary on, 92 from the row's start (float32: no difference; short rows: slower), of
// the same logits each time; 83 where two batches are read in turn.
template <typename T>
__device__ __forceinline__ int before_16(const T *p, int n) {
  return min(n, (int)((0 - (uintptr_t)p) & 15) / (int)sizeof(T));
}

// An entry of a teacher's row: its token's place, or -1.
struct Entry {
  int32_t id;
  float t;
};
// (The teacher's type is a branch: lists are short, and a kernel for each type would
// be three times the code.)
__device__ __forceinline__ Entry load_entry(const DistillArgs &a, int64_t n, int j) {
  Entry x = {-1, -INFINITY};
  if (j < a.top) {
    x.id = a.ids[n * a.i_stride + j];
    const int64_t at = n * a.t_stride + j;
    x.t = a.t_type == BPE_F32    ? ((const float *)a.teacher)[at]
          : a.t_type == BPE_BF16 ? (float)((const bf16_t *)a.teacher)[at]
                                 : (float)((const f16_t *)a.teacher)[at];
  }
  return x;
}

// The sum over a workgroup's threads, in each of them.
template <int NT>
__device__ __forceinline__ double group_sum(double x, double *lds) {
  x = wave_sum(x);
  if (NT == 64) return x;
  __syncthreads();
  if (lane_id() == 0) lds[wave_id()] = x;
  __syncthreads();
  x = 0.0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) x += lds[w];
  return x;
}

// ---- warm rows ------------------------------------------------------------------
// A loss is T^2 times a divergence that falls with T^2 where the listed tokens are
// (nearly) all that the student gives anything to, and a gradient T times a difference
// that falls with T.  From sums in 32 bits, which are off by some 2^-23, a loss of
// 0.005 over 1,000 of 1,000 tokens came out off by 0.5% at T = 32, by its double at
// 256, and negative at 4,096.  So above kDistillWarm, where the listed tokens hold
// more than 3 / 4 of the student's sum, both come from the tokens' differences, each
// of which is exact in 64 bits: with e_j = exp((t_j - largest t) / T), f_j the same of
// the student's listed z_j, d_j = ((t_j - largest t) - (z_j - largest z)) / T, mean
// and sums over the list weighted by e,
//   loss / T^2 = log(1 + sum e_j (exp(x_j) - 1 - x_j) / sum e_j) + log(1 + rest / sum f_j)
//   x_j = mean d - d_j,   log(q_j / P_j) = x_j - loss / T^2
// with rest the student's sum less sum f_j.  No term of the first logarithm is negative,
// so e's roundings (32 bits) are relative to it.  The rest is the sum over all logits,
// read again now that the largest is known, less that over the listed ones: of the
// same 32-bit values, added in 64 bits, so that what is listed leaves nothing.  (With
// more rest the loss is T^2 / 4 at least, and sums in 32 bits are near enough.)
struct Near {
  double mean, loss;  // (loss: infinite or NaN where a listed logit is; of the row / T^2)
};
// get(j, &e, &f, &d): entry j's, and whether it holds a token with e > 0.  held: sum f.
template <typename TS, int NT, typename F>
__device__ __forceinline__ Near near_teacher(F get, int top, const TS *z, int V, float zm, float k, double held,
                                             double *lds) {
  constexpr int E = 16 / sizeof(TS);
  const int tid = threadIdx.x;
  float e, f;
  double d, weight = 0.0, sum = 0.0, all = 0.0;
  for (int j = tid; j < top; j += NT) {
    if (!get(j, &e, &f, &d)) continue;
    weight += (double)e;
    sum += (double)e * d;
  }
  weight = group_sum<NT>(weight, lds);
  Near r;
  r.mean = group_sum<NT>(sum, lds) / weight;
  sum = 0.0;
  for (int j = tid; j < top; j += NT) {
    if (!get(j, &e, &f, &d)) continue;
    const double x = r.mean - d;
    sum += (double)e * (expm1(x) - x);
  }
  sum = group_sum<NT>(sum, lds) / weight;
  for (int v = tid * E; v < V; v += NT * E) {
    if (v + E <= V) {
      const Vec<TS, E> y = load_vec<TS, E>(z + v);
#pragma unroll
      for (int i = 0; i < E; ++i) all += (double)power((float)y.v[i] - zm, k);
    } else {
      for (int i = v; i < V; ++i) all += (double)power((float)z[i] - zm, k);
    }
  }
  all = group_sum<NT>(all, lds);
  r.loss = log1p(sum) + log1p((all - held) / held);
  return r;
}

// A workgroup per row: one pass over the logits with a running maximum and sum
// per thread, joined over the workgroup; the listed logits are gathered before.
// 4,096 rows of 128,256 bfloat16 logits, 1.05 GB, take 184 us, 5.7 TB/s, bound by
// memory (the vector instructions alone would take about two thirds of that).  Few
// rows are bound by what one CU reads: 48 rows of 32,256 6.6 us, one of 128,256 11.1
// (workgroups of 1,024 threads were no faster from 1 to 1,500 rows, and slower for
// many).
// With e_j = exp((t_j - largest t) / T), the loss is
//   T^2 (sum e_j ((t_j - largest t) - (z_j - largest z)) / (T sum e_j) + log (sum z / sum t))
// whose logarithm and sum are in 64 bits: it is the difference of values larger
// than itself where the student is near the teacher.  WARM: see above.
template <typename TS, int NT, bool WARM>
__global__ void __launch_bounds__(NT) k_distill(DistillArgs a) {
  constexpr int E = 16 / sizeof(TS), U = 4, STEP = NT * E;
  constexpr int W = NT / 64;
  __shared__ Soft soft_z[W], soft_t[W];
  __shared__ double terms[W];
  const int tid = threadIdx.x, lane = lane_id(), wave = wave_id();
  const int64_t n = blockIdx.x;
  const TS *z = (const TS *)a.student + n * a.s_stride;
  const int V = (int)a.vocab;
  const float k = kLog2e / a.temperature;
  uint32_t status = 0;
  auto valid = [&](const Entry &x) { return x.id >= 0 && x.id < V; };
  const Entry first = load_entry(a, n, tid);
  const float z_first = valid(first) ? (float)z[first.id] : 0.f;
  Soft x = kNothing;
  auto add = [&](const Vec<TS, E> &v) {
    float m = x.m;
#pragma unroll
    for (int e = 0; e < E; ++e) m = fmaxf(m, (float)v.v[e]);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += power((float)v.v[e] - m, k);
    x.s = x.s * power(x.m - m, k) + s;
    x.m = m;
  };
  // whole lines: what comes before the row's first 16-byte boundary is added alone
  const int head = sizeof(TS) == 2 && NT > 64 ? before_16(z, V) : 0;
  if (tid < head) {
    Vec<TS, E> y;
#pragma unroll
    for (int e = 0; e < E; ++e) y.v[e] = e == 0 ? z[tid] : (TS)-INFINITY;
    add(y);
  }
  int v = head;
  for (; v + STEP * U <= V; v += STEP * U) {
    Vec<TS, E> y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) y[u] = load_vec<TS, E>(z + v + u * STEP + tid * E);
#pragma unroll
    for (int u = 0; u < U; ++u) add(y[u]);
  }
  for (v += tid * E; v < V; v += STEP) {
    Vec<TS, E> y;
    if (v + E <= V) {
      y = load_vec<TS, E>(z + v);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) y.v[e] = v + e < V ? z[v + e] : (TS)-INFINITY;
    }
    add(y);
  }
  Soft t = kNothing;
  for (int j = tid; j < a.top; j += NT) {
    const Entry y = j == tid ? first : load_entry(a, n, j);
    if (y.id < -1 || y.id >= V) status |= BPE_STATUS_BAD_ID;
    if (!valid(y)) continue;
    const float m = fmaxf(t.m, y.t);
    t.s = t.s * power(t.m - m, k) + power(y.t - m, k);
    t.m = m;
  }
  x = wave_soft(x, k);
  t = wave_soft(t, k);
  if (W > 1) {
    if (lane == 0) {
      soft_z[wave] = x;
      soft_t[wave] = t;
    }
    __syncthreads();
    x = wave_soft(lane < W ? soft_z[lane] : kNothing, k);
    t = wave_soft(lane < W ? soft_t[lane] : kNothing, k);
  }
  const double by = 1.0 / (double)a.temperature;
  double sum = 0.0, held = 0.0;
  for (int j = tid; j < a.top; j += NT) {
    const Entry y = j == tid ? first : load_entry(a, n, j);
    if (!valid(y)) continue;
    const float zj = j == tid ? z_first : (float)z[y.id];
    const float e = power(y.t - t.m, k);
    if (e != 0.f) sum += (double)e * (((double)y.t - t.m) - ((double)zj - x.m));
    if (WARM && e != 0.f) held += (double)power(zj - x.m, k);
  }
  double warm = INFINITY;
  if (WARM) {
    held = group_sum<NT>(held, terms);
    if (held > 0.75 * (double)x.s) {  // (the same in every thread)
      auto get = [&](int j, float *e, float *f, double *d) {
        const Entry y = load_entry(a, n, j);
        if (!valid(y)) return false;
        const float zj = (float)z[y.id];
        *e = power(y.t - t.m, k);
        *f = power(zj - x.m, k);
        *d = (((double)y.t - t.m) - ((double)zj - x.m)) * by;
        return *e != 0.f;
      };
      warm = near_teacher<TS, NT>(get, a.top, z, V, x.m, k, held, terms).loss;
    }
    if (W > 1) __syncthreads();  // (terms)
  }
  sum = wave_sum(sum);
  if (W > 1) {
    if (lane == 0) terms[wave] = sum;
    __syncthreads();
  }
  if (tid == 0) {
    if (W > 1) {
      sum = 0.0;
      for (int w = 0; w < W; ++w) sum += terms[w];
    }
    const bool some = x.s != 0.f && t.s != 0.f;
    const double T = a.temperature;
    const double loss = WARM && warm < INFINITY ? warm : sum * by / t.s + log((double)x.s / t.s);
    a.losses[n] = some ? (float)(T * T * loss) : 0.f;
    float *o = a.stats + n * 4;
    o[0] = x.m;
    o[1] = x.s;
    o[2] = t.m;
    o[3] = t.s;
  }
  if (status) atomicOr(a.status, (int32_t)status);
}

// A workgroup per row and slab of logits: all of them as if nothing were listed,
// then the listed ones of the slab again.  (Few are listed: asked for at every
// logit they would cost more.)  A token that is listed twice gets the same value
// from both entries: each adds up all of the token's, in their order.  Which ones
// are is known from two bits for each of the slab's logits: listed, and listed by
// another entry too (adding up over the list for every entry took 118 us instead of
// 28 for 16,000 rows of 876 with lists of 200).  4,096 rows of 128,256 bfloat16
// logits, 2.1 GB, take 380 us, 5.5 TB/s, bound by memory; with the table as a word
// per logit, 32 KB of LDS more, 418.  WARM (of rows that are one slab: what is listed
// may be overwritten by another one's workgroup): see above.
template <typename TS, typename TG, int NT, int S, bool STREAM, bool WARM>
__global__ void __launch_bounds__(NT) k_distill_grad(DistillArgs a) {
  constexpr int E = sizeof(TS) == 2 && sizeof(TG) == 2 ? 8 : 4;
  constexpr int U = 4;
  __shared__ uint32_t seen[S / 32], twice[S / 32];
  extern __shared__ __align__(16) int32_t lds[];
  const int top8 = (a.top + 7) / 8 * 8;
  int32_t *ids = lds;
  float *parts = (float *)(ids + top8), *listed = parts + top8;  // (their logits)
  float *theirs = listed + top8;                                 // (WARM: the teacher's)
  const int tid = threadIdx.x;
  const uint32_t slabs = (uint32_t)((a.vocab + S - 1) / S);
  const uint32_t row = blockIdx.x / slabs, slab = blockIdx.x - row * slabs;
  const int64_t n = row;
  const int v0 = (int)(slab * S);
  const int count = (int)min<int64_t>(S, a.vocab - v0);
  const TS *z = (const TS *)a.student + n * a.s_stride + v0;
  TG *g = (TG *)a.grad + n * a.g_stride + v0;
  const float zm = a.in_stats[n * 4], zs = a.in_stats[n * 4 + 1];
  const float tm = a.in_stats[n * 4 + 2], ts = a.in_stats[n * 4 + 3];
  const bool some = zs != 0.f && ts != 0.f;
  const float k = kLog2e / a.temperature;
  const float c = some ? a.dloss[n] * a.temperature : 0.f;
  const float by_zs = 1.f / zs, by_ts = 1.f / ts;
  auto share = [&](float x) { return power(x - zm, k) * by_zs; };
  // an entry's place in the slab, or a number past it
  auto place = [&](int32_t id) { return (uint32_t)id - (uint32_t)v0; };
  bool bad = false;
  // (the list is filled up to whole groups of 8 with entries that hold no token)
  for (int j = tid; j < top8; j += NT) {
    const Entry y = load_entry(a, n, j);
    bad |= y.id < -1 || y.id >= a.vocab;
    ids[j] = y.id;
    parts[j] = y.id >= 0 ? power(y.t - tm, k) * by_ts : 0.f;
    if (place(y.id) < (uint32_t)count) listed[j] = (float)z[place(y.id)];
    if (WARM) theirs[j] = y.t;
  }
  for (int i = tid; i < S / 32; i += NT) seen[i] = twice[i] = 0;
  if (bad && slab == 0) atomicOr(a.status, BPE_STATUS_BAD_ID);
  auto gradient = [&](const Vec<TS, E> &x) {
    Vec<TG, E> y;
#pragma unroll
    for (int e = 0; e < E; ++e) y.v[e] = from_f32<TG>(some ? c * share((float)x.v[e]) : 0.f);
    return y;
  };
  Near near = {0.0, INFINITY};
  if (WARM) {
    __syncthreads();
    const double by = 1.0 / (double)a.temperature;
    auto get = [&](int j, float *e, float *f, double *d) {
      if (place(ids[j]) >= (uint32_t)count) return false;
      *e = power(theirs[j] - tm, k);
      *f = power(listed[j] - zm, k);
      *d = (((double)theirs[j] - tm) - ((double)listed[j] - zm)) * by;
      return *e != 0.f;
    };
    float e, f;
    double d, held = 0.0;
    for (int j = tid; j < a.top; j += NT)
      if (get(j, &e, &f, &d)) held += (double)f;
    held = group_sum<NT>(held, nullptr);
    if (some && held > 0.75 * (double)zs) near = near_teacher<TS, NT>(get, a.top, z, count, zm, k, held, nullptr);
  }
  // (the barrier: the listed logits are read before any is overwritten)
  auto claim = [&] {
    __syncthreads();
    for (int j = tid; j < a.top; j += NT) {
      const uint32_t at = place(ids[j]), bit = 1u << (at & 31);
      if (at < (uint32_t)count && atomicOr(&seen[at >> 5], bit) & bit) atomicOr(&twice[at >> 5], bit);
    }
  };
  int v = 0;
  for (; v + NT * E * U <= count; v += NT * E * U) {
    Vec<TS, E> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = load_vec<TS, E>(z + v + (u * NT + tid) * E);
    if (v == 0) claim();
#pragma unroll
    for (int u = 0; u < U; ++u) store_vec<TG, E, STREAM>(g + v + (u * NT + tid) * E, gradient(x[u]));
  }
  if (v == 0) claim();
  for (v += tid * E; v < count; v += NT * E) {
    if (v + E <= count) {
      store_vec<TG, E, STREAM>(g + v, gradient(load_vec<TS, E>(z + v)));
    } else {
      for (int e = v; e < count; ++e) g[e] = from_f32<TG>(some ? c * share((float)z[e]) : 0.f);
    }
  }
  __syncthreads();
  if (!some) return;
  // the entries that list a token, in their order
  auto same_token = [&](int32_t id, auto entry) {
    for (int i = 0; i < a.top; i += 8) {
      typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
      const i32x4 lo = *(const i32x4 *)&ids[i], hi = *(const i32x4 *)&ids[i + 4];
      uint32_t same = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) same |= (uint32_t)(lo[e] == id) << e | (uint32_t)(hi[e] == id) << (e + 4);
      for (; same; same &= same - 1) entry(i + __ffs(same) - 1);
    }
  };
  for (int j = tid; j < a.top; j += NT) {
    const int32_t id = ids[j];
    const uint32_t at = place(id);
    if (at >= (uint32_t)count) continue;
    float p = parts[j];
    const bool more = twice[at >> 5] >> (at & 31) & 1;
    if (WARM && near.loss < INFINITY) {
      // q - P by the token's first entry that the teacher gives anything to, less its
      // other entries' P: the same bits from each of them
      int j0 = parts[j] != 0.f ? j : -1;
      double others = 0.0;
      if (more) {
        j0 = -1;
        same_token(id, [&](int i) {
          if (parts[i] == 0.f) return;
          if (j0 < 0) j0 = i;
          else others += (double)parts[i];
        });
      }
      if (j0 >= 0) {
        const double d = (((double)theirs[j0] - tm) - ((double)listed[j0] - zm)) / (double)a.temperature;
        g[at] = from_f32<TG>(c * (float)((double)parts[j0] * expm1(near.mean - d - near.loss) - others));
        continue;
      }
    }
    if (more) {
      p = 0.f;
      same_token(id, [&](int i) { p += parts[i]; });
    }
    g[at] = from_f32<TG>(c * (share(listed[j]) - p));
  }
}

template <typename TS, int NT>
hipError_t distill_rows(const DistillArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)a.rows);
  if (a.temperature > kDistillWarm)
    hipLaunchKernelGGL((k_distill<TS, NT, true>), grid, dim3(NT), 0, stream, a);
  else
    hipLaunchKernelGGL((k_distill<TS, NT, false>), grid, dim3(NT), 0, stream, a);
  return hipGetLastError();
}
template <typename TS>
hipError_t distill_as(const DistillArgs &a, hipStream_t stream) {
  return a.vocab <= kDistillNarrow ? distill_rows<TS, 64>(a, stream) : distill_rows<TS, kDistillThreads>(a, stream);
}

template <typename TS, typename TG, int NT, int S, bool WARM>
hipError_t grad_slabs(const DistillArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.vocab + S - 1) / S * a.rows));
  const size_t lds = (a.top + 7) / 8 * 8 * (WARM ? 4 : 3) * sizeof(int32_t);
  const bool big = a.rows * a.vocab * (int64_t)sizeof(TG) >= kStreamBytes;
  if (big)
    hipLaunchKernelGGL((k_distill_grad<TS, TG, NT, S, true, WARM>), grid, dim3(NT), lds, stream, a);
  else
    hipLaunchKernelGGL((k_distill_grad<TS, TG, NT, S, false, WARM>), grid, dim3(NT), lds, stream, a);
  return hipGetLastError();
}
template <typename TS, typename TG>
hipError_t grad_launch(const DistillArgs &a, hipStream_t stream) {
  if (a.vocab > kDistillNarrow) return grad_slabs<TS, TG, kDistillThreads, kDistillSlab, false>(a, stream);
  return a.temperature > kDistillWarm ? grad_slabs<TS, TG, 64, kDistillNarrow, true>(a, stream)
                                      : grad_slabs<TS, TG, 64, kDistillNarrow, false>(a, stream);
}
template <typename TS>
hipError_t grad_as(const DistillArgs &a, int gt, hipStream_t stream) {
  if (gt == BPE_F32) return grad_launch<TS, float>(a, stream);
  if (gt == BPE_BF16) return grad_launch<TS, bf16_t>(a, stream);
  return grad_launch<TS, f16_t>(a, stream);
}

}  // namespace

hipError_t launch_distill(const DistillArgs &a, int st, hipStream_t stream) {
  if (st == BPE_F32) return distill_as<float>(a, stream);
  if (st == BPE_BF16) return distill_as<bf16_t>(a, stream);
  return distill_as<f16_t>(a, stream);
}

hipError_t launch_distill_grad(const DistillArgs &a, int st, int gt, hipStream_t stream) {
  if (st == BPE_F32) return grad_as<float>(a, gt, stream);
  if (st == BPE_BF16) return grad_as<bf16_t>(a, gt, stream);
  return grad_as<f16_t>(a, gt, stream);
}

}  // namespace bpe
