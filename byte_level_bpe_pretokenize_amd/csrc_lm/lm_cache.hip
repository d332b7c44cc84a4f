// lm_cache.hip -- a paged cache held in 8 or 4 bits: tokens quantised into their
// slots, and read back by block table.
#include "lm_device.h"

namespace bpe {
namespace {

constexpr int CT = kCacheThreads;
constexpr int E = kCacheVec;

__device__ __forceinline__ int32_t divide(const Divisor &d, int32_t x) {
  return d.d == 1 ? x : (int32_t)(__umulhi((uint32_t)x, d.magic) >> d.shift);
}

// The first m (1 to E) elements at p; zeros behind them.
template <typename T>
__device__ __forceinline__ Vec<T, E> load_some(const T *p, int m) {
  if (m >= E) return load_vec<T, E>(p);
  Vec<T, E> r;
#pragma unroll
  for (int e = 0; e < E; ++e) r.v[e] = e < m ? p[e] : (T)0.f;
  return r;
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// Bytes in device memory, at any address.
typedef uint16_t b2 __attribute__((aligned(1)));
typedef uint32_t b4 __attribute__((aligned(1)));
typedef uint32_t b8 __attribute__((ext_vector_type(2), aligned(1)));

// The largest of `lanes` (a power of two, the same in every lane) neighbouring
// lanes' values, in each of them; every lane active.  Lanes 1 and 2 away by quad,
// then, since quads and halves agree within, by mirroring 8 and 16 lanes.
template <int CTRL>
__device__ __forceinline__ float other(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float lanes_max(float x, int lanes) {
  x = fmaxf(x, other<0xB1>(x));
  if (lanes > 2) x = fmaxf(x, other<0x4E>(x));
  if (lanes > 4) x = fmaxf(x, other<0x141>(x));
  if (lanes > 8) x = fmaxf(x, other<0x140>(x));
  if (lanes > 16) x = fmaxf(x, __shfl_xor(x, 16, 64));
  if (lanes > 32) x = fmaxf(x, __shfl_xor(x, 32, 64));
  return x;
}

// The codes of E numbers within the format's range (up to float32's rounding of
// its ends, which rounds back to them), in the first bytes of w.
template <int F>
__device__ __forceinline__ void encode(const float *y, uint32_t *w) {
  if (F == BPE_E4M3) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
      w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], w[i], true);
    }
    return;
  }
  // adding 1.5 * 2^23 rounds to a whole number, to nearest even, in the low bits
  uint32_t b[E];
  {
#pragma clang fp contract(off)
#pragma unroll
    for (int e = 0; e < E; ++e) b[e] = __float_as_uint(y[e] + 12582912.f);
  }
  if (F == BPE_INT8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = __builtin_amdgcn_perm(b[4 * i + 1], b[4 * i], 0x0c0c0400);
      const uint32_t hi = __builtin_amdgcn_perm(b[4 * i + 3], b[4 * i + 2], 0x0c0c0400);
      w[i] = __builtin_amdgcn_perm(hi, lo, 0x05040100);
    }
  } else {
    w[0] = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) w[0] |= (b[e] & 15u) << 4 * e;
  }
}

// The scale and lowest value of a group that has infinities, NaN or magnitudes past
// 2^126, and its elements as they are to be held.
template <int F>
__device__ __forceinline__ void rare(float *y, int m, int lanes, float *scale, float *low) {
  float lo = INFINITY, hi = -INFINITY;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (!finite(y[e])) continue;
    if (F == BPE_UINT4) y[e] = fminf(fmaxf(y[e], -0x1p126f), 0x1p126f);
    if (e < m) {
      lo = fminf(lo, F == BPE_UINT4 ? y[e] : -fabsf(y[e]));
      hi = fmaxf(hi, F == BPE_UINT4 ? y[e] : fabsf(y[e]));
    }
  }
  lo = -lanes_max(-lo, lanes);
  hi = lanes_max(hi, lanes);
  const bool some = lo <= hi;
  *low = some && F == BPE_UINT4 ? lo : 0.f;
  *scale = !some ? 0.f
           : F == BPE_UINT4 ? (hi - lo) * (1.0f / 15.0f)
                            : hi * (F == BPE_E4M3 ? 1.0f / 448.0f : 1.0f / 127.0f);
}

// A group's elements are held by group / E neighbouring lanes.  Their range by
// exchange between these lanes, the codes by one multiplication each (the
// inverse is rounded once per group) instead of a division.
// A workgroup has whole tokens, about four vectors a thread, whose loads all go
// first: 60,000 tokens of 16 heads of 128 in bfloat16 to int8, 377 MB, take 75 to 81
// us from run to run, 4.6 to 5.0 TB/s (a copy makes 4.8), bound by memory; one vector
// at a time, exchanged through LDS and stored by bytes, took 116.  To 4 bits, 315 MB,
// 76, 4.1 TB/s.  Heads of 77, whose last lanes store bytes: 90 us, 2.5 TB/s (4 bits
// 97, 2.0); of 96 in groups of 64, a quarter of whose lanes have nothing: 69, 4.1
// (69, 3.5).  64 tokens: 4.7 us, a chain of three dependent accesses.
template <typename T, int F, bool WHOLE>
__global__ void __launch_bounds__(CT) k_cache_write(CacheArgs a) {
  static_assert(E == 8, "group / 8 lanes");
  constexpr int U = 4;
  const int lanes = 1 << (a.group_log2 - 3);  // of a group
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int count = (int)min<int64_t>(a.tokens, a.n - t0) * a.per_token.d;
  uint32_t status = 0;
  for (int base = 0; base < count; base += CT * U) {
    Vec<T, E> v[U];
    int64_t slot[U];
    int head[U], l[U], m[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // (lanes past the end take part in the exchange, with the last group's values)
      const int i = base + u * CT + tid;
      const int j = i < count ? i : count - lanes + (i & (lanes - 1));
      const int token = divide(a.per_token, j);
      const int k = j - token * a.per_token.d;  // lane of the token
      head[u] = divide(a.per_head, k);
      l[u] = k - head[u] * a.per_head.d;        // lane of the head
      m[u] = a.c.dim - l[u] * E;                // elements there
      slot[u] = a.slots[t0 + token];
      const T *x = (const T *)a.x + (t0 + token) * a.t_stride + head[u] * a.h_stride + l[u] * E;
      // (a head's last group may end before its last lanes)
      if (m[u] >= E) v[u] = load_vec<T, E>(x);
      else if (WHOLE || m[u] <= 0) v[u] = Vec<T, E>{};
      else v[u] = load_some(x, m[u]);
      if (i >= count) m[u] = 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float y[E], most = 0.f, zero = 0.f;
      // (a NaN drops out of the maximum; it and infinities show in the sum)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        y[e] = (float)v[u].v[e];
        most = fmaxf(most, fabsf(y[e]));
        zero = fmaf(y[e], 0.f, zero);
      }
      const bool odd = zero != 0.f || (F == BPE_UINT4 && most > 0x1p126f);
      float scale, low = 0.f;
      if (F == BPE_UINT4) {
        float lo = INFINITY, hi = -INFINITY;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          lo = fminf(lo, WHOLE || e < m[u] ? y[e] : INFINITY);
          hi = fmaxf(hi, WHOLE || e < m[u] ? y[e] : -INFINITY);
        }
        if (WHOLE && m[u] <= 0) {  // (the values there are no element's)
          lo = INFINITY;
          hi = -INFINITY;
        }
        low = -lanes_max(-lo, lanes);
        scale = (lanes_max(hi, lanes) - low) * (1.0f / 15.0f);
      } else {
        scale = lanes_max(most, lanes) * (F == BPE_E4M3 ? 1.0f / 448.0f : 1.0f / 127.0f);
      }
      const bool any_odd = __any(odd);
      if (any_odd) {
        if (zero != 0.f && m[u] > 0 && slot[u] >= 0) status |= BPE_STATUS_NOT_FINITE;
        rare<F>(y, m[u], lanes, &scale, &low);
      }
      if (scale < 0x1p-120f) scale = 0.f;
      const float inverse = scale > 0.f ? 1.0f / scale : 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = (F == BPE_UINT4 ? y[e] - low : y[e]) * inverse;
      if (any_odd) {
        constexpr float top = F == BPE_E4M3 ? 448.f : F == BPE_INT8 ? 127.f : 15.f;
        constexpr float bottom = F == BPE_UINT4 ? 0.f : -top;
#pragma unroll
        for (int e = 0; e < E; ++e)  // (a NaN is one, or an infinity in a group of scale 0)
          y[e] = y[e] == y[e] ? fminf(fmaxf(y[e], bottom), top) : 0.f;
      }
      if (slot[u] < -1 || slot[u] >= a.c.n_slots) status |= BPE_STATUS_BAD_SLOT;
      if (m[u] <= 0 || slot[u] < 0 || slot[u] >= a.c.n_slots) continue;
      uint32_t w[2];
      encode<F>(y, w);
      uint8_t *q = (uint8_t *)a.c.codes + slot[u] * a.c.codes_stride + head[u] * a.row_bytes +
                   l[u] * (F == BPE_UINT4 ? E / 2 : E);
      if (WHOLE || m[u] >= E) {
        if (F == BPE_UINT4) *(b4 *)q = w[0];
        else *(b8 *)q = b8{w[0], w[1]};
      } else if (F == BPE_UINT4) {
        w[0] &= (1u << 4 * m[u]) - 1u;
#pragma unroll
        for (int e = 0; e < E / 2; ++e)
          if (2 * e < m[u]) q[e] = (uint8_t)(w[0] >> 8 * e);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (e < m[u]) q[e] = (uint8_t)(w[e >> 2] >> 8 * (e & 3));
      }
      if ((l[u] & (lanes - 1)) == 0) {
        float *s = a.c.scales + slot[u] * a.c.scales_stride +
                   (head[u] * a.groups + (l[u] >> (a.group_log2 - 3))) * (F == BPE_UINT4 ? 2 : 1);
        s[0] = scale;
        if (F == BPE_UINT4) s[1] = low;
      }
    }
  }
  if (status) atomicOr(a.status, (int32_t)status);
}

// ---- reading: N elements a lane (cache_read_vec) ----

struct Step {
  float scale, low;
};

// The values of N codes (of N / 2 bytes for BPE_UINT4: the lower and the upper
// halves apart, since a byte to a float is one instruction).
template <int F, typename T, int N, typename S>
__device__ __forceinline__ Vec<T, N> decode(const uint32_t *w, S step) {
  Vec<T, N> r;
  uint32_t b[2];
  if (F == BPE_UINT4) {
    b[0] = w[0] & 0x0f0f0f0fu;
    b[1] = w[0] >> 4 & 0x0f0f0f0fu;
  }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    float y;
    const Step x = step(e);
    if (F == BPE_E4M3) {
      const int s = e & 3;
      y = s == 0   ? __builtin_amdgcn_cvt_f32_fp8(w[e >> 2], 0)
          : s == 1 ? __builtin_amdgcn_cvt_f32_fp8(w[e >> 2], 1)
          : s == 2 ? __builtin_amdgcn_cvt_f32_fp8(w[e >> 2], 2)
                   : __builtin_amdgcn_cvt_f32_fp8(w[e >> 2], 3);
      y *= x.scale;
    } else if (F == BPE_INT8) {
      y = (float)(int8_t)(w[e >> 2] >> 8 * (e & 3)) * x.scale;
    } else {
      y = fmaf((float)(b[e & 1] >> 8 * (e >> 1) & 0xffu), x.scale, x.low);
    }
    r.v[e] = from_f32<T>(y);
  }
  return r;
}

// The codes of the N elements from c on of a head's row q; of BPE_UINT4 c may be odd
// where they are the head's last.
template <int F, int N, bool WHOLE>
__device__ __forceinline__ void load_codes(const uint8_t *q, int c, uint32_t *w) {
  if (F == BPE_UINT4) {
    const uint8_t *at = q + (c >> 1);
    w[0] = N == 8 ? *(const b4 *)at : (uint32_t)*(const b2 *)at;
    if (!WHOLE) {
      const uint32_t after = q[(c + N - 1) >> 1];
      if (c & 1) w[0] = w[0] >> 4 | after << (4 * N - 4);
    }
  } else if (N == 8) {
    const b8 x = *(const b8 *)(q + c);
    w[0] = x.x;
    w[1] = x.y;
  } else {
    w[0] = *(const b4 *)(q + c);
  }
}
// Those of a head of dim < N elements.
template <int F, int N>
__device__ __forceinline__ void load_few(const uint8_t *q, int dim, uint32_t *w) {
  w[0] = w[1] = 0;
#pragma unroll
  for (int e = 0; e < (F == BPE_UINT4 ? N / 2 : N); ++e)
    if ((F == BPE_UINT4 ? 2 * e : e) < dim) w[e >> 2] |= (uint32_t)q[e] << 8 * (e & 3);
}

// A workgroup has up to 64 tokens in a row of the packed batch.  Their slots
// first, a lane each: the request by the offsets, the block by the table.  Then
// the tokens' vectors side by side, four a thread, whose loads all go first.
// 384,000 tokens of 16 heads of 128 from 4 bits to bfloat16, 2.0 GB, take 395 us,
// 5.1 TB/s, bound by memory (760 with one vector at a time, loaded by bytes; a
// profiler's trace, which keeps launches apart, has 439 for the same).  1,800 tokens of
// 16 heads of 64: 4.5 us, a chain of five dependent accesses.  Heads of no whole
// vectors: 60,000 tokens of 64 heads of 77 in e4m3 3.9 TB/s (4 bits 2.5), and of 80
// 5.1 (4.2).
template <typename T, int F, int N, bool WHOLE, bool STREAM>
__global__ void __launch_bounds__(CT) k_cache_read(CacheArgs a) {
  constexpr int64_t kNot = INT64_MIN;  // no request's
  __shared__ int64_t slots[kCacheTokens];
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int tokens = (int)min<int64_t>(a.tokens, a.n - t0);
  uint32_t status = 0;
  // what is wrong with the offsets, a share of them per thread of the launch
  for (int64_t r = (int64_t)blockIdx.x * CT + tid; r < a.R; r += (int64_t)gridDim.x * CT) {
    const int64_t lo = a.off[r], hi = a.off[r + 1];
    if (lo < 0 || hi < lo || hi > a.n) status |= BPE_STATUS_BAD_ID_OFFSETS;
    if (a.start && a.start[r] < 0) status |= BPE_STATUS_BAD_LENGTH;
  }
  if (uniform_wave_id() == 0) {
    // the first requests that end behind the workgroup's first and last token,
    // and between them the first that ends behind each token
    const int64_t r0 = wave_lower_bound(a.off + 1, a.R, t0 + 1);
    const int64_t r1 = wave_lower_bound(a.off + 1, a.R, t0 + tokens);
    if (tid < tokens) {
      const int64_t t = t0 + tid;
      const int64_t lo = cache_request(a.off, r0, r1, t);
      int64_t slot = kNot;
      if (lo < a.R && a.off[lo] >= 0 && a.off[lo] <= t) {
        const int64_t p = t - a.off[lo] + (a.start ? max(a.start[lo], 0) : 0);
        slot = -1;
        if (p > INT32_MAX) status |= BPE_STATUS_BAD_LENGTH;
        else
          slot = cache_slot(a.table + lo * a.stride, a.width, a.bs.d, a.c.n_slots, p,
                            divide(a.bs, (int32_t)p), &status);
      }
      slots[tid] = slot;
    }
  }
  __syncthreads();
  const int count = tokens * a.per_token.d;
  constexpr int U = 4;
  for (int base = 0; base < count; base += CT * U) {
    // All loads first, unconditional ones, so that they are in flight together.
    // Heads of no whole vectors: the last vector is the head's last N elements, some
    // of which the one before it has too (both store the same); it may have two
    // groups' elements.
    int64_t at[U], slot[U];
    int edge[U];  // the first element of the second group
    uint32_t w[U][2];
    Step first[U], second[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(base + u * CT + tid, count - 1);
      const int token = divide(a.per_token, i);
      const int k = i - token * a.per_token.d;
      const int head = divide(a.per_head, k);
      int c = (k - head * a.per_head.d) * N;
      if (!WHOLE) c = max(min(c, a.c.dim - N), 0);
      slot[u] = slots[token];
      at[u] = (t0 + token) * a.t_stride + head * a.h_stride + c;
      const uint8_t *q = (const uint8_t *)a.c.codes + slot[u] * a.c.codes_stride + head * a.row_bytes;
      const float *s = a.c.scales + slot[u] * a.c.scales_stride + head * a.groups * (F == BPE_UINT4 ? 2 : 1);
      if (slot[u] < 0) {  // (any place that is there)
        q = (const uint8_t *)a.off - (F == BPE_UINT4 ? c >> 1 : c);
        s = (const float *)a.off - (c >> a.group_log2) * (F == BPE_UINT4 ? 2 : 1);
      }
      if (WHOLE || a.c.dim >= N) load_codes<F, N, WHOLE>(q, c, w[u]);
      else load_few<F, N>(q, a.c.dim, w[u]);
      const int g = c >> a.group_log2, h = WHOLE ? g : min(c + N - 1, a.c.dim - 1) >> a.group_log2;
      auto load_step = [&](int g) {
        return F == BPE_UINT4 ? Step{s[2 * g], s[2 * g + 1]} : Step{s[g], 0.f};
      };
      first[u] = load_step(g);
      if (!WHOLE) second[u] = load_step(slot[u] < 0 ? g : h);
      edge[u] = (h << a.group_log2) - c;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Vec<T, N> y = decode<F, T, N>(w[u], [&](int e) { return WHOLE || e < edge[u] ? first[u] : second[u]; });
      if (slot[u] < 0) y = Vec<T, N>{};
      if (base + u * CT + tid >= count || slot[u] == kNot) continue;
      T *out = (T *)a.out + at[u];
      if (WHOLE || a.c.dim >= N) {
        store_vec<T, N, STREAM>(out, y);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (e < a.c.dim) out[e] = y.v[e];
      }
    }
  }
  if (status) atomicOr(a.status, (int32_t)status);
}

template <typename T, int F>
hipError_t write_launch(const CacheArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)cache_workgroups(a)), wg(CT);
  if (a.c.dim % E == 0) hipLaunchKernelGGL((k_cache_write<T, F, true>), grid, wg, 0, stream, a);
  else hipLaunchKernelGGL((k_cache_write<T, F, false>), grid, wg, 0, stream, a);
  return hipGetLastError();
}
template <typename T, int F>
hipError_t read_launch(const CacheArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)cache_workgroups(a)), wg(CT);
  constexpr int N = 16 / sizeof(T);
  const bool big = a.n * a.c.heads * a.c.dim * (int64_t)sizeof(T) >= kStreamBytes;
  if (a.c.dim % N != 0)
    hipLaunchKernelGGL((k_cache_read<T, F, 8, false, false>), grid, wg, 0, stream, a);
  else if (big)
    hipLaunchKernelGGL((k_cache_read<T, F, N, true, true>), grid, wg, 0, stream, a);
  else
    hipLaunchKernelGGL((k_cache_read<T, F, N, true, false>), grid, wg, 0, stream, a);
  return hipGetLastError();
}

template <typename T>
hipError_t write_as(const CacheArgs &a, hipStream_t stream) {
  if (a.c.format == BPE_E4M3) return write_launch<T, BPE_E4M3>(a, stream);
  if (a.c.format == BPE_INT8) return write_launch<T, BPE_INT8>(a, stream);
  return write_launch<T, BPE_UINT4>(a, stream);
}
template <typename T>
hipError_t read_as(const CacheArgs &a, hipStream_t stream) {
  if (a.c.format == BPE_E4M3) return read_launch<T, BPE_E4M3>(a, stream);
  if (a.c.format == BPE_INT8) return read_launch<T, BPE_INT8>(a, stream);
  return read_launch<T, BPE_UINT4>(a, stream);
}

}  // namespace

hipError_t launch_cache_write(const CacheArgs &a, int xt, hipStream_t stream) {
  if (xt == BPE_F32) return write_as<float>(a, stream);
  if (xt == BPE_BF16) return write_as<bf16_t>(a, stream);
  return write_as<f16_t>(a, stream);
}

hipError_t launch_cache_read(const CacheArgs &a, int ot, hipStream_t stream) {
  if (ot == BPE_F32) return read_as<float>(a, stream);
  if (ot == BPE_BF16) return read_as<bf16_t>(a, stream);
  return read_as<f16_t>(a, stream);
}

}  // namespace bpe
