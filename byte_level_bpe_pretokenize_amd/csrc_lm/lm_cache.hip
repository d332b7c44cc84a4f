// lm_cache.hip -- a paged cache held in 8 or 4 bits: tokens quantised into their
// slots, and read back by block table.
#include <float.h>

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
template <typename T>
__device__ __forceinline__ void store_some(T *p, const Vec<T, E> &x, int m) {
  if (m >= E) {
    store_vec<T, E>(p, x);
    return;
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (e < m) p[e] = x.v[e];
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// The codes of E numbers that are within the format's range, as bytes.
template <int F>
__device__ __forceinline__ Vec<uint8_t, E> encode(const float *y) {
  Vec<uint8_t, E> r;
  if (F == BPE_E4M3) {
    int32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
      w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], w[i], true);
    }
    __builtin_memcpy(&r, w, 8);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) r.v[e] = (uint8_t)(int32_t)rintf(y[e]);
  }
  return r;
}

// A group's elements are held by group / E neighbouring lanes.  Their range by
// exchange between these lanes, the codes by one multiplication each (the
// inverse is rounded once per group).  A workgroup has whole tokens.
template <typename T, int F>
__global__ void __launch_bounds__(CT) k_cache_write(CacheArgs a) {
  const int lanes = 1 << (a.group_log2 - 3);  // of a group
  static_assert(E == 8, "group / 8 lanes");
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int count = (int)min<int64_t>(a.tokens, a.n - t0) * a.per_token.d;
  uint32_t status = 0;
  for (int i = threadIdx.x; i - (int)threadIdx.x < count; i += CT) {
    // (lanes past the end take part in the exchange)
    const bool in = i < count;
    const int j = in ? i : 0;
    const int token = divide(a.per_token, j);
    const int k = j - token * a.per_token.d;  // lane of the token
    const int head = divide(a.per_head, k);
    const int l = k - head * a.per_head.d;    // lane of the head
    const int group = l >> (a.group_log2 - 3);
    const int c = l * E;                      // first element
    const int m = in ? a.c.dim - c : 0;       // elements there
    const T *x = (const T *)a.x + (t0 + token) * a.t_stride + head * a.h_stride + c;
    const int64_t slot = in ? a.slots[t0 + token] : -1;
    Vec<T, E> v = {};
    if (m > 0) v = load_some(x, m);
    float y[E];
    bool all_finite = true;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      y[e] = (float)v.v[e];
      all_finite &= finite(y[e]);
    }
    if (!all_finite && slot >= 0) status |= BPE_STATUS_NOT_FINITE;
    float scale, low = 0.f;
    if (F == BPE_UINT4) {
      float lo = INFINITY, hi = -INFINITY;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (finite(y[e])) y[e] = fminf(fmaxf(y[e], -0x1p126f), 0x1p126f);
        if (e < m && finite(y[e])) {
          lo = fminf(lo, y[e]);
          hi = fmaxf(hi, y[e]);
        }
      }
      for (int d = 1; d < lanes; d <<= 1) {
        lo = fminf(lo, __shfl_xor(lo, d, 64));
        hi = fmaxf(hi, __shfl_xor(hi, d, 64));
      }
      const bool some = lo <= hi;
      low = some ? lo : 0.f;
      scale = some ? (hi - lo) * (1.0f / 15.0f) : 0.f;
    } else {
      float most = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (finite(y[e])) most = fmaxf(most, fabsf(y[e]));
      for (int d = 1; d < lanes; d <<= 1) most = fmaxf(most, __shfl_xor(most, d, 64));
      scale = most * (F == BPE_E4M3 ? 1.0f / 448.0f : 1.0f / 127.0f);
    }
    if (scale < 0x1p-120f) scale = 0.f;
    const float inverse = scale > 0.f ? 1.0f / scale : 0.f;
    constexpr float top = F == BPE_E4M3 ? 448.f : F == BPE_INT8 ? 127.f : 15.f;
    constexpr float bottom = F == BPE_UINT4 ? 0.f : -top;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      y[e] = (F == BPE_UINT4 ? y[e] - low : y[e]) * inverse;
      // (a NaN is one, or an infinity in a group of scale 0)
      y[e] = y[e] == y[e] ? fminf(fmaxf(y[e], bottom), top) : 0.f;
    }
    if (slot < -1 || slot >= a.c.n_slots) status |= BPE_STATUS_BAD_SLOT;
    if (m <= 0 || slot < 0 || slot >= a.c.n_slots) continue;
    const Vec<uint8_t, E> codes = encode<F>(y);
    uint8_t *q = (uint8_t *)a.c.codes + slot * a.c.codes_stride + (int64_t)head * a.row_bytes;
    if (F == BPE_UINT4) {
      Vec<uint8_t, E / 2> h;
#pragma unroll
      for (int e = 0; e < E / 2; ++e)
        h.v[e] = (uint8_t)(codes.v[2 * e] | (2 * e + 1 < m ? codes.v[2 * e + 1] << 4 : 0));
      q += c / 2;
#pragma unroll
      for (int e = 0; e < E / 2; ++e)
        if (2 * e < m) q[e] = h.v[e];
    } else {
      q += c;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e < m) q[e] = codes.v[e];
    }
    if ((l & (lanes - 1)) == 0) {
      float *s = a.c.scales + slot * a.c.scales_stride +
                 ((int64_t)head * a.groups + group) * (F == BPE_UINT4 ? 2 : 1);
      s[0] = scale;
      if (F == BPE_UINT4) s[1] = low;
    }
  }
  if (status) atomicOr(a.status, (int32_t)status);
}

// The values of E codes (of E / 2 bytes for BPE_UINT4).
template <int F, typename T>
__device__ __forceinline__ Vec<T, E> decode(const uint32_t *w, float scale, float low) {
  Vec<T, E> r;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    float y;
    if (F == BPE_E4M3) {
      const int s = e & 3;
      y = s == 0   ? __builtin_amdgcn_cvt_f32_fp8(w[e >> 2], 0)
          : s == 1 ? __builtin_amdgcn_cvt_f32_fp8(w[e >> 2], 1)
          : s == 2 ? __builtin_amdgcn_cvt_f32_fp8(w[e >> 2], 2)
                   : __builtin_amdgcn_cvt_f32_fp8(w[e >> 2], 3);
      y *= scale;
    } else if (F == BPE_INT8) {
      y = (float)(int8_t)(w[e >> 2] >> 8 * (e & 3)) * scale;
    } else {
      y = fmaf((float)(w[0] >> 4 * e & 15), scale, low);
    }
    r.v[e] = from_f32<T>(y);
  }
  return r;
}

// A workgroup has up to 64 tokens in a row of the packed batch.  Their slots
// first, a lane each: the request by the offsets, the block by the table.  Then
// the tokens' vectors side by side.
template <typename T, int F>
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
  for (int i = tid; i < count; i += CT) {
    const int token = divide(a.per_token, i);
    const int k = i - token * a.per_token.d;
    const int head = divide(a.per_head, k);
    const int c = (k - head * a.per_head.d) * E;
    const int m = a.c.dim - c;
    const int64_t slot = slots[token];
    if (slot == kNot) continue;
    Vec<T, E> y = {};
    if (slot >= 0) {
      const uint8_t *q = (const uint8_t *)a.c.codes + slot * a.c.codes_stride +
                         (int64_t)head * a.row_bytes;
      constexpr int B = F == BPE_UINT4 ? E / 2 : E;
      Vec<uint8_t, B> w = {};
      q += F == BPE_UINT4 ? c / 2 : c;
      const int bytes = F == BPE_UINT4 ? (m + 1) / 2 : m;
#pragma unroll
      for (int e = 0; e < B; ++e)
        if (e < bytes) w.v[e] = q[e];
      uint32_t ww[2] = {};
      __builtin_memcpy(ww, &w, B);
      const float *s = a.c.scales + slot * a.c.scales_stride +
                       ((int64_t)head * a.groups + (c >> a.group_log2)) * (F == BPE_UINT4 ? 2 : 1);
      y = decode<F, T>(ww, s[0], F == BPE_UINT4 ? s[1] : 0.f);
    }
    store_some((T *)a.out + (t0 + token) * a.t_stride + head * a.h_stride + c, y, m);
  }
  if (status) atomicOr(a.status, (int32_t)status);
}

template <typename T, int F>
hipError_t write_launch(const CacheArgs &a, hipStream_t stream) {
  hipLaunchKernelGGL((k_cache_write<T, F>), dim3((unsigned)cache_workgroups(a)), dim3(CT), 0, stream, a);
  return hipGetLastError();
}
template <typename T, int F>
hipError_t read_launch(const CacheArgs &a, hipStream_t stream) {
  hipLaunchKernelGGL((k_cache_read<T, F>), dim3((unsigned)cache_workgroups(a)), dim3(CT), 0, stream, a);
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
