// lm_logits.hip -- penalties for repeated tokens, biases and grammar masks on
// the logits of the next token.
#include "lm_device.h"

namespace bpe {
namespace {

constexpr int LWG = 256;
constexpr uint32_t kPrompt = 1u << 31;  // the token occurs in the prompt
constexpr uint32_t kBiased = 1u << 30;  // the row has a bias for it
constexpr uint32_t kCount = kBiased - 1;

// [lo, hi) of row b of a ragged list of n entries; an offset outside [0, n] or
// a decreasing pair gives an empty row and sets *bad.
__device__ __forceinline__ void ragged(const int64_t *off, int64_t b, int64_t n, int64_t *lo,
                                       int64_t *hi, bool *bad) {
  *lo = off[b];
  *hi = off[b + 1];
  if (*lo < 0 || *hi < *lo || *hi > n) {
    *bad = true;
    *lo = *hi = 0;
  }
}

// Calls f(v) for the IDs p[0 .. n), 4 per thread and step (one 16-byte load),
// the workgroup's threads side by side.
template <typename F>
__device__ __forceinline__ void each_id(const int32_t *p, int64_t n, F f) {
  for (int64_t i = (int64_t)threadIdx.x * 4; i < n; i += LWG * 4) {
    if (i + 4 <= n) {
      const Vec<int32_t, 4> x = load_vec<int32_t, 4>(p + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) f(x.v[e]);
    } else {
      for (int64_t q = i; q < n; ++q) f(p[q]);
    }
  }
}

// One workgroup per row and slab of S logits.  The slab's logits and mask bits
// are loaded first; while they are on their way the row's whole history is
// read and what falls into the slab is counted in LDS, one word per token:
// its count among the generated IDs, a bit for the prompt, a bit for a bias.
// Then each thread finishes its own logits.  A row's history is read once per
// slab (from L2), so that no counts of rows * vocab words exist in memory.
template <typename TI, typename TO, int S>
__global__ void __launch_bounds__(LWG) k_logits(bpe_logits_args a) {
  constexpr int E = 4;                 // logits per vector: 16 bytes of float32
  constexpr int U = S / (LWG * E);     // vectors per thread
  __shared__ uint32_t tab[S];
  const int tid = threadIdx.x;
  // a row's slabs are `rows` workgroups apart: where that is a multiple of the
  // XCDs' number they run on one XCD and share the row's history in its L2
  const unsigned slab = blockIdx.x / (unsigned)a.rows;
  const int64_t b = blockIdx.x - slab * (unsigned)a.rows;
  const int64_t v0 = (int64_t)slab * S;
  const int n = (int)min<int64_t>(S, a.vocab - v0);
  const TI *x = (const TI *)a.logits + b * a.logits_stride + v0;
  Vec<TI, E> in[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = (u * LWG + tid) * E;
    if (c + E <= n) {
      in[u] = load_vec<TI, E>(x + c);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) in[u].v[e] = c + e < n ? x[c + e] : (TI)0.f;
    }
  }
  uint32_t status = 0;
  uint32_t allow[U];
  int32_t mrow = a.mask_row ? a.mask_row[b] : -1;
  if (a.mask_row && (mrow < -1 || mrow >= a.n_masks)) {
    status |= BPE_STATUS_BAD_MASK_ROW;
    mrow = -1;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = (u * LWG + tid) * E;
    allow[u] = ~0u;
    if (mrow >= 0 && c < n)
      allow[u] = a.mask[mrow * a.mask_stride + ((v0 + c) >> 5)] >> (c & 31);
  }
  const float rep = a.repetition ? a.repetition[b] : 1.f;
  const float freq = a.frequency ? a.frequency[b] : 0.f;
  const float pres = a.presence ? a.presence[b] : 0.f;
  for (int i = tid * 4; i < S; i += LWG * 4) store_vec(&tab[i], Vec<uint32_t, 4>{});
  __syncthreads();
  bool bad_off = false, bad_id = false;
  if (a.prompt_off) {
    int64_t lo, hi;
    ragged(a.prompt_off, b, a.n_prompt, &lo, &hi, &bad_off);
    each_id(a.prompt_ids + lo, hi - lo, [&](int32_t v) {
      if (v >= v0 && v < v0 + n) tab[v - v0] = kPrompt;
      bad_id |= v < 0 || v >= a.vocab;
    });
    __syncthreads();
  }
  if (a.made_len) {
    int64_t len = a.made_len[b];
    if (len < 0 || len > a.made_width) {
      status |= BPE_STATUS_BAD_LENGTH;
      len = len < 0 ? 0 : a.made_width;
    }
    each_id(a.made_ids + b * a.made_stride, len, [&](int32_t v) {
      if (v >= v0 && v < v0 + n) atomicAdd(&tab[v - v0], 1u);
      bad_id |= v < 0 || v >= a.vocab;
    });
  }
  int64_t blo = 0, bhi = 0;
  if (a.bias_off) {
    ragged(a.bias_off, b, a.n_bias, &blo, &bhi, &bad_off);
    for (int64_t i = blo + tid; i < bhi; i += LWG) {
      const int32_t v = a.bias_ids[i];
      if (v >= v0 && v < v0 + n) atomicOr(&tab[v - v0], kBiased);
      bad_id |= v < 0 || v >= a.vocab;
      if (i > blo && a.bias_ids[i - 1] >= v) status |= BPE_STATUS_BAD_BIAS;
    }
  }
  if (slab == 0) {  // every slab sees the same lists: one reports
    if (bad_off) status |= BPE_STATUS_BAD_ID_OFFSETS;
    if (bad_id) status |= BPE_STATUS_BAD_ID;
    if (status) atomicOr(a.status, (int32_t)status);
  }
  __syncthreads();
  TO *out = (TO *)a.out + b * a.out_stride + v0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = (u * LWG + tid) * E;
    if (c >= n) continue;
    const Vec<uint32_t, E> t = load_vec<uint32_t, E>(&tab[c]);
    Vec<TO, E> r;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float y = (float)in[u].v[e];
      const uint32_t w = t.v[e];
      if (w) {
        if (w & ~kBiased) y = y > 0.f ? y / rep : y * rep;
        if (w & kCount) y -= freq * (float)(w & kCount) + pres;
        if (w & kBiased) {
          int64_t lo = blo, hi = bhi;  // the last entry with an ID <= v
          while (hi - lo > 1) {
            const int64_t mid = (lo + hi) >> 1;
            if (a.bias_ids[mid] <= v0 + c + e) lo = mid;
            else hi = mid;
          }
          y += a.bias_values[lo];
        }
      }
      if (!((allow[u] >> e) & 1u)) y = -INFINITY;
      r.v[e] = from_f32<TO>(y);
    }
    if (c + E <= n) {
      store_vec<TO, E>(out + c, r);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (c + e < n) out[c + e] = r.v[e];
    }
  }
}

template <typename TI, typename TO>
hipError_t logits_as(const bpe_logits_args &a, hipStream_t stream) {
  constexpr int S = kLogitSlab;
  hipLaunchKernelGGL((k_logits<TI, TO, S>),
                     dim3((unsigned)((a.vocab + S - 1) / S * a.rows)), dim3(LWG), 0, stream, a);
  return hipGetLastError();
}

template <typename TI>
hipError_t logits_from(const bpe_logits_args &a, hipStream_t stream) {
  if (a.out_type == BPE_F32) return logits_as<TI, float>(a, stream);
  if (a.out_type == BPE_BF16) return logits_as<TI, bf16_t>(a, stream);
  return logits_as<TI, f16_t>(a, stream);
}

}  // namespace

hipError_t launch_logits(const bpe_logits_args &a, hipStream_t stream) {
  if (a.logits_type == BPE_F32) return logits_from<float>(a, stream);
  if (a.logits_type == BPE_BF16) return logits_from<bf16_t>(a, stream);
  return logits_from<f16_t>(a, stream);
}

}  // namespace bpe
