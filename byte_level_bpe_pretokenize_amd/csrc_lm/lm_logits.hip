// lm_logits.hip -- penalties for repeated tokens, biases and grammar masks on
// the logits of the next token.
#include "lm_device.h"

namespace bpe {
namespace {

constexpr uint32_t kPrompt = 1u << 31;  // the token occurs in the prompt
constexpr uint32_t kBiased = 1u << 30;  // the row has a bias for it
constexpr int kSlotShift = 21;          // the bias's slot, kBiasSlots - 1 at most
constexpr uint32_t kBiasSlots = 512;
constexpr uint32_t kCount = (1u << kSlotShift) - 1;

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

// 4 IDs of a list p[0 .. n) from i on: one 16-byte load where they are there.
// Past the list's end a lane gets -1.
__device__ __forceinline__ Vec<int32_t, 4> load_ids(const int32_t *p, int64_t i, int64_t n) {
  if (i + 4 <= n) return load_vec<int32_t, 4>(p + i);
  Vec<int32_t, 4> x;
#pragma unroll
  for (int e = 0; e < 4; ++e) x.v[e] = i + e < n ? p[i + e] : -1;
  return x;
}

// One workgroup per row and slab of S logits, in three steps.
// 1. The logits are loaded; while they are on their way the row's whole lists
//    are read (each thread's first IDs of all three together) and what falls
//    into the slab is counted in LDS, one word per token: its count among the
//    generated IDs, a bit for the prompt, a bit and a slot for a bias.  Who
//    counts a token first queues it.
// 2. The queued tokens, side by side in full waves, get their logits, which go
//    where their counts were, and a bit each that says so.
// 3. Each thread takes its own logits, or those of step 2, masks and stores
//    them.
// A row's lists are read once per slab (from L2), so that no counts of rows *
// vocab words exist in memory.  Left in step 3, the divisions and searches of
// step 2 are executed for nearly every vector of a wave for one lane's sake
// (80 us instead of 40).  Lists that do not fit one step of the workgroup have
// no queue: every word is looked at instead.
// Bound by memory with short lists: 256 rows of 128,256 bfloat16 logits to
// float32, 198 MB, take 39 us, 5.0 TB/s (a plain conversion 30 us).  Bound by
// the longest list with long ones: its IDs are read by one workgroup per slab.
template <typename TI, typename TO, int NT, int S, bool STREAM>
__global__ void __launch_bounds__(NT, 8) k_logits(bpe_logits_args a) {
  constexpr int E = 4;             // logits per vector: 16 bytes of float32
  constexpr int U = S / (NT * E);  // vectors per thread
  constexpr int LU = 4, STEP = NT * 4;  // list loads in flight, IDs per step
  __shared__ __align__(16) uint32_t tab[S];
  __shared__ __align__(16) uint32_t done[S / 32];
  constexpr int Q = S / 8;         // places in the queue
  __shared__ uint16_t queue[Q];
  __shared__ float biases[kBiasSlots];
  __shared__ int32_t queued;
  const int tid = threadIdx.x;
  // a row's slabs are `rows` workgroups apart: where that is a multiple of the
  // XCDs' number they are on one XCD and share the row's lists in its L2
  const uint32_t slab = blockIdx.x / (uint32_t)a.rows;
  const int64_t b = blockIdx.x - slab * (uint32_t)a.rows;
  const uint32_t v0 = slab * S;
  const int n = (int)min<int64_t>(S, a.vocab - v0);
  const TI *x = (const TI *)a.logits + b * a.logits_stride + v0;
  Vec<TI, E> in[U];
  if (n == S) {
#pragma unroll
    for (int u = 0; u < U; ++u) in[u] = load_vec<TI, E>(x + (u * NT + tid) * E);
  }
  uint32_t status = 0;
  bool bad_off = false, bad_id = false;
  int64_t plo = 0, phi = 0, blo = 0, bhi = 0, made = 0;
  if (a.prompt_off) ragged(a.prompt_off, b, a.n_prompt, &plo, &phi, &bad_off);
  if (a.bias_off) ragged(a.bias_off, b, a.n_bias, &blo, &bhi, &bad_off);
  if (a.made_len) {
    made = a.made_len[b];
    if (made < 0 || made > a.made_width) {
      status |= BPE_STATUS_BAD_LENGTH;
      made = made < 0 ? 0 : a.made_width;
    }
  }
  int32_t mrow = a.mask_row ? a.mask_row[b] : -1;
  if (mrow < -1 || (a.mask_row && mrow >= a.n_masks)) {
    status |= BPE_STATUS_BAD_MASK_ROW;
    mrow = -1;
  }
  const int32_t *pp = a.prompt_ids + plo, *mp = a.made_ids + b * a.made_stride;
  const int64_t np = phi - plo, nb = bhi - blo;
  // lists that do not fit one step: the words are looked at instead of a queue
  const bool scan = np > STEP || made > STEP || nb > NT;
  const bool wide = nb > kBiasSlots;  // slots repeat: values are searched for
  for (int i = tid * 4; i < S; i += NT * 4) lds_store16(&tab[i], u32x4{});
  for (int i = tid * 4; i < S / 32; i += NT * 4) lds_store16(&done[i], u32x4{});
  if (tid == 0) queued = 0;
  Vec<int32_t, 4> p0[1], m0[1];
  int32_t bv = -1, bprev = -1;
  float bval = 0.f;
  if (tid * 4 < np) p0[0] = load_ids(pp, tid * 4, np);
  if (tid * 4 < made) m0[0] = load_ids(mp, tid * 4, made);
  if (tid < nb) {
    bv = a.bias_ids[blo + tid];
    bval = a.bias_values[blo + tid];
    if (tid > 0) bprev = a.bias_ids[blo + tid - 1];
  }
  uint32_t allow[U];
  const uint32_t *mask = a.mask + mrow * a.mask_stride + (v0 >> 5);
  if (mrow >= 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = (u * NT + tid) * E;
      if (c < n) allow[u] = mask[c >> 5] >> (c & 31);
    }
  }
  __syncthreads();
  auto enqueue = [&](uint32_t k, uint32_t before) {
    if (before != 0) return;
    const int32_t at = atomicAdd(&queued, 1);
    if (at < Q) queue[at] = (uint16_t)k;
  };
  // (the counts of all of a thread's IDs are in flight before the first answer
  // is looked at)
  auto count = [&](const auto &y, int64_t i, int64_t len, bool prompt) {
    constexpr int L = sizeof(y) / sizeof(y[0]);
    uint32_t before[L * 4];
#pragma unroll
    for (int l = 0; l < L * 4; ++l) {
      const uint32_t k = (uint32_t)y[l / 4].v[l % 4] - v0;
      before[l] = 1;
      if (k < (uint32_t)n) before[l] = prompt ? atomicOr(&tab[k], kPrompt) : atomicAdd(&tab[k], 1u);
    }
    if (!scan) {
#pragma unroll
      for (int l = 0; l < L * 4; ++l) enqueue((uint32_t)y[l / 4].v[l % 4] - v0, before[l]);
    }
    if (slab == 0) {
#pragma unroll
      for (int l = 0; l < L * 4; ++l)
        bad_id |= (uint32_t)y[l / 4].v[l % 4] >= (uint32_t)a.vocab && i + l / 4 * STEP + l % 4 < len;
    }
  };
  // the same for a list too long for the queue: no answers
  auto count_only = [&](const auto &y, int64_t i, int64_t len, bool prompt) {
    constexpr int L = sizeof(y) / sizeof(y[0]);
#pragma unroll
    for (int l = 0; l < L * 4; ++l) {
      const uint32_t id = (uint32_t)y[l / 4].v[l % 4], k = id - v0;
      if (k < (uint32_t)n) {
        if (prompt) atomicOr(&tab[k], kPrompt);
        else atomicAdd(&tab[k], 1u);
      }
      if (slab == 0) bad_id |= id >= (uint32_t)a.vocab && i + l / 4 * STEP + l % 4 < len;
    }
  };
  auto bias = [&](int32_t v, int32_t prev, float val, int64_t i) {
    const uint32_t k = (uint32_t)v - v0, slot = (uint32_t)i % kBiasSlots;
    if (k < (uint32_t)n) {
      const uint32_t before = atomicOr(&tab[k], kBiased | slot << kSlotShift);
      if (!scan) enqueue(k, before);
      biases[slot] = val;
    }
    bad_id |= (uint32_t)v >= (uint32_t)a.vocab;
    if (i > 0 && prev >= v) status |= BPE_STATUS_BAD_BIAS;
  };
  if (tid * 4 < np) count(p0, tid * 4, np, true);
  if (tid * 4 < made) count(m0, tid * 4, made, false);
  if (tid < nb) bias(bv, bprev, bval, tid);
  int64_t from = STEP;
  for (; from + STEP * LU <= np; from += STEP * LU) {
    Vec<int32_t, 4> y[LU];
#pragma unroll
    for (int l = 0; l < LU; ++l) y[l] = load_vec<int32_t, 4>(pp + from + l * STEP + tid * 4);
    count_only(y, from + tid * 4, np, true);
  }
  for (; from < np; from += STEP) {
    const Vec<int32_t, 4> y[1] = {load_ids(pp, from + tid * 4, np)};
    count_only(y, from + tid * 4, np, true);
  }
  for (int64_t i = STEP + tid * 4; i < made; i += STEP) {
    const Vec<int32_t, 4> y[1] = {load_ids(mp, i, made)};
    count_only(y, i, made, false);
  }
  for (int64_t i = NT + tid; i < nb; i += NT)
    bias(a.bias_ids[blo + i], a.bias_ids[blo + i - 1], a.bias_values[blo + i], i);
  if (slab == 0) {  // every slab sees the same lists: one reports
    if (bad_off) status |= BPE_STATUS_BAD_ID_OFFSETS;
    if (bad_id) status |= BPE_STATUS_BAD_ID;
    if (status) atomicOr(a.status, (int32_t)status);
  }
  __syncthreads();
  if (scan || queued) {
    const float rep = a.repetition ? a.repetition[b] : 1.f;
    const float freq = a.frequency ? a.frequency[b] : 0.f;
    const float pres = a.presence ? a.presence[b] : 0.f;
    // the logit of the slab's token k, whose word is w
    auto listed = [&](float y, uint32_t w, uint32_t k) {
      if (w & (kPrompt | kCount)) y = y > 0.f ? y / rep : y * rep;
      if (w & kCount) y -= freq * (float)(w & kCount) + pres;
      if (w & kBiased) {
        // (two biases of one token, which the status reports, can mix slots)
        float bias = 0.f;
        if (!wide) {
          const uint32_t slot = (w >> kSlotShift) % kBiasSlots;
          if (slot < nb) bias = biases[slot];
        } else {
          int64_t lo = blo, hi = bhi;  // the last entry with an ID <= v
          while (hi - lo > 1) {
            const int64_t mid = (lo + hi) >> 1;
            if (a.bias_ids[mid] <= (int32_t)(v0 + k)) lo = mid;
            else hi = mid;
          }
          bias = a.bias_values[lo];
        }
        y += bias;
      }
      return y;
    };
    if (scan || queued > Q) {
#pragma unroll 1
      for (int u = 0; u < U; ++u) {
        const int c = (u * NT + tid) * E;
        if (c >= n) break;
        const u32x4 t = lds_load16(&tab[c]);
        uint32_t bits = 0;
#pragma unroll 1
        for (int e = 0; e < E; ++e) {
          const uint32_t w = e == 0 ? t.x : e == 1 ? t.y : e == 2 ? t.z : t.w;
          if (w == 0) continue;
          tab[c + e] = __float_as_uint(listed((float)x[c + e], w, c + e));
          bits |= 1u << e;
        }
        if (bits) atomicOr(&done[c >> 5], bits << (c & 31));
      }
    } else {
      for (int j = tid; j < queued; j += NT) {
        const uint32_t k = queue[j];
        tab[k] = __float_as_uint(listed((float)x[k], tab[k], k));
        atomicOr(&done[k >> 5], 1u << (k & 31));
      }
    }
  }
  __syncthreads();
  TO *out = (TO *)a.out + b * a.out_stride + v0;
  if (n == S) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = (u * NT + tid) * E;
      const uint32_t bits = done[c >> 5] >> (c & 31) & 15u;
      float y[E];
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = (float)in[u].v[e];
      if (bits) {
        const u32x4 t = lds_load16(&tab[c]);
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = (bits >> e) & 1u ? __uint_as_float(t[e]) : y[e];
      }
      if (mrow >= 0) {
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = (allow[u] >> e) & 1u ? y[e] : -INFINITY;
      }
      Vec<TO, E> r;
#pragma unroll
      for (int e = 0; e < E; ++e) r.v[e] = from_f32<TO>(y[e]);
      store_vec<TO, E, STREAM>(out + c, r);
    }
  } else {
    // the row's last slab, element by element
    for (int c = tid; c < n; c += NT) {
      float y = (float)x[c];
      if ((done[c >> 5] >> (c & 31)) & 1u) y = __uint_as_float(tab[c]);
      if (mrow >= 0 && !((mask[c >> 5] >> (c & 31)) & 1u)) y = -INFINITY;
      out[c] = from_f32<TO>(y);
    }
  }
}

template <typename TI, typename TO, int NT, int S, bool STREAM>
hipError_t logits_launch(const bpe_logits_args &a, hipStream_t stream) {
  hipLaunchKernelGGL((k_logits<TI, TO, NT, S, STREAM>),
                     dim3((unsigned)((a.vocab + S - 1) / S * a.rows)), dim3(NT), 0, stream, a);
  return hipGetLastError();
}

template <typename TI, typename TO, bool STREAM>
hipError_t logits_wide_or_not(const bpe_logits_args &a, hipStream_t stream) {
  return logits_wide(a) ? logits_launch<TI, TO, kLogitWideThreads, kLogitWideSlab, STREAM>(a, stream)
                        : logits_launch<TI, TO, kLogitThreads, kLogitSlab, STREAM>(a, stream);
}

template <typename TI, typename TO>
hipError_t logits_as(const bpe_logits_args &a, hipStream_t stream) {
  const bool big = a.rows * a.vocab * (int64_t)sizeof(TO) >= kStreamBytes;
  return big ? logits_wide_or_not<TI, TO, true>(a, stream)
             : logits_wide_or_not<TI, TO, false>(a, stream);
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
