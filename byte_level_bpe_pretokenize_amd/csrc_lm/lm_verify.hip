// lm_verify.hip -- drafted tokens against the target's probabilities, and the
// token drawn after those that stand.
#include "lm_device.h"

namespace bpe {
namespace {

constexpr int VT = kVerifyThreads;
constexpr int VW = VT / 64;

// A probability; what is none counts as 0.
__device__ __forceinline__ double probability(float x) {
  return x > 0.f && x < INFINITY ? (double)x : 0.0;
}

// A workgroup per request, in one launch.
// 1. Each row's draft is looked at, a thread each; the least row that does not
//    stand is the one to draw from.
// 2. The row's weights are added up in 64 bits, each wave a region of its own
//    (whole steps of 64 vectors), lanes strided within it.
// 3. The region in which the running sum passes the sampled share of the total is
//    read again (from L2), a run of elements per thread, and the element found by
//    a scan.
// Which sums decide is fixed by the sizes alone.  Steps 2 and 3 add in different
// orders; where that leaves no element past the share in the region, its last
// element of positive weight is the one.
template <typename T, bool DRAFT>
__global__ void __launch_bounds__(VT) k_verify(VerifyArgs a) {
  constexpr int E = 16 / sizeof(T);
  constexpr int STEP = 64 * E;
  __shared__ double sums[VW];
  __shared__ double red[VW];
  __shared__ int32_t s_row, s_hit, s_last;
  const int tid = threadIdx.x, lane = lane_id(), wave = uniform_wave_id();
  const int64_t r = blockIdx.x;
  int64_t lo = a.off[r], hi = a.off[r + 1];
  uint32_t status = 0;
  if (lo < 0 || hi < lo || hi > a.n_rows) {
    status = BPE_STATUS_BAD_ID_OFFSETS;
    hi = lo;
  }
  if (lo == hi) {
    if (tid == 0) {
      a.counts[r] = 0;
      if (status) atomicOr(a.status, (int32_t)status);
    }
    return;
  }
  const int n_drafts = (int)(hi - lo - 1);
  const T *P = (const T *)a.target, *Q = (const T *)a.draft;
  if (tid == 0) {
    s_row = n_drafts;
    s_hit = s_last = INT_MAX;
  }
  __syncthreads();
  for (int s = 0; s < n_drafts; s += VT) {
    const int i = s + tid;
    if (i < n_drafts) {
      const int32_t x = a.ids[lo + i];
      bool stands = false;
      if (x >= 0 && x < a.vocab) {
        const double p = probability((float)P[(lo + i) * a.t_stride + x]);
        const double q = DRAFT ? probability((float)Q[(lo + i) * a.d_stride + x]) : 1.0;
        stands = (double)a.accept[lo + i] * q < p;
      }
      if (!stands) atomicMin(&s_row, i);
    }
    __syncthreads();
    if (s_row < min(s + VT, n_drafts)) break;
  }
  const int j = s_row;
  const bool rejected = j < n_drafts;
  const int32_t drafted = rejected ? a.ids[lo + j] : -1;
  if (rejected && tid == 0 && (drafted < 0 || drafted >= a.vocab)) status |= BPE_STATUS_BAD_ID;
  for (int64_t i = tid; i < hi - lo; i += VT)
    if (i != j) a.tokens[lo + i] = i < j ? a.ids[lo + i] : -1;
  const T *p = P + (lo + j) * a.t_stride, *q = DRAFT ? Q + (lo + j) * a.d_stride : nullptr;
  const int V = (int)a.vocab;
  const int region = (V + VW * STEP - 1) / (VW * STEP) * STEP;
  // the weights of E tokens from v on; zeros past the end
  auto weights = [&](int v, bool less, double *w) {
    Vec<T, E> x = {}, y = {};
    if (v + E <= V) {
      x = load_vec<T, E>(p + v);
      if (DRAFT && less) y = load_vec<T, E>(q + v);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (v + e < V) {
          x.v[e] = p[v + e];
          if (DRAFT && less) y.v[e] = q[v + e];
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      w[e] = probability((float)x.v[e]);
      if (DRAFT && less) w[e] = fmax(w[e] - probability((float)y.v[e]), 0.0);
      if (!DRAFT && less && v + e == drafted) w[e] = fmax(w[e] - 1.0, 0.0);
    }
  };
  double total = 0.0;
  bool less = rejected;
  for (;;) {
    double sum = 0.0;
    const int end = min(V, (wave + 1) * region);
    for (int v = wave * region + lane * E; v < end; v += STEP) {
      double w[E];
      weights(v, less, w);
#pragma unroll
      for (int e = 0; e < E; ++e) sum += w[e];
    }
    sum = wave_sum(sum);
    if (lane == 0) sums[wave] = sum;
    __syncthreads();
    total = 0.0;
    for (int w = 0; w < VW; ++w) total += sums[w];
    if (total > 0.0 || !less) break;
    less = false;  // nothing is left of the difference: the target's own row
    __syncthreads();
  }
  int32_t token = -1;
  if (total > 0.0) {
    // (past the upper end, NaN included, the last token of positive weight)
    const float u = a.sample[r];
    const double share = u < 1.f ? fmax((double)u, 0.0) * total : total;
    int at = 0;
    double before = 0.0, run = 0.0;
    bool found = false;
    for (int w = 0; w < VW; ++w) {
      if (!found && sums[w] > 0.0) {
        at = w;
        before = run;
      }
      run += sums[w];
      found |= run > share;
    }
    const int begin = at * region, end = min(V, begin + region);
    for (int v0 = begin; v0 < end; v0 += VT * E) {
      const int v = v0 + tid * E;
      double w[E], sum = 0.0, all;
#pragma unroll
      for (int e = 0; e < E; ++e) w[e] = 0.0;
      if (v < end) weights(v, less, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (v + e >= end) w[e] = 0.0;
        sum += w[e];
      }
      double x = before + block_excl_sum<double, VT>(sum, red, &all);
      before += all;
      int hit = INT_MAX, last = -1;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x += w[e];
        if (w[e] > 0.0) {
          last = v + e;
          if (x > share && hit == INT_MAX) hit = v + e;
        }
      }
      if (hit < INT_MAX) atomicMin(&s_hit, hit);
      if (last >= 0) atomicMin(&s_last, INT_MAX - 1 - last);
      __syncthreads();
      if (s_hit < INT_MAX) break;
    }
    token = s_hit < INT_MAX ? s_hit : INT_MAX - 1 - s_last;
  } else {
    status |= BPE_STATUS_NO_TOKEN;
  }
  if (tid == 0) {
    a.tokens[lo + j] = token;
    a.counts[r] = j + (token >= 0);
    if (status) atomicOr(a.status, (int32_t)status);
  }
}

template <typename T>
hipError_t verify_as(const VerifyArgs &a, hipStream_t stream) {
  if (a.draft)
    hipLaunchKernelGGL((k_verify<T, true>), dim3((unsigned)a.R), dim3(VT), 0, stream, a);
  else
    hipLaunchKernelGGL((k_verify<T, false>), dim3((unsigned)a.R), dim3(VT), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_verify(const VerifyArgs &a, int type, hipStream_t stream) {
  if (type == BPE_F32) return verify_as<float>(a, stream);
  if (type == BPE_BF16) return verify_as<bf16_t>(a, stream);
  return verify_as<f16_t>(a, stream);
}

}  // namespace bpe
