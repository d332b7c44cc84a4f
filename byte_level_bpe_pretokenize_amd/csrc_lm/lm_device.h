// lm_device.h -- element types and vector accesses shared by the kernels of
// the operators on token IDs.
#pragma once

// (each source uses some of the shared scans and searches)
#pragma clang diagnostic ignored "-Wunused-function"
#include "../csrc/bpe_device.h"
#include "lm_internal.h"

namespace bpe {
namespace {

typedef __bf16 bf16_t;
typedef _Float16 f16_t;

// N consecutive elements at any element's address: one wide access (the
// hardware takes unaligned global accesses, so rows of odd width need no path
// of their own).
template <typename T, int N>
struct Vec {
  T v[N];
};
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> load_vec(const T *p) {
  Vec<T, N> r;
  __builtin_memcpy(&r, p, sizeof(r));
  return r;
}
template <typename T, int N>
__device__ __forceinline__ void store_vec(T *p, const Vec<T, N> &x) {
  __builtin_memcpy(p, &x, sizeof(x));
}

// The wave's number as a value that the compiler keeps in a scalar register.
__device__ __forceinline__ int uniform_wave_id() {
  return __builtin_amdgcn_readfirstlane(wave_id());
}

// float32 to T, rounded to nearest even.
template <typename T>
__device__ __forceinline__ T from_f32(float x) {
  return (T)x;
}

}  // namespace
}  // namespace bpe
