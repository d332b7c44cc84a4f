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

// N consecutive elements.
template <typename T, int N>
struct Vec {
  T v[N];
};

// Words of a vector in device memory, at any element's address: the hardware
// takes unaligned global accesses, so rows of odd width need no path of their
// own.  (One access of one vector value: from a struct the compiler makes
// single stores, and merges those with the tail's.)
typedef uint16_t g2 __attribute__((aligned(2)));
typedef uint32_t g4 __attribute__((aligned(2)));
typedef uint32_t g8 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t g16 __attribute__((ext_vector_type(4), aligned(2)));
template <int BYTES>
struct Word;
template <>
struct Word<2> { typedef g2 type; };
template <>
struct Word<4> { typedef g4 type; };
template <>
struct Word<8> { typedef g8 type; };
template <>
struct Word<16> { typedef g16 type; };

// STREAM: data that the caches should not keep.
template <typename T, int N, bool STREAM = false>
__device__ __forceinline__ Vec<T, N> load_vec(const T *p) {
  constexpr int B = sizeof(Vec<T, N>), W = B < 16 ? B : 16;
  typedef typename Word<W>::type word;
  word w[B / W];
#pragma unroll
  for (int i = 0; i < B / W; ++i)
    w[i] = STREAM ? __builtin_nontemporal_load((const word *)p + i) : ((const word *)p)[i];
  Vec<T, N> r;
  __builtin_memcpy(&r, w, B);
  return r;
}
template <typename T, int N, bool STREAM = false>
__device__ __forceinline__ void store_vec(T *p, const Vec<T, N> &x) {
  constexpr int B = sizeof(Vec<T, N>), W = B < 16 ? B : 16;
  typedef typename Word<W>::type word;
  word w[B / W];
  __builtin_memcpy(w, &x, B);
#pragma unroll
  for (int i = 0; i < B / W; ++i)
    if (STREAM) __builtin_nontemporal_store(w[i], (word *)p + i);
    else ((word *)p)[i] = w[i];
}

// 16 bytes in LDS, aligned.
__device__ __forceinline__ u32x4 lds_load16(const void *p) { return *(const u32x4 *)p; }
__device__ __forceinline__ void lds_store16(void *p, u32x4 x) { *(u32x4 *)p = x; }

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
