// Rows of logits: loads and stores of 16-byte vectors at any element, and sums
// over a wavefront (gfx950).  Internal header.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "mbok_device.h"

namespace mbok {

typedef uint32_t row_words_any __attribute__((ext_vector_type(4), aligned(2)));

// A 16-byte vector of logits as loaded, kept packed.
template <typename T>
struct RowVec {
  static constexpr int N = 16 / (int)sizeof(T);
  uint32_t w[4];
  __device__ __forceinline__ float at(int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    const uint32_t bits = w[e >> 1];
    if constexpr (std::is_same<T, __bf16>::value)
      return __uint_as_float((e & 1) ? bits & 0xffff0000u : bits << 16);
    return f16_bits_to_f32((uint16_t)((e & 1) ? bits >> 16 : bits & 0xffffu));
  }
  // Unknown to the compiler from here on: it does not keep what an earlier pass
  // unpacked (twice the registers of the packed row).
  __device__ __forceinline__ void forget() {
    asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3]));
  }
};

// Elements v N .. v N + N - 1 of a row of V; past the end -inf.
template <typename T>
__device__ __forceinline__ RowVec<T> load_row(const T* row, int v, int V) {
  constexpr int N = RowVec<T>::N;
  if ((v + 1) * N <= V)
    return __builtin_bit_cast(RowVec<T>, *reinterpret_cast<const row_words_any*>(row + v * N));
  T r[N];
#pragma unroll
  for (int e = 0; e < N; ++e) r[e] = v * N + e < V ? row[v * N + e] : (T)-INFINITY;
  return __builtin_bit_cast(RowVec<T>, r);
}

// The gradient of one vector of logits: N values of OT, 8 or 16 bytes.  stream:
// past the caches, for rows that start 16-byte aligned (2048 x 32000 bf16 policy
// step 61.8 -> 56.6 us; rows at any element, 2048 x 12345 fp32, 45.2 -> 47.1).
template <typename OT, int N>
__device__ __forceinline__ void store_row(OT* row, int v, int V, const float (&d)[N],
                                          bool stream) {
  OT o[N];
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = (OT)d[e];
  if ((v + 1) * N <= V) {
    constexpr int W = N * (int)sizeof(OT) / 4;  // dwords: 2 or 4
    typedef uint32_t words __attribute__((ext_vector_type(W)));
    typedef uint32_t words_any __attribute__((ext_vector_type(W), aligned(2)));
    words w;
    __builtin_memcpy(&w, o, sizeof(w));
    if (stream) __builtin_nontemporal_store(w, reinterpret_cast<words*>(row + v * N));
    else *reinterpret_cast<words_any*>(row + v * N) = w;
    return;
  }
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (v * N + e < V) row[v * N + e] = o[e];
}

__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int s = 32; s; s >>= 1) v = fmaxf(v, __shfl_xor(v, s));
  return v;
}
__device__ __forceinline__ int lanes_max(int v) {
#pragma unroll
  for (int s = 32; s; s >>= 1) v = max(v, __shfl_xor(v, s));
  return v;
}
__device__ __forceinline__ double lanes_sum(double v) {
#pragma unroll
  for (int s = 32; s; s >>= 1) v += __shfl_xor(v, s);
  return v;
}

}  // namespace mbok
