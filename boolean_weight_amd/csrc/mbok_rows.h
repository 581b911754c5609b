// Rows of logits: loads and stores of 16-byte vectors at any element, and sums
// over a wavefront (gfx950).  Internal header.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "mbok_device.h"

namespace mbok {

typedef uint32_t row_words_any __attribute__((ext_vector_type(4), aligned(2)));

// A 16-byte vector of logits as loaded.
template <typename T>
struct RowVec {
  static constexpr int N = 16 / (int)sizeof(T);
  T v[N];
};

// Elements v N .. v N + N - 1 of a row of V; past the end -inf.
template <typename T>
__device__ __forceinline__ RowVec<T> load_row(const T* row, int v, int V) {
  constexpr int N = RowVec<T>::N;
  if ((v + 1) * N <= V)
    return __builtin_bit_cast(RowVec<T>, *reinterpret_cast<const row_words_any*>(row + v * N));
  RowVec<T> r;
#pragma unroll
  for (int e = 0; e < N; ++e) r.v[e] = v * N + e < V ? row[v * N + e] : (T)-INFINITY;
  return r;
}

// The gradient of one vector of logits: N values of OT, 8 to 32 bytes.
template <typename OT, int N>
__device__ __forceinline__ void store_row(OT* row, int v, int V, const float (&d)[N]) {
  OT o[N];
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = (OT)d[e];
  if ((v + 1) * N <= V) {
    constexpr int W = N * (int)sizeof(OT) / 4;  // dwords: 2 or 4
    typedef uint32_t words __attribute__((ext_vector_type(W)));
    typedef uint32_t words_any __attribute__((ext_vector_type(W), aligned(2)));
    words w;
    __builtin_memcpy(&w, o, sizeof(w));
    *reinterpret_cast<words_any*>(row + v * N) = w;
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
__device__ __forceinline__ double lanes_sum(double v) {
#pragma unroll
  for (int s = 32; s; s >>= 1) v += __shfl_xor(v, s);
  return v;
}

}  // namespace mbok
