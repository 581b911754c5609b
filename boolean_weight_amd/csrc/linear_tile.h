// The many-token tiles of the layer with its epilogue: product_tile's sums through
// LDS to the outputs.  Internal header.
//
// The sums of 64 tokens at a time go through LDS as fp32, so that a thread holds 8
// consecutive outputs of a token: whole 16-byte accesses to Y, R and the
// pre-activations, one set of bias values per thread.
#pragma once

#include "mbok_linear.h"
#include "mfma_tile.h"

namespace mbok {
namespace {

// 8 bf16 or fp32 values of a row from p, `live` of them inside it
template <bool F32>
__device__ __forceinline__ void load8(const void* base, int64_t at, int live, float (&v)[8]) {
  if constexpr (F32) {
    typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
    const float* p = reinterpret_cast<const float*>(base) + at;
    if (live == 8) {
      const f32x4_any a = *reinterpret_cast<const f32x4_any*>(p),
                      b = *reinterpret_cast<const f32x4_any*>(p + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < live ? p[e] : 0.f;
  } else {
    const u32x4 w = load_piece(reinterpret_cast<const uint16_t*>(base) + at, live, false);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = __uint_as_float((e & 1) ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
  }
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, int64_t at, int live, const float (&v)[8]) {
  if constexpr (F32) {
    typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
    float* p = reinterpret_cast<float*>(base) + at;
    if (live == 8) {
      *reinterpret_cast<f32x4_any*>(p) = f32x4_any{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4_any*>(p + 4) = f32x4_any{v[4], v[5], v[6], v[7]};
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < live) p[e] = v[e];
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(base) + at;
    if (live == 8) {
      *reinterpret_cast<u32x4_any*>(p) = u32x4_any{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]),
                                                   bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < live) p[e] = to_bf16(v[e]);
  }
}

// The outputs of a tile, 32 TI tokens of each wavefront row in TI passes; the sums
// of C shares of the contraction are added in their order.
template <typename P, bool F32, int C>
__device__ __forceinline__ void linear_outputs(const f32x16 (&acc)[P::TI][2], int wt, int wn,
                                               int part, const LinearOut& out, int T, int t0,
                                               int n0, float* smem) {
  constexpr int kThreads = P::threads * C, kPieces = P::BN / 8, kRows = 32 * P::WT;
  constexpr int kShare = P::lds / sizeof(float);
  constexpr int kStep = kThreads / kPieces;  // rows the workgroup takes at a time
  static_assert(kThreads % kPieces == 0 && kRows % kStep == 0, "tile shape");
  static_assert(sizeof(float) * kRows * P::FS <= P::lds, "the pass fits in LDS");
  const int tid = threadIdx.x, lane = tid & 63;
  const int c = 8 * (tid % kPieces), col = n0 + c;
  const int live = max(0, min(8, out.m - col));
  float bias[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) bias[e] = e < live ? out.bias_at(col + e) : 0.f;
#pragma unroll
  for (int i = 0; i < P::TI; ++i) {
    if (i) __syncthreads();  // the pass before has been read
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        smem[part * kShare + (32 * wt + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) * P::FS + 32 * (2 * wn + j) +
             (lane & 31)] = acc[i][j][r];
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kRows / kStep; ++s) {
      const int row = s * kStep + tid / kPieces;
      const int64_t t = t0 + 32 * (P::TI * (row >> 5) + i) + (row & 31);
      if (t >= T || live == 0) continue;
      float y[8], z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        z[e] = smem[row * P::FS + c + e];
#pragma unroll
        for (int p = 1; p < C; ++p) z[e] += smem[p * kShare + row * P::FS + c + e];
        z[e] += bias[e];
      }
      if (out.R) load8<F32>(out.R, t * out.ldr + col, live, y);
      if (out.pre) store8<false>(out.pre, t * out.ldpre + col, live, z);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float unused;
        const float a = layer_activation<false>(out.act, z[e], unused);
        y[e] = out.R ? y[e] + a : a;
      }
      store8<F32>(out.Y, t * out.ldy + col, live, y);
    }
  }
}

template <typename AT, int K, typename P, bool TWO, bool F32, int C = 1>
__device__ __forceinline__ void linear_tile(const uint32_t* __restrict__ bits,
                                            const AT* __restrict__ scales,
                                            const uint16_t* __restrict__ X, int64_t ldx,
                                            const LinearOut& out, int T, int m_pad, int G, int t0,
                                            int n0, uint16_t* smem) {
  product_tile<AT, K, P, TWO, false, C>(
      bits, scales, X, ldx, T, m_pad, G, t0, n0, smem,
      [&](const f32x16 (&acc)[P::TI][2], int wt, int wn, int part) {
        linear_outputs<P, F32, C>(acc, wt, wn, part, out, T, t0, n0,
                                  reinterpret_cast<float*>(smem));
      });
}

}  // namespace
}  // namespace mbok
