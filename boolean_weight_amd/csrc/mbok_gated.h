// The gated feed-forward block's stacked layer and its epilogue (gfx950).
// Internal header.
//
// Stacked row 16 u + r is gate row 8 u + r, stacked row 16 u + 8 + r up row
// 8 u + r (r = 0..7), so every 16-row tile of the packed layer holds both
// values of 8 outputs and the epilogue H = act(g) (.) u needs nothing from
// another tile.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mbok.h"

namespace mbok {

// exp and the reciprocal through the hardware's base-2 instructions (1 ulp
// each): far below the bf16 rounding of every value formed from them.
__device__ __forceinline__ float fast_exp(float x) {
  return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f);
}

constexpr float kGeluC = 0.79788456080286535588f;  // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// 1 / (1 + exp(-v)); exact limits 0 and 1
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.f + fast_exp(-v));
}

// act(g); with DERIV also act'(g).  The tanh form of GELU is g sigmoid(2 y),
// y = sqrt(2/pi) (g + 0.044715 g^3), because (1 + tanh y) / 2 = sigmoid(2 y).
template <bool DERIV>
__device__ __forceinline__ float activation(int act, float g, float& deriv) {
  if (act == MBOK_ACT_SILU) {
    const float s = sigmoid(g);
    // s is exactly 1 for large g and exactly 0 for very negative g; infinite g
    // gives NaN (infinity times 0), as the formula does
    if (DERIV) deriv = s * fmaf(g, 1.f - s, 1.f);
    return g * s;
  }
  const float g2 = g * g;
  const float s = sigmoid(2.f * kGeluC * g * fmaf(kGeluB, g2, 1.f));
  if (DERIV) {
    // g^3 overflows long after 1 - s or s is 0: the product is dropped there
    const float t = s * (1.f - s);
    const float slope = 2.f * kGeluC * g * fmaf(3.f * kGeluB, g2, 1.f);
    deriv = t == 0.f ? s : fmaf(t, slope, s);
  }
  return g * s;
}

__device__ __forceinline__ uint16_t to_bf16(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);  // nearest-even
}

// Receives the block's outputs: H, and the pre-activations unless pre is null.
struct GatedOut {
  static constexpr int kItems = 8;  // outputs of a 16-row tile
  uint16_t* H;
  int64_t ldh;
  uint16_t* pre;
  int64_t ldpre;
  int m, act;

  // output `row` of token t; rows past m are only the padding of pre
  __device__ __forceinline__ void put(int64_t t, int row, float g, float u) const {
    if (row < m) {
      float unused;
      H[t * ldh + row] = to_bf16(activation<false>(act, g, unused) * u);
    }
    if (pre) {
      uint16_t* p = pre + t * ldpre + 16 * (row >> 3) + (row & 7);
      p[0] = row < m ? to_bf16(g) : (uint16_t)0;
      p[8] = row < m ? to_bf16(u) : (uint16_t)0;
    }
  }

  // item e of a 16-row tile (the decode kernels' epilogue)
  template <typename Sum>
  __device__ __forceinline__ void item(int token, int tile, int e, Sum&& sum) const {
    const int row = 8 * tile + e;
    if (row >= ((m + 7) & ~7)) return;  // the packed layer's own padding tiles
    put(token, row, sum(e), sum(8 + e));
  }
};

}  // namespace mbok
