// The layer's epilogue Y = R + act(z), z = X W_hat^T + b (gfx950).  Internal header.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mbok_device.h"
#include "mbok_gated.h"

namespace mbok {

// act(z); with DERIV also act'(z)
template <bool DERIV>
__device__ __forceinline__ float layer_activation(int act, float z, float& deriv) {
  if (act == MBOK_ACT_NONE) {
    if (DERIV) deriv = 1.f;
    return z;
  }
  return activation<DERIV>(act, z, deriv);
}

// Receives the layer's sums.  bias, R and pre may be null; R has Y's type.
struct LinearOut {
  static constexpr int kItems = 16;  // outputs of a 16-row tile
  void* Y;
  int64_t ldy;
  const void* R;
  int64_t ldr;
  uint16_t* pre;
  int64_t ldpre;
  const void* bias;
  int m, act;
  int y_f32, bias_dtype;

  __device__ __forceinline__ float bias_at(int row) const {
    if (!bias) return 0.f;
    if (bias_dtype == MBOK_F32) return reinterpret_cast<const float*>(bias)[row];
    const uint16_t b = reinterpret_cast<const uint16_t*>(bias)[row];
    return bias_dtype == MBOK_BF16 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b);
  }

  // item e of a 16-row tile (the decode kernels' epilogue)
  template <typename Sum>
  __device__ __forceinline__ void item(int token, int tile, int e, Sum&& sum) const {
    const int row = 16 * tile + e;
    if (row >= m) return;
    const float b = bias_at(row);
    float r = 0.f;
    if (R) {
      const int64_t at = token * ldr + row;
      r = y_f32 ? reinterpret_cast<const float*>(R)[at]
                : bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(R)[at]);
    }
    const float z = sum(e) + b;
    if (pre) pre[token * ldpre + row] = to_bf16(z);
    float unused;
    float y = layer_activation<false>(act, z, unused);
    if (R) y += r;
    if (y_f32) reinterpret_cast<float*>(Y)[token * ldy + row] = y;
    else reinterpret_cast<uint16_t*>(Y)[token * ldy + row] = to_bf16(y);
  }
};

}  // namespace mbok
