// The gated feed-forward block's entry points below the C ABI: the forward's
// dispatch and the backward pass (gfx950).
//
// With H = act(g) (.) u and s the gradient of H:
//     dg = s u act'(g),  du = s act(g),  dX = dg Wg + du Wu.
// The first two are one pass over pre and dH (bound by memory: 2 + 1 values
// read and 2 written per output, 2048 x 11008 in 36 us); dX is the transposed product of the stacked
// layer, whose rows are the columns of dpre = (dg, du) in the stacked order.
// dg and du are rounded to bf16 once: they are the matrix-core operand of dX
// and of the scale gradients, and the gradients a caller keeps.
#include "mbok_device.h"
#include "mbok_gated.h"
#include "mbok_launch.h"
#include "mbok_levels.h"

namespace mbok {
namespace {

__device__ __forceinline__ float lane_value(const u32x4& v, int e) {
  return bf16_bits_to_f32((e & 1) ? v[e >> 1] >> 16 : v[e >> 1] & 0xffffu);
}

// One thread: 8 outputs of one token, i.e. one 16-column tile of pre and dpre.
__global__ void __launch_bounds__(256) gated_backward_kernel(
    const uint16_t* pre, int64_t ldpre, const uint16_t* __restrict__ dH, int64_t lddh,
    uint16_t* dpre, int64_t lddpre, int m, int64_t items, int act) {
  const int tiles = (m + 7) / 8;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx >= items) return;
  const int64_t t = idx / tiles;
  const int tile = (int)(idx - t * tiles);
  const u32x4* p = reinterpret_cast<const u32x4*>(pre + t * ldpre + 16 * tile);
  const u32x4 gv = p[0], uv = p[1];
  const uint16_t* h = dH + t * lddh + 8 * tile;
  const int live = min(8, m - 8 * tile);
  const u32x4 sv = load_piece(h, live, m >= 8);  // dH rows start anywhere
  uint32_t dg[8], du[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float s = lane_value(sv, c), g = lane_value(gv, c), u = lane_value(uv, c);
    float slope;
    const float a = activation<true>(act, g, slope);
    dg[c] = c < live ? to_bf16(s * u * slope) : 0u;
    du[c] = c < live ? to_bf16(s * a) : 0u;
  }
  u32x4* o = reinterpret_cast<u32x4*>(dpre + t * lddpre + 16 * tile);
  o[0] = u32x4{dg[0] | dg[1] << 16, dg[2] | dg[3] << 16, dg[4] | dg[5] << 16, dg[6] | dg[7] << 16};
  o[1] = u32x4{du[0] | du[1] << 16, du[2] | du[3] << 16, du[4] | du[5] << 16, du[6] | du[7] << 16};
}

}  // namespace

int launch_gated(const mbok_desc* d, const void* packed, const void* X, int64_t T, int64_t ldx,
                 int act, void* H, int64_t ldh, void* pre, int64_t ldpre, int passes,
                 hipStream_t stream) {
  const mbok_desc stacked = gated_stacked(d);
  const GatedOut out = {reinterpret_cast<uint16_t*>(H), ldh, reinterpret_cast<uint16_t*>(pre),
                        ldpre, d->m, act};
  return launch_gated_stacked(&stacked, packed, X, T, ldx, out, passes, stream);
}

int launch_gated_backward(const mbok_desc* d, const void* packed, const void* pre, int64_t ldpre,
                          const void* dH, int64_t lddh, int64_t T, int act, void* dpre,
                          int64_t lddpre, void* dX, int64_t lddx, void* ws, int passes,
                          hipStream_t stream) {
  const int64_t items = T * ((d->m + 7) / 8);
  const int64_t blocks = (items + 255) / 256;
  if (blocks > UINT32_MAX / 256) return MBOK_ERR_SHAPE;  // a launch has 2^32 threads at most
  hipLaunchKernelGGL(gated_backward_kernel, dim3((unsigned)blocks), dim3(256), 0, stream,
                     reinterpret_cast<const uint16_t*>(pre), ldpre,
                     reinterpret_cast<const uint16_t*>(dH), lddh,
                     reinterpret_cast<uint16_t*>(dpre), lddpre, d->m, items, act);
  if (hipGetLastError() != hipSuccess) return MBOK_ERR_HIP;
  if (!dX) return MBOK_OK;
  const mbok_desc stacked = gated_stacked(d);
  return launch_gemmt(&stacked, packed, dpre, T, lddpre, dX, lddx, ws, passes, stream);
}

}  // namespace mbok
