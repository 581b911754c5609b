// The gated feed-forward block H = act(X Wg^T) (.) (X Wu^T) for many tokens on
// the matrix cores (gfx950).
//
// "Highly Efficient and Effective LLMs with Multi-Boolean Architectures",
// Paper-Notes reading note, 关键设计: W_hat = sum_k alpha_k (.) B_k with
// group-wise scales.  Both projections are one stacked layer (mbok_gated.h), so
// the block is one product with 256 tokens x 256 stacked rows (128 outputs) per
// workgroup and an epilogue in registers.
//
// Bound: the matrix cores (4 T m n operations against a few bytes per weight),
// here at ~2.1 GHz under this load: 11008 x 4096, K = 3, 2048 tokens with the
// pre-activations 332 us, 1112 TFLOP/s, matrix cores 63% busy.
// The product is product_tile of mfma_tile.h.
//
// A wavefront's two 32-row blocks are 32 gate rows and the same 32 up rows: the
// unpacking thread of stacked row 64 b + 16 u + 8 h + r writes its weights to
// LDS row 64 b + 32 h + 8 u + r, so a lane holds both values of an output.  The
// outputs go through LDS (free by then) to whole 16-byte stores.
//
// Few tokens or few rows take smaller tiles (see launch_k).  Cutting the last
// partial round of whole tiles into halves and quarters was measured slower
// than running it whole (11008 x 4096, 2048 tokens, 688 tiles on 256 compute
// units: 346 against 328 us; a half copies the same activations for half the
// products).
#include "mbok_gated.h"
#include "mfma_tile.h"

namespace mbok {
namespace {

// The outputs of the wavefront (wt, wn): first H, then (training) the
// pre-activations.
template <typename P>
__device__ __forceinline__ void gated_outputs(const f32x16 (&acc)[P::TI][2], int wt, int wn,
                                              const GatedOut& out, int T, int t0, int n0,
                                              uint16_t* smem) {
  constexpr int TI = P::TI, kThreads = P::threads, kBT = P::BT;
  const int tid = threadIdx.x, lane = tid & 63;
  const int o0 = n0 / 2;                     // first output of the tile
  const int oc = wn * 32 + (lane & 31);      // the lane's output in the tile
  const bool inside = o0 + oc < out.m;
  const int tb = wt * 32 * TI + 4 * (lane >> 5);
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float unused;
      const float h = activation<false>(out.act, acc[i][0][r], unused) * acc[i][1][r];
      smem[(tb + 32 * i + 8 * (r >> 2) + (r & 3)) * P::HS + oc] = to_bf16(h);
    }
  __syncthreads();
  constexpr int HP = P::BN / 16;  // 16-byte pieces of a row of H
  for (int e = tid; e < kBT * HP; e += kThreads) {
    const int t = e / HP, c = 8 * (e % HP);
    if (t0 + t >= T || o0 + c >= out.m) continue;
    const u32x4 v = *reinterpret_cast<const u32x4*>(smem + t * P::HS + c);
    uint16_t* dst = out.H + (int64_t)(t0 + t) * out.ldh + o0 + c;
    if (o0 + c + 8 <= out.m) {
      *reinterpret_cast<u32x4_any*>(dst) = v;
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (o0 + c + q < out.m)
          dst[q] = (uint16_t)((q & 1) ? v[q >> 1] >> 16 : v[q >> 1] & 0xffffu);
    }
  }
  if (!out.pre) return;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      uint16_t* p = smem + (tb + 32 * i + 8 * (r >> 2) + (r & 3)) * P::PS + 16 * (oc >> 3) +
                    (oc & 7);
      p[0] = inside ? to_bf16(acc[i][0][r]) : (uint16_t)0;
      p[8] = inside ? to_bf16(acc[i][1][r]) : (uint16_t)0;
    }
  __syncthreads();
  constexpr int PP = P::BN / 8;
  const int m2 = 2 * ((out.m + 7) & ~7);
  for (int e = tid; e < kBT * PP; e += kThreads) {
    const int t = e / PP, c = 8 * (e % PP);
    if (t0 + t < T && n0 + c < m2)
      *reinterpret_cast<u32x4*>(out.pre + (int64_t)(t0 + t) * out.ldpre + n0 + c) =
          *reinterpret_cast<const u32x4*>(smem + t * P::PS + c);
  }
}

// TWO with the pre-activations: 11008 x 4096, 2048 tokens 607 us, 64 tokens 76 us
template <typename AT, int K, typename P, bool TWO>
__global__ void __launch_bounds__(P::threads) gated_mfma_kernel(
    const uint32_t* __restrict__ bits, const AT* __restrict__ scales,
    const uint16_t* __restrict__ X, int64_t ldx, GatedOut out, int T, int m_pad, int G, int ntx,
    int nty) {
  extern __shared__ __attribute__((aligned(16))) uint16_t smem[];
  const int tile = tile_of_block(blockIdx.x, ntx, nty);
  const int t0 = (tile / ntx) * P::BT, n0 = (tile % ntx) * P::BN;
  product_tile<AT, K, P, TWO, true>(bits, scales, X, ldx, T, m_pad, G, t0, n0, smem,
                                    [&](const f32x16 (&acc)[P::TI][2], int wt, int wn, int) {
                                      gated_outputs<P>(acc, wt, wn, out, T, t0, n0, smem);
                                    });
}

template <typename AT, int K, bool TWO>
void launch_k(const Geom& geo, const void* packed, const uint16_t* X, int64_t T, int64_t ldx,
              const GatedOut& out, hipStream_t stream) {
  const uint32_t* bits = reinterpret_cast<const uint32_t*>(packed);
  const AT* scales = reinterpret_cast<const AT*>(reinterpret_cast<const char*>(packed) +
                                                 geo.bits_bytes);
  auto tiles = [&](int bt, int bn) { return ((T + bt - 1) / bt) * ((geo.m + bn - 1) / bn); };
  auto go = [&](auto tile) {
    using P = decltype(tile);
    const int ntx = (geo.m + P::BN - 1) / P::BN, nty = (int)((T + P::BT - 1) / P::BT);
    hipLaunchKernelGGL((gated_mfma_kernel<AT, K, P, TWO>), dim3((unsigned)ntx * (unsigned)nty),
                       dim3(P::threads), P::lds, stream, bits, scales, X, ldx, out, (int)T,
                       geo.RB * kRowBlock, geo.G, ntx, nty);
  };
  // Whole tiles where they occupy more than half of the compute units; else
  // 128 x 128 (two workgroups per compute unit) where those fill the part,
  // else, and always for up to 64 tokens, 64 x 64 (five per compute unit).
  if (T > 64 && tiles(256, 256) > 128) go(Tile<2, 4, 4>{});
  else if (T > 64 && tiles(128, 128) >= 256) go(Tile<2, 2, 2>{});
  else go(Tile<2, 1, 1>{});
}

template <typename AT, bool TWO>
void launch_t(const Geom& geo, const void* packed, const uint16_t* X, int64_t T, int64_t ldx,
              const GatedOut& out, hipStream_t stream) {
  switch (geo.K) {
    case 1: launch_k<AT, 1, TWO>(geo, packed, X, T, ldx, out, stream); break;
    case 2: launch_k<AT, 2, TWO>(geo, packed, X, T, ldx, out, stream); break;
    case 3: launch_k<AT, 3, TWO>(geo, packed, X, T, ldx, out, stream); break;
    default: launch_k<AT, 4, TWO>(geo, packed, X, T, ldx, out, stream); break;
  }
}

}  // namespace

// d: the stacked layer.  The kernel's offsets inside the layer's signs and
// inside a tile's activations are 32 bits.
int launch_gated_mfma(const mbok_desc* d, const void* packed, const void* X, int64_t T,
                      int64_t ldx, const GatedOut& out, int passes, hipStream_t stream) {
  const Geom geo = make_geom(d);
  if (geo.bits_bytes / 4 >= (int64_t(1) << 32)) return MBOK_ERR_SHAPE;
  if (ldx >= (int64_t(1) << 32) / 512) return MBOK_ERR_INVALID_ARG;
  const uint16_t* x = reinterpret_cast<const uint16_t*>(X);
  auto go = [&](auto scale) {
    using AT = decltype(scale);
    if (passes == 2) launch_t<AT, true>(geo, packed, x, T, ldx, out, stream);
    else launch_t<AT, false>(geo, packed, x, T, ldx, out, stream);
  };
  if (d->alpha_dtype == MBOK_F16) go(uint16_t{});
  else go(float{});
  return hipGetLastError() == hipSuccess ? MBOK_OK : MBOK_ERR_HIP;
}

}  // namespace mbok
