// The layer Y = R + act(X W_hat^T + b) for many tokens on the matrix cores
// (gfx950): product_tile of mfma_tile.h with an epilogue that adds the bias,
// applies the activation and adds the residual in fp32 and rounds once.
//
// Bound: the matrix cores.  (11008 x 4096, K = 3, 2048 tokens with bias, gelu and kept
// pre-activations: 189 us, 980 TFLOP/s, the cores busy 55% of the cycles; product alone
// 176.)
#include "linear_tile.h"

namespace mbok {
namespace {

using Whole = Tile<2, 4, 4>;
using Half = Tile<2, 4, 2>;  // half of a whole tile's tokens, all of its rows
static_assert(Whole::threads == Half::threads && Whole::BN == Half::BN && Half::lds <= Whole::lds,
              "both in one launch");

// The first `full` workgroups take whole tiles (of P), the others (P is Whole) halves
// of the rest, 16 for every 8 tiles: workgroup b runs on XCD b % 8, and the two halves
// of a tile stay on one XCD, whose L2 then reads their weights once.
template <typename AT, int K, typename P, bool TWO, bool F32>
__global__ void __launch_bounds__(P::threads) linear_mfma_kernel(
    const uint32_t* __restrict__ bits, const AT* __restrict__ scales,
    const uint16_t* __restrict__ X, int64_t ldx, LinearOut out, int T, int m_pad, int G, int ntx,
    int nty, int full) {
  extern __shared__ __attribute__((aligned(16))) uint16_t smem[];
  const int b = blockIdx.x;
  if (!std::is_same<P, Whole>::value || b < full) {
    const int even = full & ~7;
    const int p = b < even ? (b & 7) * (even >> 3) + (b >> 3) : b;
    const int tile = tile_at(p, ntx, nty);
    linear_tile<AT, K, P, TWO, F32>(bits, scales, X, ldx, out, T, m_pad, G, (tile / ntx) * P::BT,
                                    (tile % ntx) * P::BN, smem);
  } else if constexpr (std::is_same<P, Whole>::value) {
    const int h = b - full;
    const int p = full + (h >> 4) * 8 + (h & 7);
    if (p >= ntx * nty) return;
    const int tile = tile_at(p, ntx, nty);
    const int t0 = (tile / ntx) * Whole::BT + ((h >> 3) & 1) * Half::BT;
    if (t0 >= T) return;
    linear_tile<AT, K, Half, TWO, F32>(bits, scales, X, ldx, out, T, m_pad, G, t0,
                                       (tile % ntx) * Whole::BN, smem);
  }
}

constexpr int kUnits = 256;  // compute units

template <typename AT, int K, bool TWO>
void launch_k(const Geom& geo, const void* packed, const uint16_t* X, int64_t T, int64_t ldx,
              const LinearOut& out, hipStream_t stream) {
  const uint32_t* bits = reinterpret_cast<const uint32_t*>(packed);
  const AT* scales = reinterpret_cast<const AT*>(reinterpret_cast<const char*>(packed) +
                                                 geo.bits_bytes);
  auto tiles = [&](int bt, int bn) { return ((T + bt - 1) / bt) * ((geo.m + bn - 1) / bn); };
  auto go = [&](auto tile, int64_t full, int64_t halves) {
    using P = decltype(tile);
    const int ntx = (geo.m + P::BN - 1) / P::BN, nty = (int)((T + P::BT - 1) / P::BT);
    auto run = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)(full + halves)), dim3(P::threads), P::lds, stream,
                         bits, scales, X, ldx, out, (int)T, geo.RB * kRowBlock, geo.G, ntx, nty,
                         (int)full);
    };
    if (out.y_f32) run(linear_mfma_kernel<AT, K, P, TWO, true>);
    else run(linear_mfma_kernel<AT, K, P, TWO, false>);
  };
  auto all = [&](auto tile) {
    using P = decltype(tile);
    go(tile, tiles(P::BT, P::BN), 0);
  };
  // (Calls of few tiles run in shares of the contraction instead, linear_shares.hip.)  Up
  // to 64 tokens take tiles of 64 x 64.  More: rounds of 256 whole tiles, then what is
  // left of them in halves where those make one round (half a whole tile takes 63% of
  // its time: 11008 x 4096, K = 3, 2048 tokens, 344 tiles, 218 -> 189 us; 4096 x 11008,
  // 128 tiles, 205 -> 189) or nearly fill it (11008 x 4096, 512 tokens, 86 tiles: 79 -> 71
  // us; 5120 x 5120, K = 2, 1000 tokens, 80 tiles: 80 -> 76; 8192 x 1024, K = 2, 1000 tokens,
  // 128 tiles: 24, 128 x 128 in shares 28), else whole; without a whole round and with
  // fewer tiles, 128 x 128 where those fill the part, else 64 x 64.
  const int64_t whole = tiles(256, 256), rest = whole % kUnits;
  if (T <= 64) all(Tile<2, 1, 1>{});
  else if (rest > kUnits / 2) all(Whole{});
  else if (whole > rest || rest >= 80) go(Whole{}, whole - rest, (rest + 7) / 8 * 16);
  else if (tiles(128, 128) >= kUnits) all(Tile<2, 2, 2>{});
  else all(Tile<2, 1, 1>{});
}

template <typename AT, bool TWO>
void launch_t(const Geom& geo, const void* packed, const uint16_t* X, int64_t T, int64_t ldx,
              const LinearOut& out, hipStream_t stream) {
  switch (geo.K) {
    case 1: launch_k<AT, 1, TWO>(geo, packed, X, T, ldx, out, stream); break;
    case 2: launch_k<AT, 2, TWO>(geo, packed, X, T, ldx, out, stream); break;
    case 3: launch_k<AT, 3, TWO>(geo, packed, X, T, ldx, out, stream); break;
    default: launch_k<AT, 4, TWO>(geo, packed, X, T, ldx, out, stream); break;
  }
}

}  // namespace

// The kernel's offsets inside the layer's signs and inside a tile's activations
// are 32 bits.
int launch_linear_mfma(const mbok_desc* d, const void* packed, const void* X, int64_t T,
                       int64_t ldx, const LinearOut& out, int passes, hipStream_t stream) {
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
