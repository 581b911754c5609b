// The layer Y = R + act(X W_hat^T + b) for many tokens on the matrix cores
// (gfx950): product_tile of mfma_tile.h with an epilogue that adds the bias,
// applies the activation and adds the residual in fp32 and rounds once.
//
// Bound: the matrix cores.  The sums of 64 tokens at a time go through LDS as
// fp32, so that a thread holds 8 consecutive outputs of a token: whole 16-byte
// accesses to Y, R and the pre-activations, one set of bias values per thread.
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

// The outputs of a tile, 32 TI tokens of each wavefront row in TI passes.
template <typename P, bool F32>
__device__ __forceinline__ void linear_outputs(const f32x16 (&acc)[P::TI][2], int wt, int wn,
                                               const LinearOut& out, int T, int t0, int n0,
                                               float* smem) {
  constexpr int kThreads = P::threads, kPieces = P::BN / 8, kRows = 32 * P::WT;
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
        smem[(32 * wt + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) * P::FS + 32 * (2 * wn + j) +
             (lane & 31)] = acc[i][j][r];
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kRows / kStep; ++s) {
      const int row = s * kStep + tid / kPieces;
      const int64_t t = t0 + 32 * (P::TI * (row >> 5) + i) + (row & 31);
      if (t >= T || live == 0) continue;
      float y[8], z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = smem[row * P::FS + c + e] + bias[e];
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

template <typename AT, int K, typename P, bool TWO, bool F32>
__device__ __forceinline__ void linear_tile(const uint32_t* __restrict__ bits,
                                            const AT* __restrict__ scales,
                                            const uint16_t* __restrict__ X, int64_t ldx,
                                            const LinearOut& out, int T, int m_pad, int G, int t0,
                                            int n0, uint16_t* smem) {
  product_tile<AT, K, P, TWO, false>(bits, scales, X, ldx, T, m_pad, G, t0, n0, smem,
                                     [&](const f32x16 (&acc)[P::TI][2], int wt, int wn) {
                                       linear_outputs<P, F32>(acc, wt, wn, out, T, t0, n0,
                                                              reinterpret_cast<float*>(smem));
                                     });
}

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
  // Up to 64 tokens take tiles of 64 x 64.  More: rounds of 256 whole tiles, then
  // what is left of them in halves where those make one round (half a whole tile
  // takes 63% of its time: 11008 x 4096, K = 3, 2048 tokens, 344 tiles, 218 -> 189
  // us; 4096 x 11008, 128 tiles, 205 -> 189) or nearly fill it (11008 x 4096, 512
  // tokens, 86 tiles: 79 -> 71 us; 5120 x 5120, K = 2, 1000 tokens, 80 tiles: 80 -> 76;
  // 512 tokens, 40 tiles: 58 -> 74), else whole; without a whole round and with
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
