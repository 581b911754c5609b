// The layer Y = R + act(X W_hat^T + b) for some hundred tokens on the matrix cores
// (gfx950): few tiles, each walked by several sets of wavefronts.
//
// A tile of 64 x 64 outputs takes 0.42 us per 64 columns on two wavefronts, which
// leave most of a compute unit idle, and a batch of some hundred tokens has too few
// tiles to fill the part with them.  Here a workgroup's wavefronts divide the scale
// groups between them, each set with its own LDS buffers, and the sums meet in LDS
// in a fixed order.  Bound by no unit alone: a set of two wavefronts reads 24 KB and
// writes 16 KB of LDS per 64 columns, active in 40% of the cycles, the matrix cores in
// 22% (4096 x 11008, K = 3, 256 tokens); a set waits for its own steps.
#include "linear_tile.h"

namespace mbok {
namespace {

template <typename AT, int K, typename P, int C, bool TWO>
__global__ void __launch_bounds__(P::threads* C) linear_shares_kernel(
    const uint32_t* __restrict__ bits, const AT* __restrict__ scales,
    const uint16_t* __restrict__ X, int64_t ldx, LinearOut out, int T, int m_pad, int G, int ntx,
    int nty) {
  extern __shared__ __attribute__((aligned(16))) uint16_t smem[];
  const int tile = tile_of_block(blockIdx.x, ntx, nty);
  const int t0 = (tile / ntx) * P::BT, n0 = (tile % ntx) * P::BN;
  product_tile<AT, K, P, TWO, false, C>(
      bits, scales, X, ldx, T, m_pad, G, t0, n0, smem,
      [&](const f32x16 (&acc)[P::TI][2], int wt, int wn, int part) {
        float* sums = reinterpret_cast<float*>(smem);
        if (out.y_f32) linear_outputs<P, true, C>(acc, wt, wn, part, out, T, t0, n0, sums);
        else linear_outputs<P, false, C>(acc, wt, wn, part, out, T, t0, n0, sums);
      });
}

// The first form whose tiles run in one round takes the call.  (us, K = 3, forms 0, 1,
// 2 and the tiles without shares: 4096 x 11008, 64 to 256 tokens, 64 to 256 tiles of 64 x
// 64: 43-46, 52-55, 86, 72-78; 320 tokens 87, 73, 85, 96; 700, 192 tiles of 128 x 128: 127,
// 119, 88, 112; 1000 173, 151, 103, 112.  11008 x 4096, 200: 52, 47, 37, 44; 320, 258 of 128 x
// 128: 71, 60, 76, 59.  2000 x 640, 700: 13, 10, 11, 11.)  cost: 1e-5 us per column of the round.
struct Form {
  int tokens, rows, shares, round, cost;
};
constexpr Form kForms[] = {{64, 64, 4, 256, 350}, {64, 64, 2, 512, 620}, {128, 128, 2, 256, 740}};

int form_of(const Geom& geo, int64_t T) {
  for (int i = 0; i < 3; ++i) {
    const Form& f = kForms[i];
    const int64_t tiles =
        (T + f.tokens - 1) / f.tokens * (((int64_t)geo.m + f.rows - 1) / f.rows);
    if (geo.G >= f.shares && tiles <= f.round) return i;
  }
  return -1;
}

template <typename AT, int K, bool TWO>
void launch_k(int form, const Geom& geo, const void* packed, const uint16_t* X, int64_t T,
              int64_t ldx, const LinearOut& out, hipStream_t stream) {
  const uint32_t* bits = reinterpret_cast<const uint32_t*>(packed);
  const AT* scales = reinterpret_cast<const AT*>(reinterpret_cast<const char*>(packed) +
                                                 geo.bits_bytes);
  auto go = [&](auto tile, auto shares) {
    using P = decltype(tile);
    constexpr int C = decltype(shares)::value;
    const int ntx = (geo.m + P::BN - 1) / P::BN, nty = (int)((T + P::BT - 1) / P::BT);
    hipLaunchKernelGGL((linear_shares_kernel<AT, K, P, C, TWO>), dim3((unsigned)(ntx * nty)),
                       dim3(P::threads * C), P::lds * C, stream, bits, scales, X, ldx, out, (int)T,
                       geo.RB * kRowBlock, geo.G, ntx, nty);
  };
  using std::integral_constant;
  if (form == 0) go(Tile<2, 1, 1>{}, integral_constant<int, 4>{});
  else if (form == 1) go(Tile<2, 1, 1>{}, integral_constant<int, 2>{});
  else go(Tile<2, 2, 2>{}, integral_constant<int, 2>{});
}

template <typename AT, bool TWO>
void launch_t(int form, const Geom& geo, const void* packed, const uint16_t* X, int64_t T,
              int64_t ldx, const LinearOut& out, hipStream_t stream) {
  switch (geo.K) {
    case 1: launch_k<AT, 1, TWO>(form, geo, packed, X, T, ldx, out, stream); break;
    case 2: launch_k<AT, 2, TWO>(form, geo, packed, X, T, ldx, out, stream); break;
    case 3: launch_k<AT, 3, TWO>(form, geo, packed, X, T, ldx, out, stream); break;
    default: launch_k<AT, 4, TWO>(form, geo, packed, X, T, ldx, out, stream); break;
  }
}

}  // namespace

int linear_shares_cost(const mbok_desc* d, int64_t T) {
  const int form = form_of(make_geom(d), T);
  return form < 0 ? 0 : kForms[form].cost;
}

int launch_linear_shares(const mbok_desc* d, const void* packed, const void* X, int64_t T,
                         int64_t ldx, const LinearOut& out, int passes, hipStream_t stream) {
  const Geom geo = make_geom(d);
  const int form = form_of(geo, T);
  const uint16_t* x = reinterpret_cast<const uint16_t*>(X);
  auto go = [&](auto scale) {
    using AT = decltype(scale);
    if (passes == 2) launch_t<AT, true>(form, geo, packed, x, T, ldx, out, stream);
    else launch_t<AT, false>(form, geo, packed, x, T, ldx, out, stream);
  };
  if (d->alpha_dtype == MBOK_F16) go(uint16_t{});
  else go(float{});
  return hipGetLastError() == hipSuccess ? MBOK_OK : MBOK_ERR_HIP;
}

}  // namespace mbok
