// The gated feed-forward block H = act(X Wg^T) (.) (X Wu^T) for one token,
// two tokens, and up to eight tokens on large layers (gfx950): the fp4 x fp8
// matrix-core products of f4_body.h on the stacked layer, whose 16-row tiles
// hold 8 gate rows and the same 8 up rows, with the activation and the
// product applied where a tile's wavefront sums are added.  The two
// projections, the activation and the product are one kernel and the fp32
// pre-activations never leave it.  Bound as there by the read of the signs (two
// 11008 x 4096, K = 3: 8.6 us for one token, 38 MB; 13.9 us for 8 tokens,
// where the bf16 +-1 kernel takes 20.6).
#include "f4_body.h"
#include "mbok_gated.h"

namespace mbok {
namespace {

template <typename AT, int K, int NT, bool EARLY>
__global__ void __launch_bounds__(f4_max_waves(K) * kWave) gated_f4_kernel(
    const uint4* __restrict__ bits, const uint16_t* __restrict__ x, int G, int tiles,
    int slab_groups, int grid, int nw, int tpw, int textra, GatedOut out) {
  gemv_f4_body<AT, K, NT, EARLY>(bits, x, G, tiles, slab_groups, grid, nw, tpw, textra, out);
}

template <typename AT, int K, int NT, bool EARLY>
__global__ void __launch_bounds__(f4_max_waves(K, 2) * kWave) gated_f4_pair_kernel(
    const uint4* __restrict__ bits, const uint16_t* __restrict__ x, int G, int tiles,
    int slab_groups, int grid, int nw, int tpw, int textra, GatedOut out, int ldx) {
  f4_tokens_body<AT, K, NT, 2, EARLY>(bits, x, ldx, G, tiles, slab_groups, grid, nw, tpw, textra,
                                      out);
}

template <typename AT, int K, int NT, bool EARLY>
__global__ void __launch_bounds__(f4g_waves(1) * kWave) gated_f4g_kernel(
    const uint4* __restrict__ bits, const uint16_t* __restrict__ X, int G, int tiles,
    int slab_groups, int grid, int nw, int tpw, int textra, GatedOut out, int T, int ldx) {
  f4g_body<AT, K, NT, 1, EARLY>(bits, X, G, tiles, slab_groups, grid, nw, tpw, textra, out, T,
                                ldx);
}

// Work split of launch_f4_k (gemv_f4.hip) for `waves` wavefronts at most
struct F4Split {
  int nslabs, slab, NW, tiles, grid, slots;
};
F4Split f4_split(const Geom& geo, int waves) {
  F4Split s;
  const int max_slab = kF4GroupsPerWave * waves;
  s.nslabs = (geo.G + max_slab - 1) / max_slab;
  s.slab = (geo.G + s.nslabs - 1) / s.nslabs;
  s.NW = (s.slab + kF4GroupsPerWave - 1) / kF4GroupsPerWave;
  s.tiles = geo.RB * (kRowBlock / 16);
  s.grid = s.tiles < 256 ? s.tiles : 256;
  if (s.grid * kF4J < s.tiles) s.grid = (s.tiles + kF4J - 1) / kF4J;
  s.slots = (s.tiles + s.grid - 1) / s.grid;
  return s;
}

// calls f with the tile slots of a kernel that holds `slots` tiles per workgroup
template <typename F>
void by_slots(int slots, F&& f) {
  if (slots <= 1) f(std::integral_constant<int, 1>{});
  else if (slots <= 2) f(std::integral_constant<int, 2>{});
  else if (slots <= 4) f(std::integral_constant<int, 4>{});
  else if (slots <= 6) f(std::integral_constant<int, 6>{});
  else f(std::integral_constant<int, 8>{});
}

enum Form { kOne, kPair, kOctet };

template <typename AT, int K>
int launch_k(Form form, const Geom& geo, const void* packed, const void* X, int T, int ldx,
             const GatedOut& out, hipStream_t stream) {
  const F4Split s = f4_split(
      geo, form == kOne ? f4_max_waves(K) : form == kPair ? f4_max_waves(K, 2) : f4g_waves(1));
  const uint4* bits = reinterpret_cast<const uint4*>(packed);
  const uint16_t* x = reinterpret_cast<const uint16_t*>(X);
  by_slots(s.slots, [&](auto slots) {
    constexpr int NT = decltype(slots)::value;
    auto go = [&](auto kernel, auto... more) {
      hipLaunchKernelGGL(kernel, dim3(s.grid), dim3(s.NW * kWave), 0, stream, bits, x, geo.G,
                         s.tiles, s.slab, s.grid, s.NW, s.tiles / s.grid, s.tiles % s.grid, out,
                         more...);
    };
    // the first tile's signs go out behind the activations when there is
    // more than one tile (or, one token, more than one column slab)
    if constexpr (NT == 1) {
      if (form == kOne && s.nslabs > 1) go(gated_f4_kernel<AT, K, 1, true>);
      else if (form == kOne) go(gated_f4_kernel<AT, K, 1, false>);
      else if (form == kPair) go(gated_f4_pair_kernel<AT, K, 1, false>, ldx);
      else go(gated_f4g_kernel<AT, K, 1, false>, T, ldx);
    } else {
      if (form == kOne) go(gated_f4_kernel<AT, K, NT, true>);
      else if (form == kPair) go(gated_f4_pair_kernel<AT, K, NT, true>, ldx);
      else go(gated_f4g_kernel<AT, K, NT, true>, T, ldx);
    }
  });
  return hipGetLastError() == hipSuccess ? MBOK_OK : MBOK_ERR_HIP;
}

template <typename AT>
int launch_t(Form form, const Geom& geo, const void* packed, const void* X, int T, int ldx,
             const GatedOut& out, hipStream_t stream) {
  switch (geo.K) {
    case 1: return launch_k<AT, 1>(form, geo, packed, X, T, ldx, out, stream);
    case 2: return launch_k<AT, 2>(form, geo, packed, X, T, ldx, out, stream);
    case 3: return launch_k<AT, 3>(form, geo, packed, X, T, ldx, out, stream);
    default: return launch_k<AT, 4>(form, geo, packed, X, T, ldx, out, stream);
  }
}

}  // namespace

int gated_f4_max_tokens() { return kF4gTokens; }

int launch_gated_f4(const mbok_desc* stacked, const void* packed, const void* X, int64_t T,
                    int64_t ldx, const GatedOut& out, hipStream_t stream) {
  if (T < 1 || T > kF4gTokens || (T > 1 && (T - 1) * ldx + stacked->n > INT32_MAX))
    return MBOK_ERR_SHAPE;
  const Geom geo = make_geom(stacked);
  const Form form = T == 1 ? kOne : T == 2 ? kPair : kOctet;
  const int ld = T == 1 ? stacked->n : (int)ldx;
  if (stacked->alpha_dtype == MBOK_F16)
    return launch_t<uint16_t>(form, geo, packed, X, (int)T, ld, out, stream);
  return launch_t<float>(form, geo, packed, X, (int)T, ld, out, stream);
}

}  // namespace mbok
