// The fp4 x fp8 matrix-core products of f4_body.h for one token, two tokens and
// up to eight with an epilogue of the caller's (see RowsOut), where a tile's
// wavefront sums are added (gfx950).  Internal header.
#pragma once

#include "f4_body.h"

namespace mbok {
namespace {

template <typename AT, int K, int NT, bool EARLY, typename Out>
__global__ void __launch_bounds__(f4_max_waves(K) * kWave) f4_one_kernel(
    const uint4* __restrict__ bits, const uint16_t* __restrict__ x, int G, int tiles,
    int slab_groups, int grid, int nw, int tpw, int textra, Out out) {
  gemv_f4_body<AT, K, NT, EARLY>(bits, x, G, tiles, slab_groups, grid, nw, tpw, textra, out);
}

template <typename AT, int K, int NT, bool EARLY, typename Out>
__global__ void __launch_bounds__(f4_max_waves(K, 2) * kWave) f4_pair_kernel(
    const uint4* __restrict__ bits, const uint16_t* __restrict__ x, int G, int tiles,
    int slab_groups, int grid, int nw, int tpw, int textra, Out out, int ldx) {
  f4_tokens_body<AT, K, NT, 2, EARLY>(bits, x, ldx, G, tiles, slab_groups, grid, nw, tpw, textra,
                                      out);
}

template <typename AT, int K, int NT, bool EARLY, typename Out>
__global__ void __launch_bounds__(f4g_waves(1) * kWave) f4_octet_kernel(
    const uint4* __restrict__ bits, const uint16_t* __restrict__ X, int G, int tiles,
    int slab_groups, int grid, int nw, int tpw, int textra, Out out, int T, int ldx) {
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

// One token; two; up to eight.
enum F4Form { kOne, kPair, kOctet };

template <typename AT, int K, typename Out>
int launch_f4_k(F4Form form, const Geom& geo, const void* packed, const void* X, int T, int ldx,
             const Out& out, hipStream_t stream) {
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
      if (form == kOne && s.nslabs > 1) go(f4_one_kernel<AT, K, 1, true, Out>);
      else if (form == kOne) go(f4_one_kernel<AT, K, 1, false, Out>);
      else if (form == kPair) go(f4_pair_kernel<AT, K, 1, false, Out>, ldx);
      else go(f4_octet_kernel<AT, K, 1, false, Out>, T, ldx);
    } else {
      if (form == kOne) go(f4_one_kernel<AT, K, NT, true, Out>);
      else if (form == kPair) go(f4_pair_kernel<AT, K, NT, true, Out>, ldx);
      else go(f4_octet_kernel<AT, K, NT, true, Out>, T, ldx);
    }
  });
  return hipGetLastError() == hipSuccess ? MBOK_OK : MBOK_ERR_HIP;
}

template <typename AT, typename Out>
int launch_f4_t(F4Form form, const Geom& geo, const void* packed, const void* X, int T, int ldx,
             const Out& out, hipStream_t stream) {
  switch (geo.K) {
    case 1: return launch_f4_k<AT, 1>(form, geo, packed, X, T, ldx, out, stream);
    case 2: return launch_f4_k<AT, 2>(form, geo, packed, X, T, ldx, out, stream);
    case 3: return launch_f4_k<AT, 3>(form, geo, packed, X, T, ldx, out, stream);
    default: return launch_f4_k<AT, 4>(form, geo, packed, X, T, ldx, out, stream);
  }
}

// d: the layer whose sums go to `out`; 1 to kF4gTokens tokens
template <typename Out>
int launch_f4_forms(const mbok_desc* d, const void* packed, const void* X, int64_t T, int64_t ldx,
                    const Out& out, hipStream_t stream) {
  if (T < 1 || T > kF4gTokens || (T > 1 && (T - 1) * ldx + d->n > INT32_MAX))
    return MBOK_ERR_SHAPE;
  const Geom geo = make_geom(d);
  const F4Form form = T == 1 ? kOne : T == 2 ? kPair : kOctet;
  const int ld = T == 1 ? d->n : (int)ldx;
  if (d->alpha_dtype == MBOK_F16)
    return launch_f4_t<uint16_t>(form, geo, packed, X, (int)T, ld, out, stream);
  return launch_f4_t<float>(form, geo, packed, X, (int)T, ld, out, stream);
}

}  // namespace
}  // namespace mbok
