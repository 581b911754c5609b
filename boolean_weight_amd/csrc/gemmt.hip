// Transposed product dX = dY . W_hat for T gradient rows on the matrix cores
// (gfx950): the activation gradient of a Boolean-kernel layer.
//
// "Highly Efficient and Effective LLMs with Multi-Boolean Architectures",
// gist.science summaries, training sections: gradients flow through the
// Boolean weights; Paper-Notes reading note, 关键设计: W_hat = sum_k alpha_k
// (.) B_k, one scale per (row, 128-column group, kernel).
//     dX[t, j] = sum_i dY[t, i] W_hat[i, j]
//
// The contraction runs over the rows of W_hat, in steps of one 64-row block
// of the packed layout.  A step's dY tile (BT tokens x 64 rows) and W_hat tile
// (64 rows x 256 columns, formed from signs and scales and rounded to bf16)
// live in LDS, double-buffered; a thread forms 32 columns of one row.  The
// W_hat tile is stored as it is formed, row by row, and the matrix operand
// (8 consecutive rows of one column per lane) is read with the transposing
// LDS load ds_read_b64_tr_b16: of 16 lanes, lane s supplies the address of 4
// columns 4 (s & 3) .. of row s >> 2, and receives column s of the 4 rows.
//
// Rows past m have zero weights, and dY is read inside its m columns only: a
// partial last row block is a step of its own with element-wise loads.
#include <stdint.h>

#include <type_traits>

#include "mbok_device.h"
#include "mbok_launch.h"
#include "mbok_levels.h"

namespace mbok {
namespace {

typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t u32x4_any;  // dY rows start anywhere
typedef __attribute__((ext_vector_type(4))) short i16x4;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;

constexpr int kBN = 256;       // columns per workgroup tile
constexpr int kThreads = 512;  // 8 wavefronts
constexpr int kAStride = 72;   // bf16 elements per LDS row of dY (64 + 8)
constexpr int kWStride = 272;  // bf16 elements per LDS row of W_hat (256 + 16)

// Token rows of a tile and how the 8 wavefronts share it: WT wavefronts along
// the tokens, 8 / WT along the columns, each TI x TJ blocks of 32 x 32.
template <int TI_, int TJ_, int WT_>
struct Tile {
  static constexpr int TI = TI_, TJ = TJ_, WT = WT_, WN = 8 / WT_;
  static constexpr int BT = 32 * TI * WT;
  static_assert(32 * TJ * WN == kBN, "256 columns");
  static constexpr int kA = BT * kAStride, kW = kRowBlock * kWStride;  // elements
  static constexpr size_t kLds = 2 * (size_t)(kA + kW) * sizeof(uint16_t);
};

// 8 rows (k0 .. k0 + 7) of one column per lane: two transposing reads
__device__ __forceinline__ bf16x8 read_tr(const uint16_t* p) {
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p);
  const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 4 * kWStride));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

template <typename AT, int K, typename TL, bool PART>
__global__ void __launch_bounds__(kThreads) gemmt_kernel(
    const uint32_t* __restrict__ bits, const AT* __restrict__ scales,
    const uint16_t* __restrict__ dY, int64_t lddy, uint16_t* __restrict__ dX, int64_t lddx,
    float* __restrict__ part, int T, int m, int n, int RB, int slices) {
  constexpr int TI = TL::TI, TJ = TL::TJ, BT = TL::BT;
  constexpr int NA = (BT * 8 + kThreads - 1) / kThreads;  // 16-byte pieces of dY per thread
  extern __shared__ __attribute__((aligned(16))) uint16_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int G = n / kGroup;
  const int ntx = (n + kBN - 1) / kBN, nty = (T + BT - 1) / BT;
  const int ntiles = ntx * nty;
  // workgroup -> (slice, tile): consecutive positions on one XCD
  int p = blockIdx.x;
  const int nb = ntiles * slices;
  if ((nb & 7) == 0) p = (p & 7) * (nb >> 3) + (p >> 3);
  const int slice = p / ntiles;
  const int tile = tile_at(p - slice * ntiles, ntx, nty);
  const int t0 = (tile / ntx) * BT, j0 = (tile % ntx) * kBN;
  const int rb0 = (int)((int64_t)RB * slice / slices);
  const int rb1 = (int)((int64_t)RB * (slice + 1) / slices);
  // steps over whole row blocks; a partial last block is the tail
  const int full_end = min(rb1, m / kRowBlock);
  const int S = full_end - rb0;  // may be 0 or less
  const bool tail = rb1 > full_end;

  // unpack role: row `lane` of the step's block, 32-column word `wave` of the tile
  const int gw = min(j0 / kGroup + (wave >> 2), G - 1);
  const int uword = wave & 3;
  // dY copy role: piece u = token tid / 8 + 64 u, rows 8 (tid % 8) ..
  const int apart = tid & 7;
  const bool a_live = BT * 8 >= kThreads || tid < BT * 8;
  const uint16_t* arow[NA];
#pragma unroll
  for (int u = 0; u < NA; ++u) {
    const int t = min(t0 + (tid >> 3) + 64 * u, T - 1);  // extra tokens are never stored
    arow[u] = dY + (int64_t)t * lddy + 8 * apart;
  }

  struct StepRegs {
    u32x4 x[NA];
    uint32_t w[K];
    AT a[K];
  };
  StepRegs R0, R1;
  auto load_w = [&](int rb, StepRegs& R) {
    const int64_t c = ((int64_t)rb * G + gw) * K * kRowBlock;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      R.w[k] = bits[(c + k * kRowBlock + lane) * 4 + uword];
      R.a[k] = scales[c + k * kRowBlock + lane];
    }
  };
  auto load = [&](int rb, StepRegs& R) {
    if (a_live) {
#pragma unroll
      for (int u = 0; u < NA; ++u)
        R.x[u] = *reinterpret_cast<const u32x4_any*>(arow[u] + (int64_t)rb * kRowBlock);
    }
    load_w(rb, R);
  };
  // the partial last block: dY element by element inside its m columns
  auto load_tail = [&](int rb, StepRegs& R) {
    const int i0 = rb * kRowBlock + 8 * apart;
#pragma unroll
    for (int u = 0; u < NA; ++u) {
      uint32_t e[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        e[q] = a_live && i0 + q < m ? arow[u][(int64_t)rb * kRowBlock + q] : 0u;
      R.x[u] = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
    }
    load_w(rb, R);
  };

  f32x16 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  const int wt = wave / TL::WN, wn = wave % TL::WN;
  // dY operand: token lane % 32, rows 8 (lane / 32) ..; W_hat operand: see read_tr
  const int aoff = (wt * 32 * TI + (lane & 31)) * kAStride + (lane >> 5) * 8;
  const int woff = (8 * (lane >> 5) + ((lane & 15) >> 2)) * kWStride + wn * 32 * TJ +
                   16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  auto abuf = [&](int b) { return smem + b * (TL::kA + TL::kW); };
  auto wbuf = [&](int b) { return smem + b * (TL::kA + TL::kW) + TL::kA; };

  Levels L;
  uint32_t V[4];
  auto begin_store = [&](const StepRegs& R) {
    if (K <= 3) {
      float af[K];
#pragma unroll
      for (int k = 0; k < K; ++k) af[k] = alpha_to_f32<AT>(R.a[k]);
      L = make_levels<K, false>(af);
      word_selectors<K>(R.w, V);
    }
  };
  // quarter q of a step's stores: 8 columns of W_hat, up to one dY piece
  auto store = [&](int b, const StepRegs& R, int q) {
    if (q < NA && a_live)
      *reinterpret_cast<u32x4*>(abuf(b) + ((tid >> 3) + 64 * q) * kAStride + 8 * apart) = R.x[q];
    uint32_t out[4];
    if (K <= 3) {
      unpack_two_quads(V, q >> 1, 2 * (q & 1), L, out);
    } else {
      float af[K];
      uint32_t o32[16];
#pragma unroll
      for (int k = 0; k < K; ++k) af[k] = alpha_to_f32<AT>(R.a[k]);
      unpack_word_k4<false>(R.w, af, o32);
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = o32[4 * q + e];
    }
    *reinterpret_cast<u32x4*>(wbuf(b) + lane * kWStride + wave * 32 + 8 * q) =
        u32x4{out[0], out[1], out[2], out[3]};
  };
  // products of buffer b; between(q) runs after sub-step q
  auto mma = [&](int b, auto&& between) {
    const uint16_t* as = abuf(b) + aoff;
    const uint16_t* ws = wbuf(b) + woff;
    bf16x8 pa[2][TI], pb[2][TJ];
    auto frags = [&](int q) {
#pragma unroll
      for (int i = 0; i < TI; ++i)
        pa[q & 1][i] = *reinterpret_cast<const bf16x8*>(as + i * 32 * kAStride + 16 * q);
#pragma unroll
      for (int j = 0; j < TJ; ++j) pb[q & 1][j] = read_tr(ws + 16 * q * kWStride + 32 * j);
    };
    frags(0);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q < 3) frags(q + 1);
#pragma unroll
      for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int i = 0; i < TI; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(pa[q & 1][i], pb[q & 1][j],
                                                              acc[i][j], 0, 0, 0);
      between(q);
    }
  };
  auto store_all = [&](int b, const StepRegs& R) {
    begin_store(R);
#pragma unroll
    for (int q = 0; q < 4; ++q) store(b, R, q);
  };

  if (S > 0) {
    const int last = full_end - 1;
    load(rb0, R0);
    load(min(rb0 + 1, last), R1);
    store_all(0, R0);
    __syncthreads();
    // step s is multiplied from buffer s % 2 while step s + 1 is stored and
    // step s + 2 loaded (indices clamped at the end; the extras are unused)
    for (int s = 0; s < S; s += 2) {
      load(min(rb0 + s + 2, last), R0);
      begin_store(R1);
      mma(0, [&](int q) { store(1, R1, q); });
      __syncthreads();
      if (s + 1 >= S) break;
      load(min(rb0 + s + 3, last), R1);
      begin_store(R0);
      mma(1, [&](int q) { store(0, R0, q); });
      __syncthreads();
    }
  }
  if (tail) {
    load_tail(full_end, R0);
    store_all(0, R0);
    __syncthreads();
    mma(0, [](int) {});
  }

  // C layout: lane l, register r -> token 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int col = j0 + (wn * TJ + j) * 32 + (lane & 31);
      if (col >= n) continue;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int t = t0 + (wt * TI + i) * 32 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        if (t >= T) continue;
        if (PART) {
          part[((int64_t)slice * T + t) * n + col] = acc[i][j][r];
        } else {
          dX[(int64_t)t * lddx + col] =
              __builtin_bit_cast(uint16_t, (__bf16)acc[i][j][r]);
        }
      }
    }
}

// dX = sum of the slices' partial sums in order, rounded once; 8 columns per thread
__global__ void __launch_bounds__(256) gemmt_reduce_kernel(const float* __restrict__ part,
                                                           uint16_t* __restrict__ dX,
                                                           int64_t lddx, int T, int n,
                                                           int slices) {
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  const int64_t total = (int64_t)T * n;
  if (e >= total) return;
  float s[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 v = *reinterpret_cast<const float4*>(part + e + 4 * h);
    s[4 * h] = v.x, s[4 * h + 1] = v.y, s[4 * h + 2] = v.z, s[4 * h + 3] = v.w;
  }
  for (int k = 1; k < slices; ++k)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 v = *reinterpret_cast<const float4*>(part + k * total + e + 4 * h);
      s[4 * h] += v.x, s[4 * h + 1] += v.y, s[4 * h + 2] += v.z, s[4 * h + 3] += v.w;
    }
  const int64_t t = e / n, j = e - t * n;
  *reinterpret_cast<u32x4*>(dX + t * lddx + j) =
      u32x4{bf16_pair(s[0], s[1]), bf16_pair(s[2], s[3]), bf16_pair(s[4], s[5]),
            bf16_pair(s[6], s[7])};
}

constexpr int kUnits = 256;  // workgroups that fill the part (one per compute unit)

int tile_tokens(int64_t T) { return T <= 32 ? 32 : T <= 64 ? 64 : T <= 128 ? 128 : 256; }

// Slices of the row blocks: as many as keep the workgroups within one round
int gemmt_slices(const Geom& geo, int64_t T) {
  const int bt = tile_tokens(T);
  const int64_t tiles = ((geo.n + kBN - 1) / kBN) * ((T + bt - 1) / bt);
  int64_t s = kUnits / tiles;
  if (s > geo.RB / 2) s = geo.RB / 2;  // two steps each at least
  return s < 1 ? 1 : (int)s;
}

template <typename AT, int K>
int launch_k(const Geom& geo, const void* packed, const uint16_t* dY, int64_t T, int64_t lddy,
             uint16_t* dX, int64_t lddx, float* part, int slices, hipStream_t stream) {
  const uint32_t* bits = reinterpret_cast<const uint32_t*>(packed);
  const AT* scales = reinterpret_cast<const AT*>(reinterpret_cast<const char*>(packed) +
                                                 geo.bits_bytes);
  auto go = [&](auto tl, auto partial) {
    using TL = decltype(tl);
    constexpr bool P = decltype(partial)::value;
    const int64_t blocks = (int64_t)((geo.n + kBN - 1) / kBN) * ((T + TL::BT - 1) / TL::BT) * slices;
    hipLaunchKernelGGL((gemmt_kernel<AT, K, TL, P>), dim3((unsigned)blocks), dim3(kThreads),
                       TL::kLds, stream, bits, scales, dY, lddy, dX, lddx, part, (int)T, geo.m,
                       geo.n, geo.RB, slices);
  };
  auto by_tile = [&](auto partial) {
    switch (tile_tokens(T)) {
      case 32: go(Tile<1, 1, 1>{}, partial); break;
      case 64: go(Tile<2, 1, 1>{}, partial); break;
      case 128: go(Tile<4, 1, 1>{}, partial); break;
      default: go(Tile<4, 2, 2>{}, partial); break;
    }
  };
  if (slices > 1) {
    by_tile(std::true_type{});
    const int64_t threads = T * geo.n / 8;
    hipLaunchKernelGGL(gemmt_reduce_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0,
                       stream, part, dX, lddx, (int)T, geo.n, slices);
  } else {
    by_tile(std::false_type{});
  }
  return hipGetLastError() == hipSuccess ? MBOK_OK : MBOK_ERR_HIP;
}

template <typename AT>
int launch_t(const Geom& geo, const void* packed, const void* dY, int64_t T, int64_t lddy,
             void* dX, int64_t lddx, float* part, int slices, hipStream_t stream) {
  const uint16_t* g = reinterpret_cast<const uint16_t*>(dY);
  uint16_t* o = reinterpret_cast<uint16_t*>(dX);
  switch (geo.K) {
    case 1: return launch_k<AT, 1>(geo, packed, g, T, lddy, o, lddx, part, slices, stream);
    case 2: return launch_k<AT, 2>(geo, packed, g, T, lddy, o, lddx, part, slices, stream);
    case 3: return launch_k<AT, 3>(geo, packed, g, T, lddy, o, lddx, part, slices, stream);
    default: return launch_k<AT, 4>(geo, packed, g, T, lddy, o, lddx, part, slices, stream);
  }
}

}  // namespace

size_t gemmt_workspace_bytes(const mbok_desc* d, int64_t T) {
  const Geom geo = make_geom(d);
  const int s = gemmt_slices(geo, T);
  return s > 1 ? (size_t)s * (size_t)T * (size_t)geo.n * sizeof(float) : 0;
}

int launch_gemmt(const mbok_desc* d, const void* packed, const void* dY, int64_t T, int64_t lddy,
                 void* dX, int64_t lddx, void* ws, hipStream_t stream) {
  const Geom geo = make_geom(d);
  const int slices = ws ? gemmt_slices(geo, T) : 1;
  float* part = reinterpret_cast<float*>(ws);
  if (d->alpha_dtype == MBOK_F16)
    return launch_t<uint16_t>(geo, packed, dY, T, lddy, dX, lddx, part, slices, stream);
  return launch_t<float>(geo, packed, dY, T, lddy, dX, lddx, part, slices, stream);
}

}  // namespace mbok
