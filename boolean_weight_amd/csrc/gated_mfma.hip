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
// pre-activations 332 us, 1112 TFLOP/s, matrix cores 63% busy.  8 wavefronts of 128 tokens x 64 rows (2 per
// SIMD); the contraction runs in steps of 64 columns.  A step's activations
// are copied from memory to LDS without passing registers, its weights are
// formed from signs and scales, rounded to bf16 and stored, both
// double-buffered in rows of 128 bytes.  What the design is about is keeping
// the matrix cores fed: one matrix instruction takes 32 cycles, in which its
// wavefront can issue a few vector instructions for free (measured: 4 to 5
// beside every matrix instruction of both wavefronts cost 4%, 8 cost 37%), so
// the weights' forming and the next operands' reads are laid between them a
// few at a time, and the barrier of a step stands before the last quarter of
// its products, whose operands are in registers by then.
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
#include <stdint.h>

#include <type_traits>

#include "mbok_device.h"
#include "mbok_gated.h"
#include "mbok_launch.h"
#include "mbok_levels.h"

namespace mbok {
namespace {

typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t u32x4_any;  // H rows start anywhere

constexpr int kBK = 64;  // columns per step

// A workgroup's tile: WT wavefronts along the tokens and WN along the stacked
// rows, each TI blocks of 32 tokens x 2 blocks of 32 rows.
template <int WT_, int WN_, int TI_>
struct Tile {
  static constexpr int WT = WT_, WN = WN_, TI = TI_;
  static constexpr int threads = 64 * WT * WN, BT = 32 * TI * WT, BN = 64 * WN;
  static constexpr int NU = BT * 8 / threads;     // 16-byte pieces of activations each
  static constexpr int kX = BT * kBK, kW = BN * kBK;  // bf16 elements
  static constexpr int HS = BN / 2 + 8, PS = BN + 8;  // LDS rows of the outputs
  static constexpr size_t lds =
      2 * (size_t)(2 * (kX + kW) > BT * PS ? 2 * (kX + kW) : BT * PS);
  static_assert(lds <= 160 * 1024 && NU * threads == BT * 8, "tile shape");
  static_assert(threads == 2 * BN, "a thread unpacks one 32-column word of a row");
};

// TWO: each 64 columns are two steps with the same activations, the levels
// rounded to bf16 and then the bf16 rounding of what that left (16 significant
// bits together): twice the matrix work (11008 x 4096, 2048 tokens with the
// pre-activations 607 us, 64 tokens 76 us).
template <typename AT, int K, typename P, bool TWO>
__device__ __forceinline__ void gated_tile(const uint32_t* __restrict__ bits,
                                           const AT* __restrict__ scales,
                                           const uint16_t* __restrict__ X, int64_t ldx,
                                           const GatedOut& out, int T, int m_pad, int G, int t0,
                                           int n0, uint16_t* smem) {
  constexpr int TI = P::TI, NU = P::NU, kThreads = P::threads, kBT = P::BT;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int S = (TWO ? 4 : 2) * G;  // steps
  auto block = [](int s) { return TWO ? s >> 1 : s; };  // 64 columns of a step
  auto xbuf = [&](int b) { return smem + b * (P::kX + P::kW); };
  auto wbuf = [&](int b) { return smem + b * (P::kX + P::kW) + P::kX; };

  // A row of either tile is 8 pieces of 16 bytes, piece c of row r at position
  // c ^ (r / 2 & 7): the 64 banks are 16 such positions, two rows.
  // unpacking: one 32-column word of one row; rows past the packed layer read
  // its last row (their sums are never stored)
  const int trow = tid >> 1, word = tid & 1;
  const int lrow = (trow & ~63) + 32 * ((trow >> 3) & 1) + 8 * ((trow >> 4) & 3) + (trow & 7);
  const int wput = lrow * kBK;
  const int wkey = (lrow >> 1) & 7;
  // the tile's first row block and, in 32-bit offsets from it, the thread's
  // chunk of (row, group 0, kernel 0)
  const int rb0 = min(n0, m_pad - kRowBlock) / kRowBlock;
  const int row = min(n0 + trow, m_pad - 1);
  const uint32_t chunk = (uint32_t)(row / kRowBlock - rb0) * (uint32_t)(G * K * kRowBlock) +
                         (uint32_t)(row % kRowBlock);
  const uint32_t woff = chunk * 16u + 4u * word, soff = chunk * (uint32_t)sizeof(AT);
  const char* tile_w = reinterpret_cast<const char*>(bits) +
                       (int64_t)rb0 * G * K * kRowBlock * 16;
  const char* tile_s = reinterpret_cast<const char*>(scales) +
                       (int64_t)rb0 * G * K * kRowBlock * (int64_t)sizeof(AT);
  // activations: piece u of the step is token tid / 8 + threads / 8 u, position
  // tid % 8 (threads / 8 is a multiple of 16: the piece is the same for every u);
  // tokens past T read the last one (never stored)
  const int xrow = tid >> 3;
  const int xpiece = (tid & 7) ^ ((xrow >> 1) & 7);
  const uint16_t* tile_x = X + (int64_t)t0 * ldx;
  uint32_t xoff[NU];
#pragma unroll
  for (int u = 0; u < NU; ++u)
    xoff[u] = (uint32_t)((int64_t)min(xrow + kThreads / 8 * u, T - 1 - t0) * ldx * 2) +
              16 * xpiece;
  auto copy_x = [&](int s, int b) {
#pragma unroll
    for (int u = 0; u < NU; ++u)
      copy_to_lds(tile_x + block(s) * kBK, xoff[u], xbuf(b) + (u * kThreads + wave * kWave) * 8);
  };
  struct Signs {
    uint32_t w[K];
    AT a[K];
  };
  Signs R0, R1;
  auto load_w = [&](int s, Signs& R) {
    const int g = block(s) >> 1;
    const char* wb = tile_w + (int64_t)g * (K * kRowBlock * 16) + 8 * (block(s) & 1);
    const char* sb = tile_s + (int64_t)g * (int)(K * kRowBlock * sizeof(AT));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      R.w[k] = *reinterpret_cast<const uint32_t*>(wb + woff + k * kRowBlock * 16);
      R.a[k] = *reinterpret_cast<const AT*>(sb + soff + k * kRowBlock * (int)sizeof(AT));
    }
  };

  // one step's weights in kChunks pieces of a few instructions; the levels of
  // a scale group serve its two steps (TWO: are formed for each of the four)
  constexpr int kChunks = 24;
  float af[K];
  uint32_t pairs[2], V[4], lo = 0, hi = 0, o4[4];
  Levels L;
  auto put = [&](int b, int p) {
    *reinterpret_cast<u32x4*>(wbuf(b) + wput + 8 * ((4 * word + p) ^ wkey)) =
        u32x4{o4[0], o4[1], o4[2], o4[3]};
  };
  auto form = [&](int b, const Signs& R, int c, bool levels, bool lo_levels) {
    if (levels && c == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) af[k] = alpha_to_f32<AT>(R.a[k]);
    }
    if constexpr (K <= 3) {
      if (levels && c < 2)
        pairs[c] = lo_levels ? upper_pair<K, true>(af, c) : upper_pair<K>(af, c);
      if (levels && c == 2) L = pack_levels<K>(pairs[0], pairs[1]);
      if (c >= 3 && c < 6) word_selectors_part<K>(R.w, V, c - 3);
      const int h = (c - 8) >> 1;  // quad of the word
      if (c >= 8) {
        if ((c & 1) == 0) {
          const uint32_t sel = quad_selector<K>(V, h >> 2, h & 3);
          lo = quad_low(L, sel);
          hi = quad_high(L, sel);
        } else {
          quad_pairs(lo, hi, o4 + 2 * (h & 1));
          if (h & 1) put(b, h >> 1);
        }
      }
    } else if (c >= 8 && (c & 3) == 0) {
      const int p = (c - 8) >> 2;
      uint32_t o32[16];
      if (lo_levels) unpack_word_k4<true>(R.w, af, o32);
      else unpack_word_k4<false>(R.w, af, o32);
#pragma unroll
      for (int e = 0; e < 4; ++e) o4[e] = o32[4 * p + e];
      put(b, p);
    }
  };

  f32x16 acc[TI][2];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  const int wt = wave / P::WN, wn = wave % P::WN;
  // operand of a 32-row block: row lane % 32, columns 16 q + 8 (lane / 32) ..
  const int lbase = (lane & 31) * kBK;
  auto opos = [&](int q) { return lbase + 8 * ((2 * q + (lane >> 5)) ^ ((lane >> 1) & 7)); };
  bf16x8 pa[2][TI], pb[2][2];
  auto read_x = [&](int b, int q, int i) {
    pa[q & 1][i] = *reinterpret_cast<const bf16x8*>(xbuf(b) + opos(q) + (wt * TI + i) * 32 * kBK);
  };
  auto read_w = [&](int b, int q, int j) {
    pb[q & 1][j] = *reinterpret_cast<const bf16x8*>(wbuf(b) + opos(q) + (wn * 2 + j) * 32 * kBK);
  };
  constexpr int NX = TI * 2;
  // products of sub-step q one at a time; the operands of sub-step nq (buffer
  // b) are read and work(x) runs after product x
  auto products = [&](int q, int b, int nq, auto&& work) {
#pragma unroll
    for (int x = 0; x < NX; ++x) {
      const int i = x % TI, j = x / TI;
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(pa[q & 1][i], pb[q & 1][j], acc[i][j], 0,
                                                          0, 0);
      if (x < 2) read_w(b, nq, x);
      if (x < TI) read_x(b, nq, x);
      work(x);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  auto at = [&](int s) { return min(s, S - 1); };  // the extra steps at the end are unused
  copy_x(0, 0);
  load_w(0, R0);
  load_w(1, R1);
#pragma unroll
  for (int c = 0; c < kChunks; ++c) form(0, R0, c, true, false);
  copies_done();
  pin<K>(R1);
  __syncthreads();
  copy_x(1, 1);
  load_w(at(2), R0);
#pragma unroll
  for (int j = 0; j < 2; ++j) read_w(0, 0, j);
#pragma unroll
  for (int i = 0; i < TI; ++i) read_x(0, 0, i);
  // Step s: its products from buffer b = s % 2 while the weights of step s + 1
  // are formed from R in the other; even steps of the contraction begin a
  // scale group (TWO: odd ones are the residues').
  auto step = [&](int s, int b, Signs& R) {
#pragma unroll
    for (int q = 0; q < 3; ++q)
      products(q, b, q + 1, [&](int x) {
        const int y = q * NX + x;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          if (c * 3 * NX / kChunks == y) form(b ^ 1, R, c, TWO || b == 1, TWO && b == 0);
      });
    copies_done();
    __syncthreads();
    copy_x(at(s + 2), b);
    load_w(at(s + 3), R);
    __builtin_amdgcn_sched_barrier(0);
    products(3, b ^ 1, 0, [](int) {});
  };
  for (int s = 0; s < S; s += 2) {
    step(s, 0, R1);
    step(s + 1, 1, R0);
  }
  copies_done();

  // ---- outputs.  C layout: lane l, register r -> token 8 (r / 4) + 4 (l / 32) +
  // r % 4, row l % 32.  First H, then (training) the pre-activations.
  __syncthreads();
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

template <typename AT, int K, typename P, bool TWO>
__global__ void __launch_bounds__(P::threads) gated_mfma_kernel(
    const uint32_t* __restrict__ bits, const AT* __restrict__ scales,
    const uint16_t* __restrict__ X, int64_t ldx, GatedOut out, int T, int m_pad, int G, int ntx,
    int nty) {
  extern __shared__ __attribute__((aligned(16))) uint16_t smem[];
  const int b = blockIdx.x, blocks = ntx * nty;
  // XCD b % 8 takes consecutive positions of the tile order (as far as 8 divides)
  const int even = blocks & ~7;
  const int p = b < even ? (b & 7) * (even >> 3) + (b >> 3) : b;
  const int tile = tile_at(p, ntx, nty);
  gated_tile<AT, K, P, TWO>(bits, scales, X, ldx, out, T, m_pad, G, (tile / ntx) * P::BT,
                            (tile % ntx) * P::BN, smem);
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
