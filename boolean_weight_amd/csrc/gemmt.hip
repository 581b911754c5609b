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
// Bound: the matrix cores (2 T m n operations; 4096 x 11008, K = 3, 2048
// tokens: 172 us, 1072 TFLOP/s, matrix cores 63% busy), for few tokens the
// steps of a slice, one LDS round trip each (5120 x 5120, 16 tokens: 12.7 us
// against 1.8 us of reading).  256 columns because a weight is then formed once
// per 256 tokens; the tokens of a tile by tile_tokens, the slices by
// gemmt_split.  dY rows that are not 16-byte aligned go by way of registers, of
// which 9 to 30 of a 256-token tile then go through scratch memory (4001 rows x
// 4096 columns, 2048 tokens: 96 us, 4000 rows 81 us, without the joining).
//
// Rows past m have zero weights, and dY is read inside its m columns only: a
// partial last row block is a step of its own with element-wise loads.
#include <stdint.h>

#include <type_traits>

#include "mbok_device.h"
#include "mbok_launch.h"
#include "mbok_levels.h"
#include "mbok_sums.h"

namespace mbok {
namespace {

typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t u32x4_any;  // dY rows start anywhere
typedef __attribute__((ext_vector_type(4))) short i16x4;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;

constexpr int kBN = 256;       // columns per workgroup tile
constexpr int kThreads = 512;  // 8 wavefronts
constexpr int kAStride = kRowBlock;  // bf16 elements per LDS row of dY
// LDS image of W_hat's 64 x 256 tile: pairs of rows, each 1 KB of 64-byte
// granules (32 columns) alternating between its two rows and 128 bytes of
// padding, so that a granule of four consecutive rows covers the 64 banks once
// and every operand's address is the lane's plus a constant.  The 16-byte
// pieces of a granule are in the order piece ^ (row / 4 & 3): the 16 lanes (rows)
// of a 16-byte write then meet 16 different bank groups.
constexpr int kWPair = 576;  // bf16 elements per pair of rows

// Token rows of a tile and how the 8 wavefronts share it: WT wavefronts along
// the tokens, 8 / WT along the columns, each TI x TJ blocks of 32 x 32.
template <int TI_, int TJ_, int WT_>
struct Tile {
  static constexpr int TI = TI_, TJ = TJ_, WT = WT_, WN = 8 / WT_;
  static constexpr int BT = 32 * TI * WT;
  static_assert(32 * TJ * WN == kBN, "256 columns");
  static constexpr int kA = BT * kAStride, kW = kRowBlock / 2 * kWPair;  // elements
  static constexpr size_t kLds = 2 * (size_t)(kA + kW) * sizeof(uint16_t);
};

// 8 rows (k0 .. k0 + 7) of one column per lane: two transposing reads, of rows
// k0 .. k0 + 3 and k0 + 4 .. k0 + 7 (p4)
__device__ __forceinline__ bf16x8 read_tr(const uint16_t* p, const uint16_t* p4) {
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p);
  const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p4);
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// SLICED: every tile is (full = 0), which leaves the other epilogue out.
// TWO: each row block is two steps, W_hat's levels rounded to bf16 and then the
// bf16 rounding of what that left (16 significant bits together), with the same
// dY tile: twice the matrix work (4096 x 11008, 2048 tokens 310 us).
template <typename AT, int K, typename TL, bool ALIGNED, bool SLICED, bool TWO>
__global__ void __launch_bounds__(kThreads) gemmt_kernel(
    const uint32_t* __restrict__ bits, const AT* __restrict__ scales,
    const uint16_t* __restrict__ dY, int64_t lddy, uint16_t* __restrict__ dX, int64_t lddx,
    float* __restrict__ part, int T, int m, int n, int RB, int full, int rest, int slices) {
  constexpr int TI = TL::TI, TJ = TL::TJ, BT = TL::BT;
  constexpr int NA = (BT * 8 + kThreads - 1) / kThreads;  // 16-byte pieces of dY per thread
  extern __shared__ __attribute__((aligned(16))) uint16_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int G = n / kGroup;
  const int ntx = (n + kBN - 1) / kBN, nty = (T + BT - 1) / BT;
  // workgroup -> tile and slice: the first `full` workgroups a whole tile each,
  // the others slices of the last `rest` tiles, slice by slice (unit u of them
  // has its own partial sums); consecutive positions on one XCD in either part
  int p = blockIdx.x, unit = -1, slice = 0;
  if (!SLICED && p < full) {
    if ((full & 7) == 0) p = (p & 7) * (full >> 3) + (p >> 3);
  } else {
    unit = p - full;
    const int nu = rest * slices;
    if ((nu & 7) == 0) unit = (unit & 7) * (nu >> 3) + (unit >> 3);
    slice = unit / rest;
    p = full + unit - slice * rest;
  }
  const int parts = SLICED || unit >= 0 ? slices : 1;
  const int tile = tile_at(p, ntx, nty);
  const int t0 = (tile / ntx) * BT, j0 = (tile % ntx) * kBN;
  const int rb0 = (int)((uint32_t)RB * slice / parts);  // RB < 2^26, 32 slices at most
  const int rb1 = (int)((uint32_t)RB * (slice + 1) / parts);
  // steps over whole row blocks; a partial last block is the tail
  const int full_end = min(rb1, m / kRowBlock);
  const int S = (full_end - rb0) * (TWO ? 2 : 1);  // may be 0 or less
  const bool tail = rb1 > full_end;

  // unpack role: row `lane` of the step's block, 32-column word `wave` of the tile
  const int gw = min(j0 / kGroup + (wave >> 2), G - 1);
  const int uword = wave & 3;
  // dY copy role: piece u = token tid / 8 + 64 u, at LDS position tid % 8 of
  // its row, which holds the 8 rows apart = position ^ (token / 2 & 7) ..
  const int arow8 = tid >> 3;
  const int apart = (tid & 7) ^ ((arow8 >> 1) & 7);
  const bool a_live = BT * 8 >= kThreads || wave < BT * 8 / kWave;  // whole wavefronts
  // byte offsets inside the tile's tokens (ALIGNED: 32 bits hold them)
  const uint16_t* tile_dy = dY + (int64_t)t0 * lddy;
  typename std::conditional<ALIGNED, uint32_t, int64_t>::type arow[NA];
#pragma unroll
  for (int u = 0; u < NA; ++u) {
    const int t = min(arow8 + 64 * u, T - 1 - t0);  // extra tokens are never stored
    arow[u] = (int64_t)t * lddy * 2 + 16 * apart;
  }
  auto dy_at = [&](int u, int rb) {
    return reinterpret_cast<const uint16_t*>(reinterpret_cast<const char*>(tile_dy) + arow[u]) +
           (int64_t)rb * kRowBlock;
  };
  auto abuf = [&](int b) { return smem + b * (TL::kA + TL::kW); };
  auto wbuf = [&](int b) { return smem + b * (TL::kA + TL::kW) + TL::kA; };

  struct StepRegs {
    u32x4 x[ALIGNED ? 1 : NA];
    uint32_t w[K];
    AT a[K];
  };
  StepRegs R0, R1;
  auto load_w = [&](int rb, StepRegs& R) {
    // the wavefront's chunks: uniform bases, so only 32-bit lane offsets are vectors
    const int64_t c = ((int64_t)rb * G + gw) * K * kRowBlock;
    const uint32_t* wb = bits + c * 4 + uword;
    const AT* sb = scales + c;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      R.w[k] = wb[(uint32_t)(lane + k * kRowBlock) * 4u];
      R.a[k] = sb[(uint32_t)(lane + k * kRowBlock)];
    }
  };
  // dY of a whole row block, to its LDS buffer: straight from memory when its
  // rows are 16-byte aligned (the copy is in flight until the next barrier),
  // else by way of registers
  auto load_a = [&](int rb, int b, StepRegs& R) {
    if (a_live) {
#pragma unroll
      for (int u = 0; u < NA; ++u) {
        if constexpr (ALIGNED) {
          copy_to_lds(tile_dy + (int64_t)rb * kRowBlock, arow[u],
                      abuf(b) + (u * kThreads + wave * 64) * 8);
        } else {
          R.x[u] = *reinterpret_cast<const u32x4_any*>(dy_at(u, rb));
        }
      }
    }
  };
  // the partial last block: dY element by element inside its m columns
  auto store_a_tail = [&](int rb, int b) {
    if (!a_live) return;
    const int i0 = rb * kRowBlock + 8 * apart;
#pragma unroll
    for (int u = 0; u < NA; ++u)
      *reinterpret_cast<u32x4*>(abuf(b) + (u * kThreads + tid) * 8) =
          load_piece(dy_at(u, rb), max(0, min(8, m - i0)), m >= 8);
  };

  f32x16 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  const int wt = wave / TL::WN, wn = wave % TL::WN;
  // A dY row in LDS is 8 pieces of 16 bytes, piece c of token r at position
  // c ^ (r / 2 & 7): the 64 banks are 16 such positions, and the 16 lanes of a
  // 16-byte read meet each once.
  // dY operand: token lane % 32, rows 16 q + 8 (lane / 32) ..; W_hat operand: rows
  // 16 q + 8 (lane / 32) + 4 h + (lane / 4 & 3), see read_tr
  const int arr = (wt * 32 * TI + (lane & 31)) * kAStride;
  auto aoff = [&](int q) { return arr + 8 * ((2 * q + (lane >> 5)) ^ ((lane >> 1) & 7)); };
  const int wl = (lane & 15) >> 2;  // row of the four
  const int wpiece = (2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ (2 * (lane >> 5));
  const int wbase = (4 * (lane >> 5) + (wl >> 1)) * kWPair + 32 * (wl & 1) + 4 * (lane & 1) +
                    wn * TJ * 64;
  const int woff[2] = {wbase + 8 * wpiece, wbase + 2 * kWPair + 8 * (wpiece ^ 1)};
  // where the unpacking thread's columns go: row `lane`, granule `wave`
  const int wput = (lane >> 1) * kWPair + 32 * (lane & 1) + 64 * wave;
  const int wkey = (lane >> 2) & 3;

  // One step's W_hat, from its signs and scales to LDS, in kChunks pieces of a
  // few vector instructions each: levels, selectors, then
  // half a quad at a time.
  constexpr int kChunks = 24;
  float af[K];
  uint32_t pairs[4], flipped[3], V[4], lo = 0, hi = 0, out[4];
  Levels L;
  auto w_piece = [&](int b, int q) {
    *reinterpret_cast<u32x4*>(wbuf(b) + wput + 8 * (q ^ wkey)) =
        u32x4{out[0], out[1], out[2], out[3]};
  };
  // lo: the residues' step
  auto form = [&](int b, const StepRegs& R, int c, bool lo_levels) {
    if (c == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) af[k] = alpha_to_f32<AT>(R.a[k]);
    }
    if constexpr (!ALIGNED) {
      if (c < 4 && c < NA && a_live)
        *reinterpret_cast<u32x4*>(abuf(b) + (c * kThreads + tid) * 8) = R.x[c];
    }
    if constexpr (K <= 3) {
      if (c < 2) pairs[c] = lo_levels ? upper_pair<K, true>(af, c) : upper_pair<K>(af, c);
      if (c == 2) L = pack_levels<K>(pairs[0], pairs[1]);
      if (c >= 3 && c < 6) word_selectors_part<K>(R.w, V, c - 3);
    } else {
      if (c < 4) pairs[c] = lo_levels ? k4_pair<true>(af, c) : k4_pair(af, c);
      if (c == 4) L = k4_levels(pairs);
      if (c == 4) k4_words(R.w, flipped);
      if (c >= 5 && c < 8) word_selectors_part<3>(flipped, V, c - 5);
    }
    if (c >= 8) {
      const int quad = (c - 8) >> 1;  // of the word; piece quad / 2
      if ((c & 1) == 0) {
        const uint32_t sel = quad_selector<K <= 3 ? K : 3>(V, quad >> 2, quad & 3);
        lo = quad_low(L, sel);
        hi = K <= 3 ? quad_high(L, sel) : k4_high(L, sel, R.w[K - 1], quad);
      } else {
        quad_pairs(lo, hi, out + 2 * (quad & 1));
        if (quad & 1) w_piece(b, quad >> 1);
      }
    }
  };
  auto form_all = [&](int b, const StepRegs& R, bool lo_levels) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) form(b, R, c, lo_levels);
  };

  bf16x8 pa[2][TI], pb[2][TJ];
  auto read_a = [&](int b, int q, int i) {
    pa[q & 1][i] = *reinterpret_cast<const bf16x8*>(abuf(b) + aoff(q) + i * 32 * kAStride);
  };
  auto read_w = [&](int b, int q, int j) {
    pb[q & 1][j] = read_tr(wbuf(b) + woff[0] + 8 * q * kWPair + 64 * j,
                           wbuf(b) + woff[1] + 8 * q * kWPair + 64 * j);
  };
  // Products of sub-step q (16 rows), one at a time; after product x the
  // operands of sub-step q + 1 whose turn it is are read from buffer b (next
  // sub-step's or the next step's), and work(x) runs.  Each product takes the
  // matrix core 32 cycles, in which the wavefront issues up to 8 other vector
  // instructions; the fences keep the compiler from gathering those (it put
  // 40 in a row, and the wavefronts of a SIMD, in step after a barrier, then
  // left the matrix core idle: 4096 x 11008, 2048 tokens, 228 -> 210 us).
  constexpr int NX = TI * TJ;
  auto products = [&](int q, int b, int nq, auto&& work) {
#pragma unroll
    for (int x = 0; x < NX; ++x) {
      const int i = x % TI, j = x / TI;
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(pa[q & 1][i], pb[q & 1][j], acc[i][j], 0,
                                                          0, 0);
      if (nq >= 0) {
        if (x < TJ) read_w(b, nq, x);
        if (x < TI) read_a(b, nq, x);
        if (x == NX - 1) {
#pragma unroll
          for (int y = NX; y < TI; ++y) read_a(b, nq, y);
        }
      }
      work(x);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto first_operands = [&](int b) {
#pragma unroll
    for (int j = 0; j < TJ; ++j) read_w(b, 0, j);
#pragma unroll
    for (int i = 0; i < TI; ++i) read_a(b, 0, i);
  };

  if (S > 0) {
    const int last = full_end - 1;
    // the row block of a step; the extra steps at the end are unused
    auto at = [&](int s) { return min(rb0 + (TWO ? s >> 1 : s), last); };
    load_a(at(0), 0, R0);
    load_w(at(0), R0);
    if constexpr (!ALIGNED) load_a(at(1), 1, R1);
    load_w(at(1), R1);
    form_all(0, R0, false);
    copies_done();
    pin<K>(R1);
    __syncthreads();
    load_a(ALIGNED ? at(1) : at(2), 1, R0);
    load_w(at(2), R0);
    first_operands(0);
    // Step s: its products from buffer b = s % 2, while W_hat of step s + 1 is
    // formed from R in the other buffer.  The barrier stands before the last
    // quarter of the products, whose operands are in registers by then: the
    // next step's first operands, and the copies and loads of the steps
    // after it, are in flight during that quarter.
    auto step = [&](int s, int b, StepRegs& R) {
#pragma unroll
      for (int q = 0; q < 3; ++q)
        products(q, b, q + 1, [&](int x) {
          const int y = q * NX + x;
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (c * 3 * NX / kChunks == y) form(b ^ 1, R, c, TWO && b == 0);
        });
      copies_done();
      __syncthreads();
      load_a(ALIGNED ? at(s + 2) : at(s + 3), b, R);
      load_w(at(s + 3), R);
      __builtin_amdgcn_sched_barrier(0);
      products(3, b ^ 1, 0, [](int) {});
    };
    for (int s = 0; s < S; s += 2) {
      step(s, 0, R1);
      if (s + 1 >= S) break;
      step(s + 1, 1, R0);
    }
    copies_done();
  }
  if (tail) {
    __syncthreads();
    load_w(full_end, R0);
    store_a_tail(full_end, 0);
    if constexpr (!ALIGNED) {
      // form() stores the registers' dY too: here it is what is in place already
#pragma unroll
      for (int u = 0; u < NA; ++u)
        if (a_live) R0.x[u] = *reinterpret_cast<const u32x4*>(abuf(0) + (u * kThreads + tid) * 8);
    }
#pragma unroll
    for (int pass = 0; pass < (TWO ? 2 : 1); ++pass) {
      if (pass) __syncthreads();
      form_all(0, R0, pass == 1);
      __syncthreads();
      first_operands(0);
#pragma unroll
      for (int q = 0; q < 4; ++q) products(q, 0, q < 3 ? q + 1 : -1, [](int) {});
    }
  }

  // C layout: lane l, register r -> token 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32
  const int tb = wt * TI * 32 + 4 * (lane >> 5), cb = wn * TJ * 32 + (lane & 31);
  if (SLICED || unit >= 0) {
    float* dst = part + (int64_t)unit * (min(T, BT) * kBN);
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int t = tb + 32 * i + 8 * (r >> 2) + (r & 3);
          if (t0 + t < T) dst[t * kBN + cb + 32 * j] = acc[i][j][r];
        }
    return;
  }
  // rounded and, through LDS (free by now), to whole 16-byte stores
  constexpr int OS = kBN + 8;
  static_assert((size_t)BT * OS * 2 <= TL::kLds, "the output tile fits the buffers");
  __syncthreads();
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        smem[(tb + 32 * i + 8 * (r >> 2) + (r & 3)) * OS + cb + 32 * j] =
            __builtin_bit_cast(uint16_t, (__bf16)acc[i][j][r]);
  __syncthreads();
  for (int e = tid; e < BT * (kBN / 8); e += kThreads) {
    const int t = e / (kBN / 8), c = 8 * (e % (kBN / 8));
    if (t0 + t < T && j0 + c < n)
      *reinterpret_cast<u32x4*>(dX + (int64_t)(t0 + t) * lddx + j0 + c) =
          *reinterpret_cast<const u32x4*>(smem + t * OS + c);
  }
}

// The tiles that were sliced: the slices' partial sums added in order and rounded
// once; 4 columns per thread.  Blocks past theirs take a caller's column sums.
__global__ void __launch_bounds__(256) gemmt_reduce_kernel(const float* __restrict__ part,
                                                           uint16_t* __restrict__ dX,
                                                           int64_t lddx, int T, int n, int bt,
                                                           int full, int rest, int slices,
                                                           ColumnSums sums) {
  if ((int)blockIdx.y >= rest) {
    column_sums(sums, ((int)blockIdx.y - rest) * (int)gridDim.x + (int)blockIdx.x);
    return;
  }
  // a block takes 4 rows of one tile; all offsets are below kUnits tiles' worth
  const int idx = blockIdx.y, rows = min(T, bt), stride = rest * rows * kBN;
  const int row = blockIdx.x * 4 + (threadIdx.x >> 6), col = (threadIdx.x & 63) * 4;
  if (row >= rows) return;
  const float* src = part + (idx * rows + row) * kBN + col;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < slices; k += 8) {  // eight loads at a time
    float4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      v[u] = k + u < slices ? *reinterpret_cast<const float4*>(src + (k + u) * stride)
                            : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < 8; ++u) s[0] += v[u].x, s[1] += v[u].y, s[2] += v[u].z, s[3] += v[u].w;
  }
  // where it goes: after the loads, which the divisions would hold up (2.5 -> 2.1 us);
  // what a tile has outside T x n was not written, and is not stored
  const int ntx = (n + kBN - 1) / kBN, nty = (T + bt - 1) / bt;
  const int tile = tile_at(full + idx, ntx, nty);
  const int t = (tile / ntx) * bt + row, j = (tile % ntx) * kBN + col;
  if (t >= T || j >= n) return;
  *reinterpret_cast<uint2*>(dX + (int64_t)t * lddx + j) =
      make_uint2(bf16_pair(s[0], s[1]), bf16_pair(s[2], s[3]));
}

__global__ void __launch_bounds__(256) column_sums_kernel(ColumnSums sums) {
  column_sums(sums, (int)blockIdx.x);
}

constexpr int kUnits = 256;  // workgroups that fill the part (one per compute unit)

// Tokens per tile: as many as there are, up to 256, but fewer where tiles and
// slices of at least four steps would leave most compute units idle: below 96
// workgroups (K = 3, us, never fewer / as it is: 2048 tokens of 256 x 512 17.4 /
// 14.5, 512 of 512 x 512 13.9 / 10.5, 796 of 34 x 512 8.6 / 6.5, 300 of 640 x
// 1024 15.3 / 11.4).  Limits of 64 and 128 are within 1 us of it there; one of
// 192 is faster where 96 to 191 workgroups are left (257 tokens of 2048 x 2048
// 27.2 against 22.2, 200 of 1024 x 4096 24.0 against 18.1).
int tile_tokens(const Geom& geo, int64_t T) {
  const int64_t cols = (geo.n + kBN - 1) / kBN, most = geo.RB < 8 ? 1 : geo.RB / 4;
  int bt = T <= 32 ? 32 : T <= 64 ? 64 : T <= 128 ? 128 : 256;
  while (bt > 32 && cols * ((T + bt - 1) / bt) * most < 96) bt /= 2;
  return bt;
}

// Whole rounds of whole tiles; the row blocks of the tiles that are left in
// as many slices as keep them within one more round, of two steps at least.
// (4096 x 11008, 2048 tokens: 344 tiles, 256 whole and 88 in two slices.)
struct Split {
  int bt, full, rest, slices;
};
Split gemmt_split(const Geom& geo, int64_t T, bool workspace) {
  Split s;
  s.bt = tile_tokens(geo, T);
  const int64_t tiles = ((geo.n + kBN - 1) / kBN) * ((T + s.bt - 1) / s.bt);
  s.full = (int)tiles;
  s.rest = 0;
  s.slices = 1;
  if (!workspace || tiles % kUnits == 0) return s;
  const int64_t rest = tiles % kUnits;
  int64_t k = kUnits / rest;
  if (k > geo.RB / 2) k = geo.RB / 2;
  if (k > 32) k = 32;  // what the joining kernel adds per output
  if (k > 1) {
    s.full = (int)(tiles - rest);
    s.rest = (int)rest;
    s.slices = (int)k;
  }
  return s;
}

template <typename AT, int K>
int launch_k(const Geom& geo, const void* packed, const uint16_t* dY, int64_t T, int64_t lddy,
             uint16_t* dX, int64_t lddx, float* part, const Split& s, bool two,
             const ColumnSums* sums, hipStream_t stream) {
  // straight copies to LDS take 16-byte aligned rows at 32-bit offsets
  const bool aligned =
      ((uintptr_t)dY & 15) == 0 && (lddy % 8) == 0 && lddy < (int64_t(1) << 32) / 512;
  const uint32_t* bits = reinterpret_cast<const uint32_t*>(packed);
  const AT* scales = reinterpret_cast<const AT*>(reinterpret_cast<const char*>(packed) +
                                                 geo.bits_bytes);
  auto go = [&](auto tl) {
    using TL = decltype(tl);
    auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)(s.full + s.rest * s.slices)), dim3(kThreads),
                         TL::kLds, stream, bits, scales, dY, lddy, dX, lddx, part, (int)T, geo.m,
                         geo.n, geo.RB, s.full, s.rest, s.slices);
    };
    if (two) {
      if (aligned) launch(gemmt_kernel<AT, K, TL, true, false, true>);
      else launch(gemmt_kernel<AT, K, TL, false, false, true>);
    } else if (s.full == 0) {
      if (aligned) launch(gemmt_kernel<AT, K, TL, true, true, false>);
      else launch(gemmt_kernel<AT, K, TL, false, true, false>);
    } else {
      if (aligned) launch(gemmt_kernel<AT, K, TL, true, false, false>);
      else launch(gemmt_kernel<AT, K, TL, false, false, false>);
    }
  };
  switch (s.bt) {
    case 32: go(Tile<1, 1, 1>{}); break;
    case 64: go(Tile<2, 1, 1>{}); break;
    case 128: go(Tile<4, 1, 1>{}); break;
    default: go(Tile<4, 2, 2>{}); break;
  }
  if (s.slices > 1) {
    const int rows = T < s.bt ? (int)T : s.bt;
    const int per = (rows + 3) / 4;
    int more = sums ? (sum_blocks(*sums) + per - 1) / per : 0;
    if (s.rest + more > 65535) more = 0;  // a grid has that many rows: a launch of their own
    hipLaunchKernelGGL(gemmt_reduce_kernel, dim3(per, s.rest + more), dim3(256), 0, stream, part,
                       dX, lddx, (int)T, geo.n, s.bt, s.full, s.rest, s.slices,
                       sums ? *sums : ColumnSums{});
    if (more) sums = nullptr;
  }
  if (sums) {
    return launch_column_sums(*sums, stream);
  }
  return hipGetLastError() == hipSuccess ? MBOK_OK : MBOK_ERR_HIP;
}

template <typename AT>
int launch_t(const Geom& geo, const void* packed, const void* dY, int64_t T, int64_t lddy,
             void* dX, int64_t lddx, float* part, const Split& s, bool two,
             const ColumnSums* sums, hipStream_t stream) {
  const uint16_t* g = reinterpret_cast<const uint16_t*>(dY);
  uint16_t* o = reinterpret_cast<uint16_t*>(dX);
  switch (geo.K) {
    case 1: return launch_k<AT, 1>(geo, packed, g, T, lddy, o, lddx, part, s, two, sums, stream);
    case 2: return launch_k<AT, 2>(geo, packed, g, T, lddy, o, lddx, part, s, two, sums, stream);
    case 3: return launch_k<AT, 3>(geo, packed, g, T, lddy, o, lddx, part, s, two, sums, stream);
    default: return launch_k<AT, 4>(geo, packed, g, T, lddy, o, lddx, part, s, two, sums, stream);
  }
}

}  // namespace

size_t gemmt_workspace_bytes(const mbok_desc* d, int64_t T) {
  const Split s = gemmt_split(make_geom(d), T, true);
  return s.slices > 1 ? (size_t)s.rest * s.slices * (T < s.bt ? T : s.bt) * kBN * sizeof(float) : 0;
}

int launch_column_sums(const ColumnSums& sums, hipStream_t stream) {
  hipLaunchKernelGGL(column_sums_kernel, dim3(sum_blocks(sums)), dim3(256), 0, stream, sums);
  return hipGetLastError() == hipSuccess ? MBOK_OK : MBOK_ERR_HIP;
}

int launch_gemmt(const mbok_desc* d, const void* packed, const void* dY, int64_t T, int64_t lddy,
                 void* dX, int64_t lddx, void* ws, int passes, hipStream_t stream,
                 const ColumnSums* sums) {
  const Geom geo = make_geom(d);
  const Split s = gemmt_split(geo, T, ws != nullptr);
  float* part = reinterpret_cast<float*>(ws);
  const bool two = passes == 2;
  if (d->alpha_dtype == MBOK_F16)
    return launch_t<uint16_t>(geo, packed, dY, T, lddy, dX, lddx, part, s, two, sums, stream);
  return launch_t<float>(geo, packed, dY, T, lddy, dX, lddx, part, s, two, sums, stream);
}

}  // namespace mbok
