// Gradient of the group scales on the matrix cores (gfx950).
//
// "Highly Efficient and Effective LLMs with Multi-Boolean Architectures",
// Paper-Notes reading note, 关键设计: W_hat = sum_k alpha_k (.) B_k with one
// scale per (row, 128-column group, kernel), so
//     dalpha_k[i, g] = sum_{j in g} b_k[i, j] dW[i, j],
//     dW[i, j] = sum_t dY[t, i] X[t, j].
//
// A workgroup forms a 256 x 256 tile of dW (8 wavefronts of 64 rows x 128
// columns: one row block and one scale group each) and contracts it with the
// signs in registers; dW never leaves them.  The contraction runs over the
// tokens in steps of 64; both operands are token-major, so a step's dY and X
// tiles are copied to LDS as they are, without passing registers where they are
// aligned and whole (double-buffered), and both matrix
// operands (8 consecutive tokens of one row or column per lane) are read with
// the transposing LDS load: of 16 lanes, lane s supplies the address of 4
// columns 4 (s & 3) .. of token s >> 2, and receives column s of the 4 tokens.
//
// Bound: the matrix cores (2 T m n operations; 4096 x 11008, K = 3, 2048
// tokens: 168 us, 1099 TFLOP/s, matrix cores 63% busy; dY rows that are not
// 16-byte aligned pass registers: 4001 x 4096 117 us against 70).  A tile of
// 256 x 256 reads each operand once per 256 columns or rows of the other.
//
// Contraction with the signs: lane l holds column l % 32 of each of the
// group's four 32-column words for 32 rows, so per (row, word, kernel) one
// shift brings the column's bit to the sign position and flips the sum's sign;
// the 32 lanes of a row are then added with lane exchanges that halve the
// number of rows per lane each time.
#include <stdint.h>

#include <type_traits>

#include "mbok_device.h"
#include "mbok_lanes.h"
#include "mbok_launch.h"
#include "mbok_levels.h"

namespace mbok {
namespace {

typedef __attribute__((ext_vector_type(4))) short i16x4;

constexpr int kTile = 256;     // rows and columns of a tile
constexpr int kSteps = 64;     // tokens per step
constexpr int kThreads = 512;
// LDS image of a step's 64 tokens x 256 columns: pairs of tokens, each 1 KB of
// 64-byte granules (32 columns) alternating between its two tokens and 128
// bytes of padding, so that a granule of four consecutive tokens covers the 64
// banks once and every operand's address is the lane's plus a constant.
constexpr int kPair = 576;                    // bf16 elements per pair of tokens
constexpr int kBuf = kSteps / 2 * kPair;
constexpr size_t kLdsBytes = 4 * (size_t)kBuf * sizeof(uint16_t);
static_assert(kLdsBytes >= 8 * MBOK_MAX_K * kRowBlock * 16, "the sign chunks fit the buffers");

// 8 tokens of one column per lane: two transposing reads, of 4 tokens each
__device__ __forceinline__ bf16x8 read_tr(const uint16_t* p) {
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p);
  const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 2 * kPair));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Sum of v[0..15] over the 32 lanes of each half wavefront: the lane returns
// the sum of v[r], r = its lane bits 4, 3, 2, 1 from high to low.
__device__ __forceinline__ float sum_rows(f32x16 v, int lane) {
  // bit 4 by swapping 16-lane rows: even rows keep v[0..7], odd rows v[8..15]
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    uint32_t a = __float_as_uint(v[r]), b = __float_as_uint(v[r + 8]);
    swap16(a, b);
    v[r] = __uint_as_float(a) + __uint_as_float(b);
  }
#pragma unroll
  for (int h = 4; h >= 1; h >>= 1) {
    const bool up = (lane & (2 * h)) != 0;
#pragma unroll
    for (int r = 0; r < h; ++r) {
      const float a = v[r], b = v[r + h];
      const float give = up ? a : b, keep = up ? b : a;
      v[r] = keep + __shfl_xor(give, 2 * h);
    }
  }
  return v[0] + __shfl_xor(v[0], 1);
}

template <int K>
__global__ void __launch_bounds__(kThreads) scale_grad_kernel(
    const uint4* __restrict__ bits, const uint16_t* __restrict__ dY, int64_t lddy,
    const uint16_t* __restrict__ X, int64_t ldx, float* __restrict__ out, int T, int m, int n,
    int RB, int slices, int accumulate, int aligned) {
  extern __shared__ __attribute__((aligned(16))) uint16_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wi = wave >> 1, wj = wave & 1;
  const int G = n / kGroup;
  const int ntx = (n + kTile - 1) / kTile, nty = (m + kTile - 1) / kTile;
  const int ntiles = ntx * nty;
  int p = blockIdx.x;
  const int nb = ntiles * slices;
  if ((nb & 7) == 0) p = (p & 7) * (nb >> 3) + (p >> 3);
  const int slice = p / ntiles;
  const int tile = tile_at(p - slice * ntiles, ntx, nty);
  const int i0 = (tile / ntx) * kTile, j0 = (tile % ntx) * kTile;
  const int steps = (T + kSteps - 1) / kSteps;
  const int s0 = (int)((int64_t)steps * slice / slices);
  const int s1 = (int)((int64_t)steps * (slice + 1) / slices);
  const int full_end = min(s1, T / kSteps);  // steps of 64 live tokens
  const bool tail = s1 > full_end;

  // copy role: piece u = token ct + 16 u of the step, 8 columns cc ..
  const int ct = 2 * wave + ((lane >> 2) & 1);
  const int cc = 8 * (4 * (lane >> 3) + (lane & 3));
  // columns past n read the last ones (their sums are never stored)
  const int xc = min(j0 + cc, n - 8);
  const int ia = i0 + cc;                   // first row index of the dY piece
  const int live = max(0, min(8, m - ia));  // of which inside m
  const int yc = min(ia, m - 1);
  auto ybuf = [&](int b) { return smem + 2 * b * kBuf; };
  auto xbuf = [&](int b) { return smem + (2 * b + 1) * kBuf; };
  auto slot = [&](int u) { return (8 * u + wave) * kPair; };  // the wavefront's pair

  struct Regs {
    u32x4 y[4];
  };
  Regs R0, R1;
  auto load_dy = [&](const uint16_t* q) { return load_piece(q, live, m >= 8); };
  auto load_y = [&](int s, Regs& R, auto edge) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint16_t* q = dY + ((int64_t)s * kSteps + ct + 16 * u) * lddy + yc;
      if constexpr (decltype(edge)::value) R.y[u] = load_dy(q);
      else R.y[u] = u32x4(*reinterpret_cast<const u32x4_unaligned*>(q));
    }
  };
  auto store_y = [&](int b, const Regs& R, int u) {
    *reinterpret_cast<u32x4*>(ybuf(b) + slot(u) + lane * 8) = R.y[u];
  };
  // a step of 64 live tokens straight to LDS, at 32-bit offsets from the step
  auto copy_x = [&](int s, int b) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      copy_to_lds(X + ((int64_t)s * kSteps + 16 * u) * ldx, (uint32_t)(ct * ldx + xc) * 2u,
                  xbuf(b) + slot(u));
  };
  auto copy_y = [&](int s, int b) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      copy_to_lds(dY + ((int64_t)s * kSteps + 16 * u) * lddy, (uint32_t)(ct * lddy + yc) * 2u,
                  ybuf(b) + slot(u));
  };
  // the last, partial step: tokens past T are zero in both operands
  auto store_tail = [&](int s, int b) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t t = (int64_t)s * kSteps + ct + 16 * u;
      u32x4 y = u32x4{0u, 0u, 0u, 0u}, x = y;
      if (t < T) {
        y = load_dy(dY + t * lddy + yc);
        x = *reinterpret_cast<const u32x4*>(X + t * ldx + xc);
      }
      *reinterpret_cast<u32x4*>(ybuf(b) + slot(u) + lane * 8) = y;
      *reinterpret_cast<u32x4*>(xbuf(b) + slot(u) + lane * 8) = x;
    }
  };

  f32x16 acc[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  // operand of a 32-column block: tokens 16 q + 8 (lane / 32) + 4 h .., columns
  // as read_tr's lanes take them
  const int tl = (lane & 15) >> 2;  // token of the four
  const int toff = (4 * (lane >> 5) + (tl >> 1)) * kPair + 32 * (tl & 1) +
                   16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  bf16x8 pa[2][2], pb[2][4];
  auto read_y = [&](int b, int q, int i) {
    pa[q & 1][i] = read_tr(ybuf(b) + toff + wi * 128 + 8 * q * kPair + 64 * i);
  };
  auto read_x = [&](int b, int q, int j) {
    pb[q & 1][j] = read_tr(xbuf(b) + toff + wj * 256 + 8 * q * kPair + 64 * j);
  };
  // products of sub-step q (16 tokens) one at a time, the operands of the next
  // (nq, from buffer b) read between them; work(x) runs after product x
  auto products = [&](int q, int b, int nq, auto&& work) {
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int i = x & 1, j = x >> 1;
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(pa[q & 1][i], pb[q & 1][j], acc[i][j], 0,
                                                          0, 0);
      if (nq >= 0) {
        if (x < 2) read_y(b, nq, x);
        if (x < 4) read_x(b, nq, x);
      }
      work(x);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto first_operands = [&](int b) {
#pragma unroll
    for (int i = 0; i < 2; ++i) read_y(b, 0, i);
#pragma unroll
    for (int j = 0; j < 4; ++j) read_x(b, 0, j);
  };

  // Step s multiplies buffer s % 2.  The barrier stands before the last
  // quarter of its products, whose operands are in registers by then: the next
  // step's first operands and the copies of the step after it are in flight
  // during that quarter.  DIRECT: dY goes straight to LDS too; otherwise
  // (unaligned rows, a tile across the last row) by way of registers, loaded
  // two steps before they are stored.
  auto walk = [&](auto direct_c, auto edge) {
    constexpr bool DIRECT = decltype(direct_c)::value;
    const int S = full_end - s0;
    if (S <= 0) return;
    const int last = full_end - 1;
    auto at = [&](int s) { return min(s0 + s, last); };  // the extra steps at the end are unused
    copy_x(at(0), 0);
    if constexpr (DIRECT) {
      copy_y(at(0), 0);
    } else {
      load_y(at(0), R0, edge);
      load_y(at(1), R1, edge);
#pragma unroll
      for (int u = 0; u < 4; ++u) store_y(0, R0, u);
    }
    copies_done();
    __syncthreads();
    copy_x(at(1), 1);
    if constexpr (DIRECT) copy_y(at(1), 1);
    else load_y(at(2), R0, edge);
    first_operands(0);
    auto step = [&](int s, int b, Regs& R) {
#pragma unroll
      for (int q = 0; q < 3; ++q)
        products(q, b, q + 1, [&](int x) {
          if constexpr (!DIRECT) {
            if (q == 1 && x >= 4) store_y(b ^ 1, R, x - 4);
          }
        });
      copies_done();
      __syncthreads();
      copy_x(at(s + 2), b);
      if constexpr (DIRECT) copy_y(at(s + 2), b);
      else load_y(at(s + 3), R, edge);
      __builtin_amdgcn_sched_barrier(0);
      products(3, b ^ 1, 0, [](int) {});
    };
    for (int s = 0; s < S; s += 2) {
      step(s, 0, R1);
      if (s + 1 >= S) break;
      step(s + 1, 1, R0);
    }
    copies_done();
  };
  if (i0 + kTile > m)
    walk(std::false_type{}, std::true_type{});
  else if (aligned)
    walk(std::true_type{}, std::false_type{});
  else
    walk(std::false_type{}, std::false_type{});
  if (tail) {
    __syncthreads();
    store_tail(full_end, 0);
    __syncthreads();
    first_operands(0);
#pragma unroll
    for (int q = 0; q < 4; ++q) products(q, 0, q < 3 ? q + 1 : -1, [](int) {});
  }

  // the wavefront's row block and group: sign chunks to LDS (the buffers are
  // free once every wavefront has read its last operands)
  __syncthreads();
  const int rb = i0 / kRowBlock + wi, g = j0 / kGroup + wj;
  if (rb >= RB || g >= G) return;
  uint4* chunk = reinterpret_cast<uint4*>(smem) + wave * (K * kRowBlock);
  const int64_t c0 = ((int64_t)rb * G + g) * K * kRowBlock;
#pragma unroll
  for (int k = 0; k < K; ++k) chunk[k * kRowBlock + lane] = bits[c0 + k * kRowBlock + lane];
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the wavefront's own LDS writes

  const int c = lane & 31;
  const int sh = 31 - (8 * (c & 3) + (c >> 2));  // brings the column's bit to bit 31
  float* dst = out + (slices > 1 ? (int64_t)slice * K * m * G : 0);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      f32x16 v;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        const uint4 w = chunk[k * kRowBlock + row];
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
        // a set bit (+1) sets the sign bit: the sum is negated at the end
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s += __uint_as_float(__float_as_uint(acc[i][j][r]) ^ ((ww[j] << sh) & 0x80000000u));
        v[r] = s;
      }
      const float sum = -sum_rows(v, lane);
      const int r = (lane >> 1) & 15;  // lane bits 4 .. 1
      const int row = rb * kRowBlock + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
      if ((lane & 1) == 0 && row < m) {
        float* q = dst + ((int64_t)k * m + row) * G + g;
        *q = accumulate && slices == 1 ? *q + sum : sum;
      }
    }
  }
}

// out (+)= the slices' partial sums in order
__global__ void __launch_bounds__(256) scale_grad_reduce_kernel(const float* __restrict__ part,
                                                                float* __restrict__ out,
                                                                int64_t count, int slices,
                                                                int accumulate) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= count) return;
  float s = 0.f;
  for (int k = 0; k < slices; k += 8) {  // eight loads at a time, added in order
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = k + u < slices ? part[(int64_t)(k + u) * count + e] : 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) s += v[u];
  }
  out[e] = accumulate ? out[e] + s : s;
}

constexpr int kUnits = 256;  // workgroups that fill the part (one per compute unit)

int grad_slices(const Geom& geo, int64_t T) {
  const int64_t tiles = (int64_t)((geo.n + kTile - 1) / kTile) * ((geo.m + kTile - 1) / kTile);
  int64_t s = kUnits / tiles;
  const int64_t steps = (T + kSteps - 1) / kSteps;
  if (s > steps / 2) s = steps / 2;  // two steps each at least
  if (s > 32) s = 32;                // what the joining kernel adds per scale
  return s < 1 ? 1 : (int)s;
}

}  // namespace

size_t scale_grad_workspace_bytes(const mbok_desc* d, int64_t T) {
  const Geom geo = make_geom(d);
  const int s = grad_slices(geo, T);
  return s > 1 ? (size_t)s * geo.K * (size_t)geo.m * geo.G * sizeof(float) : 0;
}

int launch_scale_grad(const mbok_desc* d, const void* packed, const void* dY, int64_t T,
                      int64_t lddy, const void* X, int64_t ldx, float* dalpha, bool accumulate,
                      void* ws, hipStream_t stream) {
  const Geom geo = make_geom(d);
  const int slices = ws ? grad_slices(geo, T) : 1;
  // straight copies of dY to LDS take 16-byte aligned rows
  const int aligned = ((uintptr_t)dY & 15) == 0 && (lddy % 8) == 0;
  // and 32-bit offsets over 16 rows: leading dimensions past that are refused
  if (lddy >= (int64_t(1) << 26) || ldx >= (int64_t(1) << 26)) return MBOK_ERR_INVALID_ARG;
  const int64_t blocks = (int64_t)((geo.n + kTile - 1) / kTile) *
                         ((geo.m + kTile - 1) / kTile) * slices;
  float* out = slices > 1 ? reinterpret_cast<float*>(ws) : dalpha;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kThreads), kLdsBytes, stream,
                       reinterpret_cast<const uint4*>(packed),
                       reinterpret_cast<const uint16_t*>(dY), lddy,
                       reinterpret_cast<const uint16_t*>(X), ldx, out, (int)T, geo.m, geo.n,
                       geo.RB, slices, accumulate ? 1 : 0, aligned);
  };
  switch (geo.K) {
    case 1: go(scale_grad_kernel<1>); break;
    case 2: go(scale_grad_kernel<2>); break;
    case 3: go(scale_grad_kernel<3>); break;
    default: go(scale_grad_kernel<4>); break;
  }
  if (slices > 1) {
    const int64_t count = (int64_t)geo.K * geo.m * geo.G;
    hipLaunchKernelGGL(scale_grad_reduce_kernel, dim3((unsigned)((count + 255) / 256)), dim3(256),
                       0, stream, out, dalpha, count, slices, accumulate ? 1 : 0);
  }
  return hipGetLastError() == hipSuccess ? MBOK_OK : MBOK_ERR_HIP;
}

}  // namespace mbok
