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
// tiles are copied to LDS as they are (double-buffered) and both matrix
// operands (8 consecutive tokens of one row or column per lane) are read with
// the transposing LDS load: of 16 lanes, lane s supplies the address of 4
// columns 4 (s & 3) .. of token s >> 2, and receives column s of the 4 tokens.
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

typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t u32x4_any;  // dY rows start anywhere
typedef __attribute__((ext_vector_type(4))) short i16x4;

constexpr int kTile = 256;     // rows and columns of a tile
constexpr int kSteps = 64;     // tokens per step
constexpr int kThreads = 512;
constexpr int kStride = 272;   // bf16 elements per LDS row (256 + 16)
constexpr int kBuf = kSteps * kStride;
constexpr size_t kLdsBytes = 4 * (size_t)kBuf * sizeof(uint16_t);
static_assert(kLdsBytes >= 8 * MBOK_MAX_K * kRowBlock * 16, "the sign chunks fit the buffers");

// 8 tokens of one column per lane: two transposing reads
__device__ __forceinline__ bf16x8 read_tr(const uint16_t* p) {
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p);
  const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 4 * kStride));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Sum of v[0..15] over the 32 lanes of each half wavefront: the lane returns
// the sum of v[r], r = its lane bits 4, 3, 2, 1 from high to low.
__device__ __forceinline__ float sum_rows(float (&v)[16], int lane) {
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
      const float give = up ? v[r] : v[r + h];
      const float keep = up ? v[r + h] : v[r];
      v[r] = keep + __shfl_xor(give, 2 * h);
    }
  }
  return v[0] + __shfl_xor(v[0], 1);
}

template <int K>
__global__ void __launch_bounds__(kThreads) scale_grad_kernel(
    const uint4* __restrict__ bits, const uint16_t* __restrict__ dY, int64_t lddy,
    const uint16_t* __restrict__ X, int64_t ldx, float* __restrict__ out, int T, int m, int n,
    int RB, int slices, int accumulate) {
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

  // copy role: piece u = token tid / 32 + 16 u of the step, 8 columns 8 (tid % 32) ..
  const int ct = tid >> 5, cc = 8 * (tid & 31);
  // columns past n read the last ones (their sums are never stored)
  const uint16_t* xp = X + (int64_t)ct * ldx + min(j0 + cc, n - 8);
  const int ia = i0 + cc;               // first row index of the dY piece
  const int live = max(0, min(8, m - ia));  // of which inside m
  const uint16_t* yp = dY + (int64_t)ct * lddy + min(ia, m - 1);

  struct Regs {
    u32x4 y[4], x[4];
  };
  Regs R0, R1;
  auto load_dy = [&](const uint16_t* q, bool edge) {
    if (!edge || live == 8) return u32x4(*reinterpret_cast<const u32x4_any*>(q));
    uint32_t e[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) e[c] = c < live ? q[c] : 0u;
    return u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
  };
  auto load = [&](int s, Regs& R, bool edge) {
    const int64_t t = (int64_t)s * kSteps;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      R.y[u] = load_dy(yp + (t + 16 * u) * lddy, edge);
      R.x[u] = *reinterpret_cast<const u32x4*>(xp + (t + 16 * u) * ldx);
    }
  };
  // the last, partial step: tokens past T are zero in both operands
  auto load_tail = [&](int s, Regs& R) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t t = (int64_t)s * kSteps + 16 * u;
      R.y[u] = R.x[u] = u32x4{0u, 0u, 0u, 0u};
      if (t + ct < T) {
        R.y[u] = load_dy(yp + t * lddy, true);
        R.x[u] = *reinterpret_cast<const u32x4*>(xp + t * ldx);
      }
    }
  };
  auto ybuf = [&](int b) { return smem + 2 * b * kBuf; };
  auto xbuf = [&](int b) { return smem + (2 * b + 1) * kBuf; };
  auto store = [&](int b, const Regs& R, int u) {
    *reinterpret_cast<u32x4*>(ybuf(b) + (ct + 16 * u) * kStride + cc) = R.y[u];
    *reinterpret_cast<u32x4*>(xbuf(b) + (ct + 16 * u) * kStride + cc) = R.x[u];
  };

  f32x16 acc[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  const int off = (8 * (lane >> 5) + ((lane & 15) >> 2)) * kStride + 16 * ((lane >> 4) & 1) +
                  4 * (lane & 3);
  auto mma = [&](int b, auto&& between) {
    const uint16_t* ys = ybuf(b) + off + wi * 64;
    const uint16_t* xs = xbuf(b) + off + wj * 128;
    bf16x8 pa[2][2], pb[2][4];
    auto frags = [&](int q) {
#pragma unroll
      for (int i = 0; i < 2; ++i) pa[q & 1][i] = read_tr(ys + 16 * q * kStride + 32 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) pb[q & 1][j] = read_tr(xs + 16 * q * kStride + 32 * j);
    };
    frags(0);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q < 3) frags(q + 1);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(pa[q & 1][i], pb[q & 1][j],
                                                              acc[i][j], 0, 0, 0);
      between(q);
    }
  };

  auto walk = [&](auto edge_c) {
    constexpr bool edge = decltype(edge_c)::value;
    const int S = full_end - s0;
    if (S <= 0) return;
    const int last = full_end - 1;
    load(s0, R0, edge);
    load(min(s0 + 1, last), R1, edge);
#pragma unroll
    for (int u = 0; u < 4; ++u) store(0, R0, u);
    __syncthreads();
    for (int s = 0; s < S; s += 2) {
      load(min(s0 + s + 2, last), R0, edge);
      mma(0, [&](int q) { store(1, R1, q); });
      __syncthreads();
      if (s + 1 >= S) break;
      load(min(s0 + s + 3, last), R1, edge);
      mma(1, [&](int q) { store(0, R0, q); });
      __syncthreads();
    }
  };
  if (i0 + kTile <= m)
    walk(std::false_type{});
  else
    walk(std::true_type{});
  if (tail) {
    load_tail(full_end, R0);
#pragma unroll
    for (int u = 0; u < 4; ++u) store(0, R0, u);
    __syncthreads();
    mma(0, [](int) {});
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
      float v[16];
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
  float s = part[e];
  for (int k = 1; k < slices; ++k) s += part[k * count + e];
  out[e] = accumulate ? out[e] + s : s;
}

constexpr int kUnits = 256;  // workgroups that fill the part (one per compute unit)

int grad_slices(const Geom& geo, int64_t T) {
  const int64_t tiles = (int64_t)((geo.n + kTile - 1) / kTile) * ((geo.m + kTile - 1) / kTile);
  int64_t s = kUnits / tiles;
  const int64_t steps = (T + kSteps - 1) / kSteps;
  if (s > steps / 4) s = steps / 4;  // four steps each at least
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
  const int64_t blocks = (int64_t)((geo.n + kTile - 1) / kTile) *
                         ((geo.m + kTile - 1) / kTile) * slices;
  float* out = slices > 1 ? reinterpret_cast<float*>(ws) : dalpha;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kThreads), kLdsBytes, stream,
                       reinterpret_cast<const uint4*>(packed),
                       reinterpret_cast<const uint16_t*>(dY), lddy,
                       reinterpret_cast<const uint16_t*>(X), ldx, out, (int)T, geo.m, geo.n,
                       geo.RB, slices, accumulate ? 1 : 0);
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
