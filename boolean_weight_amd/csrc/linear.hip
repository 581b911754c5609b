// The layer with its epilogue, Y = R + act(X W_hat^T + b): dispatch by token
// count, and the backward pass (gfx950).
//
// With s the gradient of Y:
//     dz = s act'(z),  db = sum_t dz,  dX = dz W_hat,  dR = s.
// The first two are one pass over s and z (bound by memory: two values read and
// one written per output) that adds each column's values in fp32 before they
// are rounded; dX is the transposed product, whose operand is the rounded dz, or s
// itself without an activation: bf16, as the matrix instructions and the scales'
// gradients take it, half a step of 2^-8 beside the levels' and dX's own (the
// two-term form leaves the levels' out).  (2048 x 11008: 28 us, 4.9 TB/s; with dX of
// 4096 columns, K = 3, 195-200.)
#include "mbok_launch.h"
#include "mbok_levels.h"
#include "mbok_linear.h"
#include "mbok_sums.h"

namespace mbok {
namespace {

__device__ __forceinline__ float piece_value(const u32x4& v, int e) {
  return __uint_as_float((e & 1) ? v[e >> 1] & 0xffff0000u : v[e >> 1] << 16);
}

constexpr int kColumns = 256;                 // of one workgroup: 32 pieces of 8
constexpr int kRowLanes = 8;                  // rows it takes at a time
constexpr int kThreads = kColumns / 8 * kRowLanes;

// Rows slice * step .. of 256 columns.  ACT: dz of an activation, written to
// dpre; else dz = dY.  SUM: the columns' sums to sums[slice][m], or, of a single
// slice, to dbias.
template <bool ACT, bool SUM>
__global__ void __launch_bounds__(kThreads) linear_backward_kernel(
    const uint16_t* pre, int64_t ldpre, const uint16_t* dY, int64_t lddy, uint16_t* dpre,
    int64_t lddpre, int64_t T, int step, int m, int act, float* __restrict__ sums,
    int accumulate) {
  const int piece = threadIdx.x % (kColumns / 8), lane_row = threadIdx.x / (kColumns / 8);
  const int col = (int)blockIdx.x * kColumns + 8 * piece;
  const int live = max(0, min(8, m - col));
  const int64_t r0 = (int64_t)blockIdx.y * step, r1 = min(T, r0 + step);
  float sum[8] = {};
  if (live > 0) {
    constexpr int U = 4;  // rows in flight
    for (int64_t r = r0 + lane_row; r < r1; r += U * kRowLanes) {
      u32x4 s[U], z[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t t = r + u * kRowLanes;
        if (t >= r1) continue;
        s[u] = load_piece(dY + t * lddy + col, live, m >= 8);
        if (ACT) z[u] = load_piece(pre + t * ldpre + col, live, m >= 8);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t t = r + u * kRowLanes;
        if (t >= r1) continue;
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          d[e] = piece_value(s[u], e);
          if (ACT) {
            float slope;
            activation<true>(act, piece_value(z[u], e), slope);
            d[e] *= slope;
          }
          if (SUM) sum[e] += d[e];
        }
        if (ACT) {
          uint16_t* o = dpre + t * lddpre + col;
          if (live == 8) {
            *reinterpret_cast<u32x4_unaligned*>(o) =
                u32x4_unaligned{bf16_pair(d[0], d[1]), bf16_pair(d[2], d[3]),
                                bf16_pair(d[4], d[5]), bf16_pair(d[6], d[7])};
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (e < live) o[e] = to_bf16(d[e]);
          }
        }
      }
    }
  }
  if (!SUM) return;
  __shared__ float part[kRowLanes][kColumns + 4];
#pragma unroll
  for (int e = 0; e < 8; ++e) part[lane_row][8 * piece + e] = sum[e];
  __syncthreads();
  const int c = (int)blockIdx.x * kColumns + (int)threadIdx.x;
  if (c >= m) return;
  float total = 0.f;
#pragma unroll
  for (int i = 0; i < kRowLanes; ++i) total += part[i][threadIdx.x];
  float* out = sums + (int64_t)blockIdx.y * m + c;
  *out = accumulate ? *out + total : total;
}

// Slices of the rows: enough for about 1500 workgroups, of at least 16 rows, two
// for each thread (a slope takes some 40 instructions: 109 rows of 94 columns in one
// slice 19 us).  More than one slice needs a workspace for its sums, and their
// adding: up to 32 rows stay one.
struct RowSplit {
  int slices, step;
};
RowSplit row_split(int m, int64_t T, bool whole) {
  const int cols = (m + kColumns - 1) / kColumns;
  const int64_t want = (1500 + cols - 1) / cols, most = T <= 32 ? 1 : T / 16;
  const int64_t n = whole ? 1 : (want < most ? want : most);
  const int64_t step = (T + n - 1) / n;
  return RowSplit{(int)((T + step - 1) / step), (int)step};
}

// More than 16 tokens on the few-token products: the tiles' kernels walk their
// contraction step by step whatever the token count, and a small layer has few tiles;
// the few-token kernel spreads the contraction over wavefronts, of which each has at
// least a group to take, so that below 8 groups it is no faster than with 8.  (us,
// few-token products / tiles, K = 3: 4096 x 11008 33 and 64 tokens 29 / 43, 128 46 / 43,
// 200 83 / 45; 11008 x 4096 33 33 / 19; 2000 x 640 200 9.7 / 6.9; K = 2: 4096 x 4096 128 15 /
// 18, 200 28 / 19; 1000 x 2048 512 10.5 / 11.3, 700 18 / 12; 64 x 11008 1000 18 / 42; K = 4:
// 724 x 1408 320 8.5 / 10.3, 450 14 / 10.)  560: tiles without shares.
bool in_chunks(const mbok_desc* d, int64_t T, int passes, int shares) {
  const int64_t tiles = (int64_t)(shares ? shares : 560) * passes;
  return linear_chunks_cost(d, T) * (d->n < 1024 ? 1024 : d->n) < tiles * d->n;
}

}  // namespace

// The few-token rule of the gated block (gemm.hip): T = 1 and 2 and, on layers of
// at least 2^26 sign bits 3 to 6, of 2^27 7 and 8 tokens on the fp4 x fp8 forms.
int launch_linear(const mbok_desc* d, const void* packed, const void* X, int64_t T, int64_t ldx,
                  const LinearOut& out, int passes, hipStream_t stream) {
  if (T > skinny_max_tokens()) {
    // what both kernels' 32-bit offsets take, alike
    if ((int64_t)d->K * ((d->m + kRowBlock - 1) / kRowBlock * kRowBlock) * (d->n / 32) >
        (int64_t)UINT32_MAX)
      return MBOK_ERR_SHAPE;
    if (ldx >= (int64_t(1) << 32) / 512) return MBOK_ERR_INVALID_ARG;
    const int shares = linear_shares_cost(d, T);
    if (in_chunks(d, T, passes, shares))
      return launch_linear_chunks(d, packed, X, T, ldx, out, stream);
    if (shares) return launch_linear_shares(d, packed, X, T, ldx, out, passes, stream);
    return launch_linear_mfma(d, packed, X, T, ldx, out, passes, stream);
  }
  if (T == 1) return launch_linear_f4(d, packed, X, T, ldx, out, stream);
  if ((T - 1) * ldx + d->n <= INT32_MAX) {
    const int64_t work = (int64_t)d->K * d->m * d->n;
    if (T == 2 || (T <= 6 && work >= (int64_t(1) << 26)) ||
        (T <= 8 && work >= (int64_t(1) << 27)))
      return launch_linear_f4(d, packed, X, T, ldx, out, stream);
  }
  return launch_linear_skinny(d, packed, X, T, ldx, out, stream);
}

// the product's partial sums, then the slices' sums of dbias, which its last kernel
// adds
size_t product_bytes(const mbok_desc* d, int64_t T) {
  return (gemmt_workspace_bytes(d, T) + 255) / 256 * 256;
}

size_t linear_backward_workspace_bytes(const mbok_desc* d, int64_t T) {
  const RowSplit s = row_split(d->m, T, false);
  if (s.slices == 1) return gemmt_workspace_bytes(d, T);
  return product_bytes(d, T) + (size_t)s.slices * d->m * sizeof(float);
}

int launch_linear_backward(const mbok_desc* d, const void* packed, const LinearGrad& g, int64_t T,
                           int act, int accumulate, void* ws, int passes, hipStream_t stream) {
  const bool with_act = act != MBOK_ACT_NONE;
  // without a sum the rows split freely
  const RowSplit s = row_split(d->m, T, g.dbias && !ws);
  const bool sliced = s.slices > 1;
  // what is left of dbias after the first kernel: the slices' sums, or, of up to 127
  // rows without an activation (and without a workspace), the rows of dY themselves
  ColumnSums tail = {g.dY, g.lddy, 1, (int)T, d->m, accumulate, g.dbias};
  const bool direct = !with_act && (T < 128 || !ws);
  bool has_tail = g.dbias && direct;
  if (with_act || (g.dbias && !direct)) {
    float* sums = sliced && g.dbias
                      ? reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + product_bytes(d, T))
                      : g.dbias;
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((d->m + kColumns - 1) / kColumns, s.slices), dim3(kThreads),
                         0, stream, reinterpret_cast<const uint16_t*>(g.pre), g.ldpre,
                         reinterpret_cast<const uint16_t*>(g.dY), g.lddy,
                         reinterpret_cast<uint16_t*>(g.dpre), g.lddpre, T, s.step, d->m, act, sums,
                         sliced ? 0 : accumulate);
    };
    if (!with_act) go(linear_backward_kernel<false, true>);
    else if (g.dbias) go(linear_backward_kernel<true, true>);
    else go(linear_backward_kernel<true, false>);
    if (hipGetLastError() != hipSuccess) return MBOK_ERR_HIP;
    if (g.dbias && sliced) {
      tail = {sums, d->m, 0, s.slices, d->m, accumulate, g.dbias};
      has_tail = true;
    }
  }
  if (!g.dX) return has_tail ? launch_column_sums(tail, stream) : MBOK_OK;
  return launch_gemmt(d, packed, with_act ? g.dpre : g.dY, T, with_act ? g.lddpre : g.lddy, g.dX,
                      g.lddx, ws, passes, stream, has_tail ? &tail : nullptr);
}

}  // namespace mbok
