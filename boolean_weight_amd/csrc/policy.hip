// Log-probabilities of the tokens of a batch, their gradient, the clipped
// policy loss with a KL term and the loss of paired log ratios (gfx950).
//
// With q = softmax(z / tau) over a row and its token a:
//     logp = z_a / tau - log sum exp(z / tau),  d logp / d z_v = ([v = a] - q_v) / tau.
// Policy loss (Schulman et al., "Proximal Policy Optimization Algorithms";
// the KL term in the form exp(x) - x - 1 with x = ref - logp, which is never
// negative and has the KL divergence as its mean): ratio r = exp(logp - old),
//     loss = w (-min(r A, clip(r, 1 - lo, 1 + hi) A) + beta (exp(x) - x - 1)).
// Preference loss (Rafailov et al., "Direct Preference Optimization"): h = beta
// (S_chosen - S_rejected) - margin with S the sum (or mean) of logp - ref over
// a sequence's tokens,
//     loss = w ((1 - s) log(1 + exp(-h)) + s log(1 + exp(h))).
//
// Bound: the row of logits, read once and (gradient) written once.  As in the
// distillation loss one workgroup takes a row and keeps it in registers, so
// maximum, sum and gradient cost one read.  (2048 rows of 32000 bf16 logits with the
// gradient: 56-60 us, 4.4-4.7 TB/s of the 262 MB; logp alone 28-32 us, its gradient 37
// behind it, 49 where nothing of the row is cached; 301 rows of 12345 fp32 ones 10-11 us;
// 512 rows of 128000 bf16 ones, 16 vectors per thread, 63, of 152000, read again, 94.)
// The ratio stands next to a border (1 + hi), so what is formed from the row's
// sum is float64.
#include <math.h>

#include <type_traits>

#include "mbok_launch.h"
#include "mbok_rows.h"

namespace mbok {
namespace {

constexpr int kMaxThreads = 1024;
constexpr float kLn2 = 0.693147180559945309417f;

struct RowStats {
  float zmax;     // largest logit
  float inv_sum;  // 1 / sum exp((z - zmax) / tau)
  float rest;     // 1 - q_a
  float pad;
};
static_assert(sizeof(RowStats) == MBOK_LOGP_STATS * sizeof(float), "stats row");

struct RowShape {
  int V;
  float tau, c;  // c = log2(e) / tau
  bool stream;   // gradient rows start 16-byte aligned (see store_row)
};

// Reduction buffers of one row's workgroup.
struct RowLds {
  float top[kMaxThreads / kWave];
  double sum[kMaxThreads / kWave];
  float slope, inv_sum, rest;
};

// exp((z - zmax) / tau) of a vector.  The scaled argument is one fma, z c - k with
// k = zmax c rounded, where k is small (the factor 2^(zmax c - k) that all
// exponentials of the row then lack is 1 to 2^-17, and is put back where their
// sum is used alone), else subtracted first.
struct Exps {
  float zmax, c, k;
  bool near;
  __device__ __forceinline__ Exps(float zmax_, float c_)
      : zmax(zmax_), c(c_), k(zmax_ * c_), near(fabsf(k) < 256.f) {}
  // log of the row's sum of true exponentials from the sum of these
  __device__ __forceinline__ double log_sum(double S) const {
    const double fix = near ? (double)kLn2 * ((double)k - (double)zmax * (double)c) : 0.0;
    return log(S) + fix;
  }
  template <typename T, int N>
  __device__ __forceinline__ void operator()(const RowVec<T>& x, float (&e)[N]) const {
    if (near) {
#pragma unroll
      for (int i = 0; i < N; ++i) e[i] = __builtin_amdgcn_exp2f(fmaf(x.at(i), c, -k));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) e[i] = __builtin_amdgcn_exp2f((x.at(i) - zmax) * c);
    }
  }
};

// the larger of three, NaN dropped (fmaxf quiets its operands first)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// What the first wavefront forms of a row: log-probability, loss and its slope.
struct Policy {
  const float *adv, *old, *ref, *weight;
  double low, high;
  float kl;
  float *loss, *dlogp;

  // the loss of row t and d loss / d logp, without the weight
  __device__ __forceinline__ double of(int64_t t, double logp, double& slope) const {
    const double A = (double)adv[t];
    // without old the present logp is its own: 1, or NaN where there is none
    const double r = old ? exp(logp - (double)old[t]) : logp != logp ? logp : 1.0;
    // an advantage of 0 gains nothing at any ratio, an infinite one included
    double gain = 0.0;
    slope = 0.0;
    if (A != 0.0 || r != r) {
      const bool clipped = A > 0.0 ? r > high : r < low;
      gain = (clipped ? (A > 0.0 ? high : low) : r) * A;
      if (!clipped) slope = -r * A;
    }
    double loss = -gain;
    if (ref && kl != 0.f) {  // 0 times an infinite divergence is no KL term
      // x of +inf: a token at -inf that the reference finds possible (y - x is no number)
      const double x = (double)ref[t] - logp, y = expm1(x);
      loss += (double)kl * (y == INFINITY ? y : y - x);
      slope -= (double)kl * y;
    }
    return loss;
  }
};
struct NoLoss {};

// Wavefronts per SIMD.  A held row of 8 vectors and the loss in float64 take 72 registers,
// 7 of them; 8 spill 2 values of fp32 logits, 3 of bf16 and 82 of fp16 ones.  (Policy
// step, us, 7 / 8: 2048 x 32000 fp16 55 / 102, bf16 57 / 60, 600 x 9000 bf16 9.1 / 9.8, 2048 x
// 16000 fp32 55 / 54.  Of 1024 threads 7 leave one row on a compute unit instead of two:
// 2048 x 60000 bf16 130 / 107, fp16 127 / 179.)
template <typename ZT>
constexpr int row_waves(int nv, int threads, bool grad) {
  if (nv > 8) return 4;
  const bool f16 = std::is_same<ZT, _Float16>::value;
  return grad && nv == 8 && (f16 || (sizeof(ZT) == 2 && threads < 1024)) ? 7 : 8;
}

// LOSS: Policy or NoLoss (log-probabilities alone).  GRAD: with dZ.
template <typename ZT, typename OT, int NV, int THREADS, bool GRAD, typename Loss>
__global__ void __launch_bounds__(THREADS, row_waves<ZT>(NV, THREADS, GRAD)) row_kernel(
    const ZT* Z, int64_t ldz, const int32_t* __restrict__ label, RowShape s,
    float* __restrict__ logp_out, RowStats* __restrict__ stats, OT* dZ, int64_t lddz, Loss loss) {
  constexpr int N = RowVec<ZT>::N;
  constexpr bool POLICY = std::is_same<Loss, Policy>::value;
  __shared__ RowLds lds;
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int lane = tid & (kWave - 1), wave = tid / kWave, nw = nt / kWave;
  const ZT* row = Z + t * ldz;
  OT* drow = GRAD ? dZ + t * lddz : nullptr;
  const int nvec = (s.V + N - 1) / N;
  const int a = label[t];
  const bool there = a >= 0 && a < s.V;
  float w = 1.f;
  if constexpr (POLICY) w = loss.weight ? loss.weight[t] : 1.f;
  auto zeros = [&] {
    const float zero[N] = {};
    for (int v = tid; v < nvec; v += nt) store_row<OT, N>(drow, v, s.V, zero, s.stream);
  };

  // a row without a token, or one that nothing is asked of
  if (!there || (POLICY && w == 0.f && !logp_out && !stats)) {
    if (GRAD) zeros();
    if (tid == 0) {
      if (logp_out) logp_out[t] = 0.f;
      if (stats) stats[t] = RowStats{};
      if constexpr (POLICY) {
        loss.loss[t] = 0.f;
        if (loss.dlogp) loss.dlogp[t] = 0.f;
      }
    }
    return;
  }

  RowVec<ZT> held[NV > 0 ? NV : 1];
  if (NV > 0) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int v = tid + u * nt;
      if (v < nvec) held[u] = load_row(row, v, s.V);
    }
  }
  const float za = (float)row[a];

  // largest logit (a NaN is dropped here: it makes the sum below NaN)
  float top = -INFINITY;
  auto max_of = [&](const RowVec<ZT>& x) {
#pragma unroll
    for (int e = 0; e < N; e += 2) top = max3(top, x.at(e), x.at(e + 1));
  };
  if (NV > 0) {
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (tid + u * nt < nvec) max_of(held[u]);
  } else {
    for (int v = tid; v < nvec; v += nt) max_of(load_row(row, v, s.V));
  }
  top = lanes_max(top);
  if (lane == 0) lds.top[wave] = top;
  __syncthreads();
  top = lds.top[0];
  for (int i = 1; i < nw; ++i) top = fmaxf(top, lds.top[i]);

  // sum of exponentials; a thread adds at most 128 terms in fp32
  const Exps exps(top, s.c);
  double sum = 0.0;
  if (NV > 0) {
    float part = 0.f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (tid + u * nt >= nvec) continue;
      held[u].forget();
      float e[N];
      exps(held[u], e);
#pragma unroll
      for (int i = 0; i < N; ++i) part += e[i];
    }
    sum = (double)part;
  } else {
    for (int v = tid; v < nvec; v += nt) {
      float e[N], part = 0.f;
      exps(load_row(row, v, s.V), e);
#pragma unroll
      for (int i = 0; i < N; ++i) part += e[i];
      sum += (double)part;
    }
  }
  sum = lanes_sum(sum);
  if (lane == 0) lds.sum[wave] = sum;
  __syncthreads();

  if (wave == 0) {
    double S = 0.0;
    for (int i = 0; i < nw; ++i) S += lds.sum[i];
    const double logp = ((double)za - (double)top) / (double)s.tau - exps.log_sum(S);
    const float rest = (float)-expm1(logp);
    if (lane == 0) {
      if (logp_out) logp_out[t] = (float)logp;
      if (stats) stats[t] = RowStats{top, (float)(1.0 / S), rest, 0.f};
    }
    if constexpr (POLICY) {
      double slope = 0.0;
      const double l = loss.of(t, logp, slope);
      if (lane == 0) {
        loss.loss[t] = w == 0.f ? 0.f : (float)((double)w * l);
        if (loss.dlogp) loss.dlogp[t] = w == 0.f ? 0.f : (float)((double)w * slope);
        lds.slope = w == 0.f ? 0.f : (float)((double)w * slope / (double)s.tau);
        lds.inv_sum = (float)(1.0 / S);
        lds.rest = rest;
      }
    }
  }
  if (!GRAD) return;
  __syncthreads();

  const float A = lds.slope;
  if (A == 0.f) {  // clipped, or weight 0: a row that holds a NaN as well
    zeros();
    return;
  }
  const float f = -A * lds.inv_sum;
  auto put = [&](int v, float (&e)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] *= f;
    if (v == a / N) {  // the token's own, from 1 - q_a
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i == a % N) e[i] = A * lds.rest;
    }
    store_row<OT, N>(drow, v, s.V, e, s.stream);
  };
  if (NV > 0) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int v = tid + u * nt;
      if (v >= nvec) continue;
      held[u].forget();
      float e[N];
      exps(held[u], e);
      put(v, e);
    }
  } else {
    for (int v = tid; v < nvec; v += nt) {
      float e[N];
      exps(load_row(row, v, s.V), e);
      put(v, e);
    }
  }
}

// dZ of sum_t dlogp_t logp_t, from the statistics of an earlier pass
template <typename ZT, typename OT>
__global__ void __launch_bounds__(kMaxThreads) logp_backward_kernel(
    const ZT* Z, int64_t ldz, const int32_t* __restrict__ label, RowShape s,
    const RowStats* __restrict__ stats, const float* __restrict__ dlogp, OT* dZ, int64_t lddz) {
  constexpr int N = RowVec<ZT>::N;
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, nt = blockDim.x;
  const ZT* row = Z + t * ldz;
  OT* drow = dZ + t * lddz;
  const int nvec = (s.V + N - 1) / N;
  const int a = label[t];
  const float g = dlogp[t];
  if (a < 0 || a >= s.V || g == 0.f) {
    const float zero[N] = {};
    for (int v = tid; v < nvec; v += nt) store_row<OT, N>(drow, v, s.V, zero, s.stream);
    return;
  }
  const RowStats st = stats[t];
  const Exps exps(st.zmax, s.c);
  const float A = g / s.tau, f = -A * st.inv_sum;
  for (int v = tid; v < nvec; v += nt) {
    float e[N];
    exps(load_row(row, v, s.V), e);
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] *= f;
    if (v == a / N) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i == a % N) e[i] = A * st.rest;
    }
    store_row<OT, N>(drow, v, s.V, e, s.stream);
  }
}

// A pair's rows begin at the largest offset up to its own, so that pairs share no rows
// (and no two workgroups write one's slope) whatever the offsets hold.  Up to kNearPairs
// every wavefront looks through the offsets before its pair itself; beyond, one
// workgroup first leaves each pair's largest where its loss goes, kScanPairs to a thread.
// (Slopes of 256 rows a pair, us, each pair from its own offset / so: 8 pairs 3.7 / 3.9,
// 1024 6.0 / 6.3; with the second kernel 4096 13.8 / 17.0, 65536 159 / 178.)
constexpr int kNearPairs = 1024;
constexpr int kScanThreads = 1024, kScanPairs = 8;
typedef int i32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
__global__ void __launch_bounds__(kScanThreads) pair_starts_kernel(
    const int32_t* __restrict__ offsets, int64_t pairs, float* __restrict__ starts) {
  __shared__ int tops[kScanThreads / kWave];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  int carry = 0;  // largest offset before this pass's pairs
  for (int64_t base = 0; base < pairs; base += kScanThreads * kScanPairs) {
    const int64_t p0 = base + tid * kScanPairs;
    int own[kScanPairs], upto[kScanPairs];  // a pair's first offset; the thread's up to its second
    int top = 0;
    if (p0 + kScanPairs <= pairs) {
#pragma unroll
      for (int i = 0; i < kScanPairs; i += 2) {
        const i32x4_any v = *reinterpret_cast<const i32x4_any*>(offsets + 2 * (p0 + i));
        own[i] = v[0], upto[i] = v[1], own[i + 1] = v[2], upto[i + 1] = v[3];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kScanPairs; ++i) {
        const bool there = p0 + i < pairs;
        own[i] = there ? offsets[2 * (p0 + i)] : 0;
        upto[i] = there ? offsets[2 * (p0 + i) + 1] : 0;
      }
    }
#pragma unroll
    for (int i = 0; i < kScanPairs; ++i) upto[i] = top = max(top, max(own[i], upto[i]));
#pragma unroll
    for (int s = 1; s < kWave; s <<= 1) {
      const int up = __shfl_up(top, s);
      if (lane >= s) top = max(top, up);
    }
    const int left = __shfl_up(top, 1);
    if (lane == kWave - 1) tops[wave] = top;
    __syncthreads();
    int before = lane ? max(carry, left) : carry;
    for (int i = 0; i < kScanThreads / kWave; ++i) {
      if (i < wave) before = max(before, tops[i]);
      carry = max(carry, tops[i]);
    }
#pragma unroll
    for (int i = kScanPairs - 1; i >= 0; --i)
      own[i] = max(own[i], i ? max(before, upto[i - 1]) : before);
    if (p0 + kScanPairs <= pairs) {
#pragma unroll
      for (int i = 0; i < kScanPairs; i += 4)
        *reinterpret_cast<f32x4_any*>(starts + p0 + i) =
            f32x4_any{__int_as_float(own[i]), __int_as_float(own[i + 1]),
                      __int_as_float(own[i + 2]), __int_as_float(own[i + 3])};
    } else {
#pragma unroll
      for (int i = 0; i < kScanPairs; ++i)
        if (p0 + i < pairs) starts[p0 + i] = __int_as_float(own[i]);
    }
    __syncthreads();  // tops has been read
  }
}

// One pair of sequences per workgroup: sequence 2 p chosen, 2 p + 1 rejected.
constexpr int kPairThreads = 256;
__global__ void __launch_bounds__(kPairThreads) preference_kernel(
    const int32_t* __restrict__ offsets, const float* __restrict__ logp,
    const float* __restrict__ ref, const int32_t* __restrict__ label, int64_t T,
    const float* __restrict__ weight, mbok_preference_desc d, bool near,
    float* __restrict__ loss, float* __restrict__ dlogp) {
  __shared__ double red[4][kPairThreads / kWave];
  const int64_t p = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  int start = max(0, offsets[2 * p]);
  if (near) {
    int top = start;
    const int end = 2 * (int)p;  // loads past the pair's own offset read that
    for (int i = lane; i - lane < end; i += 8 * kWave) {
#pragma unroll
      for (int u = 0; u < 8; ++u) top = max(top, offsets[min(i + u * kWave, end)]);
    }
    if (__ballot(top > start)) start = lanes_max(top);
  } else {
    start = __float_as_int(loss[p]);
  }
  // bounds inside [0, T] and in order, whatever the offsets hold
  int64_t at[3];
  at[0] = min((int64_t)start, T);
  for (int i = 1; i < 3; ++i) at[i] = max(at[i - 1], min((int64_t)offsets[2 * p + i], T));
  auto counted = [&](int64_t r) { return !label || (label[r] >= 0 && label[r] < d.vocab); };
  double sum[2], count[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    double s = 0.0;
    int n = 0;
    for (int64_t r = at[q] + tid; r < at[q + 1]; r += kPairThreads)
      if (counted(r)) {
        s += (double)logp[r] - (ref ? (double)ref[r] : 0.0);
        ++n;
      }
    s = lanes_sum(s);
    const double c = lanes_sum((double)n);
    if (lane == 0) {
      red[2 * q][wave] = s;
      red[2 * q + 1][wave] = c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    sum[q] = count[q] = 0.0;
    for (int i = 0; i < kPairThreads / kWave; ++i) {
      sum[q] += red[2 * q][i];
      count[q] += red[2 * q + 1][i];
    }
    count[q] = d.mean ? fmax(count[q], 1.0) : 1.0;
  }
  const double beta = (double)d.beta, s = (double)d.smoothing;
  const double h = beta * (sum[0] / count[0] - sum[1] / count[1]) - (double)d.margin;
  const double w = weight ? (double)weight[p] : 1.0;
  const double soft = log1p(exp(-fabs(h)));
  // 0 times an infinite h is 0 here: smoothing 0 leaves the other term out
  const double up = (1.0 - s) * (soft + fmax(-h, 0.0)),
               down = s > 0.0 ? s * (soft + fmax(h, 0.0)) : 0.0;
  if (tid == 0) loss[p] = w == 0.0 ? 0.f : (float)(w * (h != h ? h : up + down));
  if (!dlogp) return;
  const double sig = 1.0 / (1.0 + exp(-h));  // exp overflows to 0 here
  const double other = 1.0 / (1.0 + exp(h));
  const double dh = w == 0.0 ? 0.0 : w * beta * (s * sig - (1.0 - s) * other);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float slope = (float)((q ? -dh : dh) / count[q]);
    for (int64_t r = at[q] + tid; r < at[q + 1]; r += kPairThreads)
      dlogp[r] = counted(r) ? slope : 0.f;
  }
}

RowShape shape_of(int V, float tau, const RowArgs& a) {
  const int size = a.dz_dtype == MBOK_F32 ? 4 : 2;
  const bool stream = ((uintptr_t)a.dZ & 15) == 0 && (a.lddz * size) % 16 == 0;
  return RowShape{V, tau, (float)(1.4426950408889634074 / (double)tau), stream};
}

// Threads of a row's workgroup for `want` vectors each, 256 to 1024 (256 for each
// of MBOK_MAX_DISTILL_ROWS rows are 2^31).
int row_threads(int64_t T, int nvec, int want) {
  int threads = 256;
  while (threads < kMaxThreads && threads * want < nvec && T * threads * 2 <= UINT32_MAX)
    threads *= 2;
  return threads;
}

// A row's workgroup: with many rows the fewest threads that hold it in 8 vectors
// each (3 or 4 resident rows per compute unit hide one another's reductions: 1024 x
// 32000 bf16 logits, policy step, 27.3 us with 512 threads, 30.5 with 1024); with
// few the fewest that do in 4 (32000 bf16, 64 rows 8.9 us with 1024 threads, 10.4
// with 512; 16000, 301 rows 9.5 with 512, 9.9 with 1024 of 2 vectors).
template <typename ZT, typename OT, bool GRAD, typename Loss>
int launch_rows(const RowArgs& a, const RowShape& s, float* logp, float* stats, const Loss& loss,
                hipStream_t stream) {
  const int nvec = (s.V + RowVec<ZT>::N - 1) / RowVec<ZT>::N;
  auto go = [&](auto nv, auto threads) {
    hipLaunchKernelGGL(
        (row_kernel<ZT, OT, decltype(nv)::value, decltype(threads)::value, GRAD, Loss>),
        dim3((unsigned)a.T), dim3(decltype(threads)::value), 0, stream,
        reinterpret_cast<const ZT*>(a.Z), a.ldz, a.label, s, logp,
        reinterpret_cast<RowStats*>(stats), reinterpret_cast<OT*>(a.dZ), a.lddz, loss);
  };
  auto row = [&](auto threads, auto nv) {
    constexpr int64_t n = decltype(threads)::value;
    if (nvec > n * decltype(nv)::value || a.T * n > UINT32_MAX) return false;
    go(nv, threads);
    return true;
  };
  using std::integral_constant;
  const integral_constant<int, 256> t256;
  const integral_constant<int, 512> t512;
  const integral_constant<int, 1024> t1024;
  const integral_constant<int, 2> v2;
  const integral_constant<int, 4> v4;
  const integral_constant<int, 8> v8;
  const integral_constant<int, 16> v16;
  const integral_constant<int, 0> again;
  const bool many = a.T >= 512;
  if (row(t256, v2) || row(t256, v4) || (many && row(t256, v8)) || row(t512, v4) ||
      (many && row(t512, v8)) || row(t1024, v4) || row(t1024, v8) || row(t1024, v16)) {
  } else if (a.T * 1024 <= UINT32_MAX) {
    go(again, t1024);
  } else {  // a launch has fewer than 2^32 threads
    go(again, t256);
  }
  return hipGetLastError() == hipSuccess ? MBOK_OK : MBOK_ERR_HIP;
}

// calls f with the logit and gradient types of the call
template <typename F>
int by_types(const RowArgs& a, F&& f) {
  const bool same = !a.dZ || a.dz_dtype == a.z_dtype;
  switch (a.z_dtype) {
    case MBOK_F32: return same ? f(float{}, float{}) : f(float{}, __bf16{});
    case MBOK_F16: return same ? f(_Float16{}, _Float16{}) : f(_Float16{}, __bf16{});
    default: return f(__bf16{}, __bf16{});
  }
}

}  // namespace

int launch_logp(const mbok_logp_desc* d, const RowArgs& a, float* logp, float* stats,
                hipStream_t stream) {
  const RowShape s = shape_of(d->vocab, d->temperature, a);
  auto go = [&](auto z) {
    return launch_rows<decltype(z), decltype(z), false>(a, s, logp, stats, NoLoss{}, stream);
  };
  switch (a.z_dtype) {
    case MBOK_F32: return go(float{});
    case MBOK_F16: return go(_Float16{});
    default: return go(__bf16{});
  }
}

int launch_policy(const mbok_policy_desc* d, const RowArgs& a, const float* advantage,
                  const float* old_logp, const float* ref_logp, const float* weight, float* loss,
                  float* logp, float* stats, float* dlogp, hipStream_t stream) {
  const RowShape s = shape_of(d->vocab, d->temperature, a);
  const Policy p = {advantage, old_logp, ref_logp, weight, 1.0 - (double)d->clip_low,
                    1.0 + (double)d->clip_high, d->kl, loss, dlogp};
  return by_types(a, [&](auto z, auto o) {
    if (a.dZ) return launch_rows<decltype(z), decltype(o), true>(a, s, logp, stats, p, stream);
    return launch_rows<decltype(z), decltype(o), false>(a, s, logp, stats, p, stream);
  });
}

int launch_logp_backward(const mbok_logp_desc* d, const RowArgs& a, const float* stats,
                         const float* dlogp, hipStream_t stream) {
  const RowShape s = shape_of(d->vocab, d->temperature, a);
  return by_types(a, [&](auto z, auto o) {
    using ZT = decltype(z);
    using OT = decltype(o);
    const int nvec = (s.V + RowVec<ZT>::N - 1) / RowVec<ZT>::N;
    const int threads = row_threads(a.T, nvec, 4);
    hipLaunchKernelGGL((logp_backward_kernel<ZT, OT>), dim3((unsigned)a.T), dim3(threads), 0,
                       stream, reinterpret_cast<const ZT*>(a.Z), a.ldz, a.label, s,
                       reinterpret_cast<const RowStats*>(stats), dlogp,
                       reinterpret_cast<OT*>(a.dZ), a.lddz);
    return hipGetLastError() == hipSuccess ? MBOK_OK : MBOK_ERR_HIP;
  });
}

int launch_preference(const mbok_preference_desc* d, const int32_t* offsets, int64_t pairs,
                      const float* logp, const float* ref_logp, const int32_t* label, int64_t T,
                      const float* weight, float* loss, float* dlogp, hipStream_t stream) {
  const bool near = pairs <= kNearPairs;
  if (!near) {
    hipLaunchKernelGGL(pair_starts_kernel, dim3(1), dim3(kScanThreads), 0, stream, offsets, pairs,
                       loss);
    if (hipGetLastError() != hipSuccess) return MBOK_ERR_HIP;
  }
  hipLaunchKernelGGL(preference_kernel, dim3((unsigned)pairs), dim3(kPairThreads), 0, stream,
                     offsets, logp, ref_logp, label, T, weight, *d, near, loss, dlogp);
  return hipGetLastError() == hipSuccess ? MBOK_OK : MBOK_ERR_HIP;
}

}  // namespace mbok
