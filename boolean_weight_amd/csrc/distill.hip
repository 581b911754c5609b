// Distillation loss from a teacher's top logits, and its gradient (gfx950).
//
// "Highly Efficient and Effective LLMs with Multi-Boolean Architectures",
// gist.science summaries, training sections: the kernels are finetuned by
// distillation from the full-precision model.  Per row, with q = softmax(z /
// tau) over the vocabulary and the teacher's listed (index v_j, logit l_j):
//     loss = w tau^2 [ sum_j p_j (log p_j - log q_{v_j}) + p_r log(p_r / q_r) ]
//     dz_v = w tau [ q_v (s - [v not listed] p_r / q_r) - sum_{j: v_j = v} p_j ]
// where p is the softmax of the listed l / tau (then p_r = 0 and s = 1), or
// with t_lse exp(l / tau - t_lse) and p_r = 1 - sum p the mass of what is not
// listed; s = sum p + p_r is 1 as well unless p_r is cut off at 0 (an index
// listed twice, a t_lse that is too small) or its class drops out.  Where what
// is not listed lies far below the largest logit, its sum R is taken relative
// to its own largest logit zu: log q_r keeps its digits at any distance, and
// the factor of exp((z_v - zu) / tau) in dz_v,
//     s exp((zu - zmax) / tau) / S - p_r / R,
// stays below s + p_r where p_r / q_r overflows.
//
// Bound: the row of logits, read once and (gradient) written once.  One
// workgroup takes one row and keeps it in registers as loaded (NV 16-byte
// vectors per thread), so the maximum, the sum of exponentials and the
// gradient cost one read (2048 rows of 32000 bf16 logits with the gradient:
// 74 us, 3.5 TB/s read and written, against 53 us for a copy).  What is left:
// ~12 vector instructions per logit, and 118 registers with 8 vectors, so two
// rows per compute unit to hide one's arithmetic behind the other's traffic.
// 16 vectors of 16-bit logits (vocabularies of 65537 to 131072) do not all fit
// with what else is live: 55 to 60 registers go through scratch memory (512 x
// 128256 with the gradient 127 us, 2.1 TB/s).  Rows of more than 16 vectors for
// each of 1024 threads are read again for each pass (512 x 262144 186 us).
// Rows start at any element: the 16-byte accesses need no alignment on this
// part, and the last, partial vector of a row goes element by element.
//
// Membership of a token in the list is one bit per token in LDS.  The main
// pass writes every dz_v as if v had no p_j; after a barrier the threads of
// the listed entries write theirs again, adding the p of every entry with the
// same index in list order, so equal indices need no atomics and all writers
// of an element write the same bits.
#include <math.h>

#include <type_traits>

#include "mbok_device.h"
#include "mbok_launch.h"

namespace mbok {
namespace {

constexpr int kMaxThreads = 1024;
constexpr float kLn2 = 0.693147180559945309417f;

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<_Float16>(_Float16 v) { return (float)v; }
template <>
__device__ __forceinline__ float to_f32<__bf16>(__bf16 v) { return (float)v; }

// A 16-byte vector of logits as loaded.
template <typename T>
struct Vec {
  static constexpr int N = 16 / (int)sizeof(T);
  T v[N];
};

// Elements v N .. v N + N - 1 of a row of V; past the end -inf.
template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T* row, int v, int V) {
  constexpr int N = Vec<T>::N;
  if ((v + 1) * N <= V)
    return __builtin_bit_cast(Vec<T>, *reinterpret_cast<const u32x4_any*>(row + v * N));
  Vec<T> r;
#pragma unroll
  for (int e = 0; e < N; ++e) r.v[e] = v * N + e < V ? row[v * N + e] : (T)-INFINITY;
  return r;
}

// Vec of the gradient: N values of OT for one vector of logits, 8 to 32 bytes.
template <typename OT, int N>
__device__ __forceinline__ void store_vec(OT* row, int v, int V, const float (&d)[N]) {
  OT o[N];
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = (OT)d[e];
  if ((v + 1) * N <= V) {
    constexpr int W = N * (int)sizeof(OT) / 4;  // dwords: 2 or 4
    typedef uint32_t words __attribute__((ext_vector_type(W)));
    typedef uint32_t words_any __attribute__((ext_vector_type(W), aligned(2)));
    words w;
    __builtin_memcpy(&w, o, sizeof(w));
    *reinterpret_cast<words_any*>(row + v * N) = w;
    return;
  }
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (v * N + e < V) row[v * N + e] = o[e];
}

struct Sum2 {
  double a, b;
};

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int s = 32; s; s >>= 1) v = fmaxf(v, __shfl_xor(v, s));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int s = 32; s; s >>= 1) v += __shfl_xor(v, s);
  return v;
}

__device__ __forceinline__ float teacher_logit(const void* l, int dtype, int64_t i) {
  if (dtype == MBOK_F32) return reinterpret_cast<const float*>(l)[i];
  if (dtype == MBOK_F16) return (float)reinterpret_cast<const _Float16*>(l)[i];
  return (float)reinterpret_cast<const __bf16*>(l)[i];
}

// Statistics of a row, as stats holds them
struct RowStats {
  float zmax;    // largest logit
  float listed;  // s / S: s q_v = exp((z_v - zmax) / tau) listed for listed v
  float tmax;    // largest listed teacher logit (no t_lse)
  float inv_n;   // 1 / sum exp((l - tmax) / tau); 0: no teacher weight, NaN: no number
  // dz_v = w tau exp((z_v - zu) / tau) unlisted for the others
  float zu, unlisted;
  float pad[2];
};
static_assert(sizeof(RowStats) == MBOK_DISTILL_STATS * sizeof(float), "stats row");

struct DistillRow {
  int V, top;
  float tau, c_hi, c_lo;  // log2(e) / tau as an fp32 pair
};

// exp(d / tau), d <= 0, carried to fp32 accuracy: the rounding of the scaled
// argument to first order (for the few listed entries).
__device__ __forceinline__ float exp_listed(float d, const DistillRow& r) {
  const float a = d * r.c_hi;
  const float lo = fmaf(d, r.c_hi, -a) + d * r.c_lo;
  const float e = __builtin_amdgcn_exp2f(a);
  return a < -126.f ? 0.f : fmaf(e * kLn2, lo, e);
}

// exp(x) to about 1 ulp of fp32 for a float64 x: the argument's low part to
// first order.
__device__ __forceinline__ float exp_fine(double x) {
  const double a = x * 1.4426950408889634074;
  const float hi = (float)a;
  const float e = __builtin_amdgcn_exp2f(hi);
  return hi < -126.f ? 0.f : fmaf(e * kLn2, (float)(a - (double)hi), e);
}

// The lists of one row in LDS: index (or -1), then p, then one bit per token.
struct RowLds {
  int* idx;
  float* p;
  uint32_t* bits;
};

__device__ __forceinline__ RowLds row_lds(void* base, int top) {
  RowLds s;
  s.idx = reinterpret_cast<int*>(base);
  s.p = reinterpret_cast<float*>(s.idx + top);
  s.bits = reinterpret_cast<uint32_t*>(s.p + top);
  return s;
}

// Index of entry j, -1 where there is none
__device__ __forceinline__ int entry_index(const int32_t* t_index, int64_t at, int V) {
  const int v = t_index[at];
  return v >= 0 && v < V ? v : -1;
}

// Sets the bits of the listed tokens; true for a thread that met a bit set
// before (an index listed twice).  The bits were cleared before a barrier.
__device__ __forceinline__ bool mark_entry(uint32_t* bits, int v) {
  const uint32_t m = 1u << (v & 31);
  return (atomicOr(&bits[v >> 5], m) & m) != 0;
}

// The gradient of the listed entries, after the main pass of the same
// workgroup and a barrier: base scale A = w tau.
template <typename ZT, typename OT>
__device__ __forceinline__ void write_entries(const RowLds& s, const DistillRow& r,
                                              const float* zl, OT* drow, const RowStats& st,
                                              float A, bool twice) {
  for (int j = threadIdx.x; j < r.top; j += blockDim.x) {
    const int v = s.idx[j];
    if (v < 0) continue;
    float p = 0.f;
    if (twice) {
      for (int i = 0; i < r.top; ++i)
        if (s.idx[i] == v) p += s.p[i];
    } else {
      p = s.p[j];
    }
    const float e = __builtin_amdgcn_exp2f((zl[j] - st.zmax) * r.c_hi);
    drow[v] = (OT)(fmaf(e, st.listed, -p) * A);
  }
}

// The main pass's dz = exp((z - zu) / tau) A of a vector.  For 16-bit gradients
// the factor is folded into the exponent, exp2(z c + k), where zu is small
// enough for k's rounding (2^-24 of |k|) to stay far below theirs; it takes
// two instructions fewer.
template <typename OT>
struct GradScale {
  float A, zu, c, k;
  uint32_t sign;
  bool fold;  // the same for the whole row
  __device__ __forceinline__ GradScale(float A_, float zu_, const DistillRow& r)
      : A(A_), zu(zu_), c(r.c_hi), k(0.f), sign(__float_as_uint(A_) & 0x80000000u) {
    const float shift = zu * c;
    fold = sizeof(OT) == 2 && fabsf(shift) < 256.f;
    // A = 0 goes through the exponent as well (log2 0 = -inf gives 0), NaN stays
    if (fold) k = __builtin_amdgcn_logf(fabsf(A)) - shift;
  }
  template <typename ZT, int N>
  __device__ __forceinline__ void operator()(const Vec<ZT>& x, float (&d)[N]) const {
    if (fold) {
#pragma unroll
      for (int e = 0; e < N; ++e)
        d[e] = __uint_as_float(
            __float_as_uint(__builtin_amdgcn_exp2f(fmaf(to_f32(x.v[e]), c, k))) ^ sign);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) d[e] = __builtin_amdgcn_exp2f((to_f32(x.v[e]) - zu) * c) * A;
    }
  }
};

// REST: with t_lse (one kernel for both: 512 x 128256 bf16 logits without, 136
// against 127 us)
template <typename ZT, typename OT, int NV, bool GRAD, bool REST>
__global__ void __launch_bounds__(kMaxThreads) distill_kernel(
    const ZT* Z, int64_t ldz, const void* __restrict__ t_logits, int t_dtype,
    const int32_t* __restrict__ t_index, int64_t ldt, const float* __restrict__ t_lse,
    const float* __restrict__ weight, DistillRow r, float* __restrict__ loss,
    RowStats* __restrict__ stats, OT* dZ, int64_t lddz) {
  constexpr int N = Vec<ZT>::N;
  extern __shared__ __attribute__((aligned(16))) uint32_t smem[];
  __shared__ float red_f[kMaxThreads / kWave];
  __shared__ double red_d[2 * kMaxThreads / kWave];
  __shared__ RowStats sh;
  __shared__ int twice_any;
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int lane = tid & (kWave - 1), wave = tid / kWave, nw = nt / kWave;
  const ZT* row = Z + t * ldz;
  OT* drow = GRAD ? dZ + t * lddz : nullptr;
  const float w = weight ? weight[t] : 1.f;
  const int nvec = (r.V + N - 1) / N;

  if (w == 0.f) {
    if (GRAD) {
      const float zero[N] = {};
      for (int v = tid; v < nvec; v += nt) store_vec<OT, N>(drow, v, r.V, zero);
    }
    if (tid == 0) {
      loss[t] = 0.f;
      if (stats) stats[t] = RowStats{};
    }
    return;
  }

  // the row
  Vec<ZT> held[NV > 0 ? NV : 1];
  if (NV > 0) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int v = tid + u * nt;
      if (v < nvec) held[u] = load_vec(row, v, r.V);
    }
  }
  auto each = [&](auto&& f) {
    if (NV > 0) {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int v = tid + u * nt;
        if (v < nvec) f(v, held[u]);
      }
    } else {
      for (int v = tid; v < nvec; v += nt) f(v, load_vec(row, v, r.V));
    }
  };

  // the lists: index, raw teacher logit (in p's place), student logit
  const RowLds s = row_lds(smem, r.top);
  const int nbits = (r.V + 31) / 32;
  float* zl = reinterpret_cast<float*>(s.bits + nbits);
  for (int i = tid; i < nbits; i += nt) s.bits[i] = 0u;
  if (tid == 0) twice_any = 0;
  for (int j = tid; j < r.top; j += nt) {
    const int v = entry_index(t_index, t * ldt + j, r.V);
    s.idx[j] = v;
    s.p[j] = v < 0 ? -INFINITY : teacher_logit(t_logits, t_dtype, t * ldt + j);
    zl[j] = v < 0 ? 0.f : to_f32(row[v]);
  }

  auto listed_at = [&](int v) { return s.bits[(v * N) >> 5] >> ((v * N) & 31); };
  // largest logit (a NaN is dropped here: it makes the sum below NaN)
  float mx = -INFINITY;
  each([&](int, const Vec<ZT>& x) {
#pragma unroll
    for (int e = 0; e < N; ++e) mx = fmaxf(mx, to_f32(x.v[e]));
  });
  mx = wave_max(mx);
  if (lane == 0) red_f[wave] = mx;
  __syncthreads();  // also: lists and cleared bits are in LDS
  mx = red_f[0];
  for (int i = 1; i < nw; ++i) mx = fmaxf(mx, red_f[i]);

  bool twice = false;
  for (int j = tid; j < r.top; j += nt)
    if (s.idx[j] >= 0) twice |= mark_entry(s.bits, s.idx[j]);
  if (twice) twice_any = 1;
  __syncthreads();

  // Sums of exponentials: all, and (with t_lse) the unlisted ones.  The scaled
  // argument (z - max) c is one fma, z c - k with k = max c rounded, where k is
  // small (2^klo then corrects the sums for that rounding, |klo| <= 2^-17: to
  // first order), else subtracted first.  That c is log2(e) / tau rounded
  // (2^-24 relative at most) moves log sum by at most 2^-24 E_q[(max - z) / tau]
  // <= 2^-24 log V, since that mean is the entropy of q less log sum.  (Carrying
  // it exactly cost two instructions per logit, the subtraction one: 2048 x
  // 32000 bf16 with gradient 76.5 -> 74.1 us.)
  // A thread adds at most 128 terms in fp32: a row that is read again adds each
  // vector's sums in float64.
  float sum_z = 0.f, sum_r = 0.f;
  double far_z = 0.0, far_r = 0.0;
  auto next_vector = [&] {
    if (NV > 0) return;
    far_z += (double)sum_z;
    far_r += (double)sum_r;
    sum_z = sum_r = 0.f;
  };
  const float k = mx * r.c_hi;
  const bool near = fabsf(k) < 256.f;
  auto sum = [&](auto near_c) {
    auto ex = [&](ZT z) {
      return __builtin_amdgcn_exp2f(decltype(near_c)::value ? fmaf(to_f32(z), r.c_hi, -k)
                                                            : (to_f32(z) - mx) * r.c_hi);
    };
    each([&](int v, const Vec<ZT>& x) {
      const uint32_t m = REST ? listed_at(v) : 0u;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float y = ex(x.v[e]);
        sum_z += y;
        if (REST) sum_r += (m >> e) & 1u ? 0.f : y;
      }
      next_vector();
    });
  };
  if (near) sum(std::true_type{});
  else sum(std::false_type{});
  {
    const double fix =
        near ? 1.0 - (double)kLn2 * ((double)mx * (double)r.c_hi - (double)k) : 1.0;
    const double dz = wave_sum((double)sum_z + far_z) * fix;
    const double dr = REST ? wave_sum((double)sum_r + far_r) * fix : 0.0;
    if (lane == 0) {
      red_d[2 * wave] = dz;
      red_d[2 * wave + 1] = dr;
    }
  }
  __syncthreads();

  // What is not listed has next to nothing relative to the largest logit: its sum
  // again, relative to its own largest (0 if that is -inf).  Below 2^-30, so
  // that what the first sum and the gradient flush, exponentials below 2^-126,
  // is less than 2^-96 of the rest.  (2048 x 32000 bf16 78 us, 114 when every row
  // is read again.  Taking the unlisted maximum of every row in the first pass
  // instead: 512 x 128256 bf16 139 -> 169 us.)
  float zu = mx;
  if (REST) {
    double R = 0.0;
    for (int i = 0; i < nw; ++i) R += red_d[2 * i + 1];
    if (R < 0x1p-30) {
      zu = -INFINITY;
      for (int v = tid; v < nvec; v += nt) {
        const Vec<ZT> x = load_vec(row, v, r.V);
        const uint32_t m = listed_at(v);
#pragma unroll
        for (int e = 0; e < N; ++e) zu = fmaxf(zu, (m >> e) & 1u ? -INFINITY : to_f32(x.v[e]));
      }
      zu = wave_max(zu);
      if (lane == 0) red_f[wave] = zu;
      __syncthreads();  // also: every thread has its R
      zu = red_f[0];
      for (int i = 1; i < nw; ++i) zu = fmaxf(zu, red_f[i]);
      if (!(zu > -INFINITY)) zu = 0.f;
      double far = 0.0;
      for (int v = tid; v < nvec; v += nt) {
        const Vec<ZT> x = load_vec(row, v, r.V);
        const uint32_t m = listed_at(v);
        float part = 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e)
          part += (m >> e) & 1u ? 0.f
                                : __builtin_amdgcn_exp2f((to_f32(x.v[e]) - zu) * r.c_hi);
        far += (double)part;
      }
      far = wave_sum(far);
      if (lane == 0) red_d[2 * wave + 1] = far;
      __syncthreads();
    }
  }

  // the first wavefront: teacher, loss, statistics
  if (wave == 0) {
    // S: the row's sum, relative to zmax; R: the unlisted part's, relative to zu
    double S = 0.0, R = 0.0;
    for (int i = 0; i < nw; ++i) {
      S += red_d[2 * i];
      R += red_d[2 * i + 1];
    }
    const double inv_tau = 1.0 / (double)r.tau;
    const double up =
        zu == mx ? 1.0 : R > 0.0 ? exp(((double)zu - (double)mx) * inv_tau) : 0.0;
    RowStats st = {};
    st.zmax = mx;
    st.zu = zu;
    double log_n, shift, Nsum = 1.0;  // log p_j = (l_j - shift) / tau - log_n
    if (REST) {
      shift = 0.0;
      log_n = (double)t_lse[t];
      st.inv_n = 1.f;
    } else {
      float tm = -INFINITY;
      for (int j = lane; j < r.top; j += kWave) tm = fmaxf(tm, s.p[j]);
      tm = wave_max(tm);
      st.tmax = tm;
      // a NaN was dropped from the maximum: it makes the sum NaN, beside
      // entries of -inf too; so does a maximum of +inf
      Nsum = 0.0;
      for (int j = lane; j < r.top; j += kWave) {
        const float l = s.p[j];
        if (tm > -INFINITY) Nsum += (double)exp_listed(l - tm, r);
        else if (l != l) Nsum = l;
      }
      Nsum = wave_sum(Nsum);
      log_n = log(Nsum);
      shift = (double)tm;
      st.inv_n = Nsum != 0.0 ? (float)(1.0 / Nsum) : 0.f;
    }
    const double log_s = log(S);
    double kl = 0.0, psum = 0.0;
    if (st.inv_n != 0.f) {
      for (int j = lane; j < r.top; j += kWave) {
        const float l = s.p[j];
        double p;
        double log_p = 0.0;
        if (REST) {
          log_p = (double)l * inv_tau - log_n;
          p = (double)exp_fine(log_p);
        } else {
          log_p = ((double)l - shift) * inv_tau - log_n;
          p = (double)exp_listed(l - st.tmax, r) / Nsum;
        }
        if (s.idx[j] < 0) p = 0.0;
        s.p[j] = (float)p;
        psum += p;
        const double log_q = ((double)zl[j] - (double)mx) * inv_tau - log_s;
        if (p > 0.0 || p != p) kl += p * (log_p - log_q);
      }
      kl = wave_sum(kl);
      psum = wave_sum(psum);
    } else {
      for (int j = lane; j < r.top; j += kWave) s.p[j] = 0.f;
    }
    if (S != S) kl = S;
    double mass = REST ? psum : Nsum == Nsum ? 1.0 : Nsum, take = 0.0;
    const double pr = REST ? fmax(0.0, 1.0 - psum) : 0.0;
    if (pr > 0.0 && R > 0.0) {
      kl += pr * (log(pr) - (((double)zu - (double)mx) * inv_tau + log(R) - log_s));
      mass += pr;
      take = pr / R;
    }
    if (st.inv_n == 0.f) mass = 0.0;
    st.listed = (float)(mass / S);
    st.unlisted = (float)(mass * up / S - take);
    if (lane == 0) {
      loss[t] = (float)((double)w * (double)r.tau * (double)r.tau * kl);
      sh = st;
      if (stats) stats[t] = st;
    }
  }
  if (!GRAD) return;
  __syncthreads();

  const RowStats st = sh;
  const float A = w * r.tau;
  const GradScale<OT> scale(A * st.unlisted, zu, r);
  each([&](int v, const Vec<ZT>& x) {
    float d[N];
    scale(x, d);
    store_vec<OT, N>(drow, v, r.V, d);
  });
  __syncthreads();
  if (st.inv_n != 0.f)
    write_entries<ZT, OT>(s, r, zl, drow, st, A, twice_any != 0);
}

template <typename ZT, typename OT>
__global__ void __launch_bounds__(kMaxThreads) distill_backward_kernel(
    const ZT* Z, int64_t ldz, const void* __restrict__ t_logits, int t_dtype,
    const int32_t* __restrict__ t_index, int64_t ldt, const float* __restrict__ t_lse,
    const float* __restrict__ weight, DistillRow r, const RowStats* __restrict__ stats,
    const float* __restrict__ dloss, OT* dZ, int64_t lddz) {
  constexpr int N = Vec<ZT>::N;
  extern __shared__ __attribute__((aligned(16))) uint32_t smem[];
  __shared__ int twice_any;
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, nt = blockDim.x;
  const ZT* row = Z + t * ldz;
  OT* drow = dZ + t * lddz;
  const float w = (weight ? weight[t] : 1.f), dl = dloss[t];
  const int nvec = (r.V + N - 1) / N;
  if (w == 0.f || dl == 0.f) {
    const float zero[N] = {};
    for (int v = tid; v < nvec; v += nt) store_vec<OT, N>(drow, v, r.V, zero);
    return;
  }
  const RowStats st = stats[t];
  const RowLds s = row_lds(smem, r.top);
  const int nbits = (r.V + 31) / 32;
  float* zl = reinterpret_cast<float*>(s.bits + nbits);
  for (int i = tid; i < nbits; i += nt) s.bits[i] = 0u;
  if (tid == 0) twice_any = 0;
  __syncthreads();
  bool twice = false;
  for (int j = tid; j < r.top; j += nt) {
    const int v = entry_index(t_index, t * ldt + j, r.V);
    s.idx[j] = v;
    float p = 0.f;
    if (v >= 0) {
      const float l = teacher_logit(t_logits, t_dtype, t * ldt + j);
      p = t_lse ? exp_fine((double)l * (1.0 / (double)r.tau) - (double)t_lse[t])
                : exp_listed(l - st.tmax, r) * st.inv_n;
      if (st.inv_n == 0.f) p = 0.f;
      zl[j] = to_f32(row[v]);
      twice |= mark_entry(s.bits, v);
    }
    s.p[j] = p;
  }
  if (twice) twice_any = 1;
  __syncthreads();
  const float A = w * r.tau * dl;
  const GradScale<OT> scale(A * st.unlisted, st.zu, r);
  for (int v = tid; v < nvec; v += nt) {
    const Vec<ZT> x = load_vec(row, v, r.V);
    float d[N];
    scale(x, d);
    store_vec<OT, N>(drow, v, r.V, d);
  }
  __syncthreads();
  if (st.inv_n != 0.f)
    write_entries<ZT, OT>(s, r, zl, drow, st, A, twice_any != 0);
}

DistillRow row_of(const mbok_distill_desc* d) {
  const double c = 1.4426950408889634074 / (double)d->temperature;
  const float hi = (float)c;
  return DistillRow{d->vocab, d->top, d->temperature, hi, (float)(c - (double)hi)};
}

size_t row_lds_bytes(const mbok_distill_desc* d) {
  return ((size_t)d->top * 3 + ((size_t)d->vocab + 31) / 32) * 4;
}

// Threads of a row's workgroup for `want` vectors each, 256 to 1024; a launch has
// fewer than 2^32 threads (256 for each of MBOK_MAX_DISTILL_ROWS rows are 2^31).
int row_threads(int64_t T, int nvec, int want) {
  int threads = 256;
  while (threads < kMaxThreads && threads * want < nvec && T * threads * 2 <= UINT32_MAX)
    threads *= 2;
  return threads;
}

template <typename ZT, typename OT>
int launch_rows(const mbok_distill_desc* d, const DistillArgs& a, float* loss, float* stats,
                hipStream_t stream) {
  const int nvec = (d->vocab + Vec<ZT>::N - 1) / Vec<ZT>::N;
  const size_t lds = row_lds_bytes(d);
  const DistillRow r = row_of(d);
  // 8 vectors per thread; with few rows, where latency counts, 2 (step, us, for 2
  // / 8: 32000 bf16 logits 1 row 9.6 / 10.0, 128 rows 11.1 / 11.8, 256 rows 12.6
  // / 13.5, 512 rows 23.5 / 17.7, 2048 rows 97.9 / 75.5; 12345 fp32 logits 256
  // rows 10.6 / 10.2, 512 rows 19.9 / 14.1; 4000 bf16 logits the same for both).
  // From 257 rows to 511, past one row per compute unit, 8 is the faster one
  // too (384 rows 21.9 / 16.8, fp32 18.3 / 12.8).
  const int threads = row_threads(a.T, nvec, a.T < 512 ? 2 : 8);
  const int per = (nvec + threads - 1) / threads;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)a.T), dim3(threads), lds, stream,
                       reinterpret_cast<const ZT*>(a.Z), a.ldz, a.t_logits, a.t_dtype, a.t_index,
                       a.ldt, a.t_lse, a.weight, r, loss, reinterpret_cast<RowStats*>(stats),
                       reinterpret_cast<OT*>(a.dZ), a.lddz);
  };
  auto by_nv = [&](auto grad, auto rest) {
    constexpr bool G = decltype(grad)::value, R = decltype(rest)::value;
    if (per <= 2) go(distill_kernel<ZT, OT, 2, G, R>);
    else if (per <= 4) go(distill_kernel<ZT, OT, 4, G, R>);
    else if (per <= 8) go(distill_kernel<ZT, OT, 8, G, R>);
    else if (per <= 16) go(distill_kernel<ZT, OT, 16, G, R>);
    else go(distill_kernel<ZT, OT, 0, G, R>);
  };
  auto by_rest = [&](auto grad) {
    if (a.t_lse) by_nv(grad, std::true_type{});
    else by_nv(grad, std::false_type{});
  };
  if (a.dZ) by_rest(std::true_type{});
  else by_rest(std::false_type{});
  return hipGetLastError() == hipSuccess ? MBOK_OK : MBOK_ERR_HIP;
}

template <typename ZT, typename OT>
int launch_rows_backward(const mbok_distill_desc* d, const DistillArgs& a, const float* stats,
                         const float* dloss, hipStream_t stream) {
  const int nvec = (d->vocab + Vec<ZT>::N - 1) / Vec<ZT>::N;
  // 4 vectors per thread: of 2, 4 and 8 the loss and gradient calls together
  // take 95.6, 95.4 and 97.2 us for 2048 x 32000 bf16, 23.8, 23.6 and 24.1 for
  // 512 rows, 20.2, 19.5 and 19.8 for 512 x 12345 fp32
  const int threads = row_threads(a.T, nvec, 4);
  hipLaunchKernelGGL((distill_backward_kernel<ZT, OT>), dim3((unsigned)a.T), dim3(threads),
                     row_lds_bytes(d), stream, reinterpret_cast<const ZT*>(a.Z), a.ldz,
                     a.t_logits, a.t_dtype, a.t_index, a.ldt, a.t_lse, a.weight, row_of(d),
                     reinterpret_cast<const RowStats*>(stats), dloss,
                     reinterpret_cast<OT*>(a.dZ), a.lddz);
  return hipGetLastError() == hipSuccess ? MBOK_OK : MBOK_ERR_HIP;
}

// calls f with the logit and gradient types of the call
template <typename F>
int by_types(const DistillArgs& a, F&& f) {
  const bool same = !a.dZ || a.dz_dtype == a.z_dtype;
  switch (a.z_dtype) {
    case MBOK_F32: return same ? f(float{}, float{}) : f(float{}, __bf16{});
    case MBOK_F16: return same ? f(_Float16{}, _Float16{}) : f(_Float16{}, __bf16{});
    default: return f(__bf16{}, __bf16{});
  }
}

}  // namespace

int launch_distill(const mbok_distill_desc* d, const DistillArgs& a, float* loss, float* stats,
                   hipStream_t stream) {
  return by_types(a, [&](auto z, auto o) {
    return launch_rows<decltype(z), decltype(o)>(d, a, loss, stats, stream);
  });
}

int launch_distill_backward(const mbok_distill_desc* d, const DistillArgs& a, const float* stats,
                            const float* dloss, hipStream_t stream) {
  return by_types(a, [&](auto z, auto o) {
    return launch_rows_backward<decltype(z), decltype(o)>(d, a, stats, dloss, stream);
  });
}

}  // namespace mbok
