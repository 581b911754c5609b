// One AdamW step over many tensors (gfx950).
//
// Decoupled weight decay, bias-corrected moments (Loshchilov and Hutter,
// "Decoupled Weight Decay Regularization"):
//     g' = c g,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//     p  = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// What a Boolean-kernel model trains besides signs are scales ("Highly
// Efficient and Effective LLMs with Multi-Boolean Architectures", Paper-Notes
// reading note, 训练策略), whose masters and gradients are in the order of
// mbok_pack's alpha and whose working copies sit in the packed layer, 64 rows
// of one (group, kernel) together: a workgroup turns its part of the masters
// around in LDS and writes whole lines of the packed buffer.
//
// Bound: memory, 28 bytes a parameter with fp32 states and gradients, 16 with
// 8-bit ones, beside the copy.  (29.5 M scales of 48 layers, fp32
// gradients: 203 us of 0.89 GB, 4.4 TB/s; 8-bit states 130 us of 0.54 GB, 4.1 TB/s, and
// 60 M vector instructions, which alone take 100.)
//
// 8-bit states: 256 consecutive values, one wavefront's 64 lanes x 4, share a
// power-of-two scale, so scaling is exact and the block's largest magnitude
// lies in [128, 256) of e4m3's 448.  The second moment is kept as r = sqrt(v),
// which halves the range it needs.  Codes are rounded stochastically: a step
// moves v by a thousandth, half an e4m3 step is a sixteenth to a thirty-second,
// so nearest rounding would leave most of them where they are.  The expected
// value of a code is the value: r, which the update divides by, follows its
// decay in the mean (its square up to a sixteenth slower, by the codes'
// variance).  A value r that is not 0 keeps code 1 at least, so that no m is
// divided by eps alone, down to the r whose squares are 0 in fp32 (2^-75; with fp32
// states v is 0 there, too).
#include <math.h>

#include <algorithm>
#include <type_traits>
#include <vector>

#include "mbok_adamw.h"
#include "mbok_device.h"
#include "mbok_launch.h"

namespace mbok {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 4;                      // values per thread and access
constexpr int kPass = kThreads * kVec;       // values a workgroup takes at a time
constexpr int kBlockValues = MBOK_ADAMW_BLOCK;
static_assert(kBlockValues == kWave * kVec, "a wavefront holds one block");

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(1)));

// odd multipliers of the hash (fractions of the golden ratio and of the square
// roots of 2, 3, 5 and 7)
constexpr uint32_t kH0 = 0x9E3779B1u, kH1 = 0x6A09E667u, kH2 = 0xBB67AE85u, kH3 = 0x3C6EF373u,
                   kH4 = 0xA54FF53Bu;

__device__ __forceinline__ uint32_t hash32(uint32_t h) {
  h = (h ^ (h >> 16)) * kH3;
  h = (h ^ (h >> 15)) * kH4;
  return h ^ (h >> 16);
}

// What every value's update needs, the same for a whole tensor.
struct Rule {
  float scale, b1, c1, b2, c2, keep, step, rden, eps;  // c = 1 - b, keep = 1 - lr wd
  uint32_t key;
};

// 4 values at p + i, `live` of them inside the tensor (the others 0)
__device__ __forceinline__ f32x4 load4(const float* p, int live) {
  if (live == 4) return f32x4(*reinterpret_cast<const f32x4_any*>(p));
  f32x4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < live) r[e] = p[e];
  return r;
}
__device__ __forceinline__ f32x4 load4(const _Float16* p, int live) {
  f32x4 r = {0.f, 0.f, 0.f, 0.f};
  if (live == 4) {
    const u16x4_any v = *reinterpret_cast<const u16x4_any*>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = f16_bits_to_f32(v[e]);
    return r;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < live) r[e] = (float)p[e];
  return r;
}
__device__ __forceinline__ f32x4 load4(const __bf16* p, int live) {
  f32x4 r = {0.f, 0.f, 0.f, 0.f};
  if (live == 4) {
    const u16x4_any v = *reinterpret_cast<const u16x4_any*>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = bf16_bits_to_f32(v[e]);
    return r;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < live) r[e] = (float)p[e];
  return r;
}
__device__ __forceinline__ void store4(float* p, f32x4 v, int live) {
  if (live == 4) {
    *reinterpret_cast<f32x4_any*>(p) = v;
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < live) p[e] = v[e];
}
template <typename T>
__device__ __forceinline__ void store4_half(T* p, f32x4 v, int live) {
  u16x4_any o;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = __builtin_bit_cast(uint16_t, (T)v[e]);
  if (live == 4) {
    *reinterpret_cast<u16x4_any*>(p) = o;
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < live) reinterpret_cast<uint16_t*>(p)[e] = o[e];
}
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int live) {
  if (live == 4) return *reinterpret_cast<const u32_any*>(p);
  uint32_t r = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < live) r |= (uint32_t)p[e] << (8 * e);
  return r;
}
__device__ __forceinline__ void store_codes(uint8_t* p, uint32_t v, int live) {
  if (live == 4) {
    *reinterpret_cast<u32_any*>(p) = v;
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < live) p[e] = (uint8_t)(v >> (8 * e));
}

// largest value over the wavefront, in every lane
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  auto dpp = [](uint32_t x, auto ctrl) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, 0xf, 0xf, false);
  };
  v = max(v, dpp(v, std::integral_constant<int, 0xB1>{}));   // lane ^ 1
  v = max(v, dpp(v, std::integral_constant<int, 0x4E>{}));   // lane ^ 2
  v = max(v, dpp(v, std::integral_constant<int, 0x141>{}));  // 7 - lane of 8
  v = max(v, dpp(v, std::integral_constant<int, 0x140>{}));  // 15 - lane of 16
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max((uint32_t)a[0], (uint32_t)a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max((uint32_t)b[0], (uint32_t)b[1]);
}

// The 4 values of a lane in e4m3 with the block's scale (returned in *scale; NaN
// where a value is not finite, which then stands for the whole block).  Bits
// 4 .. 19 of each value's 20 random bits are `rnd`'s; ROOT: values that are not
// negative, and not 0 keep code 1 at least.  y in [2^-6, 256): exponent and 3
// mantissa bits of y plus the random bits; below, multiples of 2^-9.
template <bool ROOT>
__device__ __forceinline__ uint32_t to_codes(f32x4 x, const uint32_t (&rnd)[4], float* scale) {
#pragma clang fp contract(off)
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
  top = wave_umax(top);
  // the scale is at least 2^-87: values far below it matter to nothing (eps)
  const uint32_t ex = max(top >> 23, 47u) - 7u;
  *scale = top >= 0x7f800000u ? __builtin_nanf("") : __uint_as_float(ex << 23);
  const float up = __uint_as_float((254u - ex) << 23);
  uint32_t codes = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float y = fabsf(x[e]) * up;
    const uint32_t bits = rnd[e] << 4 | 8u;
    const uint32_t normal = ((__float_as_uint(y) + bits) >> 20) - 960u;
    const uint32_t small = (uint32_t)(y * 512.f + (float)bits * 0x1p-20f);
    uint32_t c = y >= 0x1p-6f ? normal : small;
    if (ROOT) c = max(c, min(__float_as_uint(x[e]), 1u)) & 0x7fu;
    else c = (c & 0x7fu) | (x[e] < 0.f ? 0x80u : 0u);
    codes |= c << (8 * e);
  }
  return codes;
}

__device__ __forceinline__ f32x4 from_codes(uint32_t c, float scale) {
  const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false);
  const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
  return f32x4{a[0] * scale, a[1] * scale, b[0] * scale, b[1] * scale};
}

// One access's values and states as loaded.
template <bool EIGHT>
struct Held;
template <>
struct Held<false> {
  f32x4 p, g, m, v;
};
template <>
struct Held<true> {
  f32x4 p, g;
  uint32_t m, r;
  float ms, rs;
};

// The moments are formed without fused operations: each product and sum is
// rounded, as the elementary operations of the plain formula do.
__device__ __forceinline__ void moments(const Rule& rule, f32x4 g, f32x4& m, f32x4& v) {
#pragma clang fp contract(off)
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float x = g[e] * rule.scale;
    m[e] = m[e] * rule.b1 + x * rule.c1;
    v[e] = v[e] * rule.b2 + (x * x) * rule.c2;
  }
}

// r = sqrt(v) to the last bit for the state, 1 ulp where only p takes it
__device__ __forceinline__ float new_param(const Rule& rule, float p, float m, float r) {
  const float den = fmaf(r, rule.rden, rule.eps);
  return fmaf(-rule.step, m * __builtin_amdgcn_rcpf(den), p * rule.keep);
}

// Values start .. start + len of one tensor; put(i, p) receives the new values
// of start + i .. + 3.
template <bool EIGHT, typename GT, typename Put>
__device__ __forceinline__ void update(const AdamTensor& t, const Rule& rule, int64_t start,
                                       int len, Put&& put) {
  constexpr int U = 1;  // accesses in flight; 2: 5 wavefronts per SIMD, not 6 (8 bits 141 us, not 131)
  const GT* grad = reinterpret_cast<const GT*>(t.grad) + start;
  float* param = t.param + start;
  const int lane = threadIdx.x & (kWave - 1);
  auto load = [&](int i) {
    Held<EIGHT> h;
    const int live = min(4, len - i);
    h.p = load4(param + i, live);
    h.g = load4(grad + i, live);
    if constexpr (EIGHT) {
      h.m = load_codes(reinterpret_cast<const uint8_t*>(t.m) + start + i, live);
      h.r = load_codes(reinterpret_cast<const uint8_t*>(t.v) + start + i, live);
      const int64_t b = (start + i) / kBlockValues;
      h.ms = t.m_scale[b];
      h.rs = t.v_scale[b];
    } else {
      h.m = load4(reinterpret_cast<const float*>(t.m) + start + i, live);
      h.v = load4(reinterpret_cast<const float*>(t.v) + start + i, live);
    }
    return h;
  };
  auto finish = [&](int i, const Held<EIGHT>& h, bool inside) {
    const int live = inside ? min(4, len - i) : 0;
    f32x4 m, v, p;
    if constexpr (EIGHT) {
      m = from_codes(h.m, h.ms);
      v = from_codes(h.r, h.rs);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = v[e] * v[e];
      moments(rule, h.g, m, v);
      uint32_t low[4], high[4];
      const uint32_t seed = (uint32_t)(start + i) * kH2 + rule.key;
      f32x4 r;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        r[e] = __builtin_sqrtf(v[e]);
        p[e] = new_param(rule, h.p[e], m[e], r[e]);
        const uint32_t rnd = hash32(seed + e * kH2);
        low[e] = rnd & 0xffffu;
        high[e] = rnd >> 16;
        if (e >= live) m[e] = r[e] = 0.f;
      }
      float ms, rs;
      const uint32_t mc = to_codes<false>(m, low, &ms), rc = to_codes<true>(r, high, &rs);
      if (live > 0) {
        store_codes(reinterpret_cast<uint8_t*>(t.m) + start + i, mc, live);
        store_codes(reinterpret_cast<uint8_t*>(t.v) + start + i, rc, live);
        if (lane == 0) {
          const int64_t b = (start + i) / kBlockValues;
          t.m_scale[b] = ms;
          t.v_scale[b] = rs;
        }
      }
    } else {
      m = h.m;
      v = h.v;
      moments(rule, h.g, m, v);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        p[e] = new_param(rule, h.p[e], m[e], __builtin_amdgcn_sqrtf(v[e]));
      if (live > 0) {
        store4(reinterpret_cast<float*>(t.m) + start + i, m, live);
        store4(reinterpret_cast<float*>(t.v) + start + i, v, live);
      }
    }
    if (live > 0) {
      store4(param + i, p, live);
      put(i, p, live);
    }
  };
  for (int base = 0; base < len; base += U * kPass) {
    Held<EIGHT> held[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = base + u * kPass + (int)threadIdx.x * kVec;
      // a wavefront's lanes past the end take part in its largest value
      if (i < len) held[u] = load(i);
      else held[u] = Held<EIGHT>{};
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = base + u * kPass + (int)threadIdx.x * kVec;
      finish(i, held[u], i < len);
    }
  }
}

template <bool EIGHT, typename Put>
__device__ __forceinline__ void update_by_grad(const AdamTensor& t, const Rule& rule,
                                               int64_t start, int len, Put&& put) {
  if (t.grad_dtype == MBOK_F32) update<EIGHT, float>(t, rule, start, len, put);
  else if (t.grad_dtype == MBOK_F16) update<EIGHT, _Float16>(t, rule, start, len, put);
  else update<EIGHT, __bf16>(t, rule, start, len, put);
}

template <typename Put>
__device__ __forceinline__ void update_any(const AdamTensor& t, const Rule& rule, int64_t start,
                                           int len, Put&& put) {
  if (t.state_dtype == MBOK_F32) update_by_grad<false>(t, rule, start, len, put);
  else update_by_grad<true>(t, rule, start, len, put);
}

// A layer's scales: the new masters go to LDS by (row, group), rows an odd number
// of words apart, then 64 rows at a time to the packed buffer.
template <typename AT>
__device__ __forceinline__ void update_layer(const AdamTensor& t, const Rule& rule, int64_t start,
                                             int len, float* lds) {
  const int G = t.groups, pitch = G | 1;
  const uint32_t r0 = (uint32_t)(start / G);  // row of [K m], at most 2^26
  const int first = (int)(start - (int64_t)r0 * G);  // group of the first value
  // x / G by the reciprocal: off by x 2^-23 / G at most, where 0.5 / G is spare
  const bool quick = G < (1 << 20);
  const float inv = 1.f / (float)G;
  update_any(t, rule, start, len, [&](int i, f32x4 p, int live) {
    const uint32_t x = (uint32_t)(first + i);
    const uint32_t row = quick ? (uint32_t)(((float)x + 0.5f) * inv) : x / (uint32_t)G;
    int g = (int)(x - row * (uint32_t)G), at = (int)row * pitch + g - first;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e < live) lds[at] = p[e];
      ++at;
      if (++g == G) {
        g = 0;
        at += pitch - G;
      }
    }
  });
  __syncthreads();
  const int rows = (int)((uint32_t)(first + len + G - 1) / (uint32_t)G);
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  AT* out = reinterpret_cast<AT*>(t.out);
  for (int r = lane; r < rows; r += kWave) {
    const uint32_t row = r0 + (uint32_t)r, k = row / (uint32_t)t.rows, i = row - k * (uint32_t)t.rows;
    AT* dst = out + ((int64_t)(i / kRowBlock) * G * t.kernels + k) * kRowBlock + i % kRowBlock;
    // the part's values of this row: groups g0 .. g1
    const int g0 = r == 0 ? first : 0, g1 = min(G, first + len - r * G);
    for (int g = g0 + wave; g < g1; g += kThreads / kWave) {
      const float p = lds[r * pitch + g - first];
      AT* at = dst + (int64_t)g * t.kernels * kRowBlock;
      if constexpr (sizeof(AT) == 2) *at = (AT)p;
      else *at = p;
    }
  }
}

// the step's own numbers, from the host or (live) from device memory; false: no step (the
// skip flag, or a count below 1, as a zeroed buffer holds it: 1 - b^0 would divide by 0)
__device__ __forceinline__ bool step_of(const AdamStep& s, const float* live, const AdamTensor& t,
                                        Rule& rule) {
  double lr = s.lr, c1 = s.correct1, c2 = s.correct2;
  float scale = s.grad_scale;
  uint32_t key = s.key;
  if (live) {
    if (live[3] != 0.f || !(live[2] >= 1.f)) return false;
    lr = (double)live[0];
    scale = live[1];
    const double n = (double)live[2];
    c1 = -expm1(n * s.log_b1);
    c2 = -expm1(n * s.log_b2);
    key += (uint32_t)(int64_t)n * kH0;
  }
  rule = {scale, s.b1, s.c1, s.b2, s.c2, (float)(1.0 - lr * t.decay), (float)(lr / c1),
          (float)(1.0 / sqrt(c2)), s.eps, key + t.salt};
  return true;
}

__global__ void __launch_bounds__(kThreads) adamw_kernel(const AdamTensor* __restrict__ tensors,
                                                         const AdamPart* __restrict__ parts,
                                                         const float* __restrict__ live,
                                                         AdamStep s) {
  extern __shared__ float lds[];
  const AdamPart part = parts[blockIdx.x];
  const AdamTensor t = tensors[part.tensor];
  Rule rule;
  if (!step_of(s, live, t, rule)) return;
  if (t.groups) {
    if (t.out_dtype == MBOK_F16) update_layer<_Float16>(t, rule, part.start, part.len, lds);
    else update_layer<float>(t, rule, part.start, part.len, lds);
    return;
  }
  update_any(t, rule, part.start, part.len, [&](int i, f32x4 p, int n) {
    if (!t.out) return;
    if (t.out_dtype == MBOK_F32) store4(reinterpret_cast<float*>(t.out) + part.start + i, p, n);
    else if (t.out_dtype == MBOK_F16)
      store4_half(reinterpret_cast<_Float16*>(t.out) + part.start + i, p, n);
    else store4_half(reinterpret_cast<__bf16*>(t.out) + part.start + i, p, n);
  });
}

}  // namespace

// Parts of 4096 values (layers turn theirs around in LDS, 17 KB for 32 groups);
// smaller where there would be fewer than 1024 of them.
int adamw_part(int64_t values) {
  int part = 4096;
  while (part > kPass && values / part < 1024) part /= 2;
  return part;
}

// LDS of a part of a layer of G groups: its values, a word between rows where G is
// even (a part meets at most (part - 2) / G + 2 rows)
int adamw_layer_lds(int G, int part) { return (part + (part + G - 1) / G + 1) * 4; }

int launch_adamw(const mbok_adamw_plan* plan, const void* table, const mbok_adamw_step* step,
                 const float* live, hipStream_t stream) {
  AdamStep s;
  s.lr = step->lr;
  s.log_b1 = log(step->beta1);
  s.log_b2 = log(step->beta2);
  s.correct1 = -expm1((double)step->step * s.log_b1);
  s.correct2 = -expm1((double)step->step * s.log_b2);
  s.b1 = (float)step->beta1;
  s.c1 = (float)(1.0 - step->beta1);
  s.b2 = (float)step->beta2;
  s.c2 = (float)(1.0 - step->beta2);
  s.eps = (float)step->eps;
  s.grad_scale = step->grad_scale;
  s.key = step->seed + (live ? 0u : (uint32_t)step->step * kH0);
  const AdamTensor* tensors = reinterpret_cast<const AdamTensor*>(table);
  const AdamPart* parts = reinterpret_cast<const AdamPart*>(tensors + plan->tensors);
  hipLaunchKernelGGL(adamw_kernel, dim3((unsigned)plan->parts), dim3(kThreads),
                     (size_t)plan->lds_bytes, stream, tensors, parts, live, s);
  return hipGetLastError() == hipSuccess ? MBOK_OK : MBOK_ERR_HIP;
}

uint32_t adamw_salt(int tensor) { return (uint32_t)tensor * kH1; }

}  // namespace mbok
