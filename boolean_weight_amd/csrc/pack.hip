// Packs int8 +-1 sign planes and natural-order scales into the L64 layout
// described in include/mbok.h: one thread per 16-byte chunk (row, group,
// kernel); chunk c = ((rb*G + g)*K + k)*64 + r holds the group's 128 signs as
// four uint32 words, bit (8e + q) of word w being column 32w + 4q + e of the
// group, bit 1 = +1.  The scale of the chunk goes to value index c of the
// scale region.  Rows past m are written as zero bits and zero scales.
#include "mbok_device.h"
#include "mbok_launch.h"

namespace mbok {
namespace {

template <typename AT, bool GATED>
__global__ void __launch_bounds__(256) pack_kernel(const int8_t* __restrict__ signs,
                                                   const AT* __restrict__ alpha,
                                                   const int8_t* __restrict__ signs2,
                                                   const AT* __restrict__ alpha2, int m, int n,
                                                   int K, int RB, int row_stride, int group_stride,
                                                   uint4* __restrict__ bits,
                                                   AT* __restrict__ scales) {
  const int G = n / kGroup;
  const int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t total = (int64_t)RB * G * K * kRowBlock;
  if (c >= total) return;
  const int r = (int)(c % kRowBlock);
  int64_t t = c / kRowBlock;
  const int k = (int)(t % K);
  t /= K;
  const int g = (int)(t % G);
  const int rb = (int)(t / G);
  int i = rb * kRowBlock + r;
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  AT a = AT(0);
  // GATED: stacked row 16 u + r is row 8 u + r of the first projection for
  // r < 8, of the second for r >= 8; m is one projection's
  const bool second = GATED && (i & 8);
  if (GATED) {
    i = 8 * (i >> 4) + (i & 7);
    if (second) signs = signs2, alpha = alpha2;
  }
  if (i < m) {
    const int4* src = reinterpret_cast<const int4*>(signs + ((int64_t)k * m + i) * n +
                                                    (int64_t)g * kGroup);
#pragma unroll
    for (int v = 0; v < 8; ++v) {  // 16 signs per 16-byte load
      const int4 s = src[v];
      const uint32_t parts[4] = {(uint32_t)s.x, (uint32_t)s.y, (uint32_t)s.z, (uint32_t)s.w};
#pragma unroll
      for (int p = 0; p < 4; ++p) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          // byte b of part p is column 16v + 4p + b = 32w + 4q + e with
          // w = v/2, q = 4(v%2) + p, e = b; bit 1 when the int8 is >= 0
          const uint32_t bit = ((~parts[p]) >> (8 * b + 7)) & 1u;
          w[v >> 1] |= bit << (8 * b + 4 * (v & 1) + p);
        }
      }
    }
    a = alpha[((int64_t)k * m + i) * row_stride + (int64_t)g * group_stride];
  }
  bits[c] = make_uint4(w[0], w[1], w[2], w[3]);
  scales[c] = a;
}

// alpha[(k m + i) * row_stride + g * group_stride] is the scale of chunk
// (row i, group g, kernel k): (G, 1) for per-group scales, (1, 0) for one
// scale per row (the SVID s_out).  geo: the packed layer's geometry; m: rows
// of the sign and scale arrays.
template <typename AT, bool GATED>
int pack_typed(const Geom& geo, int m, const int8_t* signs, const void* alpha,
               const int8_t* signs2, const void* alpha2, void* packed, int row_stride,
               int group_stride, hipStream_t stream) {
  const int64_t total = (int64_t)geo.RB * geo.G * geo.K * kRowBlock;
  const int block = 256;
  const int64_t blocks = (total + block - 1) / block;
  if (blocks > 0x7fffffff) return MBOK_ERR_SHAPE;
  uint4* bits = reinterpret_cast<uint4*>(packed);
  AT* scales = reinterpret_cast<AT*>(reinterpret_cast<char*>(packed) + geo.bits_bytes);
  hipLaunchKernelGGL((pack_kernel<AT, GATED>), dim3((unsigned)blocks), dim3(block), 0, stream,
                     signs, reinterpret_cast<const AT*>(alpha), signs2,
                     reinterpret_cast<const AT*>(alpha2), m, geo.n, geo.K, geo.RB, row_stride,
                     group_stride, bits, scales);
  return hipGetLastError() == hipSuccess ? MBOK_OK : MBOK_ERR_HIP;
}

int pack_strided(const mbok_desc* d, const int8_t* signs, const void* alpha, void* packed,
                 int row_stride, int group_stride, hipStream_t stream) {
  const Geom geo = make_geom(d);
  if (d->alpha_dtype == MBOK_F16)
    return pack_typed<uint16_t, false>(geo, geo.m, signs, alpha, nullptr, nullptr, packed,
                                       row_stride, group_stride, stream);
  return pack_typed<float, false>(geo, geo.m, signs, alpha, nullptr, nullptr, packed, row_stride,
                                  group_stride, stream);
}

}  // namespace

int launch_pack(const mbok_desc* d, const int8_t* signs, const void* alpha, void* packed,
                hipStream_t stream) {
  return pack_strided(d, signs, alpha, packed, d->n / kGroup, 1, stream);
}

mbok_desc gated_stacked(const mbok_desc* d) {
  mbok_desc s = *d;
  s.m = 16 * ((d->m + 7) / 8);
  return s;
}

int launch_gated_pack(const mbok_desc* d, const int8_t* signs_gate, const void* alpha_gate,
                      const int8_t* signs_up, const void* alpha_up, void* packed,
                      hipStream_t stream) {
  const mbok_desc stacked = gated_stacked(d);
  const Geom geo = make_geom(&stacked);
  if (d->alpha_dtype == MBOK_F16)
    return pack_typed<uint16_t, true>(geo, d->m, signs_gate, alpha_gate, signs_up, alpha_up,
                                      packed, geo.G, 1, stream);
  return pack_typed<float, true>(geo, d->m, signs_gate, alpha_gate, signs_up, alpha_up, packed,
                                 geo.G, 1, stream);
}

int launch_svid_pack(const mbok_desc* d, const int8_t* signs, const void* s_out, void* packed,
                     hipStream_t stream) {
  return pack_strided(d, signs, s_out, packed, 1, 0, stream);
}

}  // namespace mbok
