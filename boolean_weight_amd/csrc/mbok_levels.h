// Tiles of W_hat as bf16 for the matrix cores (gfx950): the level values of a
// (row, group), their selection by sign bits, and the tile order, shared by the
// multi-token product and its transposed form.  Internal header.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mbok {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(16))) float f32x16;
// a native vector type keeps the activation staging in registers (a uint4
// struct member went through scratch memory)
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __bf16 ha = (__bf16)a, hb = (__bf16)b;  // nearest-even
  return (uint32_t)__builtin_bit_cast(uint16_t, ha) |
         ((uint32_t)__builtin_bit_cast(uint16_t, hb) << 16);
}

// Byte-planar bf16 levels of one (row, group): lo_a/hi_a hold the low/high
// bytes of levels 0..3, lo_b/hi_b of levels 4..7.  Level index bit k-1 is the
// sign bit of kernel k (1 = +alpha_k).
struct Levels {
  uint32_t lo_a, lo_b, hi_a, hi_b;
};

// What is left of an fp32 value after its rounding to bf16.  The difference
// is exact in fp32 (it is v's own low significand bits) and at most half a
// bf16 ulp of v, so hi + bf16(lo) carries 16 significant bits of v.
__device__ __forceinline__ float bf16_residue(float v) { return v - (float)(__bf16)v; }

// LO = false: the levels rounded to bf16 (the default product).  LO = true:
// the bf16 rounding of each level's residue, for the second pass of the
// two-pass product (hi + lo levels, ~2^-16 relative error per weight).
template <int K, bool LO = false>
__device__ __forceinline__ Levels make_levels(const float* a) {
  float l[8];
#pragma unroll
  for (int idx = 0; idx < 8; ++idx) {
    float v = (idx & 1) ? a[0] : -a[0];
    if (K >= 2) v += (idx & 2) ? a[1] : -a[1];
    if (K >= 3) v += (idx & 4) ? a[2] : -a[2];
    l[idx] = LO ? bf16_residue(v) : v;
  }
  const uint32_t p01 = bf16_pair(l[0], l[1]), p23 = bf16_pair(l[2], l[3]);
  const uint32_t p45 = bf16_pair(l[4], l[5]), p67 = bf16_pair(l[6], l[7]);
  Levels L;
  // v_perm_b32(s0, s1, sel): selector byte 0..3 picks s1 bytes, 4..7 s0 bytes
  L.lo_a = __builtin_amdgcn_perm(p23, p01, 0x06040200u);
  L.hi_a = __builtin_amdgcn_perm(p23, p01, 0x07050301u);
  L.lo_b = __builtin_amdgcn_perm(p67, p45, 0x06040200u);
  L.hi_b = __builtin_amdgcn_perm(p67, p45, 0x07050301u);
  return L;
}

// Unpack one 32-column sign word per kernel (w[k]) into 32 bf16 weights in
// natural column order: out[2q], out[2q+1] hold columns 4q..4q+3.
template <int K>
__device__ __forceinline__ void unpack_word(const uint32_t* w, const Levels& L, uint32_t* out) {
  constexpr uint32_t M = 0x11111111u;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    // nibble j = 2e + a of V holds the level index of quad q = 4a + b, element e
    uint32_t V = (w[0] >> b) & M;
    if (K >= 2) V |= ((w[1] >> b) & M) << 1;
    if (K >= 3) V |= ((w[2] >> b) & M) << 2;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int q = 4 * a + b;
      const uint32_t sel = (a ? (V >> 4) : V) & 0x0f0f0f0fu;
      const uint32_t lo = __builtin_amdgcn_perm(L.lo_b, L.lo_a, sel);
      const uint32_t hi = __builtin_amdgcn_perm(L.hi_b, L.hi_a, sel);
      out[2 * q] = __builtin_amdgcn_perm(hi, lo, 0x05010400u);
      out[2 * q + 1] = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
    }
  }
}

// K = 4 (16 levels): direct fp32 sums, then bf16 (LO: their residues).
template <bool LO = false>
__device__ __forceinline__ void unpack_word_k4(const uint32_t* w, const float* a, uint32_t* out) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) s += ((w[k] >> (8 * e + q)) & 1u) ? a[k] : -a[k];
      v[e] = LO ? bf16_residue(s) : s;
    }
    out[2 * q] = bf16_pair(v[0], v[1]);
    out[2 * q + 1] = bf16_pair(v[2], v[3]);
  }
}

// Selector words of one 32-column sign word per kernel: V[b] nibble 2e + a is
// the level index of quad q = 4a + b, element e (see unpack_word).
template <int K>
__device__ __forceinline__ void word_selectors(const uint32_t* w, uint32_t* V) {
  constexpr uint32_t M = 0x11111111u;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    uint32_t v = (w[0] >> b) & M;
    if (K >= 2) v |= ((w[1] >> b) & M) << 1;
    if (K >= 3) v |= ((w[2] >> b) & M) << 2;
    V[b] = v;
  }
}

// Quads 4a .. 4a+3 of a word (16 columns 16a .. 16a+15) as 8 bf16 pairs.
__device__ __forceinline__ void unpack_quads(const uint32_t* V, int a, const Levels& L,
                                             uint32_t* out) {
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const uint32_t sel = (a ? (V[b] >> 4) : V[b]) & 0x0f0f0f0fu;
    const uint32_t lo = __builtin_amdgcn_perm(L.lo_b, L.lo_a, sel);
    const uint32_t hi = __builtin_amdgcn_perm(L.hi_b, L.hi_a, sel);
    out[2 * b] = __builtin_amdgcn_perm(hi, lo, 0x05010400u);
    out[2 * b + 1] = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
  }
}

__device__ __forceinline__ void unpack_two_quads(const uint32_t* V, int a, int b0, const Levels& L,
                                                 uint32_t* out) {
#pragma unroll
  for (int bb = 0; bb < 2; ++bb) {
    const int b = b0 + bb;
    const uint32_t sel = (a ? (V[b] >> 4) : V[b]) & 0x0f0f0f0fu;
    const uint32_t lo = __builtin_amdgcn_perm(L.lo_b, L.lo_a, sel);
    const uint32_t hi = __builtin_amdgcn_perm(L.hi_b, L.hi_a, sel);
    out[2 * bb] = __builtin_amdgcn_perm(hi, lo, 0x05010400u);
    out[2 * bb + 1] = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
  }
}

// Tile at position p of the XCD-blocked order: pairs of token tiles, sweeping
// the row tiles (p -> token tile 2q + d, row tile tx), the last token tile
// alone when their count is odd.  Workgroup b runs on XCD b % 8, so giving
// XCD x the positions x * nfull / 8 .. of the full round puts ~16 row tiles
// x 2 token tiles on each XCD: its L2 holds those activations and weights
// instead of every XCD streaming every token tile.
__device__ __forceinline__ int tile_at(int p, int ntx, int nty) {
  const int q = p / (2 * ntx);
  const int rem = p - q * 2 * ntx;
  if (2 * q + 1 < nty) return (2 * q + (rem & 1)) * ntx + (rem >> 1);
  return 2 * q * ntx + rem;
}

}  // namespace mbok
