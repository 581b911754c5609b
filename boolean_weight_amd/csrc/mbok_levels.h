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

// 8 bf16 values at p (any 2-byte alignment) of which the first `live` lie inside
// the row and the others are returned as 0 without being read.  back: at least
// 8 values of the row end where the live ones do, so one load of those, shifted,
// serves a partial piece.
typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t u32x4_unaligned;
__device__ __forceinline__ u32x4 load_piece(const uint16_t* p, int live, bool back) {
  if (live == 8) return u32x4(*reinterpret_cast<const u32x4_unaligned*>(p));
  u32x4 r = u32x4{0u, 0u, 0u, 0u};
  if (live <= 0) return r;
  if (back) {
    const u32x4 v = *reinterpret_cast<const u32x4_unaligned*>(p + live - 8);
    const int drop = 8 - live;  // values before p: 1 .. 7
    const bool d4 = drop & 4, d2 = drop & 2, d1 = drop & 1;
    uint32_t w[5] = {d4 ? v[2] : v[0], d4 ? v[3] : v[1], d4 ? 0u : v[2], d4 ? 0u : v[3], 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = d2 ? (i < 3 ? w[i + 1] : 0u) : w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = d1 ? (w[i] >> 16 | (i < 3 ? w[i + 1] << 16 : 0u)) : w[i];
    return r;
  }
  uint32_t e[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) e[c] = c < live ? p[c] : 0u;
  return u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
}

// Copies 16 bytes per lane from memory to LDS without passing registers: lane l
// of the wavefront writes dst + 16 l (dst is the wavefront's).  The copy is in
// flight until copies_done(); a barrier after that shows it to the workgroup.
// (The compiler's builtin for this makes it wait for the copy before the next
// transposing LDS read of any buffer, i.e. at once.)  The wait counts the
// compiler inserts for its own loads stay right: loads return in order, so
// an uncounted copy in flight only makes a wait longer.
// m0 is the statement's alone: it is reserved, so the compiler takes no clobber
// of it, and nothing else in the kernels that use this writes or reads it (LDS
// accesses need none on this part).
// The source is base (the wavefront's) + off bytes (the lane's).
__device__ __forceinline__ void copy_to_lds(const void* base, uint32_t off, const uint16_t* dst) {
  const uint32_t at =
      (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint16_t*)dst;
  const uint64_t from = (uint64_t)(uintptr_t)base;
  const uint64_t sbase =
      (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)from) |
      (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(from >> 32)) << 32;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(__builtin_amdgcn_readfirstlane(at)), "v"(off), "s"(sbase)
               : "memory");
}
// Waits for every load in flight.  The builtin, not assembly: the compiler then
// knows that its own loads are done too (it otherwise waited for them again
// after the next copies were issued, and so for those).
__device__ __forceinline__ void copies_done() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0); the other counters at their maximum
  asm volatile("" ::: "memory");
}

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
//
// Flipping every sign negates a level: only those with the highest kernel's
// sign set (+) are summed and rounded, and the others are their bytes in
// reverse order with the sign bit flipped (rounding is symmetric).

// Levels 2 p and 2 p + 1 of the upper half (K = 3: p = 0, 1 for levels 4 .. 7;
// K = 2: levels 2, 3; K = 1: level 1 twice) as a bf16 pair.
template <int K, bool LO = false>
__device__ __forceinline__ uint32_t upper_pair(const float* a, int p) {
  float l[2];
  if (K == 1) {
    l[0] = l[1] = a[0];
  } else {
    const float s = K == 2 ? a[1] : (p ? a[2] + a[1] : a[2] - a[1]);
    l[0] = s - a[0];
    l[1] = s + a[0];
  }
  return LO ? bf16_pair(bf16_residue(l[0]), bf16_residue(l[1])) : bf16_pair(l[0], l[1]);
}
// v_perm_b32(s0, s1, sel): selector byte 0..3 picks s1 bytes, 4..7 s0 bytes
template <int K>
__device__ __forceinline__ Levels pack_levels(uint32_t p0, uint32_t p1) {
  Levels L;
  if (K == 3) {  // p0 = levels 4, 5; p1 = levels 6, 7
    L.lo_b = __builtin_amdgcn_perm(p1, p0, 0x06040200u);
    L.hi_b = __builtin_amdgcn_perm(p1, p0, 0x07050301u);
    L.lo_a = __builtin_amdgcn_perm(p1, p0, 0x00020406u);
    L.hi_a = __builtin_amdgcn_perm(p1, p0, 0x01030507u) ^ 0x80808080u;
  } else {  // p0 = levels 2, 3 (K = 1: level 1 twice)
    L.lo_a = __builtin_amdgcn_perm(p0, p0, K == 2 ? 0x02000002u : 0x00000000u);
    L.hi_a = __builtin_amdgcn_perm(p0, p0, K == 2 ? 0x03010103u : 0x01010101u) ^
             (K == 2 ? 0x00008080u : 0x00000080u);
    L.lo_b = L.hi_b = 0u;
  }
  return L;
}
template <int K, bool LO = false>
__device__ __forceinline__ Levels make_levels(const float* a) {
  return pack_levels<K>(upper_pair<K, LO>(a, 0), K == 3 ? upper_pair<K, LO>(a, 1) : 0u);
}

// Selector words of one 32-column sign word per kernel: bits 0 .. K - 1 of
// V[b]'s nibble 2e + a are the level index of quad q = 4a + b, element e (the
// nibble's other bits are other quads').  Two words are merged for two b at a
// time.
// (a & mask) | (b & ~mask), the compiler's own instruction: it knows which registers
// matrix instructions in flight still read or write, which it does not for assembly
// (see skinny.hip).  (0xE4: the truth table; written out, it is taken apart into three.)
__device__ __forceinline__ uint32_t bit_select(uint32_t mask, uint32_t a, uint32_t b) {
  return __builtin_amdgcn_bitop3_b32(a, b, mask, 0xE4);
}
// Holds loaded signs and scales in registers at this point of the program, so
// that their loads are not moved past a later barrier.
template <int K, typename R>
__device__ __forceinline__ void pin(R& r) {
#pragma unroll
  for (int k = 0; k < K; ++k) asm volatile("" : "+v"(r.w[k]), "+v"(r.a[k]));
}
// part 0, 1, 2 in turn (V holds what is between them)
template <int K>
__device__ __forceinline__ void word_selectors_part(const uint32_t* w, uint32_t* V, int part) {
  if (K == 1) {
    if (part == 0) {
#pragma unroll
      for (int b = 0; b < 4; ++b) V[b] = w[0] >> b;
    }
    return;
  }
  if (part == 0) {
    V[0] = bit_select(0x55555555u, w[0], w[1] << 1);  // b = 0, 2
    V[1] = bit_select(0x55555555u, w[0] >> 1, w[1]);  // b = 1, 3
  }
  if (part == 1) {
    V[2] = K == 3 ? bit_select(0x33333333u, V[0] >> 2, w[2]) : V[0] >> 2;
    if (K == 3) V[0] = bit_select(0x33333333u, V[0], w[2] << 2);
  }
  if (part == 2) {
    V[3] = K == 3 ? bit_select(0x33333333u, V[1] >> 2, w[2] >> 1) : V[1] >> 2;
    if (K == 3) V[1] = bit_select(0x33333333u, V[1], w[2] << 1);
  }
}
template <int K>
__device__ __forceinline__ void word_selectors(const uint32_t* w, uint32_t* V) {
#pragma unroll
  for (int p = 0; p < 3; ++p) word_selectors_part<K>(w, V, p);
}

// Level indices of quad 4 a + b, one per byte
template <int K>
__device__ __forceinline__ uint32_t quad_selector(const uint32_t* V, int a, int b) {
  return (a ? V[b] >> 4 : V[b]) & (K == 1 ? 0x01010101u : K == 2 ? 0x03030303u : 0x07070707u);
}
// Low and high bytes of the quad's 4 columns, and the columns as two bf16 pairs
__device__ __forceinline__ uint32_t quad_low(const Levels& L, uint32_t sel) {
  return __builtin_amdgcn_perm(L.lo_b, L.lo_a, sel);
}
__device__ __forceinline__ uint32_t quad_high(const Levels& L, uint32_t sel) {
  return __builtin_amdgcn_perm(L.hi_b, L.hi_a, sel);
}
__device__ __forceinline__ void quad_pairs(uint32_t lo, uint32_t hi, uint32_t* out) {
  out[0] = __builtin_amdgcn_perm(hi, lo, 0x05010400u);
  out[1] = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
}
template <int K>
__device__ __forceinline__ void unpack_quad(const uint32_t* V, int a, int b, const Levels& L,
                                            uint32_t* out) {
  const uint32_t sel = quad_selector<K>(V, a, b);
  quad_pairs(quad_low(L, sel), quad_high(L, sel), out);
}

// Unpack one 32-column sign word per kernel (w[k]) into 32 bf16 weights in
// natural column order: out[2q], out[2q+1] hold columns 4q..4q+3.
template <int K>
__device__ __forceinline__ void unpack_word(const uint32_t* w, const Levels& L, uint32_t* out) {
  uint32_t V[4];
  word_selectors<K>(w, V);
#pragma unroll
  for (int q = 0; q < 8; ++q) unpack_quad<K>(V, q >> 2, q & 3, L, out + 2 * q);
}

// K = 4 (16 levels).  Flipping every sign negates a level, so the 8 levels with the
// fourth kernel's sign set are kept, as for K = 3; where it is not set the other three
// signs are flipped (k4_words) and the level's sign too (k4_high).  The same sums, in
// the kernels' order, as adding them one column at a time.
// Levels 2 p and 2 p + 1 (bits: signs of kernels 0, 1, 2) as a bf16 pair.
template <bool LO = false>
__device__ __forceinline__ uint32_t k4_pair(const float* a, int p) {
  float l[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float s = (e ? a[0] : -a[0]) + ((p & 1) ? a[1] : -a[1]);
    l[e] = (s + ((p & 2) ? a[2] : -a[2])) + a[3];
  }
  return LO ? bf16_pair(bf16_residue(l[0]), bf16_residue(l[1])) : bf16_pair(l[0], l[1]);
}
__device__ __forceinline__ Levels k4_levels(const uint32_t* p) {
  Levels L;
  L.lo_a = __builtin_amdgcn_perm(p[1], p[0], 0x06040200u);
  L.hi_a = __builtin_amdgcn_perm(p[1], p[0], 0x07050301u);
  L.lo_b = __builtin_amdgcn_perm(p[3], p[2], 0x06040200u);
  L.hi_b = __builtin_amdgcn_perm(p[3], p[2], 0x07050301u);
  return L;
}
__device__ __forceinline__ void k4_words(const uint32_t* w, uint32_t* x) {
#pragma unroll
  for (int k = 0; k < 3; ++k) x[k] = ~(w[k] ^ w[3]);
}
// High bytes of quad q
__device__ __forceinline__ uint32_t k4_high(const Levels& L, uint32_t sel, uint32_t w3, int q) {
  return quad_high(L, sel) ^ ((~w3 << (7 - q)) & 0x80808080u);
}
template <bool LO = false>
__device__ __forceinline__ void unpack_word_k4(const uint32_t* w, const float* a, uint32_t* out) {
  uint32_t p[4], x[3], V[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = k4_pair<LO>(a, i);
  const Levels L = k4_levels(p);
  k4_words(w, x);
  word_selectors<3>(x, V);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t sel = quad_selector<3>(V, q >> 2, q & 3);
    quad_pairs(quad_low(L, sel), k4_high(L, sel, w[3], q), out + 2 * q);
  }
}

// Quads 4a .. 4a+3 of a word (16 columns 16a .. 16a+15) as 8 bf16 pairs.
template <int K>
__device__ __forceinline__ void unpack_quads(const uint32_t* V, int a, const Levels& L,
                                             uint32_t* out) {
#pragma unroll
  for (int b = 0; b < 4; ++b) unpack_quad<K>(V, a, b, L, out + 2 * b);
}

template <int K>
__device__ __forceinline__ void unpack_two_quads(const uint32_t* V, int a, int b0, const Levels& L,
                                                 uint32_t* out) {
#pragma unroll
  for (int bb = 0; bb < 2; ++bb) unpack_quad<K>(V, a, b0 + bb, L, out + 2 * bb);
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
