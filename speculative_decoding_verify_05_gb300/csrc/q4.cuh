// The paged cache in 4 bits: a value is a whole number n of -7 .. 7 times the scale of its 32 neighbouring dims of one
// key, an 8-bit float without a sign (5 exponent bits, 3 mantissa bits): byte c stands for
// (1 + (c & 7) / 8) 2^((c >> 3) - 20).  Why whole numbers and not the 4-bit floats (0 .5 1 1.5 2 3 4 6): scaled by
// the maximum of so small a group their even steps fit normal values at least as well (off by 9.8 % in rms, the floats by
// 10.2 %), and two of them leave a word by one logical operation.  The scale needs no second one per tensor: it
// reaches from 2^-20 to 3840, so values of 7e-6 to 26880 keep their precision whatever the tensor's range.
//
// A page holds 128 keys of one kv head in 8704 bytes: 4 planes of 128 rows of 16 bytes (32 entries), then 512 scales.
//   keys    plane q, row k: dims 32 q .. 32 q + 31 of key k;  scale of dims 32 g .. of key k at byte 4 k + g
//   values  plane q, row d: keys 32 q .. 32 q + 31 of dim d;  scale of dims 32 g .. of key k at byte 128 g + k
// Values lie transposed: both products of an attention then contract over what is contiguous in a row (dims in Q K^T,
// keys in P V), so K and V tiles are brought to bf16 by the same code, one row per thread.  Planes, so that 32
// threads with a row each read 512 consecutive bytes.
// A row's 16 bytes are 4 words of 8 entries: n + 8 of entries 0, 2, 4, 6, 1, 3, 5, 7 from the low bits up, so that a shift and
// one logical operation leave two neighbouring entries in the halves of a word.
#pragma once

#include "attention_util.cuh"

namespace spec {

constexpr int Q4_PAGE = 128;             // keys per page
constexpr int Q4_PLANE = 128 * 16;
constexpr int Q4_SCALES = 4 * Q4_PLANE;  // offset of the scales
constexpr int Q4_BYTES = Q4_SCALES + 512;

// Position (in bits) of entry e of 8 in its word.
__host__ __device__ constexpr int q4_shift(int e) { return 4 * ((e >> 1) + 4 * (e & 1)); }

// ----------------------------------------------------------------- to 4 bits
// What is stored hangs on the last bit of what it is rounded from, so the definition fixes every operation: a seventh of
// the group's largest magnitude, rounded to 3 bits behind the leading one, halves to even, is the scale; a value over
// the scale, rounded, and again to a whole number, halves to even, is the entry; both quotients rounded correctly.
struct Q4Scale {
  float scale, reciprocal;
  unsigned code;
};
// Of a finite maximum below Q4_LARGE.  Quotients by Markstein's theorem ("Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990): with the correctly rounded reciprocal of the divisor, one step by the exact remainder
// leaves the correctly rounded quotient (here the divisor has at most 4 bits, so a quotient that is no number of 24 bits lies
// at least a thirtieth of a unit from the middle of two).  The scale's reciprocal is one Newton step (y + y (1 - s y)) from the hardware's
// approximation: 1 - s y is exact (s has 4 bits), and what is rounded is 1 / s off by the square of the approximation's
// error, far less than 1 / s is from the middle of two numbers (s has 8 significands; 1/9 .. 1/15 repeat in at most 12 bits).
// (The division operator's general sequence, per value, made the append of 8192 rows wait for instructions: 48 us.)
constexpr float Q4_LARGE = 26880.f;      // 7 scales of the largest
__device__ __forceinline__ Q4Scale q4_scale(float top) {
  constexpr float seventh = 1.f / 7.f;
  const float q = __fmul_rn(top, seventh), t = __fmaf_rn(__fmaf_rn(-q, 7.f, top), seventh, q);
  unsigned i = __float_as_uint(fmaxf(t, 0x1p-20f));
  i = (i + 0x7FFFFu + ((i >> 20) & 1u)) & 0xFFF00000u;
  Q4Scale d;
  d.code = (i >> 20) - 107u * 8u;
  d.scale = __uint_as_float(i);
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d.scale));
  d.reciprocal = __fmaf_rn(__fmaf_rn(-d.scale, y, 1.f), y, y);
  return d;
}
__device__ __forceinline__ float2 q4_mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
// Whole numbers of two values, each with a scale (which leaves |x| below 7.5 scales; NaN gives 0).
__device__ __forceinline__ int2 q4_whole2(float2 x, float2 scale, float2 reciprocal) {
  const float2 q = q4_mul2(x, reciprocal), r = fma2(make_float2(-q.x, -q.y), scale, x), y = fma2(r, reciprocal, q);
  return make_int2(__float2int_rn(y.x), __float2int_rn(y.y));
}
// Any values, infinities and NaN among them: the entries of 8 values, 4 bits each in order, and the code of the scale that
// they share with the lanes up to `span` apart (a power of two).  Out of line: seldom needed.
static __device__ __noinline__ uint2 q4_any(float4 a, float4 b, int span) {
  const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));       // (NaN is passed over)
  for (int o = 1; o < span; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  unsigned i = __float_as_uint(fminf(fmaxf(__fdiv_rn(top, 7.f), 0x1p-20f), 3840.f));
  i = (i + 0x7FFFFu + ((i >> 20) & 1u)) & 0xFFF00000u;
  uint2 r = make_uint2(0u, (i >> 20) - 107u * 8u);
#pragma unroll 1
  for (int e = 0; e < 8; ++e) {
    const float x = e < 4 ? (e < 2 ? (e ? a.y : a.x) : (e & 1 ? a.w : a.z)) : (e < 6 ? (e & 1 ? b.y : b.x) : (e & 1 ? b.w : b.z));
    r.x |= (unsigned)(min(max(__float2int_rn(__fdiv_rn(x, __uint_as_float(i))), -7), 7) + 8) << (4 * e);
  }
  return r;
}

// ----------------------------------------------------------------- back to bf16
__device__ __forceinline__ uint32_t q4_fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// bf16 bits of the scales of two codes (each in the low byte of a half).
__device__ __forceinline__ uint32_t q4_scale2(uint32_t codes) { return (codes << 4) + ((107u << 7) * 0x10001u); }
// -136 times two scales, exact: 136 = 17 * 8, and 17 times a 4-bit significand has 8 bits.
__device__ __forceinline__ uint32_t q4_offset2(uint32_t scale2) { return q4_fma2(scale2, 0xC308C308u, 0x80008000u); }
// Entries 2 j and 2 j + 1 of a word as bf16: n + 8 in the mantissa of 128 makes 128 + n + 8, and (n + 136) s - 136 s is
// rounded once; n s has 3 + 4 bits, so nothing is lost.
template <int J>
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, uint32_t scale2, uint32_t offset2) {
  return q4_fma2(((w >> (4 * J)) & 0x000F000Fu) | 0x43004300u, scale2, offset2);
}

// The same times 2^-19, for the tensor cores (what comes out of them is scaled anyway), with fewer operations.  The
// bits 0 .. 255 of a bf16 are that many 2^-133 (subnormals, and the first normal numbers in the same steps), so
// entries of the low byte need no shift and no exponent put in: n + 8 or 16 (n + 8) of those steps, times s 2^114 or s
// 2^110, less 8 s 2^-19.  Two of a word's four pairs lie in the low bytes of its halves, the others after one shift by 8.
// (Four shifts and a bit more each: 16 x 1 row at 30000 keys 139 us.)
constexpr float Q4_TILE_SCALE = 0x1p19f;
__device__ __forceinline__ uint32_t q4_even2(uint32_t codes) { return (codes << 4) + (221u << 7) * 0x10001u; }
__device__ __forceinline__ uint32_t q4_odd2(uint32_t codes) { return (codes << 4) + (217u << 7) * 0x10001u; }
__device__ __forceinline__ uint32_t q4_less2(uint32_t codes) { return (codes << 4) + ((91u << 7) | 0x8000u) * 0x10001u; }
// J: the pair; by: q4_even2 or q4_odd2 of the pair's two scales for an even or odd J.
template <int J>
__device__ __forceinline__ uint32_t q4_tile_pair(uint32_t w, uint32_t w8, uint32_t by, uint32_t less) {
  return q4_fma2((J & 2 ? w8 : w) & (J & 1 ? 0x00F000F0u : 0x000F000Fu), by, less);
}

}  // namespace spec
