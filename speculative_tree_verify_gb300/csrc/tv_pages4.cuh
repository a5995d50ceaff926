// The cache in 4 bits: where a block of 16 tokens of one head holds what, and
// the rounding of values into codes (tv_pool4 in tv.h).
#pragma once

#include "tv_common.cuh"

namespace tv {

template <int D>
struct Block4 {
  static constexpr int G = D / 32;              // groups of a token, a scale each
  static constexpr int OFF_SCALE = 16 * D / 2;
  static constexpr int BYTES = OFF_SCALE + 16 * G * 2;
  // K: a word of 8 values, dimensions 8 c .. + 7 of token t
  __host__ __device__ static constexpr int k_word(int t, int c) { return t * (D / 2) + (c % 4 * G + c / 4) * 4; }
  // V: a word of 4 values of tokens t and t ^ 1 (the even one in its lower half), dimensions 4 e .. + 3
  __host__ __device__ static constexpr int v_word(int t, int e) {
    return ((t / 8 * 32 + e % 8 * 4 + t % 8 / 2) * G + e / 8) * 4;
  }
  // the word with the scales of tokens t and t ^ 1 of group g
  __host__ __device__ static constexpr int scale(int t, int g) { return OFF_SCALE + ((t / 8 * 4 + t % 8 / 2) * G + g) * 4; }
};

// the scale of the odd or the even token of a word of two
__device__ __forceinline__ float scale_f(uint32_t w, bool odd) { return __uint_as_float(odd ? w & 0xffff0000u : w << 16); }

// 8 values of a group of 32, the others' on the lanes that differ in the two
// lowest bits: the word of their codes, and the group's scale.  All lanes of a
// warp call it.
__device__ __forceinline__ uint32_t round4(const uint4& x, uint32_t& scale) {
  const uint32_t q[4] = {x.x, x.y, x.z, x.w};
  uint32_t top = __vmaxu2(__vmaxu2(q[0] & 0x7fff7fffu, q[1] & 0x7fff7fffu), __vmaxu2(q[2] & 0x7fff7fffu, q[3] & 0x7fff7fffu));
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
  top = max(top & 0xffffu, top >> 16);   // bits of max |x|: what is not finite is above all that is
  // a / 7 is never within 2^-12 of itself of a tie between two bf16 values
  // (7 times one is an odd multiple of the half step, a a whole one), so the
  // product with the reciprocal rounds to the same
  float s = __bfloat162float(__float2bfloat16_rn(__uint_as_float(top << 16) * (1.f / 7.f)));
  if (s < 0x1p-126f) s = 0.f;
  if (top >= 0x7f80u) s = __uint_as_float(0x7fc00000u);
  scale = __float_as_uint(s) >> 16;
  // x / s is a multiple of 2^-10 or so away from a half, or one: 2^-20 more
  // (the reciprocal is right to 2^-23) takes halves away from zero and nothing
  // else across.  The sum with 1.5 * 2^23 + 8 rounds to a whole number, the code
  // its lowest bits.
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  r *= 1.f + 0x1p-20f;
  uint32_t w = 0u;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    w += __float_as_uint(fmaf(__uint_as_float(q[u] << 16), r, 12582920.f)) << (8 * u);
    w += __float_as_uint(fmaf(__uint_as_float(q[u] & 0xffff0000u), r, 12582920.f)) << (8 * u + 4);
  }
  w -= 0x3f400000u;   // what 1.5 * 2^23 left of the sums, shifted left by 0, 4 and 8 bits
  return s > 0.f ? w : 0x88888888u;
}

// The 8 values that a word of codes stands for.  128 + a code is a bf16 value, less
// 136 it is n, and n s is rounded once: two values an instruction.
__device__ __forceinline__ uint4 value4(uint32_t w, float s) {
  const __nv_bfloat162 off = __float2bfloat162_rn(136.f), scale = __float2bfloat162_rn(s);   // (s is a bf16 value)
  uint32_t y[4];   // values u and u + 4
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint32_t x = (w >> (4 * u) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 v = __hmul2_rn(__hsub2_rn(*reinterpret_cast<const __nv_bfloat162*>(&x), off), scale);
    y[u] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(__byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410), __byte_perm(y[0], y[1], 0x7632),
                    __byte_perm(y[2], y[3], 0x7632));
}

}  // namespace tv
