// The 4-bit cache's format. 32 neighbouring elements of a head make a group; with least and greatest
// element lo, hi (differences, quotients and products in fp32, each rounded to nearest)
//   minimum = lo rounded down to bf16
//   scale   = (hi - minimum) / 15 rounded up to four significant bits, at least 2^-80
//   code    = the integer nearest to (x - minimum) * (1 / scale), ties to even: 0 .. 15
// and the element stands for code * scale + minimum, at most half a scale from x and what the three fp32
// roundings add, 45 * 2^-24 of a scale (a code of 15 moves by 15 * 3 half steps). The scale's four bits
// make code * scale exact in bf16, which is what attention feeds the matrix units with; they cost
// at most an eighth of the step, 4 % on average. A group that holds a NaN, an infinity or a magnitude of
// 2^30 and more has NaN as scale and minimum.
// A head's row has d / 2 bytes of codes, element 32 j + 8 t + n in nibble n of the little-endian 32-bit
// word t * d / 32 + j, so that a lane of a matrix instruction finds its elements of every group in
// neighbouring words; then (scale, minimum) of each group, bf16.
#pragma once
#include "device_common.cuh"
#include "warp_mma.cuh"

namespace rc {

constexpr int kKv4MaxDim = 256;
__host__ __device__ constexpr int kv4_row_bytes(int d) { return d / 2 + d / 8; }
// What every head's row starts on, given a plane that does: layers of one tensor may follow one another
// at any number of slots.
constexpr int kv4_align(int d) { return kv4_row_bytes(d) % 16 ? 8 : 16; }

// The least number of four significant bits that is at least x > 0, and 2^-80.
__device__ __forceinline__ float kv4_scale(float x) {
  return fmaxf(__uint_as_float((__float_as_uint(x) + 0xFFFFFu) & ~0xFFFFFu), 0x1p-80f);
}
struct Kv4Group {
  uint32_t pair;   // scale in the low half, minimum in the high half
  float low, inv;
  bool lost;
};
// ROUND: lo may have more bits than bf16. The quotient by 15 is Markstein's: the product with the
// reciprocal, corrected once by its exact remainder (right for all 2^23 significands); the reciprocal of
// four bits a Newton step from the hardware's.
template <bool ROUND>
__device__ __forceinline__ Kv4Group kv4_group(float lo, float hi) {
  Kv4Group g;
  if constexpr (ROUND) {
    const uint32_t u = __float_as_uint(lo);
    g.low = __uint_as_float((lo < 0.f ? u + 0xFFFFu : u) & 0xFFFF0000u) + 0.f;
  } else {
    g.low = lo + 0.f;
  }
  const float width = __fsub_rn(hi, g.low), by15 = 1.f / 15.f;
  const float q = __fmul_rn(width, by15);
  const float scale = kv4_scale(__fmaf_rn(__fmaf_rn(-15.f, q, width), by15, q));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(scale));
  g.inv = __fmaf_rn(__fmaf_rn(-scale, r, 1.f), r, r);
  g.lost = !(lo > -0x1p30f && hi < 0x1p30f);
  g.pair = g.lost ? 0x7FC07FC0u : (__float_as_uint(scale) >> 16) | __float_as_uint(g.low);
  return g;
}
// Eight elements' codes, the first in the lowest nibble. Adding 1.5 * 2^23 rounds to an integer, which the
// number's low bits then hold; the eight are put together with all their bits, whose sum is known.
__device__ __forceinline__ uint32_t kv4_codes(const Kv4Group& g, const float* x) {
  uint32_t w = 0, base = 0;
#pragma unroll
  for (int k = 7; k >= 0; --k) {
    const float t = __fmul_rn(__fsub_rn(x[k], g.low), g.inv);
    w = w * 16 + __float_as_uint(__fadd_rn(t, 12582912.f));
    base = base * 16 + 0x4B400000u;
  }
  return g.lost ? 0u : w - base;
}

}  // namespace rc
