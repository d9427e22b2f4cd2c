// The 4-bit cache's format. 32 neighbouring elements of a head make a group; with least and greatest
// element lo, hi (differences, quotients and products in fp32, each rounded to nearest)
//   minimum = lo rounded down to bf16
//   scale   = (hi - minimum) / 15 rounded up to four significant bits, at least 2^-80
//   code    = the integer nearest to (x - minimum) * (1 / scale), ties to even: 0 .. 15
// and the element stands for code * scale + minimum, at most half a scale from x. The scale's four bits
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

struct Kv4Group {
  uint32_t pair;   // scale in the low half, minimum in the high half
  float low, inv;
  bool lost;
};
__device__ __forceinline__ Kv4Group kv4_group(float lo, float hi) {
  Kv4Group g;
  const uint32_t u = __float_as_uint(lo);
  g.low = __uint_as_float((lo < 0.f ? u + 0xFFFFu : u) & 0xFFFF0000u) + 0.f;
  const float step = __fdiv_rn(__fsub_rn(hi, g.low), 15.f);
  const float scale =
      fmaxf(__uint_as_float((__float_as_uint(step) + 0xFFFFFu) & ~0xFFFFFu), 0x1p-80f);
  g.inv = __frcp_rn(scale);
  g.lost = !(lo > -0x1p30f && hi < 0x1p30f);
  g.pair = g.lost ? 0x7FC07FC0u : (__float_as_uint(scale) >> 16) | __float_as_uint(g.low);
  return g;
}
// x's code, in the low bits of a number of 24 bits
__device__ __forceinline__ uint32_t kv4_code(const Kv4Group& g, float x) {
  return __float_as_uint(
             __fadd_rn(__fmul_rn(__fsub_rn(x, g.low), g.inv), 12582912.f)) & 15u;
}

}  // namespace rc
