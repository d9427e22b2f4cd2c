// Per-head RMS norm and position rotation of one head row, shared by rc_qk_norm_rope and
// rc_kv_append.
//
// A head row of d elements (d a multiple of 8) is held by L lanes (4, 8 or 16 for d up to 64, 128
// or 256), two 8-element chunks per lane, both kept as fp32. The chunks of a lane are chosen so
// that every rotated pair lies inside one lane and no value crosses lanes but the norm's sum:
//   half-split pairs (e, e + r/2):  lane i < r/16 holds chunks i and i + r/16;
//   interleaved pairs (2e, 2e + 1): lane i holds chunks 2i and 2i + 1;
// either way lane i < r/16 rotates the pairs 8i .. 8i + 7. Chunks past the rotated dims follow two
// by two. A warp's loads of one chunk index are contiguous over its lanes.
#pragma once
#include "device_common.cuh"

namespace rc {

constexpr int kNormRopeMaxDim = 256;

__host__ __device__ constexpr int head_lanes(int d) { return d <= 64 ? 4 : d <= 128 ? 8 : 16; }

// 8 consecutive elements <-> fp32
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  const uint4 w = *(const uint4*)p;
  v[0] = bf16lo(w.x); v[1] = bf16hi(w.x); v[2] = bf16lo(w.y); v[3] = bf16hi(w.y);
  v[4] = bf16lo(w.z); v[5] = bf16hi(w.z); v[6] = bf16lo(w.w); v[7] = bf16hi(w.w);
}
__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = ((const float4*)p)[0], b = ((const float4*)p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *(const uint32_t*)&v;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
  *(uint4*)p = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                          pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  ((float4*)p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  ((float4*)p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// 8 elements as they are stored: one 16-byte chunk of bf16, two of fp32
template <typename T>
struct Raw {
  static constexpr int N = (int)sizeof(T) / 2;
  uint4 v[N];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = ((const uint4*)p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < N; ++i) ((uint4*)p)[i] = v[i];
  }
  __device__ __forceinline__ void get(float* f) const { load8((const T*)v, f); }
  __device__ __forceinline__ void set(const float* f) { store8((T*)v, f); }
};

// The two chunks of lane i in a row of d elements whose first r are rotated; -1: none.
struct LaneChunks {
  int c0, c1;
  bool rot;   // this lane's pairs are rotated
};
__device__ __forceinline__ LaneChunks lane_chunks(int i, int d, int r, bool interleaved) {
  LaneChunks lc;
  const int n = d >> 3, m = r >> 4;
  lc.rot = i < m;
  if (lc.rot && !interleaved) {
    lc.c0 = i;
    lc.c1 = i + m;
  } else {
    lc.c0 = 2 * i;
    lc.c1 = 2 * i + 1;
  }
  if (lc.c0 >= n) lc.c0 = -1;
  if (lc.c1 >= n) lc.c1 = -1;
  return lc;
}

// cos and sin of a lane's 8 pairs: table row = r / 2 cosines, then r / 2 sines
struct LaneAngles {
  float c[8], s[8];
};
__device__ __forceinline__ void load_angles(const float* row, int i, int r, LaneAngles& a) {
  load8(row + 8 * i, a.c);
  load8(row + (r >> 1) + 8 * i, a.s);
}

// rsqrt(mean(x^2) + eps) of a row held as chunks x and y of L lanes. Every lane of the warp calls
// it (the sum crosses lanes); lanes without a chunk hold zeros.
template <int L>
__device__ __forceinline__ float norm_scale(const float* x, const float* y, int d, float eps) {
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
#pragma unroll
  for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  return rsqrtf(__fadd_rn(__fdiv_rn(ss, (float)d), eps));
}

// (a, b) -> (a cos - b sin, b cos + a sin) on a lane's 8 pairs, each as one product and one fused
// multiply-add: written out, so that every kernel rounds alike and a key has the same bits
// whichever entry point rotated it.
__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
  const float p = a, q = b;
  a = __fmaf_rn(p, c, -__fmul_rn(q, s));
  b = __fmaf_rn(q, c, __fmul_rn(p, s));
}
__device__ __forceinline__ void rotate_pairs(float* x, float* y, bool interleaved,
                                             const LaneAngles& a) {
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      rotate_pair(x[2 * e], x[2 * e + 1], a.c[e], a.s[e]);
      rotate_pair(y[2 * e], y[2 * e + 1], a.c[e + 4], a.s[e + 4]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) rotate_pair(x[e], y[e], a.c[e], a.s[e]);
  }
}

// v_e *= scale * w_e
template <typename T>
__device__ __forceinline__ void scale8(float* v, float scale, const T* w) {
  float g[8];
  load8(w, g);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(v[e], __fmul_rn(scale, g[e]));
}

// Streaming multiprocessors of the current device.
int sm_count(const char* fn, int* out);
// Host-side checks shared by the entry points: head_dim, rotation and table.
int check_norm_rope(const char* fn, int head_dim, int rotary_dim, int64_t max_position,
                    const float* rope, float eps, bool any_weight);

}  // namespace rc
