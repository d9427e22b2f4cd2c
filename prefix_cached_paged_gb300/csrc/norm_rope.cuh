// Per-head RMS norm and position rotation of one head row, shared by rc_qk_norm_rope and
// rc_kv_append.
//
// A head row of d elements (d a multiple of 8) is held by L lanes (4, 8 or 16 for d up to 64, 128
// or 256), two 8-element chunks per lane, both kept as fp32. The chunks of a lane are chosen so
// that every rotated pair lies inside one lane and no value crosses lanes but the norm's sum:
//   half-split pairs (e, e + r/2):  lane i < r/16 holds chunks i and i + r/16;
//   interleaved pairs (2e, 2e + 1): lane i holds chunks 2i and 2i + 1;
// either way lane i < r/16 rotates the pairs 8i .. 8i + 7. Chunks past the rotated dims follow two
// by two. Where pairs are half-split, a warp's loads of one chunk index are contiguous over the lanes
// that rotate; elsewhere they take every second chunk, and the other index takes the rest.
#pragma once
#include "device_common.cuh"
#include "warp_mma.cuh"

namespace rc {

constexpr int kNormRopeMaxDim = 256;

__host__ __device__ constexpr int head_lanes(int d) { return d <= 64 ? 4 : d <= 128 ? 8 : 16; }

// Two fp32 numbers in one register pair, with the packed instructions of sm_100 and later (each
// half rounds as the scalar instruction does).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 swap2(f32x2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return pack2(hi, lo);
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
  // as four pairs of fp32, and back (rounded to nearest)
  __device__ __forceinline__ void get(f32x2 (&f)[4]) const {
    const uint32_t* w = (const uint32_t*)v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2)
        f[i] = pack2(bf16lo(w[i]), bf16hi(w[i]));
      else
        f[i] = pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
  }
  __device__ __forceinline__ void set(const f32x2 (&f)[4]) {
    uint32_t* w = (uint32_t*)v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      unpack2(f[i], lo, hi);
      if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        w[i] = *(const uint32_t*)&b;
      } else {
        w[2 * i] = __float_as_uint(lo);
        w[2 * i + 1] = __float_as_uint(hi);
      }
    }
  }
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

// cos and sin of a lane's 8 pairs, two pairs per register pair (a table row is r / 2 cosines, then
// r / 2 sines)
struct LaneAngles {
  f32x2 c[4], s[4];
  __device__ __forceinline__ void load(const float* row, int i, int r) {
    const ulonglong2* pc = (const ulonglong2*)(row + 8 * i);
    const ulonglong2* ps = (const ulonglong2*)(row + (r >> 1) + 8 * i);
    const ulonglong2 c0 = pc[0], c1 = pc[1], s0 = ps[0], s1 = ps[1];
    c[0] = c0.x; c[1] = c0.y; c[2] = c1.x; c[3] = c1.y;
    s[0] = s0.x; s[1] = s0.y; s[2] = s1.x; s[3] = s1.y;
  }
};

// A lane's 16 elements of a row: chunks c0 (x) and c1 (y); zeros where it has none.
struct LaneRow {
  f32x2 x[4], y[4];

  // rsqrt(mean(x^2) + eps) of the row held by L lanes. Every lane of the warp calls it.
  template <int L>
  __device__ __forceinline__ float norm_scale(int d, float eps) const {
    f32x2 acc = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc = fma2(x[e], x[e], acc);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc = fma2(y[e], y[e], acc);
    float lo, hi;
    unpack2(acc, lo, hi);
    float ss = __fadd_rn(lo, hi);
#pragma unroll
    for (int o = 1; o < L; o <<= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
    return rsqrtf(__fadd_rn(__fdiv_rn(ss, (float)d), eps));
  }
  // times scale * w, w the weights of the lane's elements
  __device__ __forceinline__ void scale(float scale, const LaneRow& w) {
    const f32x2 s2 = pack2(scale, scale);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = mul2(x[e], mul2(s2, w.x[e]));
      y[e] = mul2(y[e], mul2(s2, w.y[e]));
    }
  }
  // (a, b) -> (a cos - b sin, b cos + a sin), each one product and one fused multiply-add, so a key
  // has the same bits whichever entry point rotated it
  __device__ __forceinline__ void rotate(const LaneAngles& a, bool interleaved) {
    if (interleaved) {   // pair e is one register pair
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float c0, c1, s0, s1;
        unpack2(a.c[e], c0, c1);
        unpack2(a.s[e], s0, s1);
        f32x2& u = e < 2 ? x[2 * e] : y[2 * e - 4];
        f32x2& v = e < 2 ? x[2 * e + 1] : y[2 * e - 3];
        u = fma2(u, pack2(c0, c0), mul2(swap2(u), pack2(-s0, s0)));
        v = fma2(v, pack2(c1, c1), mul2(swap2(v), pack2(-s1, s1)));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f32x2 p = x[e];
        x[e] = fma2(p, a.c[e], mul2(y[e], a.s[e] ^ 0x8000000080000000ull));
        y[e] = fma2(y[e], a.c[e], mul2(p, a.s[e]));
      }
    }
  }
};

// A lane's weights (zeros where it has no chunk).
template <typename T>
__device__ __forceinline__ void load_weights(const T* w, const LaneChunks& lc, LaneRow& out) {
  Raw<T> a, b;
  a.clear();
  b.clear();
  if (lc.c0 >= 0) a.load(w + lc.c0 * 8);
  if (lc.c1 >= 0) b.load(w + lc.c1 * 8);
  a.get(out.x);
  b.get(out.y);
}

// The same operations on single registers, for a kernel that has none to spare for pairs: every
// product, sum and their order are those of LaneRow, so the results have the same bits.
struct ScalarRow {
  float x[8], y[8];

  template <typename T>
  __device__ __forceinline__ void get(const Raw<T>& a, const Raw<T>& b) {
    const uint32_t *u = (const uint32_t*)a.v, *v = (const uint32_t*)b.v;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 2) {
        x[i] = i & 1 ? bf16hi(u[i / 2]) : bf16lo(u[i / 2]);
        y[i] = i & 1 ? bf16hi(v[i / 2]) : bf16lo(v[i / 2]);
      } else {
        x[i] = __uint_as_float(u[i]);
        y[i] = __uint_as_float(v[i]);
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ void set(Raw<T>& a, Raw<T>& b) const {
    uint32_t *u = (uint32_t*)a.v, *v = (uint32_t*)b.v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        u[i] = pack2_bf16(x[2 * i], x[2 * i + 1]);
        v[i] = pack2_bf16(y[2 * i], y[2 * i + 1]);
      } else {
        u[2 * i] = __float_as_uint(x[2 * i]);
        u[2 * i + 1] = __float_as_uint(x[2 * i + 1]);
        v[2 * i] = __float_as_uint(y[2 * i]);
        v[2 * i + 1] = __float_as_uint(y[2 * i + 1]);
      }
    }
  }
  template <int L>
  __device__ __forceinline__ float norm_scale(int d, float eps) const {
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      lo = __fmaf_rn(x[e], x[e], lo);
      hi = __fmaf_rn(x[e + 1], x[e + 1], hi);
    }
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      lo = __fmaf_rn(y[e], y[e], lo);
      hi = __fmaf_rn(y[e + 1], y[e + 1], hi);
    }
    float ss = __fadd_rn(lo, hi);
#pragma unroll
    for (int o = 1; o < L; o <<= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
    return rsqrtf(__fadd_rn(__fdiv_rn(ss, (float)d), eps));
  }
  template <typename T>
  __device__ __forceinline__ static void scale8(float* v, float s, const T* w) {
    Raw<T> raw;
    raw.load(w);
    const uint32_t* u = (const uint32_t*)raw.v;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float g;
      if constexpr (sizeof(T) == 2)
        g = i & 1 ? bf16hi(u[i / 2]) : bf16lo(u[i / 2]);
      else
        g = __uint_as_float(u[i]);
      v[i] = __fmul_rn(v[i], __fmul_rn(s, g));
    }
  }
  template <typename T>
  __device__ __forceinline__ void scale(float s, const T* w, const LaneChunks& lc) {
    if (lc.c0 >= 0) scale8(x, s, w + lc.c0 * 8);
    if (lc.c1 >= 0) scale8(y, s, w + lc.c1 * 8);
  }
  __device__ __forceinline__ static void rotate_pair(float& a, float& b, float c, float s) {
    const float p = a, q = b;
    a = __fmaf_rn(p, c, -__fmul_rn(q, s));
    b = __fmaf_rn(q, c, __fmul_rn(p, s));
  }
  // c, s: the lane's 8 cosines and sines
  __device__ __forceinline__ void rotate(const float* c, const float* s, bool interleaved) {
    if (interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        rotate_pair(x[2 * e], x[2 * e + 1], c[e], s[e]);
        rotate_pair(y[2 * e], y[2 * e + 1], c[e + 4], s[e + 4]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) rotate_pair(x[e], y[e], c[e], s[e]);
    }
  }
};

// Streaming multiprocessors of the current device.
int sm_count(const char* fn, int* out);
// Host-side checks shared by the entry points: head_dim, rotation and table.
int check_norm_rope(const char* fn, int head_dim, int rotary_dim, int64_t max_position,
                    const float* rope, float eps, bool any_weight);

}  // namespace rc
