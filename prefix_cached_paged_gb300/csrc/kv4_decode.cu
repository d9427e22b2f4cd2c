// Decode attention over the cache held in 4 bits (format: kv4.cuh).
//
// score(q, k) = sum_j [ s_j sum_{e in j} q_e c_e + m_j sum_{e in j} q_e ],   o = sum_t p_t (s_tj c_te + m_tj)
// with the codes c, scales s and minima m of each group j: nothing is dequantised on the way. The work
// is bound by HBM on paper (160 bytes of a token and KV head of 128, 16 tokens x 8 query heads
// on one matrix instruction) and by instruction issue next to it: an SM has 23 bytes a clock of HBM and
// so about 3.5 instruction lanes for each code.
//
// Work split: the steps of all (row, group of KV heads) pairs in one line, cut into as many equal ranges as
// CTAs fit on the GPU at once, so long and short rows share them evenly; states of a pair that
// ranges cut are joined by a second kernel, in the order of their tokens. In a CTA a warp takes one KV
// head, so that neighbouring heads of a slot are read at the same time (their rows do not end on
// sectors), and with few KV heads several warps share a head's tokens. A warp works alone on its ring
// of cp.async stages of 32 tokens.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "host_common.h"
#include "kv4.cuh"
#include "norm_rope.cuh"

namespace rc {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxGroup = 16;
constexpr int kMaxCtas = 304;   // two for each of 152 SMs
constexpr int kTile = 32;       // tokens of a stage

struct Range {     // of one CTA: the pairs it shares with others, -1: none
  int row0, hg0, start0, last0;   // begun before it: first and last CTA
  int row1, hg1, last1;           // begun in it and not ended
  int pad;
};
struct Workspace {
  Range* range;   // [ctas]
  float* ml;      // [ctas][2][heads of a group of KV heads][2]: maximum (base 2), sum
  float* o;       // [ctas][2][heads of a group][d]
};
struct Params {
  rc_kv4_decode_args a;
  Workspace w;
  int* status;
  int G;          // query heads of a KV head
  int HG, TS;     // KV heads of a CTA, warps that share a head's tokens
  int groups;     // KV heads / HG
  int min_steps;  // of a CTA
};

template <typename T, int D, int NT>
struct Cfg {
  static constexpr int NG = D / 32, RB = kv4_row_bytes(D);
  static constexpr int CH = 4 * NG;          // bytes of a chunk: what a lane reads of a token's codes
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int QP = F32 ? 3 : 1;     // bf16 parts of a query element
  static constexpr int PP = F32 ? 3 : 2;     // of a weight
  static constexpr int PER_SM = F32 || NT > 1 ? 1 : 2;
  static constexpr int STAGES = PER_SM == 1 ? 4 : 2;
  // a stage: codes of K, (scale, minimum) of K in rows of 16 bytes, the same of V
  static constexpr int PAR = kTile * 4 * CH, VAL = PAR + kTile * 16, STAGE = 2 * VAL;
  static constexpr int WARP = STAGES * STAGE, SMEM = kWarps * WARP;
  static_assert(STAGE >= 8 * (D + 2) * 4, "a stage holds the state of 8 heads");
};

// chunk c of row r of a stage's codes lies at c ^ swizzle(r): conflict-free for K (8 rows x 4 chunks)
// and V (rows 2t, chunk g / 2)
template <int NG>
__device__ __forceinline__ int swizzle(int r) {
  return NG == 4 ? r >> 1 & 3 : (r >> 2 & 1) << 1;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  return __byte_perm(a, b, sel);
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void ldmatrix_x2_trans(uint32_t addr, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];"
               : "=r"(r0), "=r"(r1) : "r"(addr) : "memory");
}
template <int N>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&r)[N]) {
  static_assert(N == 2 || N == 4, "");
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
  else
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t lds1(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
  return r;
}
// the upper and lower halves' next bf16 part: packs and leaves the rest
__device__ __forceinline__ uint32_t take_part(float& lo, float& hi) {
  const uint32_t p = pack2_bf16(lo, hi);
  lo -= bf16lo(p);
  hi -= bf16hi(p);
  return p;
}

__device__ __forceinline__ int steps_of(const Params& p, int len, int req) {
  if (len <= 0 || len > p.a.max_seq_len || req < 0 || req >= p.a.max_reqs) return 0;
  return (len + kTile * p.TS - 1) / (kTile * p.TS);
}

// How the line of steps is cut: range c is [total c / ctas, total (c + 1) / ctas).
struct Cut {
  int64_t total;
  int ctas;
  __device__ int64_t begin(int c) const { return total * c / ctas; }
  __device__ int of(int64_t x) const { return (int)(((x + 1) * ctas - 1) / total); }
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, (Cfg<T, D, NT>::PER_SM))
kv4_decode_kernel(const __grid_constant__ Params p) {
  using C = Cfg<T, D, NT>;
  constexpr int NG = C::NG, QP = C::QP, PP = C::PP, S = C::STAGES;
  extern __shared__ __align__(16) char smem[];
  __shared__ int64_t s_sum[kWarps];
  __shared__ int64_t s_before;
  __shared__ int s_row;
  __shared__ uint4 s_meta[kWarps][S];
  const auto& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;

  // ---- the CTA's range: a scan of all rows' steps
  const int each = (a.num_rows + kThreads - 1) / kThreads;
  const int r0 = min(a.num_rows, (int)threadIdx.x * each), r1 = min(a.num_rows, r0 + each);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) mine += steps_of(p, a.seq_len[r], a.req_idx[r]);
  int64_t upto = mine;
#pragma unroll
  for (int x = 1; x < 32; x *= 2) {
    const int64_t y = __shfl_up_sync(~0u, upto, x);
    if (lane >= x) upto += y;
  }
  if (lane == 31) s_sum[warp] = upto;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) upto += total;
    total += s_sum[w];
  }
  Cut cut;
  cut.total = total * p.groups;
  cut.ctas = (int)min((int64_t)gridDim.x, max((int64_t)1, cut.total / p.min_steps));
  const bool idle = (int)blockIdx.x >= cut.ctas || total == 0;
  const int64_t begin = idle ? 0 : cut.begin(blockIdx.x);
  const int64_t end = idle ? 0 : cut.begin(blockIdx.x + 1);
  if (!idle) {
    const int64_t at = begin / p.groups;
    if (at >= upto - mine && at < upto) {
      int64_t before = upto - mine;
      int r = r0;
      for (; r + 1 < r1; ++r) {
        const int n = steps_of(p, a.seq_len[r], a.req_idx[r]);
        if (at < before + n) break;
        before += n;
      }
      s_row = r;
      s_before = before * p.groups;
    }
  }
  // rows without a token
  for (int r = blockIdx.x; r < a.num_rows; r += gridDim.x) {
    const int len = a.seq_len[r];
    if (steps_of(p, len, a.req_idx[r])) continue;
    if (len != 0 && threadIdx.x == 0) set_status(p.status, kStatusPosRange);
    for (int x = threadIdx.x; x < a.num_q_heads * D; x += kThreads)
      ((T*)a.o)[(int64_t)r * a.num_q_heads * D + x] = Elem<T>::from_f(0.f);
    if (a.lse)
      for (int x = threadIdx.x; x < a.num_q_heads; x += kThreads)
        a.lse[(int64_t)r * a.num_q_heads + x] = -INFINITY;
  }
  // the unused half of the rows of (scale, minimum) takes part in matrix products
  const uint32_t ring = smem_u32(smem) + warp * C::WARP;
  if (NG == 2)
    for (int s = 0; s < S; ++s)
      for (int v = 0; v < 2; ++v)
        *(uint2*)(smem + warp * C::WARP + s * C::STAGE + v * C::VAL + C::PAR + lane * 16 + 8) =
            make_uint2(0, 0);
  __syncthreads();
  if (threadIdx.x == 0) {
    Range rg = {-1, 0, 0, 0, -1, 0, 0, 0};
    if (!idle) {
      int r = s_row;
      const int n = max(1, steps_of(p, a.seq_len[r], a.req_idx[r]));
      const int64_t at = s_before + (begin - s_before) / n * n;   // first step of the pair
      if (at < begin) {
        rg.row0 = r;
        rg.hg0 = (int)((at - s_before) / n);
        rg.start0 = cut.of(at);
        rg.last0 = cut.of(at + n - 1);
      }
    }
    p.w.range[blockIdx.x] = rg;   // row1 follows where the pair is met
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int hw = warp % p.HG, ts = warp / p.HG;
  if (idle || ts >= p.TS) return;

  // ---- the producer's place: pair (row, hg), step of it
  const int64_t stride = (int64_t)a.num_kv_heads * C::RB;
  int row = s_row, req = a.req_idx[row], len = a.seq_len[row], steps = max(1, steps_of(p, len, req));
  int hg = min(p.groups - 1, (int)((begin - s_before) / steps)), step = (int)((begin - s_before) % steps);
  int64_t left = end - begin;   // steps to issue
  const int64_t count = left;
  int len1 = 0, req1 = 0;       // of the next row
  auto peek = [&] {
    if (row + 1 < a.num_rows) len1 = a.seq_len[row + 1], req1 = a.req_idx[row + 1];
  };
  peek();
  bool opened = true;           // first step of a pair in this CTA
  int slot = 0;
  auto load_slots = [&] {
    const int pos = (step * p.TS + ts) * kTile + lane;
    slot = pos < len ? a.req_to_token[(int64_t)req * a.max_ctx + pos] : 0;
  };
  // where the lane's 5 of a stage's 160 chunks (5 of a token: four of codes, (scale, minimum)) lie
  int from[5], dst[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const int tok = (i * 32 + lane) / 5, c = (i * 32 + lane) % 5;
    from[i] = tok | c << 8;
    dst[i] = c < 4 ? tok * 4 * C::CH + (c ^ swizzle<NG>(tok)) * C::CH : C::PAR + tok * 16;
  }
  auto issue = [&](int stage) {
    if (left > 0) {
      const int n = len - (step * p.TS + ts) * kTile;
      const bool ok = lane < n && slot >= 0 && slot < a.num_slots;
      if (lane < n && !ok) set_status(p.status, kStatusSlotRange);
      const uint32_t live = __ballot_sync(~0u, ok);
      const char* kb = (const char*)a.k_pool + (int64_t)(hg * p.HG + hw) * C::RB;
      const char* vb = (const char*)a.v_pool + (int64_t)(hg * p.HG + hw) * C::RB;
      const uint32_t base = ring + stage * C::STAGE;
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        const int tok = from[i] & 255;
        const bool in = live >> tok & 1;
        const int s = __shfl_sync(~0u, slot, tok);
        const int64_t off = in ? s * stride + (from[i] >> 8) * C::CH : 0;
        cp_async_or_zero<C::CH>(base + dst[i], kb + off, in);
        cp_async_or_zero<C::CH>(base + C::VAL + dst[i], vb + off, in);
      }
      --left;
      const bool ends = step + 1 == steps;
      if (lane == 0)
        s_meta[warp][stage] = make_uint4(row, hg << 4 | (opened ? 1 : 0) | (ends || left == 0 ? 2 : 0) |
                                                  (ends ? 4 : 0) | (step == 0 ? 8 : 0),
                                         live, steps);
      opened = ends;
      if (!ends) {
        ++step;
      } else if (left > 0) {
        step = 0;
        if (++hg == p.groups) {
          hg = 0;
          do {
            ++row, len = len1, req = req1;
            steps = steps_of(p, len, req);
            peek();
          } while (steps == 0 && row + 1 < a.num_rows);
        }
      }
      if (left > 0) load_slots();
    }
    cp_async_commit();
  };

  // ---- the consumer's state of one pair: queries, maxima and sums, outputs
  uint32_t qf[QP][NT][NG][2][2];   // query elements of the matrix steps of each group
  uint32_t qm[NT][3];              // sums of a group's query elements, in three bf16 parts
  float F[NT][2], mx[NT][2], l[NT][2];
  float O[NT][NG][2][4], M[NT][4];
  int whole = 0;                   // the pair began in this CTA
  int64_t first = 0;               // its first step here

  auto begin_pair = [&](int row, int h) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int qh = nt * 8 + g;
      float x[NG][8], most = 0.f;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
#pragma unroll
        for (int n = 0; n < 8; ++n) x[j][n] = 0.f;
        if (qh < p.G) {
          const T* src = (const T*)a.q + ((int64_t)row * a.num_q_heads + h * p.G + qh) * D + 32 * j +
                         8 * t;
          if constexpr (C::F32) {
            const float4 u = ((const float4*)src)[0], v = ((const float4*)src)[1];
            x[j][0] = u.x, x[j][1] = u.y, x[j][2] = u.z, x[j][3] = u.w;
            x[j][4] = v.x, x[j][5] = v.y, x[j][6] = v.z, x[j][7] = v.w;
          } else {
            const uint4 u = *(const uint4*)src;
            x[j][0] = bf16lo(u.x), x[j][1] = bf16hi(u.x), x[j][2] = bf16lo(u.y), x[j][3] = bf16hi(u.y);
            x[j][4] = bf16lo(u.z), x[j][5] = bf16hi(u.z), x[j][6] = bf16lo(u.w), x[j][7] = bf16hi(u.w);
          }
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) most = fmaxf(most, fabsf(x[j][n]));
      }
      most = fmaxf(most, __shfl_xor_sync(~0u, most, 1));
      most = fmaxf(most, __shfl_xor_sync(~0u, most, 2));
      // the head's elements over 2^e, below 4 in magnitude: a power of two, exact. A code's pattern
      // is the bf16 number code * 2^-133 (or 16 times that), subnormal or next to it, which times
      // an element * 2^125 is code * element * 2^-8
      const int e = min(max((int)(__float_as_uint(most) >> 23) - 127, -100), 126);
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        float s = 0.f;
#pragma unroll
        for (int n = 0; n < 8; ++n) x[j][n] *= down, s += x[j][n];
        s += __shfl_xor_sync(~0u, s, 1);
        s += __shfl_xor_sync(~0u, s, 2);
        if (t == j) sum = s;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float up = b ? 0x1p121f : 0x1p125f;
            float lo = x[j][2 * k + b] * up, hi = x[j][2 * k + b + 4] * up;
#pragma unroll
            for (int q = 0; q < QP; ++q) qf[q][nt][j][k][b] = take_part(lo, hi);
          }
      }
      float none = 0.f;
      sum *= 0x1p-8f;
#pragma unroll
      for (int k = 0; k < 3; ++k) qm[nt][k] = take_part(none, sum);
      const float f = a.sm_scale * (kLog2e * 256.f) * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        F[nt][k] = __shfl_sync(~0u, f, (2 * t + k) * 4);
        mx[nt][k] = -FLT_MAX, l[nt][k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        M[nt][k] = 0.f;
#pragma unroll
        for (int j = 0; j < NG; ++j) O[nt][j][0][k] = O[nt][j][1][k] = 0.f;
      }
    }
  };

  // scores of 16 tokens (rows 16 u ..): x[nt] = tokens g, g + 8 x heads 2t, 2t + 1
  auto scores = [&](uint32_t st, int u, float (&x)[NT][4]) {
    const int r = u * 16 + g;
    const uint32_t at = st + r * 4 * C::CH + (t ^ swizzle<NG>(r)) * C::CH;
    const uint32_t par = st + C::PAR + r * 16;
    uint32_t wa[NG], wb[NG], pa[NG], pb[NG];
    lds(at, wa);
    lds(at + 32 * C::CH, wb);
    lds(par, pa);
    lds(par + 128, pb);
    const uint32_t ma = lds1(par + 4 * t), mb = lds1(par + 128 + 4 * t);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
      mma_bf16(x[nt], ma, mb, ma, mb, qm[nt][0], qm[nt][1]);
      mma_bf16(x[nt], ma, mb, 0, 0, qm[nt][2], 0);
    }
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      float d[NT][4] = {};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t va = wa[j] >> 8 * k, vb = wb[j] >> 8 * k;
        const uint32_t a0 = va & 0x000F000Fu, a1 = vb & 0x000F000Fu;
        const uint32_t a2 = va & 0x00F000F0u, a3 = vb & 0x00F000F0u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int q = 0; q < QP; ++q)
            mma_bf16(d[nt], a0, a1, a2, a3, qf[q][nt][j][k][0], qf[q][nt][j][k][1]);
      }
      const float sa = bf16lo(pa[j]), sb = bf16lo(pb[j]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        x[nt][0] = fmaf(sa, d[nt][0], x[nt][0]);
        x[nt][1] = fmaf(sa, d[nt][1], x[nt][1]);
        x[nt][2] = fmaf(sb, d[nt][2], x[nt][2]);
        x[nt][3] = fmaf(sb, d[nt][3], x[nt][3]);
      }
    }
  };

  // outputs += weights x of 16 tokens times their values
  auto values = [&](uint32_t st, int u, float (&x)[NT][4]) {
    uint32_t b[NT][PP][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < PP; ++k) {
        b[nt][k][0] = movmatrix_trans(take_part(x[nt][0], x[nt][1]));
        b[nt][k][1] = movmatrix_trans(take_part(x[nt][2], x[nt][3]));
      }
    const int r = u * 16 + 2 * t;
    const uint32_t at = st + C::VAL + r * 4 * C::CH + ((g >> 1) ^ swizzle<NG>(r)) * C::CH;
    const uint32_t par = st + C::VAL + C::PAR + u * 256;
    uint32_t m0, m1;
    ldmatrix_x2_trans(par + (lane & 15) * 16, m0, m1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < PP; ++k) mma_bf16(M[nt], m0, 0, m1, 0, b[nt][k][0], b[nt][k][1]);
    uint32_t w0[NG], w1[NG], w2[NG], w3[NG], s01[NG], s23[NG];
    {
      uint32_t q0[NG], q1[NG];
      lds(par + 2 * t * 16, q0);
      lds(par + 2 * t * 16 + 16, q1);
#pragma unroll
      for (int j = 0; j < NG; ++j) s01[j] = mul2(prmt(q0[j], q1[j], 0x5410), 0x6F806F80u);   // 2^96
      lds(par + 2 * t * 16 + 128, q0);
      lds(par + 2 * t * 16 + 144, q1);
#pragma unroll
      for (int j = 0; j < NG; ++j) s23[j] = mul2(prmt(q0[j], q1[j], 0x5410), 0x6F806F80u);
    }
    lds(at, w0);
    lds(at + 4 * C::CH, w1);
    lds(at + 32 * C::CH, w2);
    lds(at + 36 * C::CH, w3);
    const uint32_t half = g & 1 ? 0x7632 : 0x5410;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const uint32_t v01 = prmt(w0[j], w1[j], half), v23 = prmt(w2[j], w3[j], half);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // code * 2^-133 (16 times that) times scale * 2^96: eight bits, exact
        const uint32_t va = v01 >> 8 * k, vb = v23 >> 8 * k;
        const uint32_t a0 = mul2(va & 0x000F000Fu, s01[j]), a1 = mul2(va & 0x00F000F0u, s01[j]);
        const uint32_t a2 = mul2(vb & 0x000F000Fu, s23[j]), a3 = mul2(vb & 0x00F000F0u, s23[j]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (C::F32) {   // sums in fp32, since a matrix instruction cuts its sums off
            float d[4] = {};
#pragma unroll
            for (int q = 0; q < PP; ++q) mma_bf16(d, a0, a1, a2, a3, b[nt][q][0], b[nt][q][1]);
#pragma unroll
            for (int q = 0; q < 4; ++q) O[nt][j][k][q] += d[q];
          } else {
#pragma unroll
            for (int q = 0; q < PP; ++q)
              mma_bf16(O[nt][j][k], a0, a1, a2, a3, b[nt][q][0], b[nt][q][1]);
          }
        }
      }
    }
  };

  // the state of head 2t + c of tile nt: dims 32 j + 4 g .. + 3
  auto outputs = [&](int nt, int c, int j, float4& v) {
    const float m = __shfl_sync(~0u, M[nt][c], (2 * j + 1) * 4 + t);
    v.x = fmaf(O[nt][j][0][c], 0x1p37f, m);
    v.y = fmaf(O[nt][j][0][2 + c], 0x1p33f, m);
    v.z = fmaf(O[nt][j][1][c], 0x1p37f, m);
    v.w = fmaf(O[nt][j][1][2 + c], 0x1p33f, m);
  };
  // what a pair's head gave: the outputs, or a state in the workspace
  auto store = [&](int row, int hg, int flags, int qh, int d, float4 v, float m, float den) {
    const int64_t head = (int64_t)row * a.num_q_heads + (hg * p.HG + hw) * p.G + qh;
    if (whole && (flags & 4)) {
      const float f = den == 0.f ? 0.f : 1.f / den;
      T* o = (T*)a.o + head * D + d;
      if constexpr (C::F32)
        *(float4*)o = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
      else
        *(uint2*)o = make_uint2(pack2_bf16(v.x * f, v.y * f), pack2_bf16(v.z * f, v.w * f));
      if (a.lse && d == 0) a.lse[head] = den == 0.f ? -INFINITY : kLn2 * (m + log2f(den));
    } else {
      const int64_t at = (((int64_t)blockIdx.x * 2 + (whole ? 1 : 0)) * p.HG + hw) * p.G + qh;
      *(float4*)(p.w.o + at * D + d) = v;
      if (d == 0) *(float2*)(p.w.ml + at * 2) = make_float2(m, den);
    }
  };
  auto end_pair = [&](int row, int hg, int flags, int steps, int stage) {
    if (warp == 0 && lane == 0 && whole && !(flags & 4)) {
      Range* rg = p.w.range + blockIdx.x;
      rg->row1 = row, rg->hg1 = hg, rg->last1 = cut.of(begin + first + steps - 1);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int x = 4; x < 32; x *= 2) l[nt][c] += __shfl_xor_sync(~0u, l[nt][c], x);
      if (p.TS == 1) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < NG; ++j) {
            float4 v;
            outputs(nt, c, j, v);
            const int qh = nt * 8 + 2 * t + c;
            if (qh < p.G) store(row, hg, flags, qh, 32 * j + 4 * g, v, mx[nt][c], l[nt][c]);
          }
        continue;
      }
      // warps that share a head join their states through the stage that each has just read
      float* own = (float*)(smem + warp * C::WARP + stage * C::STAGE);
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          float4 v;
          outputs(nt, c, j, v);
          *(float4*)(own + (2 * t + c) * D + 32 * j + 4 * g) = v;
        }
        if (g == 0) own[8 * D + 2 * t + c] = mx[nt][c], own[8 * D + 8 + 2 * t + c] = l[nt][c];
      }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + hw), "r"(32 * p.TS) : "memory");
      const int heads = min(8, p.G - nt * 8);
      for (int x = ts * 32 + lane; x < heads * (D / 4); x += 32 * p.TS) {
        const int qh = x / (D / 4), d = x % (D / 4) * 4;
        float m = -FLT_MAX, den = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < p.TS; ++s)
          m = fmaxf(m, ((const float*)(smem + (s * p.HG + hw) * C::WARP + stage * C::STAGE))[8 * D + qh]);
        for (int s = 0; s < p.TS; ++s) {
          const float* other = (const float*)(smem + (s * p.HG + hw) * C::WARP + stage * C::STAGE);
          const float f = ex2(other[8 * D + qh] - m);
          const float4 w = *(const float4*)(other + qh * D + d);
          den = fmaf(f, other[8 * D + 8 + qh], den);
          v.x = fmaf(f, w.x, v.x), v.y = fmaf(f, w.y, v.y);
          v.z = fmaf(f, w.z, v.z), v.w = fmaf(f, w.w, v.w);
        }
        store(row, hg, flags, nt * 8 + qh, d, v, m, den);
      }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + hw), "r"(32 * p.TS) : "memory");
    }
    // the copies that come next write what the joins read and wrote; (scale, minimum) rows of two
    // groups keep their zeros
    if (NG == 2 && p.TS > 1) {
#pragma unroll
      for (int v = 0; v < 2; ++v)
        *(uint2*)(smem + warp * C::WARP + stage * C::STAGE + v * C::VAL + C::PAR + lane * 16 + 8) =
            make_uint2(0, 0);
      __syncwarp();
    }
  };

  load_slots();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(i);
  int stage = 0;
  for (int64_t i = 0; i < count; ++i) {
    issue(stage == 0 ? S - 1 : stage - 1);
    cp_async_wait<S - 1>();
    __syncwarp();
    const uint4 meta = s_meta[warp][stage];
    const int flags = meta.y & 15, pair = (int)meta.y >> 4;
    if (flags & 1) {
      whole = flags & 8;
      first = i;
      begin_pair((int)meta.x, pair * p.HG + hw);
    }
    const uint32_t st = ring + stage * C::STAGE;
    float x[2][NT][4];
    scores(st, 0, x[0]);
    scores(st, 1, x[1]);
    // scores to base 2; tokens that are not there weigh nothing. The reference of a head's weights
    // is a running maximum that follows once a score is 2^8 times beyond it
    const bool all = meta.z == ~0u;
    bool beyond = false;
    float top[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) top[nt][c] = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float& y = x[u][nt][k];
          y *= F[nt][k & 1];
          if (!all && !(meta.z >> (u * 16 + (k >> 1) * 8 + g) & 1)) y = -INFINITY;
          top[nt][k & 1] = fmaxf(top[nt][k & 1], y);
        }
#pragma unroll
      for (int c = 0; c < 2; ++c) beyond |= top[nt][c] > mx[nt][c] + 8.f;
    }
    if (__any_sync(~0u, beyond)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int s = 4; s < 32; s *= 2)
            top[nt][c] = fmaxf(top[nt][c], __shfl_xor_sync(~0u, top[nt][c], s));
          const float now = fmaxf(mx[nt][c], top[nt][c]), f = ex2(mx[nt][c] - now);
          mx[nt][c] = now;
          l[nt][c] *= f;
          M[nt][c] *= f;
#pragma unroll
          for (int j = 0; j < NG; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) O[nt][j][k][c] *= f, O[nt][j][k][2 + c] *= f;
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[u][nt][k] = ex2(x[u][nt][k] - mx[nt][k & 1]);
          l[nt][k & 1] += x[u][nt][k];
        }
      values(st, u, x[u]);
    }
    __syncwarp();
    if (flags & 2) end_pair((int)meta.x, pair, flags, (int)meta.w, stage);
    stage = stage + 1 == S ? 0 : stage + 1;
  }
}

// Joins the states of pairs that ranges cut. The CTAs that share a pair share its heads; few states: a
// warp for each head, many: all warps.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_merge_kernel(const __grid_constant__ Params p) {
  __shared__ float so[kWarps][D], sml[kWarps][2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int E = D / 32;
  const auto& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Range rg = p.w.range[blockIdx.x];
  const int heads = p.HG * p.G;
  for (int side = 0; side < 2; ++side) {
    const int row = side ? rg.row1 : rg.row0, hg = side ? rg.hg1 : rg.hg0;
    if (row < 0) continue;
    const int start = side ? (int)blockIdx.x : rg.start0, last = side ? rg.last1 : rg.last0;
    const int n = last - start + 1;
    const bool many = n > 16;
    const int team = many ? 1 : kWarps, i0 = many ? warp : 0, di = many ? kWarps : 1;
    for (int h = (blockIdx.x - start) * team + (many ? 0 : warp); h < heads; h += n * team) {
      auto at = [&](int i) { return ((int64_t)(start + i) * 2 + (i == 0)) * heads + h; };
      float m = -FLT_MAX, den = 0.f, v[E] = {};
      for (int i = i0 + lane * di; i < n; i += 32 * di) m = fmaxf(m, p.w.ml[at(i) * 2]);
#pragma unroll
      for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, x));
#pragma unroll 4
      for (int i = i0; i < n; i += di) {
        const float2 ml = *(const float2*)(p.w.ml + at(i) * 2);
        const float f = ex2(ml.x - m);
        den = fmaf(f, ml.y, den);
        if constexpr (E == 4) {
          const float4 o = *(const float4*)(p.w.o + at(i) * D + lane * 4);
          v[0] = fmaf(f, o.x, v[0]), v[1] = fmaf(f, o.y, v[1]);
          v[2] = fmaf(f, o.z, v[2]), v[3] = fmaf(f, o.w, v[3]);
        } else {
          const float2 o = *(const float2*)(p.w.o + at(i) * D + lane * 2);
          v[0] = fmaf(f, o.x, v[0]), v[1] = fmaf(f, o.y, v[1]);
        }
      }
      if (many) {
#pragma unroll
        for (int e = 0; e < E; ++e) so[warp][lane * E + e] = v[e];
        if (lane == 0) sml[warp][0] = m, sml[warp][1] = den;
        __syncthreads();
        m = -FLT_MAX, den = 0.f;
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sml[w][0]);
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = 0.f;
        for (int w = 0; w < kWarps; ++w) {
          const float f = ex2(sml[w][0] - m);
          den = fmaf(f, sml[w][1], den);
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] = fmaf(f, so[w][lane * E + e], v[e]);
        }
        __syncthreads();
        if (warp != 0) continue;
      }
      const int64_t head = (int64_t)row * a.num_q_heads + (int64_t)hg * heads + h;
      const float f = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
      for (int e = 0; e < E; ++e)
        ((T*)a.o)[head * D + lane * E + e] = Elem<T>::from_f(v[e] * f);
      if (a.lse && lane == 0) a.lse[head] = den == 0.f ? -INFINITY : kLn2 * (m + log2f(den));
    }
  }
}

// ---------------------------------------------------------------- host side
int validate(const rc_kv4_decode_args* a, const char* fn) {
  RC_CHECK_ARG(a != nullptr, "%s: args is NULL", fn);
  RC_CHECK_ARG(a->dtype == RC_DTYPE_BF16 || a->dtype == RC_DTYPE_F32, "%s: dtype %d", fn, a->dtype);
  RC_CHECK_ARG(a->num_rows >= 0 && a->num_q_heads > 0 && a->num_kv_heads > 0 &&
                   a->num_q_heads % a->num_kv_heads == 0,
               "%s: bad head counts", fn);
  RC_CHECK_ARG(a->num_q_heads / a->num_kv_heads <= kMaxGroup, "%s: group size %d (at most %d)", fn,
               a->num_q_heads / a->num_kv_heads, kMaxGroup);
  RC_CHECK_ARG(a->head_dim == 64 || a->head_dim == 128, "%s: head_dim %d (64 or 128)", fn,
               a->head_dim);
  RC_CHECK_ARG(a->max_seq_len >= 0 && a->max_seq_len <= (1 << 24), "%s: max_seq_len %d", fn,
               a->max_seq_len);
  RC_CHECK_ARG(a->num_rows <= (1 << 20) && (int64_t)a->num_rows * a->num_q_heads < (1ll << 28),
               "%s: too many rows", fn);
  return RC_OK;
}

Params params_of(const rc_kv4_decode_args* a) {
  Params p{};
  p.a = *a;
  p.G = a->num_q_heads / a->num_kv_heads;
  // the divisor of the KV heads (up to 8) that leaves fewest warps idle, the largest of those
  int best = 0;
  for (int h = 1; h <= kWarps; ++h) {
    if (a->num_kv_heads % h) continue;
    const int busy = kWarps / h * h;
    if (busy >= best) best = busy, p.HG = h, p.TS = kWarps / h;
  }
  p.groups = a->num_kv_heads / p.HG;
  p.min_steps = 2;
  return p;
}

// CTAs that may have a range, whatever the rows hold.
int64_t most_ctas(const Params& p) {
  const int64_t steps = (p.a.max_seq_len + kTile * p.TS - 1) / (kTile * p.TS);
  return std::max<int64_t>(1, std::min<int64_t>(
      kMaxCtas, (steps * p.a.num_rows * p.groups + p.min_steps - 1) / p.min_steps));
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }
Workspace carve(void* base, const Params& p, size_t* total) {
  const size_t c = (size_t)most_ctas(p), heads = c * 2 * p.HG * p.G;
  Workspace w{};
  char* b = (char*)base;
  size_t at = 0;
  w.range = (Range*)b;
  at += align256(c * sizeof(Range));
  w.ml = (float*)(b + at);
  at += align256(heads * 8);
  w.o = (float*)(b + at);
  at += align256(heads * p.a.head_dim * 4);
  *total = at;
  return w;
}

struct Setup {
  int ctas;
};

template <typename T, int D, int NT>
cudaError_t launch_t(const Params& p, cudaStream_t s) {
  using C = Cfg<T, D, NT>;
  static PerDevice<Setup> setup;
  const Setup* st = nullptr;
  cudaError_t e = setup.get(
      [](Setup& x) {
        int dev = 0, sms = 0, per = 0;
        cudaError_t r = cudaFuncSetAttribute(kv4_decode_kernel<T, D, NT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (r == cudaSuccess) r = cudaGetDevice(&dev);
        if (r == cudaSuccess)
          r = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (r == cudaSuccess)
          r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kv4_decode_kernel<T, D, NT>,
                                                            kThreads, C::SMEM);
        x.ctas = std::max(1, std::min(kMaxCtas, sms * per));
        return r;
      },
      &st);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)std::min<int64_t>(most_ctas(p), st->ctas);
  kv4_decode_kernel<T, D, NT><<<grid, kThreads, C::SMEM, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launches(1);
  if (grid == 1 || p.a.max_seq_len <= kTile * p.TS) return cudaSuccess;   // no pair is cut
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv4_merge_kernel<T, D>, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <int D>
cudaError_t launch_d(const Params& p, cudaStream_t s) {
  if (p.a.dtype == RC_DTYPE_BF16)
    return p.G <= 8 ? launch_t<__nv_bfloat16, D, 1>(p, s) : launch_t<__nv_bfloat16, D, 2>(p, s);
  return p.G <= 8 ? launch_t<float, D, 1>(p, s) : launch_t<float, D, 2>(p, s);
}

}  // namespace
}  // namespace rc

extern "C" int rc_kv4_decode_workspace_bytes(const rc_kv4_decode_args* a, size_t* out_bytes) {
  const int v = rc::validate(a, "rc_kv4_decode_workspace_bytes");
  if (v != RC_OK) return v;
  RC_CHECK_ARG(out_bytes != nullptr, "rc_kv4_decode_workspace_bytes: out_bytes is NULL");
  const rc::Params p = rc::params_of(a);
  rc::carve(nullptr, p, out_bytes);
  return RC_OK;
}

extern "C" int rc_kv4_decode_attention(const rc_kv4_decode_args* a, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  static const char* fn = "rc_kv4_decode_attention";
  const int v = rc::validate(a, fn);
  if (v != RC_OK) return v;
  RC_CHECK_ARG(a->max_reqs > 0 && a->max_ctx > 0 && a->num_slots > 0 && a->max_seq_len <= a->max_ctx,
               "%s: bad sizes (max_seq_len must lie within the slot table)", fn);
  RC_CHECK_ARG(a->sm_scale > 0.f && std::isfinite(a->sm_scale),
               "%s: sm_scale must be positive and finite", fn);
  if (a->num_rows == 0) return RC_OK;
  RC_CHECK_ARG(a->q && a->seq_len && a->req_idx && a->req_to_token && a->k_pool && a->v_pool && a->o,
               "%s: NULL pointer", fn);
  const uintptr_t al = (uintptr_t)a->q | (uintptr_t)a->o | (uintptr_t)workspace;
  RC_CHECK_ARG((al & 15) == 0, "%s: q, o and workspace must be 16-byte aligned", fn);
  RC_CHECK_ARG((((uintptr_t)a->k_pool | (uintptr_t)a->v_pool) & (rc::kv4_align(a->head_dim) - 1)) == 0,
               "%s: planes must be multiples of %d bytes", fn, rc::kv4_align(a->head_dim));
  rc::Params p = rc::params_of(a);
  size_t need = 0;
  p.w = rc::carve(workspace, p, &need);
  RC_CHECK_ARG(workspace && workspace_bytes >= need, "%s: workspace %zu bytes < %zu needed", fn,
               workspace ? workspace_bytes : 0, need);
  p.status = rc::device_status_ptr();
  if (!p.status) return rc::fail(RC_ERR_CUDA, "%s: no device status word", fn);
  const cudaError_t e = a->head_dim == 128 ? rc::launch_d<128>(p, (cudaStream_t)stream)
                                           : rc::launch_d<64>(p, (cudaStream_t)stream);
  if (e != cudaSuccess)
    return rc::fail(RC_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return rc::check_launch(fn);
}
