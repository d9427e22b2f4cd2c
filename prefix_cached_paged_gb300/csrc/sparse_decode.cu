// Decode attention over the blocks of positions that a cheap score selects for each query row and
// KV head.
//
// A block's box (lo_d, hi_d: the least and greatest of its keys in each dimension) bounds q.k from
// above by s = sum_d (q_d >= 0 ? q_d hi_d : q_d lo_d); the largest s over the query heads of a KV head
// ranks the block. Kernels:
//   select: a cluster of CTAs per (row, KV head) scores its blocks; the first CTA finds the
//           top_blocks best and writes their numbers in ascending order;
//   attend: one CTA per (row, KV head, part of the selected tokens), softmax in fp32 with running
//           maximum and sum; the last CTA of a unit to finish joins its parts' states.
#include <algorithm>
#include <cmath>

#include "host_common.h"
#include "warp_mma.cuh"

namespace rc {
namespace {

constexpr int kMaxPart = 512;   // selected tokens per attention CTA, at most
constexpr int kMinPart = 64;    // and at least: one stage for each of its warps
constexpr int kEnoughCtas = 456;   // three per SM
constexpr int kMaxGroup = 16;   // query heads per KV head

struct Workspace {
  float* score;               // [rows * Hkv * nb], fp32
  float* tsum;                // [rows * Hkv * nb], magnitudes of their terms
  unsigned long long* rank;   // [rows * Hkv * nb], 64-bit ranks of the blocks near the border
  int* sel;                   // [rows * Hkv * top]
  int* count;                 // [rows * Hkv] parts finished
  float* plse;                // [rows * Hkv * parts * G], base 2
  float* po;                  // [rows * Hkv * parts * G * D]
};
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Params {
  rc_sparse_decode_args a;
  Workspace w;
  int nb;      // blocks of max_seq_len
  int part_tokens;   // selected tokens per attention CTA
  int parts;   // attention CTAs per (row, KV head)
  int G;
  int* status;
};

Workspace carve(void* base, const Params& p, size_t* total) {
  const int64_t units = (int64_t)p.a.num_rows * p.a.num_kv_heads;
  Workspace w{};
  char* b = (char*)base;
  size_t o = 0;
  w.score = (float*)(b + o);
  o += align256((size_t)units * p.nb * 4);
  w.tsum = (float*)(b + o);
  o += align256((size_t)units * p.nb * 4);
  w.rank = (unsigned long long*)(b + o);
  o += align256((size_t)units * p.nb * 8);
  w.sel = (int*)(b + o);
  o += align256((size_t)units * p.a.top_blocks * 4);
  w.count = (int*)(b + o);
  o += align256((size_t)units * 4);
  w.plse = (float*)(b + o);
  o += align256((size_t)units * p.parts * p.G * 4);
  w.po = (float*)(b + o);
  o += align256((size_t)units * p.parts * p.G * p.a.head_dim * 4);
  *total = o;
  return w;
}

// Visible tokens of row n; 0 for an empty row, and for one with bad data (recorded).
__device__ __forceinline__ int row_len(const Params& p, int64_t n, bool report) {
  const int L = p.a.seq_len[n], row = p.a.req_idx[n];
  if (L < 0 || L > p.a.max_seq_len || row < 0 || row >= p.a.max_reqs) {
    if (report) set_status(p.status, kStatusPosRange);
    return 0;
  }
  return L;
}

// ---------------------------------------------------------------- scores
// Scores are computed in fp32 next to t = sum_d of the magnitudes of their terms. A score's fp32
// error is at most kScoreError * t: bf16 products are exact, a matrix instruction adds 16 of them
// and its accumulator with at most 2^-23 of the largest lost per addend, and each of four chains
// has at most 4 instructions (d = 128: 16 for the 2 d products), so 4 * 17 * 2^-23 = 2^-16.9 with
// the joining sums; the fp32 path's chains are shorter. Selection recomputes in 64 bits wherever
// twice that bound reaches across the border, so the result is that of 64-bit scores.
constexpr float kScoreError = 1.0f / 65536;
constexpr int kSelThreads = 256;

// Scores of 16 blocks against the query heads of a KV head by one warp, boxes and queries straight
// from global memory into matrix fragments: the dot product does not care in which order the
// dimensions come, so lane (gid, tig) takes 16 contiguous bytes of a row where the instruction
// wants four pairs, the same ones for both operands. [q-, q+] . [lo, hi] needs no comparison:
// one of q+ = max(q, 0) and q- = min(q, 0) is zero. (0 * inf gives a NaN that the definition has
// not: a score that is not finite sends its unit to the 64-bit path.)
template <int D, int NT>
__device__ void score_tiles(const Params& p, int64_t n, int g, int have, int tile0, int tile_step,
                            float* score, float* tsum) {
  constexpr int J = D / 32;   // 32-element groups of a row
  const rc_sparse_decode_args& a = p.a;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  uint4 q[NT][J];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int h = t * 8 + gid;
    const uint4* src = (const uint4*)((const __nv_bfloat16*)a.q +
                                      (n * a.num_q_heads + (int64_t)g * p.G + h) * D);
#pragma unroll
    for (int j = 0; j < J; ++j) q[t][j] = h < p.G ? src[j * 4 + tig] : make_uint4(0, 0, 0, 0);
  }
  const __nv_bfloat16* boxes = (const __nv_bfloat16*)a.bounds +
                               ((int64_t)a.req_idx[n] * a.max_blocks * a.num_kv_heads + g) * 2 * D;
  const int64_t stride = (int64_t)a.num_kv_heads * 2 * D;
  for (int tile = tile0; tile * 16 < have; tile += tile_step) {
    const int r0 = tile * 16 + gid, r1 = r0 + 8;
    const uint4* b0 = (const uint4*)(boxes + r0 * stride);
    const uint4* b1 = (const uint4*)(boxes + r1 * stride);
    uint4 x[2 * J], y[2 * J];
#pragma unroll
    for (int j = 0; j < 2 * J; ++j) {
      x[j] = r0 < have ? b0[j * 4 + tig] : make_uint4(0, 0, 0, 0);
      y[j] = r1 < have ? b1[j * 4 + tig] : make_uint4(0, 0, 0, 0);
    }
    float best0 = -INFINITY, best1 = -INFINITY, t0 = 0.f, t1 = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float c[4][4] = {}, m[4] = {};
      constexpr uint32_t kAbs = 0x7fff7fffu;
#pragma unroll
      for (int j = 0; j < 2 * J; ++j) {
        const uint4 qq = q[t][j % J];
        uint4 w;   // q- beside lo (the first half of a row), q+ beside hi
        if (j < J)
          w = make_uint4(min_nan_bf16x2(qq.x, 0), min_nan_bf16x2(qq.y, 0), min_nan_bf16x2(qq.z, 0),
                         min_nan_bf16x2(qq.w, 0));
        else
          w = make_uint4(max_nan_bf16x2(qq.x, 0), max_nan_bf16x2(qq.y, 0), max_nan_bf16x2(qq.z, 0),
                         max_nan_bf16x2(qq.w, 0));
        mma_bf16(c[j % 4], x[j].x, y[j].x, x[j].y, y[j].y, w.x, w.y);
        mma_bf16(c[j % 4], x[j].z, y[j].z, x[j].w, y[j].w, w.z, w.w);
        mma_bf16(m, x[j].x & kAbs, y[j].x & kAbs, x[j].y & kAbs, y[j].y & kAbs, w.x & kAbs,
                 w.y & kAbs);
        mma_bf16(m, x[j].z & kAbs, y[j].z & kAbs, x[j].w & kAbs, y[j].w & kAbs, w.z & kAbs,
                 w.w & kAbs);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (t * 8 + 2 * tig + e < p.G) {
          best0 = max_nan(best0, (c[0][e] + c[1][e]) + (c[2][e] + c[3][e]));
          best1 = max_nan(best1, (c[0][2 + e] + c[1][2 + e]) + (c[2][2 + e] + c[3][2 + e]));
          t0 = max_nan(t0, m[e]);
          t1 = max_nan(t1, m[2 + e]);
        }
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      best0 = max_nan(best0, __shfl_xor_sync(0xffffffffu, best0, o));
      best1 = max_nan(best1, __shfl_xor_sync(0xffffffffu, best1, o));
      t0 = max_nan(t0, __shfl_xor_sync(0xffffffffu, t0, o));
      t1 = max_nan(t1, __shfl_xor_sync(0xffffffffu, t1, o));
    }
    if (tig == 0 && r0 < have) {
      score[r0] = best0;
      tsum[r0] = t0;
    }
    if (tig == 0 && r1 < have) {
      score[r1] = best1;
      tsum[r1] = t1;
    }
  }
}

// The fp32 form: one warp per block, lanes over the dimensions.
template <int D>
__device__ void score_blocks_f32(const Params& p, int64_t n, int g, int have, int b0, int step,
                                 float* score, float* tsum) {
  constexpr int E = D / 32;
  const rc_sparse_decode_args& a = p.a;
  const int lane = threadIdx.x & 31;
  const float* q = (const float*)a.q + (n * a.num_q_heads + (int64_t)g * p.G) * D + lane * E;
  const float* boxes = (const float*)a.bounds +
                       ((int64_t)a.req_idx[n] * a.max_blocks * a.num_kv_heads + g) * 2 * D + lane * E;
  for (int b = b0; b < have; b += step) {
    const float* box = boxes + (int64_t)b * a.num_kv_heads * 2 * D;
    float lo[E], hi[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      lo[e] = box[e];
      hi[e] = box[D + e];
    }
    float best = -INFINITY, tm = 0.f;
    for (int h = 0; h < p.G; ++h) {
      float s = 0.f, t = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float x = q[h * D + e];
        const float y = x >= 0.f ? hi[e] : lo[e];
        s = fmaf(x, y, s);
        t = fmaf(fabsf(x), fabsf(y), t);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        t += __shfl_xor_sync(0xffffffffu, t, o);
      }
      best = max_nan(best, s);
      tm = max_nan(tm, t);
    }
    if (lane == 0) {
      score[b] = best;
      tsum[b] = tm;
    }
  }
}

// ---------------------------------------------------------------- selection
// Larger score <=> larger integer.
__device__ __forceinline__ uint32_t order32(float s) {
  const int b = __float_as_int(s + 0.f);   // -0 ranks as 0
  return (uint32_t)(b < 0 ? ~b : (b | (1 << 31)));
}
__device__ __forceinline__ unsigned long long order64(double s) {
  if (!(s < 1.7976931348623157e308)) s = 1.7976931348623157e308;   // NaN, +inf
  if (s < -1.7976931348623157e308) s = -1.7976931348623157e308;
  const long long b = __double_as_longlong(s + 0.0);
  return (unsigned long long)(b < 0 ? ~b : (b | (1ll << 63)));
}

struct SelectShared {
  int hist[256];
  int wsum[2][kSelThreads / 32];
  int bin, above;
  uint32_t lo, hi;
  float tmax;
};

// Sum over the CTA (all threads get it).
__device__ __forceinline__ int block_sum(SelectShared& s, int x) {
  x = __reduce_add_sync(0xffffffffu, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.wsum[0][threadIdx.x >> 5] = x;
  __syncthreads();
  int r = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) r += s.wsum[0][w];
  return r;
}

// The k-th largest (k >= 1) of the values key(i), i < n, for which ok(i); there are at least k.
// A radix search that begins below the digits all of them share.
template <typename K, typename Key, typename Ok>
__device__ K kth_largest(SelectShared& s, int n, int k, K lo, K hi, Key key, Ok ok) {
  int shift = lo == hi ? 0 : (int)(sizeof(K) * 8) - __clzll((unsigned long long)(lo ^ hi)) +
                                 (int)(64 - sizeof(K) * 8);
  K prefix = shift >= (int)sizeof(K) * 8 ? 0 : (hi >> shift) << shift;
  while (shift > 0) {
    const int bits = min(shift, 8);
    const int low = shift - bits;
    s.hist[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kSelThreads) {
      if (!ok(i)) continue;
      const K x = key(i);
      if (shift >= (int)sizeof(K) * 8 || (x >> shift) == (prefix >> shift))
        atomicAdd(&s.hist[(int)((x >> low) & (K)((1 << bits) - 1))], 1);
    }
    __syncthreads();
    if (threadIdx.x < 32) {   // bin that holds the k-th largest, from the top
      const int lane = threadIdx.x;
      int c[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = s.hist[255 - (lane * 8 + e)];
        sum += c[e];
      }
      int run = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
      }
      int before = run - sum;
      if (before < k && run >= k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (before < k && before + c[e] >= k) {
            s.bin = 255 - (lane * 8 + e);
            s.above = before;
          }
          before += c[e];
        }
      }
    }
    __syncthreads();
    prefix |= (K)s.bin << low;
    k -= s.above;
    shift = low;
    __syncthreads();
  }
  return prefix;
}

// The 64-bit rank of block b: the largest score over the KV head's queries. One warp.
template <typename T>
__device__ unsigned long long exact_rank(const Params& p, int64_t n, int g, int b) {
  const rc_sparse_decode_args& a = p.a;
  const int lane = threadIdx.x & 31, d = a.head_dim;
  const T* box = (const T*)a.bounds +
                 ((((int64_t)a.req_idx[n] * a.max_blocks + b) * a.num_kv_heads + g) * 2) * d;
  unsigned long long rank = 0;
  for (int h = 0; h < p.G; ++h) {
    const T* q = (const T*)a.q + (n * a.num_q_heads + (int64_t)g * p.G + h) * d;
    double s = 0.0;
    for (int e = lane; e < d; e += 32) {
      const float x = Elem<T>::to_f(q[e]);
      s += (double)x * (double)Elem<T>::to_f(x >= 0.f ? box[d + e] : box[e]);
    }
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    rank = max(rank, order64(s));
  }
  return rank;
}

// A cluster of CTAs scores the blocks of one (row, KV head); its first CTA selects.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kSelThreads) sparse_select_kernel(Params p, int cluster) {
  __shared__ SelectShared sh;
  const rc_sparse_decode_args& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int64_t unit = blockIdx.x / cluster;
  const int rank = blockIdx.x - (int)unit * cluster;
  const int64_t n = unit / a.num_kv_heads;
  const int g = (int)(unit - n * a.num_kv_heads);
  const int L = row_len(p, n, rank == 0 && tid == 0 && g == 0);
  const int have = (L + a.block - 1) / a.block;
  const int take = min(have, a.top_blocks);
  float* score = p.w.score + unit * p.nb;
  float* tsum = p.w.tsum + unit * p.nb;
  const bool choose = take < have;   // else every block is taken and none is scored
  if (choose) {
    const int w0 = rank * (kSelThreads / 32) + wid, ws = cluster * (kSelThreads / 32);
    if constexpr (sizeof(T) == 2)
      score_tiles<D, NT>(p, n, g, have, w0, ws, score, tsum);
    else
      score_blocks_f32<D>(p, n, g, have, w0, ws, score, tsum);
  }
  if (cluster > 1) {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::
                     : "memory");
    if (rank) return;
  } else {
    __syncthreads();
  }
  if (tid == 0) p.w.count[unit] = 0;
  int* out = p.w.sel + unit * a.top_blocks;
  int* user = a.selected ? a.selected + unit * a.top_blocks : nullptr;
  for (int i = tid; i < a.top_blocks; i += kSelThreads) {
    const int b = !choose && i < take ? i : -1;
    if (!choose || i >= take) {
      out[i] = b;
      if (user) user[i] = b;
    }
  }
  if (!choose) return;

  // blocks [f0, f1) are scored ones; the others are forced
  const int f0 = min(a.sink_blocks, have), f1 = max(f0, have - a.recent_blocks);
  const int m = f1 - f0, k = take - (have - m);   // k of the m scored blocks are taken
  score += f0;
  tsum += f0;
  int need64 = 0;    // scored blocks whose 64-bit ranks decide
  int in = 0;        // scored blocks that are taken whatever those say
  float hi_s = 0.f, lo_s = 0.f;
  bool all64 = false;
  if (k > 0) {
    uint32_t lo = 0xffffffffu, hi = 0;
    float tmax = 0.f;
    bool finite = true;
    for (int i = tid; i < m; i += kSelThreads) {
      const float s = score[i], t = tsum[i];
      const uint32_t o = order32(s);
      lo = min(lo, o);
      hi = max(hi, o);
      tmax = fmaxf(tmax, t);
      finite = finite && fabsf(s) < INFINITY && t < INFINITY;
    }
    if (tid == 0) {
      sh.lo = 0xffffffffu;
      sh.hi = 0;
      sh.tmax = 0.f;
    }
    all64 = __syncthreads_or(!finite);
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t tb = __reduce_max_sync(0xffffffffu, __float_as_uint(tmax));   // tmax >= 0
    if (lane == 0) {
      atomicMin(&sh.lo, lo);
      atomicMax(&sh.hi, hi);
      atomicMax((unsigned int*)&sh.tmax, tb);
    }
    __syncthreads();
    if (!all64) {
      const uint32_t thr = kth_largest<uint32_t>(
          sh, m, k, sh.lo, sh.hi, [&](int i) { return order32(score[i]); },
          [](int) { return true; });
      const float ts = __uint_as_float(thr & (1u << 31) ? thr & ~(1u << 31) : ~thr);
      const float e2 = 2.f * kScoreError * 1.0001f * sh.tmax;
      hi_s = ts + e2;
      lo_s = ts - e2;
      int ci = 0, ca = 0;
      for (int i = tid; i < m; i += kSelThreads) {
        const float s = score[i];
        ci += s > hi_s;
        ca += s >= lo_s && s <= hi_s;
      }
      in = block_sum(sh, ci);
      need64 = block_sum(sh, ca);
    } else {
      need64 = m;
    }
  }
  const int rest = k - in;   // to be taken of the need64 near the border
  unsigned long long* r64 = p.w.rank + unit * p.nb + f0;
  auto near = [&](int i) { return all64 || (score[i] >= lo_s && score[i] <= hi_s); };
  unsigned long long thr64 = 0;
  int ties = 0;   // blocks of rank thr64 that are taken, the lowest-numbered ones
  const bool exact = k > 0 && need64 > rest;
  if (exact) {
    for (int i0 = wid * 32; i0 < m; i0 += kSelThreads) {
      const int i = i0 + lane;
      unsigned todo = __ballot_sync(0xffffffffu, i < m && near(i));
      while (todo) {
        const int j = __ffs(todo) - 1;
        todo &= todo - 1;
        const unsigned long long r = exact_rank<T>(p, n, g, f0 + i0 + j);
        if (lane == 0) r64[i0 + j] = r;
      }
    }
    __syncthreads();
    thr64 = kth_largest<unsigned long long>(
        sh, m, rest, 0ull, ~0ull, [&](int i) { return r64[i]; }, near);
    int c = 0;
    for (int i = tid; i < m; i += kSelThreads) c += near(i) && r64[i] > thr64;
    ties = rest - block_sum(sh, c);
  }
  // the chosen blocks in ascending order
  int done = 0, eq_done = 0;
  for (int b0 = 0; b0 < have; b0 += kSelThreads) {
    const int b = b0 + tid, i = b - f0;
    bool pick = b < have && (b < f0 || b >= f1), eq = false;
    if (b >= f0 && b < f1 && k > 0) {
      if (near(i)) {
        if (exact) {
          pick = r64[i] > thr64;
          eq = r64[i] == thr64;
        } else {
          pick = true;
        }
      } else {
        pick = score[i] > hi_s;
      }
    }
    const unsigned me = __ballot_sync(0xffffffffu, eq);
    __syncthreads();
    if (lane == 0) sh.wsum[0][wid] = __popc(me);
    __syncthreads();
    int ebase = eq_done;
    for (int w = 0; w < wid; ++w) ebase += sh.wsum[0][w];
    if (eq && ebase + __popc(me & ((1u << lane) - 1)) < ties) pick = true;
    const unsigned mp = __ballot_sync(0xffffffffu, pick);
    if (lane == 0) sh.wsum[1][wid] = __popc(mp);
    __syncthreads();
    int base = done;
    for (int w = 0; w < wid; ++w) base += sh.wsum[1][w];
    if (pick) {
      const int at = base + __popc(mp & ((1u << lane) - 1));
      out[at] = b;
      if (user) user[at] = b;
    }
#pragma unroll
    for (int w = 0; w < kSelThreads / 32; ++w) {
      done += sh.wsum[1][w];
      eq_done += sh.wsum[0][w];
    }
  }
}

// ---------------------------------------------------------------- attention
// What an attention CTA works on: tokens [t0, t1) of the selected tokens of a unit = (row, KV head),
// token t standing at position sel[t / block] * block + t % block. The newest block is selected and
// comes last, so it alone may be short and the selected tokens are the first `count`.
struct Part {
  int64_t unit, n;
  int g, L, t0, t1, parts;   // parts that have tokens (at least 1)
};
__device__ __forceinline__ bool part_of(const Params& p, Part& w) {
  const rc_sparse_decode_args& a = p.a;
  w.unit = blockIdx.x / p.parts;
  const int part = blockIdx.x - (int)w.unit * p.parts;
  w.n = w.unit / a.num_kv_heads;
  w.g = (int)(w.unit - w.n * a.num_kv_heads);
  w.L = row_len(p, w.n, false);
  const int have = (w.L + a.block - 1) / a.block;
  const int count = have <= a.top_blocks ? w.L : (a.top_blocks - 1) * a.block + w.L -
                                                     (have - 1) * a.block;
  w.parts = max(1, (count + p.part_tokens - 1) / p.part_tokens);
  w.t0 = part * p.part_tokens;
  w.t1 = min(count, w.t0 + p.part_tokens);
  return part < w.parts;
}

// Slots of the part's tokens into shared memory (-1: outside the pool, recorded).
__device__ __forceinline__ void load_slots(const Params& p, const Part& w, int* slots) {
  const rc_sparse_decode_args& a = p.a;
  const int* sel = p.w.sel + w.unit * a.top_blocks;
  const int shift = __ffs(a.block) - 1;
  for (int t = w.t0 + threadIdx.x; t < w.t1; t += blockDim.x) {
    const int pos = (sel[t >> shift] << shift) + (t & (a.block - 1));
    int s = a.req_to_token[(int64_t)a.req_idx[w.n] * a.max_ctx + pos];
    if (s < 0 || s >= a.num_slots) {
      set_status(p.status, kStatusSlotRange);
      s = -1;
    }
    slots[t - w.t0] = s;
  }
}

// The end of an attention CTA, all 128 threads: joins the four warps' states (m base 2, l, and
// unnormalised o, in shared memory) and writes the outputs, or the part's state with the CTA that
// finishes a unit last joining its parts in their order. The unit's counter was zeroed by the
// selection kernel.
template <typename T, int D>
__device__ void finish_part(const Params& p, const Part& w, const float* sm, const float* sl,
                            const float* so, int* last) {
  const rc_sparse_decode_args& a = p.a;
  const int G = p.G;
  const int64_t o0 = (w.n * a.num_q_heads + (int64_t)w.g * G) * D;
  const int64_t l0 = w.n * a.num_q_heads + (int64_t)w.g * G;
  const int part = blockIdx.x - (int)w.unit * p.parts;
  for (int x = threadIdx.x; x < G * D; x += 128) {
    const int h = x / D;
    const float M = fmaxf(fmaxf(sm[h], sm[G + h]), fmaxf(sm[2 * G + h], sm[3 * G + h]));
    float den = 0.f, num = 0.f;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float mv = sm[v * G + h];
      const float c = mv == -INFINITY ? 1.f : exp2f(mv - M);   // an empty state is all zeros
      den = fmaf(sl[v * G + h], c, den);
      num = fmaf(so[v * G * D + x], c, num);
    }
    const float o = den == 0.f ? 0.f : num / den;
    const float lse = den == 0.f ? -INFINITY : M + log2f(den);
    if (w.parts == 1) {
      ((T*)a.o)[o0 + x] = Elem<T>::from_f(o);
      if (a.lse && x % D == 0) a.lse[l0 + h] = den == 0.f ? -INFINITY : lse * kLn2;
    } else {
      const int64_t pi = (w.unit * p.parts + part) * G;
      p.w.po[pi * D + x] = o;
      if (x % D == 0) p.w.plse[pi + h] = lse;
    }
  }
  if (w.parts == 1) return;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) *last = atomicAdd(&p.w.count[w.unit], 1) == w.parts - 1;
  __syncthreads();
  if (!*last) return;
  __threadfence();
  for (int x = threadIdx.x; x < G * D; x += 128) {
    const int h = x / D;
    const int64_t pi = w.unit * p.parts * G;
    float M = -INFINITY;
    for (int c = 0; c < w.parts; ++c) M = fmaxf(M, __ldcg(&p.w.plse[pi + c * G + h]));
    float num = 0.f, den = 0.f;
    for (int c = 0; c < w.parts; ++c) {
      const float pl = __ldcg(&p.w.plse[pi + c * G + h]);
      const float k = pl == -INFINITY ? 0.f : exp2f(pl - M);
      den += k;
      num = fmaf(k, __ldcg(&p.w.po[(pi + c * G) * D + x]), num);
    }
    ((T*)a.o)[o0 + x] = Elem<T>::from_f(den == 0.f ? 0.f : num / den);
    if (a.lse && x % D == 0) a.lse[l0 + h] = den == 0.f ? -INFINITY : (M + log2f(den)) * kLn2;
  }
}

// bf16: one CTA of 4 warps per part. A warp streams every 4th stage of 16 tokens through its own
// ring: 16-byte copies of the tokens' K and V rows, completion by copy groups. The two
// contractions run on warp-level matrix instructions with the tokens as M and the KV head's query
// heads as N (NT tiles of 8): S^T = K Q^T, O^T += V^T P^T. K fragments by ldmatrix, V^T by its
// transposing form (rows padded by 16 bytes: no bank conflicts), Q^T in registers, P^T from the
// accumulators by movmatrix. P goes in as a bf16 part and its bf16 remainder, so P.V keeps 16 bits
// of the weights.
template <int D>
struct AttendCfg {
  static constexpr int TOK = 16, STAGES = 2;
  static constexpr int RB = D * 2, RS = RB + 16;
  static constexpr int STAGE = TOK * 2 * RS;
  static constexpr int RING = 4 * STAGES * STAGE;   // bytes for the CTA
};

template <int D, int NT>
__global__ void __launch_bounds__(128) sparse_attend_mma_kernel(Params p) {
  using C = AttendCfg<D>;
  constexpr int KS = D / 16;
  extern __shared__ __align__(128) char smem[];
  __shared__ float sm[4 * kMaxGroup], sl[4 * kMaxGroup];
  __shared__ int last;
  const rc_sparse_decode_args& a = p.a;
  int* slots = (int*)(smem + C::RING);
  Part w;
  if (!part_of(p, w)) return;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  const int G = p.G, n = w.t1 - w.t0;
  load_slots(p, w, slots);

  uint32_t qb[NT][KS][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int h = t * 8 + gid;
    const __nv_bfloat16* q = (const __nv_bfloat16*)a.q +
                             (w.n * a.num_q_heads + (int64_t)w.g * G + (h < G ? h : 0)) * D;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      qb[t][k][0] = h < G ? *(const uint32_t*)(q + k * 16 + tig * 2) : 0u;
      qb[t][k][1] = h < G ? *(const uint32_t*)(q + k * 16 + tig * 2 + 8) : 0u;
    }
  }
  __syncthreads();

  const uint32_t ring = smem_u32(smem) + wid * C::STAGES * C::STAGE;
  const char* kp = (const char*)a.k_pool + (int64_t)w.g * C::RB;
  const char* vp = (const char*)a.v_pool + (int64_t)w.g * C::RB;
  const int64_t slot_bytes = (int64_t)a.num_kv_heads * C::RB;
  constexpr int CPR = C::RB / 16, RPI = 32 / CPR;   // 16-byte copies per row, rows per copy step
  const int cc = (lane % CPR) * 16, rsub = lane / CPR;
  auto issue = [&](int s, int buf) {   // stage s of the part: tokens 16 s ..
    const uint32_t kd = ring + buf * C::STAGE + cc;
#pragma unroll
    for (int i = 0; i < C::TOK / RPI; ++i) {
      const int t = i * RPI + rsub, at = s * C::TOK + t;
      const int slot = at < n ? slots[at] : -1;
      const int64_t off = (int64_t)max(slot, 0) * slot_bytes + cc;
      cp_async16_or_zero(kd + t * C::RS, kp + off, slot >= 0);
      cp_async16_or_zero(kd + (C::TOK + t) * C::RS, vp + off, slot >= 0);
    }
  };

  const float qscale = a.sm_scale * kLog2e;
  const int k_row = (lane & 7) + ((lane >> 3) & 1) * 8, k_col = (lane >> 4) * 8;
  const int v_row = (lane & 7) + (lane >> 4) * 8, v_col = ((lane >> 3) & 1) * 8;
  float acc[NT][KS][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t][0] = m[t][1] = -INFINITY;
    l[t][0] = l[t][1] = 0.f;
#pragma unroll
    for (int i = 0; i < KS; ++i) acc[t][i][0] = acc[t][i][1] = acc[t][i][2] = acc[t][i][3] = 0.f;
  }
  const int stages = (n + C::TOK - 1) / C::TOK;
  if (wid < stages) issue(wid, 0);
  cp_async_commit();
  int buf = 0;
  for (int s = wid; s < stages; s += 4, buf ^= 1) {
    if (s + 4 < stages) issue(s + 4, buf ^ 1);
    cp_async_commit();
    cp_async_wait<1>();
    __syncwarp();
    const uint32_t kb = ring + buf * C::STAGE, vb = kb + C::TOK * C::RS;
    float sc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint32_t r[4];
      ldmatrix_x4(kb + k_row * C::RS + (k * 16 + k_col) * 2, r);
#pragma unroll
      for (int t = 0; t < NT; ++t) mma_bf16(sc[t], r[0], r[1], r[2], r[3], qb[t][k][0], qb[t][k][1]);
    }
    const int at = s * C::TOK + gid;
    const bool ok0 = at < n && slots[at] >= 0, ok1 = at + 8 < n && slots[at + 8] >= 0;
    uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {   // query heads 8 t + 2 tig + e
        sc[t][e] = ok0 ? sc[t][e] * qscale : -INFINITY;
        sc[t][2 + e] = ok1 ? sc[t][2 + e] * qscale : -INFINITY;
        float x = fmaxf(sc[t][e], sc[t][2 + e]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
        // the running maximum moves only when it grows by more than 2^8
        const float mo = m[t][e], mx = fmaxf(mo, x);
        const bool grow = mx > mo + 8.f;
        const float mn = grow ? mx : mo;
        const float al = grow && mo != -INFINITY ? exp2f(mo - mn) : 1.f;
        m[t][e] = mn;
        const float u = mn == -INFINITY ? 0.f : mn;   // nothing but masked tokens so far
        sc[t][e] = exp2f(sc[t][e] - u);
        sc[t][2 + e] = exp2f(sc[t][2 + e] - u);
        l[t][e] = l[t][e] * al + sc[t][e] + sc[t][2 + e];
        if (__any_sync(0xffffffffu, al != 1.f)) {
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            acc[t][i][e] *= al;
            acc[t][i][2 + e] *= al;
          }
        }
      }
      const uint32_t hx = pack2_bf16(sc[t][0], sc[t][1]), hy = pack2_bf16(sc[t][2], sc[t][3]);
      ph[t][0] = movmatrix_trans(hx);
      ph[t][1] = movmatrix_trans(hy);
      pl[t][0] = movmatrix_trans(pack2_bf16(sc[t][0] - bf16lo(hx), sc[t][1] - bf16hi(hx)));
      pl[t][1] = movmatrix_trans(pack2_bf16(sc[t][2] - bf16lo(hy), sc[t][3] - bf16hi(hy)));
    }
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      uint32_t r[4];
      ldmatrix_x4_trans(vb + v_row * C::RS + (i * 16 + v_col) * 2, r);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mma_bf16(acc[t][i], r[0], r[1], r[2], r[3], ph[t][0], ph[t][1]);
        mma_bf16(acc[t][i], r[0], r[1], r[2], r[3], pl[t][0], pl[t][1]);
      }
    }
    __syncwarp();   // the buffer may be filled again
  }
  cp_async_wait<0>();
  __syncthreads();   // the rings become the warps' states
  float* so = (float*)smem;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = l[t][e];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      const int h = t * 8 + 2 * tig + e;
      if (h < G) {
        if (gid == 0) {
          sm[wid * G + h] = m[t][e];
          sl[wid * G + h] = x;
        }
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          so[(wid * G + h) * D + i * 16 + gid] = acc[t][i][e];
          so[(wid * G + h) * D + i * 16 + 8 + gid] = acc[t][i][2 + e];
        }
      }
    }
  }
  __syncthreads();
  finish_part<__nv_bfloat16, D>(p, w, sm, sl, so, &last);
}

// fp32: one CTA of 4 warps per part, warp w takes every 4th token; lanes over the dimensions.
template <int D, int GM>
__global__ void __launch_bounds__(128) sparse_attend_f32_kernel(Params p) {
  constexpr int E = D / 32;
  extern __shared__ __align__(128) char smem[];
  __shared__ float q_s[GM * D];
  __shared__ float sm[4 * GM], sl[4 * GM];
  __shared__ int last;
  const rc_sparse_decode_args& a = p.a;
  float* so = (float*)smem;                     // [4][G][D]
  int* slots = (int*)(so + 4 * GM * D);
  Part w;
  if (!part_of(p, w)) return;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int G = p.G, n = w.t1 - w.t0;
  load_slots(p, w, slots);
  const float scale = a.sm_scale * kLog2e;
  for (int e = threadIdx.x; e < G * D; e += 128)
    q_s[e] = ((const float*)a.q)[(w.n * a.num_q_heads + (int64_t)w.g * G) * D + e] * scale;
  __syncthreads();
  float m[GM], l[GM], acc[GM][E];
#pragma unroll
  for (int h = 0; h < GM; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[h][e] = 0.f;
  }
  for (int t = wid; t < n; t += 4) {
    const int slot = slots[t];
    if (slot < 0) continue;
    const int64_t r = ((int64_t)slot * a.num_kv_heads + w.g) * D;
    float k[E], v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      k[e] = ((const float*)a.k_pool)[r + e * 32 + lane];
      v[e] = ((const float*)a.v_pool)[r + e * 32 + lane];
    }
#pragma unroll
    for (int h = 0; h < GM; ++h) {
      if (h >= G) break;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(q_s[h * D + e * 32 + lane], k[e], s);
#pragma unroll
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const float mn = fmaxf(m[h], s);
      // a score of -inf weighs nothing; a NaN reaches the output as it would in a dense softmax
      const float al = mn == -INFINITY ? 1.f : exp2f(m[h] - mn);
      const float pr = s == -INFINITY ? 0.f : exp2f(s - mn);
      m[h] = mn;
      l[h] = l[h] * al + pr;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[h][e] = fmaf(pr, v[e], acc[h][e] * al);
    }
  }
#pragma unroll
  for (int h = 0; h < GM; ++h) {
    if (h >= G) break;
    if (lane == 0) {
      sm[wid * G + h] = m[h];
      sl[wid * G + h] = l[h];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) so[(wid * G + h) * D + e * 32 + lane] = acc[h][e];
  }
  __syncthreads();
  finish_part<float, D>(p, w, sm, sl, so, &last);
}

int validate(const rc_sparse_decode_args* a, const char* fn) {
  RC_CHECK_ARG(a != nullptr, "%s: args is NULL", fn);
  RC_CHECK_ARG(a->dtype == RC_DTYPE_BF16 || a->dtype == RC_DTYPE_F32, "%s: dtype %d", fn, a->dtype);
  RC_CHECK_ARG(a->num_rows >= 0 && a->num_q_heads > 0 && a->num_kv_heads > 0 &&
                   a->num_q_heads % a->num_kv_heads == 0,
               "%s: bad head counts", fn);
  RC_CHECK_ARG(a->num_q_heads / a->num_kv_heads <= kMaxGroup, "%s: group size %d (at most %d)", fn,
               a->num_q_heads / a->num_kv_heads, kMaxGroup);
  RC_CHECK_ARG(a->head_dim == 64 || a->head_dim == 128, "%s: head_dim %d (64 or 128)", fn,
               a->head_dim);
  RC_CHECK_ARG(a->block == 16 || a->block == 32 || a->block == 64 || a->block == 128,
               "%s: block %d (16, 32, 64 or 128)", fn, a->block);
  RC_CHECK_ARG(a->max_seq_len >= 0 && a->max_seq_len <= (1 << 24), "%s: max_seq_len %d", fn,
               a->max_seq_len);
  RC_CHECK_ARG(a->top_blocks > 0 && a->top_blocks <= (1 << 20) && a->sink_blocks >= 0 &&
                   a->recent_blocks >= 1 &&
                   (int64_t)a->sink_blocks + a->recent_blocks <= a->top_blocks,
               "%s: top_blocks must hold the sink blocks and at least one recent block", fn);
  RC_CHECK_ARG((int64_t)a->num_rows * a->num_q_heads < (1ll << 28), "%s: too many rows", fn);
  return RC_OK;
}

Params params_of(const rc_sparse_decode_args* a) {
  Params p{};
  p.a = *a;
  p.G = a->num_q_heads / a->num_kv_heads;
  p.nb = std::max(1, (a->max_seq_len + a->block - 1) / a->block);
  const int64_t tokens = (int64_t)std::min(p.nb, a->top_blocks) * a->block;
  // parts as long as kMaxPart leaves enough CTAs to fill the GPU, shorter ones for few rows
  const int64_t units = (int64_t)a->num_rows * a->num_kv_heads;
  int64_t part = kMaxPart;
  while (part > kMinPart && units * ((tokens + part - 1) / part) < kEnoughCtas) part /= 2;
  p.part_tokens = (int)part;
  p.parts = (int)((tokens + part - 1) / part);
  return p;
}

// Launches an attention kernel with more dynamic shared memory than the default allows.
template <typename K>
cudaError_t launch_attend(K kernel, PerDevice<int>& setup, int max_smem, int smem, const Params& p,
                          unsigned units, cudaStream_t s) {
  const int* unused = nullptr;
  const cudaError_t e = setup.get(
      [&](int&) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem);
      },
      &unused);
  if (e != cudaSuccess) return e;
  kernel<<<units * (unsigned)p.parts, 128, smem, s>>>(p);
  return cudaGetLastError();
}
template <int D, int NT>
cudaError_t attend_bf16(const Params& p, unsigned units, cudaStream_t s) {
  static PerDevice<int> setup;
  constexpr int base = AttendCfg<D>::RING;
  static_assert(base >= 4 * 8 * NT * D * 4, "the warps' states fit the rings");
  return launch_attend(sparse_attend_mma_kernel<D, NT>, setup, base + kMaxPart * 4,
                       base + p.part_tokens * 4, p, units, s);
}
template <int D, int GM>
cudaError_t attend_f32(const Params& p, unsigned units, cudaStream_t s) {
  static PerDevice<int> setup;
  constexpr int base = 4 * GM * D * 4;
  return launch_attend(sparse_attend_f32_kernel<D, GM>, setup, base + kMaxPart * 4,
                       base + p.part_tokens * 4, p, units, s);
}

template <typename T, int D, int NT>
cudaError_t launch_select(const Params& p, unsigned units, cudaStream_t s) {
  // a CTA's 8 warps score 128 blocks (bf16) or 64 (fp32: 8 blocks a warp) before one works twice;
  // up to 8 CTAs share the work of one unit
  const int per_cta = sizeof(T) == 2 ? 128 : 64;
  int cluster = 1;
  while (cluster < 8 && cluster * per_cta < p.nb) cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(units * cluster);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sparse_select_kernel<T, D, NT>, p, cluster);
}

template <typename T, int D>
int launch(const Params& p, cudaStream_t s) {
  const unsigned units = (unsigned)(p.a.num_rows * p.a.num_kv_heads);
  cudaError_t e;
  if constexpr (sizeof(T) == 2)
    e = p.G <= 8 ? launch_select<T, D, 1>(p, units, s) : launch_select<T, D, 2>(p, units, s);
  else
    e = launch_select<T, D, 1>(p, units, s);
  if (e != cudaSuccess)
    return fail(RC_ERR_CUDA, "rc_sparse_decode_attention: launch failed: %s", cudaGetErrorString(e));
  if constexpr (sizeof(T) == 2)
    e = p.G <= 8 ? attend_bf16<D, 1>(p, units, s) : attend_bf16<D, 2>(p, units, s);
  else
    e = p.G <= 1   ? attend_f32<D, 1>(p, units, s)
        : p.G <= 4 ? attend_f32<D, 4>(p, units, s)
        : p.G <= 8 ? attend_f32<D, 8>(p, units, s)
                   : attend_f32<D, 16>(p, units, s);
  if (e != cudaSuccess)
    return fail(RC_ERR_CUDA, "rc_sparse_decode_attention: launch failed: %s", cudaGetErrorString(e));
  count_launches(2);
  return check_launch("rc_sparse_decode_attention");
}

template <typename T>
int launch_d(const Params& p, cudaStream_t s) {
  return p.a.head_dim == 128 ? launch<T, 128>(p, s) : launch<T, 64>(p, s);
}

}  // namespace
}  // namespace rc

extern "C" int rc_sparse_decode_workspace_bytes(const rc_sparse_decode_args* a, size_t* out_bytes) {
  const int v = rc::validate(a, "rc_sparse_decode_workspace_bytes");
  if (v != RC_OK) return v;
  RC_CHECK_ARG(out_bytes != nullptr, "rc_sparse_decode_workspace_bytes: out_bytes is NULL");
  const rc::Params p = rc::params_of(a);
  rc::carve(nullptr, p, out_bytes);
  return RC_OK;
}

extern "C" int rc_sparse_decode_attention(const rc_sparse_decode_args* a, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  static const char* fn = "rc_sparse_decode_attention";
  const int v = rc::validate(a, fn);
  if (v != RC_OK) return v;
  RC_CHECK_ARG(a->max_reqs > 0 && a->max_ctx > 0 && a->max_blocks > 0 && a->num_slots > 0 &&
                   a->max_seq_len <= a->max_ctx &&
                   (a->max_seq_len + a->block - 1) / a->block <= a->max_blocks,
               "%s: bad sizes (max_seq_len must lie within the slot table and the bounds)", fn);
  RC_CHECK_ARG(a->sm_scale > 0.f && std::isfinite(a->sm_scale),
               "%s: sm_scale must be positive and finite", fn);
  if (a->num_rows == 0) return RC_OK;
  RC_CHECK_ARG(a->q && a->seq_len && a->req_idx && a->req_to_token && a->k_pool && a->v_pool &&
                   a->bounds && a->o && workspace,
               "%s: NULL pointer", fn);
  const uintptr_t al = (uintptr_t)a->q | (uintptr_t)a->k_pool | (uintptr_t)a->v_pool |
                       (uintptr_t)a->bounds | (uintptr_t)a->o | (uintptr_t)workspace;
  RC_CHECK_ARG((al & 15) == 0, "%s: tensors and workspace must be 16-byte aligned", fn);
  rc::Params p = rc::params_of(a);
  RC_CHECK_ARG((int64_t)a->num_rows * a->num_kv_heads * p.parts < (1ll << 31),
               "%s: too many rows for top_blocks %d of %d tokens", fn, a->top_blocks, a->block);
  size_t need = 0;
  p.w = rc::carve(workspace, p, &need);
  RC_CHECK_ARG(workspace_bytes >= need, "%s: workspace %zu bytes < %zu needed", fn, workspace_bytes,
               need);
  p.status = rc::device_status_ptr();
  if (!p.status) return rc::fail(RC_ERR_CUDA, "%s: no device status word", fn);
  return a->dtype == RC_DTYPE_BF16 ? rc::launch_d<__nv_bfloat16>(p, (cudaStream_t)stream)
                                   : rc::launch_d<float>(p, (cudaStream_t)stream);
}
