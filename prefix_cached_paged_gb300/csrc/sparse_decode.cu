// Decode attention over the blocks of positions that a cheap score selects for each query row and
// KV head.
//
// A block's box (lo_d, hi_d: the least and greatest of its keys in each dimension) bounds q.k from
// above by s = sum_d (q_d >= 0 ? q_d hi_d : q_d lo_d); the largest s over the query heads of a KV head
// ranks the block.
//
// One kernel, one cluster of CTAs per unit = (row, KV head), so that a unit's latency-bound steps
// run beside other units' streaming and nothing but the chosen blocks' numbers leaves the SMs:
//   score:  the cluster's warps share the blocks; every score goes to the shared memory of each
//           CTA of the cluster;
//   select: each CTA finds the top_blocks best by itself (the same ones);
//   attend: each CTA streams an equal part of the selected tokens, softmax in fp32 with running
//           maximum and sum;
//   join:   the CTAs' states are joined through distributed shared memory, each CTA finishing a
//           share of the outputs.
//
// Bound by HBM (boxes of a row once, K and V of the selected tokens once per KV head) with many rows,
// by the chain of dependent steps with few. Measured, bf16, heads of 128, inputs beyond L2:
//   128 rows, 32 + 32 heads, contexts 512 .. 8192, 16 blocks of 64: 339 us, 6.4 TB/s, 95 % of the
//     copy rate; 64 rows, 32 + 8 heads, contexts 4096 .. 32768, 64 blocks: 208 us, 5.5 TB/s, 82 % (a
//     CTA scores, waits and selects for ~8 us of its ~60; four of them share an SM).
//   1 row, 64 + 8 heads, 131071 tokens, 64 blocks: 28 us: score 4, cluster barriers 5, select 4 to
//     11 (the longer where finer scores are needed), slots 1, 256 tokens 4, join 2. A fifth of the
//     stalls there is instruction fetch: every step runs once.
//   fp32, heads of 128, 4096 or 2048 selected tokens: 32 rows, 8 + 8 heads 117 us of a floor of 90; 64
//     rows, 32 + 4 heads 130 of 86; 64 rows, 32 + 2 heads 245 of 86, bound by its 16 products per key
//     element on the CUDA cores (scores summed one by one over the lanes: 146, 436, 817 us).
// On the way, for the three: separate kernels for scores, selection, attention and merge, all scores
// in 64 bits and attention on CUDA cores 1093, 1399, 334 us; scores on matrix instructions 710, 728,
// 141; attention too, the last CTA of a row merging 417, 263, 126 (the merge of 64 parts alone 80);
// one kernel 341, 227, 39; K and V halves in one ring of three (four CTAs per SM, not three) 334, 200.
#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "host_common.h"
#include "warp_mma.cuh"

namespace rc {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 128, kWarps = 4;
constexpr int kMaxGroup = 16;      // query heads per KV head
constexpr int kMaxTop = 8192;      // the list of chosen blocks is kept in shared memory
constexpr int kMaxCluster = 16;
constexpr int kSegment = 512;      // tokens whose slots are resolved at a time
constexpr int kSmemBlocks = 7500;  // blocks whose scores and ranks are kept in shared memory (90 KB)

struct Workspace {                 // used only when a unit's scores outgrow shared memory
  float* score;                    // [units * nb]
  unsigned long long* rank;        // [units * nb]
};
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Params {
  rc_sparse_decode_args a;
  Workspace w;
  int nb;        // blocks of max_seq_len
  int G;         // query heads per KV head
  int cluster;   // CTAs per unit
  int* status;
  // dynamic shared memory (see Cfg): where the scores, the histogram, the slots and the list begin
  int score_at, hist_at, slots_at, list_at;
};

// Visible tokens of row n; 0 for an empty row (whatever its req_idx: a padded batch), and for one
// with bad data (recorded).
__device__ __forceinline__ int row_len(const Params& p, int64_t n, bool report) {
  const int L = p.a.seq_len[n], row = p.a.req_idx[n];
  if (L == 0) return 0;
  if (L < 0 || L > p.a.max_seq_len || row < 0 || row >= p.a.max_reqs) {
    if (report) set_status(p.status, kStatusPosRange);
    return 0;
  }
  return L;
}

// Dynamic shared memory of a CTA: the copy rings, in whose place first the unit's 64-bit ranks, scores
// and the selection's histogram stand and in the end the states to join; then the slots of a segment;
// then the chosen blocks. With many blocks the first part outgrows the rings.
constexpr int kBins = 2048;        // counters of the selection's radix steps

template <typename T, int D, int GM>
struct Cfg {
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int STAGES = 3;
  static constexpr int TOK = 16;                              // bf16: a stage is K or V of 16 tokens
  static constexpr int RB = D * 2, RS = RB + 16;              // bytes of a row, padded
  static constexpr int TB = GM == 16 ? 2 : 4;                 // fp32: K and V of TB tokens
  static constexpr int STAGE = kBf16 ? TOK * RS : 2 * TB * D * 4;
  // 16 heads of 128 keep their queries in shared memory: 168 registers and three CTAs per SM, not 181
  // and two (64 blocks of 64 read, 160, 320 and 640 units: 101, 173, 296 us, and 140, 232, 395)
  static constexpr bool Q_SHARED = kBf16 && GM * D > 1024;
  static constexpr int QUERIES = Q_SHARED ? GM * RS : 0;
  static constexpr int STATE = GM * D * 4;                    // o of one state
  static constexpr int WEIGHTS = kWarps * STAGES * STAGE;     // fp32: 64 words per warp
  static constexpr int RING = WEIGHTS + (kBf16 ? 0 : kWarps * 256);
  static constexpr int BASE = RING > (kWarps + 1) * STATE ? RING : (kWarps + 1) * STATE;

  // Lays it out for p; returns its size.
  static int layout(Params& p) {
    const int blocks = p.nb <= kSmemBlocks ? (p.nb + 1) / 2 * 2 : 0;
    p.score_at = blocks * 8;
    p.hist_at = blocks * 12;
    p.slots_at = (std::max(BASE, p.hist_at + kBins * 4) + 127) / 128 * 128;
    p.list_at = p.slots_at + kSegment * 4 + QUERIES;   // (the queries lie after the slots)
    return p.list_at + std::min(p.nb, p.a.top_blocks) * 4;
  }
  static constexpr int MOST = (BASE > kSmemBlocks * 12 + kBins * 4 ? BASE : kSmemBlocks * 12 +
                               kBins * 4) + 128 + kSegment * 4 + QUERIES + kMaxTop * 4;
};

// ---------------------------------------------------------------- scores
// Scores are computed in fp32 next to t = sum_d of the magnitudes of their terms. A score's fp32
// error is at most kScoreError * t: bf16 products are exact, a matrix instruction that begins at
// zero adds 16 of them with at most 2^-23 of the largest lost per addend, 16 * 2^-23 of its share
// of t, and the 16 results (d = 128: 2 d products) are added in fp32, 16 * 2^-24 of t: 2^-18.4 in
// all. The fp32 path's chains are shorter. Selection looks closer wherever twice that bound reaches
// across the border, in the end in 64 bits, so the result is that of 64-bit scores.
constexpr float kScoreError = 0x1p-18f;

// Larger score <=> larger integer.
__device__ __forceinline__ uint32_t order32(float s) {
  const int b = __float_as_int(s + 0.f);   // -0 ranks as 0
  return (uint32_t)(b < 0 ? ~b : (b | (1 << 31)));
}
__device__ __forceinline__ float unorder32(uint32_t o) {
  return __uint_as_float(o & (1u << 31) ? o & ~(1u << 31) : ~o);
}
__device__ __forceinline__ unsigned long long order64(double s) {
  if (!(s < 1.7976931348623157e308)) s = 1.7976931348623157e308;   // NaN, +inf
  if (s < -1.7976931348623157e308) s = -1.7976931348623157e308;
  const long long b = __double_as_longlong(s + 0.0);
  return (unsigned long long)(b < 0 ? ~b : (b | (1ll << 63)));
}

// Where the scores of a unit's blocks [f0, f1) go (index block - f0): the shared memory of every
// CTA of the cluster, or the workspace.
struct ScoreSink {
  float* local;   // this CTA's shared memory, or the workspace
  bool shared;
  int cluster, f0, f1;
  float tmax = 0.f;   // largest t this lane saw; least and greatest score it put
  uint32_t lo = 0xffffffffu, hi = 0;
  // `parts` lanes that all have the score share the CTAs it goes to; this one is number `part`
  __device__ __forceinline__ void put(int b, float s, int part, int parts) {
    lo = min(lo, order32(s));
    hi = max(hi, order32(s));
    if (!shared || cluster == 1) {
      if (part == 0) local[b - f0] = s;
    } else {
      for (int r = part; r < cluster; r += parts)
        cg::this_cluster().map_shared_rank(local, r)[b - f0] = s;
    }
  }
};

// Scores of 16 blocks at a time against the query heads of a KV head by one warp, boxes and queries
// straight from global memory into matrix fragments: the dot product does not care in which order the
// dimensions come, so lane (gid, tig) takes 16 contiguous bytes of a row where the instruction
// wants four pairs, the same ones for both operands. [q-, q+] . [lo, hi] needs no comparison:
// one of q+ = max(q, 0) and q- = min(q, 0) is zero. (0 * inf gives a NaN that the definition has
// not: a score that is not finite sends its unit to the 64-bit path.)
template <int D, int NT>
__device__ __forceinline__ void score_tiles(const Params& p, int64_t n, int g, int tile0,
                                            int tile_step, ScoreSink& out) {
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
  for (int tile = tile0; out.f0 + tile * 16 < out.f1; tile += tile_step) {
    const int r0 = out.f0 + tile * 16 + gid, r1 = r0 + 8;
    const uint4* b0 = (const uint4*)(boxes + r0 * stride);
    const uint4* b1 = (const uint4*)(boxes + r1 * stride);
    uint4 x[2 * J], y[2 * J];
#pragma unroll
    for (int j = 0; j < 2 * J; ++j) {
      x[j] = r0 < out.f1 ? b0[j * 4 + tig] : make_uint4(0, 0, 0, 0);
      y[j] = r1 < out.f1 ? b1[j * 4 + tig] : make_uint4(0, 0, 0, 0);
    }
    float best0 = -INFINITY, best1 = -INFINITY;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float c[4] = {}, m[4] = {};
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
        float z0[4] = {}, z1[4] = {};
        mma_bf16(z0, x[j].x, y[j].x, x[j].y, y[j].y, w.x, w.y);
        mma_bf16(z1, x[j].z, y[j].z, x[j].w, y[j].w, w.z, w.w);
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] += z0[e] + z1[e];
        mma_bf16(m, x[j].x & kAbs, y[j].x & kAbs, x[j].y & kAbs, y[j].y & kAbs, w.x & kAbs,
                 w.y & kAbs);
        mma_bf16(m, x[j].z & kAbs, y[j].z & kAbs, x[j].w & kAbs, y[j].w & kAbs, w.z & kAbs,
                 w.w & kAbs);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (t * 8 + 2 * tig + e < p.G) {
          best0 = max_nan(best0, c[e]);
          best1 = max_nan(best1, c[2 + e]);
          out.tmax = max_nan(out.tmax, max_nan(m[e], m[2 + e]));   // rows past f1 are zeros
        }
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      best0 = max_nan(best0, __shfl_xor_sync(0xffffffffu, best0, o));
      best1 = max_nan(best1, __shfl_xor_sync(0xffffffffu, best1, o));
    }
    if (r0 < out.f1) out.put(r0, best0, tig, 4);
    if (r1 < out.f1) out.put(r1, best1, tig, 4);
  }
}

// The sums over a warp of V values per lane (a power of two up to 32), V - 1 exchanges instead of
// 5 V: every step hands half of the values to the other half of the lanes. Lane l gets the sum of
// value l / (32 / V).
template <int V>
__device__ __forceinline__ float sum_values(float (&a)[V]) {
  const int lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int n = V / 2; n >= 1; n /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? a[i] : a[i + n];
      a[i] = (up ? a[i + n] : a[i]) + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
#pragma unroll
  for (; o >= 1; o /= 2) a[0] += __shfl_xor_sync(0xffffffffu, a[0], o);
  return a[0];
}

// The fp32 form: one warp per block, lanes over the dimensions, GM >= G query heads. t is taken as the
// sum over the lanes of the largest head's part, which is no less.
template <int D, int GM>
__device__ __forceinline__ void score_blocks_f32(const Params& p, int64_t n, int g, int first,
                                                 int step, ScoreSink& out) {
  constexpr int E = D / 32;
  const rc_sparse_decode_args& a = p.a;
  const int lane = threadIdx.x & 31;
  const float* src = (const float*)a.q + (n * a.num_q_heads + (int64_t)g * p.G) * D + lane * E;
  float q[GM][E];
#pragma unroll
  for (int h = 0; h < GM; ++h)
#pragma unroll
    for (int e = 0; e < E; ++e) q[h][e] = h < p.G ? src[h * D + e] : 0.f;
  const float* boxes = (const float*)a.bounds +
                       ((int64_t)a.req_idx[n] * a.max_blocks * a.num_kv_heads + g) * 2 * D + lane * E;
  constexpr int NB = GM >= 8 ? 2 : 4;   // boxes at a time: one warp per scheduler has to overlap itself
  for (int b0 = out.f0 + first; b0 < out.f1; b0 += NB * step) {
    float lo[NB][E], hi[NB][E], s[NB][GM], t[NB], best[NB];
#pragma unroll
    for (int u = 0; u < NB; ++u) {   // past the end: the last box again
      const float* box = boxes + (int64_t)min(b0 + u * step, out.f1 - 1) * a.num_kv_heads * 2 * D;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        lo[u][e] = box[e];
        hi[u][e] = box[D + e];
      }
      t[u] = 0.f;
    }
#pragma unroll
    for (int h = 0; h < GM; ++h) {
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        float x = 0.f, th = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float y = q[h][e] >= 0.f ? hi[u][e] : lo[u][e];
          x = fmaf(q[h][e], y, x);
          th = fmaf(fabsf(q[h][e]), fabsf(y), th);
        }
        s[u][h] = x;
        t[u] = max_nan(t[u], h < p.G ? th : 0.f);
      }
    }
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      best[u] = sum_values<GM>(s[u]);
      if (lane / (32 / GM) >= p.G) best[u] = -INFINITY;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        t[u] += __shfl_xor_sync(0xffffffffu, t[u], o);
        if (o >= 32 / GM) best[u] = max_nan(best[u], __shfl_xor_sync(0xffffffffu, best[u], o));
      }
    }
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      out.tmax = max_nan(out.tmax, t[u]);
      if (b0 + u * step < out.f1) out.put(b0 + u * step, best[u], lane, 32);
    }
  }
}

// ---------------------------------------------------------------- selection
struct SelectShared {
  unsigned long long list[kThreads];   // keys near the k-th largest, or ranks near the border
  int index[kThreads];                 // and their blocks
  int wsum[2][kWarps];
  int bin, above, inbin, listed;
  unsigned long long kth;
  uint32_t lo, hi, tmax;               // of the scores (ordered integers), and of their t
};

// Sums of x and y over the CTA (all threads get them).
__device__ __forceinline__ void block_sum2(SelectShared& s, int& x, int& y) {
  x = __reduce_add_sync(0xffffffffu, x);
  y = __reduce_add_sync(0xffffffffu, y);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    s.wsum[0][threadIdx.x >> 5] = x;
    s.wsum[1][threadIdx.x >> 5] = y;
  }
  __syncthreads();
  x = y = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    x += s.wsum[0][w];
    y += s.wsum[1][w];
  }
}

// put(place, i) for every i < n for which is(i), in no particular order; `count` places are taken
// after. The whole CTA; few i are expected, so a warp asks for places only where it has one.
template <typename Is, typename Put>
__device__ __forceinline__ void list_those(int& count, int n, Is is, Put put) {
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int i0 = threadIdx.x & ~31; i0 < n; i0 += kThreads) {
    const bool yes = i0 + lane < n && is(i0 + lane);
    const unsigned all = __ballot_sync(0xffffffffu, yes);
    if (all) {
      int at = 0;
      if (lane == 0) at = atomicAdd(&count, __popc(all));
      at = __shfl_sync(0xffffffffu, at, 0);
      if (yes) put(at + __popc(all & ((1u << lane) - 1)), i0 + lane);
    }
  }
}

// The k-th largest (k >= 1) of the values key(i), i < n, for which ok(i), all between lo and hi;
// there are at least k, and `left` at most. Radix steps of 11 bits, beginning below the digits that
// lo and hi share, until at most one key per thread is left, whose ranks are counted: one step,
// unless most scores are alike. hist: kBins counters.
template <typename K, typename Key, typename Ok>
__device__ K kth_largest(SelectShared& s, int* hist, int n, int left, int k, K lo, K hi, Key key,
                         Ok ok) {
  constexpr int kBits = sizeof(K) * 8, kDigit = 11, kPer = kBins / kThreads;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  int shift = lo == hi ? 0 : kBits - (__clzll((unsigned long long)(lo ^ hi)) - (64 - kBits));
  K prefix = shift == kBits ? 0 : (hi >> shift) << shift;
  while (shift > 0) {
    if (left <= kThreads) {
      if (tid == 0) s.listed = 0;
      __syncthreads();
      list_those(
          s.listed, n,
          [&](int i) {
            return ok(i) && (shift == kBits || (key(i) >> shift) == (prefix >> shift));
          },
          [&](int at, int i) { s.list[at] = key(i); });
      __syncthreads();
      const int c = s.listed;
      if (tid < c) {
        const unsigned long long x = s.list[tid];
        int above = 0, equal = 0;
        for (int i = 0; i < c; ++i) {
          above += s.list[i] > x;
          equal += s.list[i] == x;
        }
        if (above < k && above + equal >= k) s.kth = x;   // the same value from every such thread
      }
      __syncthreads();
      return (K)s.kth;
    }
    const int bits = min(shift, kDigit), low = shift - bits;
#pragma unroll
    for (int i = 0; i < kPer; ++i) hist[i * kThreads + tid] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < n; i += kThreads) {
      if (!ok(i)) continue;
      const K x = key(i);
      if (shift == kBits || (x >> shift) == (prefix >> shift))
        atomicAdd(&hist[(int)((x >> low) & (K)((1 << bits) - 1))], 1);
    }
    __syncthreads();
    // the bin that holds the k-th largest, from the top: thread t has bins 2047 - 16 t downwards
    int c[kPer], sum = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      c[e] = hist[kBins - 1 - (tid * kPer + e)];
      sum += c[e];
    }
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    if (lane == 31) s.wsum[0][wid] = run;
    __syncthreads();
    int before = run - sum;
    for (int w = 0; w < wid; ++w) before += s.wsum[0][w];
    if (before < k && before + sum >= k) {
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (before < k && before + c[e] >= k) {
          s.bin = kBins - 1 - (tid * kPer + e);
          s.above = before;
          s.inbin = c[e];
        }
        before += c[e];
      }
    }
    __syncthreads();
    prefix |= (K)s.bin << low;
    k -= s.above;
    left = s.inbin;
    shift = low;
  }
  return prefix;
}

// Where many blocks tie (all keys alike, a query of zeros) every one of them is ranked so, and the
// adders of a GB300 SM for doubles are few: one row of 2048 tied blocks takes 0.45 ms, 512 units of
// 64 .. 512 tied blocks 1.2 ms.
//
// The 64-bit rank of block b: the largest score over the KV head's queries. One warp, four queries
// at a time so that their loads and sums overlap.
template <typename T, int D>
__device__ __noinline__ unsigned long long exact_rank(const Params& p, int64_t n, int g, int b) {
  constexpr int E = D / 32;
  const rc_sparse_decode_args& a = p.a;
  const int lane = threadIdx.x & 31;
  const T* box = (const T*)a.bounds +
                 ((((int64_t)a.req_idx[n] * a.max_blocks + b) * a.num_kv_heads + g) * 2) * D + lane;
  const T* q = (const T*)a.q + (n * a.num_q_heads + (int64_t)g * p.G) * D + lane;
  float lo[E], hi[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    lo[e] = Elem<T>::to_f(box[e * 32]);
    hi[e] = Elem<T>::to_f(box[D + e * 32]);
  }
  unsigned long long rank = 0;
  for (int h0 = 0; h0 < p.G; h0 += 4) {
    double s[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      s[h] = 0.0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float x = h0 + h < p.G ? Elem<T>::to_f(q[(h0 + h) * D + e * 32]) : 0.f;
        s[h] += (double)x * (double)(x >= 0.f ? hi[e] : lo[e]);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int h = 0; h < 4; ++h) s[h] += __shfl_xor_sync(0xffffffffu, s[h], o);
#pragma unroll
    for (int h = 0; h < 4; ++h)
      if (h0 + h < p.G) rank = max(rank, order64(s[h]));
  }
  return rank;
}

// The score of block b in twice the precision of fp32, one warp: every product and every sum is
// kept with its rounding error (the error-free transformations of Dekker and Knuth, accumulated as
// in Ogita, Rump and Oishi, "Accurate sum and dot product", 2005). The errors' own sum is fp32: at
// most 512 addends, each at most 2^-24 of the partial sums of a tree of depth 13, so what is lost is
// below 512 * 13 * 2^-48 * t < 2^-35 * t. Far cheaper than doubles, of which an SM adds two a clock.
constexpr float kFineError = 0x1p-34f;
__device__ __forceinline__ void two_sum(float& s, float& err, float b) {
  const float a = s;
  s = __fadd_rn(a, b);
  const float bb = __fsub_rn(s, a);
  err = __fadd_rn(err, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb)));
}
// Returned as an integer of the same order: the sum's fp32 value, then what that lacks.
template <typename T, int D>
__device__ __forceinline__ unsigned long long fine_score(const Params& p, int64_t n, int g, int b) {
  constexpr int E = D / 32, H = 4;
  const rc_sparse_decode_args& a = p.a;
  const int lane = threadIdx.x & 31;
  const T* box = (const T*)a.bounds +
                 ((((int64_t)a.req_idx[n] * a.max_blocks + b) * a.num_kv_heads + g) * 2) * D + lane;
  const T* q = (const T*)a.q + (n * a.num_q_heads + (int64_t)g * p.G) * D + lane;
  float lo[E], hi[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    lo[e] = Elem<T>::to_f(box[e * 32]);
    hi[e] = Elem<T>::to_f(box[D + e * 32]);
  }
  unsigned long long best = 0;
  for (int h0 = 0; h0 < p.G; h0 += H) {
    float s[H], c[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      s[h] = c[h] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float x = h0 + h < p.G ? Elem<T>::to_f(q[(h0 + h) * D + e * 32]) : 0.f;
        const float y = x >= 0.f ? hi[e] : lo[e];
        const float xy = __fmul_rn(x, y);
        two_sum(s[h], c[h], xy);
        if constexpr (sizeof(T) == 4) c[h] = __fadd_rn(c[h], __fmaf_rn(x, y, -xy));
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const float s2 = __shfl_xor_sync(0xffffffffu, s[h], o);
        c[h] = __fadd_rn(c[h], __shfl_xor_sync(0xffffffffu, c[h], o));
        two_sum(s[h], c[h], s2);
      }
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      float err = 0.f;
      two_sum(s[h], err, c[h]);
      if (h0 + h < p.G)
        best = max(best, (unsigned long long)order32(s[h]) << 32 | order32(err));
    }
  }
  return best;
}

// Writes first + i for every i < m for which kind(i) is 2, and for the first `ties` for which it is
// 1, in ascending order. Each warp counts in its quarter of them, then writes from where the
// earlier ones end.
template <bool kTies, typename Kind>
__device__ __forceinline__ void compact(SelectShared& sh, int m, int first, int ties, int* list,
                                        Kind kind) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int quarter = (m + kThreads - 1) / kThreads * 32;
  const int i0 = wid * quarter, i1 = min(m, i0 + quarter);
  int np = 0, ne = 0;
#pragma unroll 4
  for (int i = i0 + lane; i < i1; i += 32) {
    const int c = kind(i);
    np += c == 2;
    if (kTies) ne += c == 1;
  }
  np = __reduce_add_sync(0xffffffffu, np);
  if (kTies) ne = __reduce_add_sync(0xffffffffu, ne);
  __syncthreads();
  if (lane == 0) {
    sh.wsum[0][wid] = np;
    sh.wsum[1][wid] = ne;
  }
  __syncthreads();
  int at = 0, eq = 0;
  for (int w = 0; w < wid; ++w) {
    at += sh.wsum[0][w];
    eq += sh.wsum[1][w];
  }
  if (kTies) at += min(eq, ties);
  const unsigned below = (1u << lane) - 1;
#pragma unroll 4
  for (int i = i0; i < i1; i += 32) {
    const int c = i + lane < i1 ? kind(i + lane) : 0;
    bool pick = c == 2;
    if (kTies) {
      const unsigned me = __ballot_sync(0xffffffffu, c == 1);
      pick = pick || (c == 1 && eq + __popc(me & below) < ties);
      eq += __popc(me);
    }
    const unsigned mp = __ballot_sync(0xffffffffu, pick);
    if (pick) list[at + __popc(mp & below)] = first + i + lane;
    at += __popc(mp);
  }
  __syncthreads();
}

// The k best of a unit's scored blocks [f0, f0 + m) in ascending order into `list` (shared memory),
// by the whole CTA, 1 <= k < m: by score[b - f0] where the fp32 scores can tell, then by finer ones
// where a few blocks are near the border, then by 64-bit ranks in r64. kOwn: the scores are this
// CTA's own copy in shared memory (else in the workspace, the cluster's).
template <typename T, int D, bool kOwn>
__device__ __forceinline__ void select_blocks(const Params& p, SelectShared& sh, int* hist, int64_t n,
                                              int g, int f0, int m, int k, float* score,
                                              unsigned long long* r64, int* list) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const bool all64 = sh.tmax >= 0x7e800000u;   // 2^126: sums may overflow, or be no numbers
  const float tmax = __uint_as_float(sh.tmax);
  float hi_s = 0.f, lo_s = 0.f;
  int in = 0, close = m;   // taken whatever finer scores say; those that they decide about
  if (!all64) {
    const uint32_t thr = kth_largest<uint32_t>(
        sh, hist, m, m, k, sh.lo, sh.hi, [&](int i) { return order32(score[i]); },
        [](int) { return true; });
    const float ts = unorder32(thr);
    // (1 % for the roundings of these lines; products below the smallest normal number may be lost)
    const float e2 = 2.02f * kScoreError * tmax + 0x1p-110f;
    hi_s = ts + e2;
    lo_s = ts - e2;
    close = 0;
#pragma unroll 4
    for (int i = tid; i < m; i += kThreads) {
      const float s = score[i];
      in += s > hi_s;
      close += s >= lo_s && s <= hi_s;
    }
    block_sum2(sh, in, close);
  }
  const int rest = k - in;   // to be taken of the `close`
  auto near = [&](int i) { return all64 || (score[i] >= lo_s && score[i] <= hi_s); };
  bool clear = close == rest;
  if (kOwn && !clear && close <= kThreads && !all64) {
    if (tid == 0) sh.listed = 0;
    __syncthreads();
    list_those(sh.listed, m, near, [&](int at, int i) { sh.index[at] = i; });
    __syncthreads();
    for (int c = wid; c < close; c += kWarps) {
      const unsigned long long f = fine_score<T, D>(p, n, g, f0 + sh.index[c]);
      if (lane == 0) sh.list[c] = f;
    }
    __syncthreads();
    const unsigned long long f = tid < close ? sh.list[tid] : 0;
    if (tid < close) {
      int above = 0, equal = 0;
      for (int c = 0; c < close; ++c) {
        above += sh.list[c] > f;
        equal += sh.list[c] == f;
      }
      if (above < rest && above + equal >= rest) sh.kth = f;
    }
    __syncthreads();
    // how far above the least one taken
    const float d = __fadd_rn(__fsub_rn(unorder32(f >> 32), unorder32(sh.kth >> 32)),
                              __fsub_rn(unorder32((uint32_t)f), unorder32((uint32_t)sh.kth)));
    const float w = 2.02f * kFineError * tmax + 0x1p-120f;
    const bool mine = tid < close && d >= -w;
    const int take = __syncthreads_count(mine);
    if (take == rest) {   // no block left out is as near as the error bound
      if (tid < close) score[sh.index[tid]] = mine ? INFINITY : -INFINITY;
      __syncthreads();
      clear = true;
    }
  }
  if (clear) {
    compact<false>(sh, m, f0, 0, list, [&](int i) { return score[i] >= lo_s ? 2 : 0; });
    return;
  }
  // many blocks: the cluster's CTAs, which all stand here, share them
  const cg::cluster_group cl = cg::this_cluster();
  const int P = p.cluster, rank = (int)(blockIdx.x % P);
  for (int i0 = (rank * kWarps + wid) * 32; i0 < m; i0 += P * kThreads) {
    const int i = i0 + lane;
    unsigned todo = __ballot_sync(0xffffffffu, i < m && near(i));
    while (todo) {
      const int j = __ffs(todo) - 1;
      todo &= todo - 1;
      const unsigned long long r = exact_rank<T, D>(p, n, g, f0 + i0 + j);
      if (kOwn && P > 1) {
        if (lane < P) cl.map_shared_rank(r64, lane)[i0 + j] = r;
      } else if (lane == 0) {
        r64[i0 + j] = r;
      }
    }
  }
  if (P > 1) cl.sync(); else __syncthreads();
  const unsigned long long thr64 = kth_largest<unsigned long long>(
      sh, hist, m, close, rest, 0ull, ~0ull, [&](int i) { return r64[i]; }, near);
  int c = 0, unused = 0;
  for (int i = tid; i < m; i += kThreads) c += near(i) && r64[i] > thr64;
  block_sum2(sh, c, unused);
  compact<true>(sh, m, f0, rest - c, list, [&](int i) {
    if (!near(i)) return score[i] > hi_s ? 2 : 0;
    return r64[i] > thr64 ? 2 : r64[i] == thr64 ? 1 : 0;
  });
}

// ---------------------------------------------------------------- attention
// Weights are 2^(score - running maximum) times 2^-32: the maximum may lag by 2^8 and a unit has at most
// 2^20 tokens (kMaxTop blocks of 128), so their sum times the largest value there is stays below 2^124
// and the mean of any finite values is finite. (Subtracted in the exponent, 32 would cost the scores
// five bits.)
constexpr float kWeightScale = 0x1p-32f;
__device__ __forceinline__ float log_sum(float mx, float den) {   // natural
  return (mx + log2f(den * 0x1p32f)) * kLn2;
}

// A weight x >= 0 goes to the matrix units as three bf16 parts that make it up exactly:
// h = head_part(x), m = head_part(x - h) and x - h - m. head_part takes the top 8 of the 24 bits of
// the number just below x, so what it leaves is above 0, at most 2^-7 of x and a multiple of x's last
// bit; two steps leave at most 8 bits. With every part of a positive weight above 0 an infinite value
// stays infinite (a part of 0 or of the other sign would make a NaN of it), down to weights of 2^-117,
// whose least part may be the least number there is.
__device__ __forceinline__ float head_part(float x) {
  return __uint_as_float((max(__float_as_uint(x), 1u) - 1) & 0xffff0000u);
}
// two numbers of 8 bits as bf16
__device__ __forceinline__ uint32_t pack2_cut(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}

// One warp's running state over its tokens, bf16: every 4th stage of 16 tokens of a segment through
// its own ring: 16-byte copies of the tokens' K and V rows, completion by copy groups. The two
// contractions run on warp-level matrix instructions with the tokens as M and the KV head's query
// heads as N (NT tiles of 8): S^T = K Q^T, O^T += V^T P^T. K fragments by ldmatrix, V^T by its
// transposing form (rows padded by 16 bytes: no bank conflicts), Q^T in registers (16 heads of 128: shared memory), P^T
// from the accumulators by movmatrix, in three parts (head_part). The products of 16 tokens are summed
// from zero and added to O^T in fp32: a matrix instruction cuts its sums off, which over thousands of
// tokens in one accumulator goes one way. bf16 outputs unlike those of 64 bits, per 100 000: 64 rows of
// 64 blocks of 64 265 with two parts and one accumulator, 198 with three parts, 241 from zero, 24 with
// both (fp32 sums over fp32 weights: 77); 128 rows of 16 blocks 244, 64, 243, 24 (43). It takes 1 to 3 % of
// the time of the batches above, 6 to 10 % with 16 heads of 128 or several rows of a request, which
// read from L2 (64 rows of 4 requests 162 us, 148 before).
template <int D, int NT>
struct AttendMma {
  using C = Cfg<__nv_bfloat16, D, 8 * NT>;
  static constexpr int KS = D / 16;
  uint32_t qb[C::Q_SHARED ? 1 : NT][C::Q_SHARED ? 1 : KS][2];
  float acc[NT][KS][4], m[NT][2], l[NT][2];

  static __device__ __forceinline__ int next1(int b) { return b == 2 ? 0 : b + 1; }
  static __device__ __forceinline__ int next2(int b) { return b == 0 ? 2 : b - 1; }

  // (the queries in shared memory: before the CTA's next barrier)
  __device__ __forceinline__ void begin(const Params& p, char* smem, int64_t n, int g) {
    const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    const __nv_bfloat16* q0 = (const __nv_bfloat16*)p.a.q +
                              (n * p.a.num_q_heads + (int64_t)g * p.G) * D;
    if constexpr (C::Q_SHARED) {
      char* to = smem + p.slots_at + kSegment * 4;
      for (int x = threadIdx.x; x < NT * 8 * (D / 8); x += kThreads) {
        const int h = x / (D / 8), c = x % (D / 8);
        *(uint4*)(to + h * C::RS + c * 16) =
            h < p.G ? ((const uint4*)(q0 + h * D))[c] : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if constexpr (!C::Q_SHARED) {
        const int h = t * 8 + gid;
        const __nv_bfloat16* q = q0 + (h < p.G ? h : 0) * D;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qb[t][k][0] = h < p.G ? *(const uint32_t*)(q + k * 16 + tig * 2) : 0u;
          qb[t][k][1] = h < p.G ? *(const uint32_t*)(q + k * 16 + tig * 2 + 8) : 0u;
        }
      }
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int i = 0; i < KS; ++i) acc[t][i][0] = acc[t][i][1] = acc[t][i][2] = acc[t][i][3] = 0.f;
    }
  }

  __device__ __forceinline__ void tokens(const Params& p, char* smem, int g, const int* slots,
                                         int n) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, gid = lane >> 2;
    const uint32_t ring = smem_u32(smem) + wid * C::STAGES * C::STAGE;
    const char* kp = (const char*)p.a.k_pool + (int64_t)g * C::RB;
    const char* vp = (const char*)p.a.v_pool + (int64_t)g * C::RB;
    const int64_t slot_bytes = (int64_t)p.a.num_kv_heads * C::RB;
    constexpr int CPR = C::RB / 16, RPI = 32 / CPR;   // copies per row, rows per copy step
    const int cc = (lane % CPR) * 16, rsub = lane / CPR;
    // the stream of a warp: K of its first tokens, their V, K of the next ones, .. (half h: stage
    // wid + 4 (h / 2), K or V), three halves in flight or in use
    const int stages = (n + C::TOK - 1) / C::TOK;
    auto issue = [&](int h, int buf) {
      const int s = wid + (h >> 1) * kWarps;
      if (s < stages) {
        const char* src = h & 1 ? vp : kp;
        const uint32_t dst = ring + buf * C::STAGE + cc;
#pragma unroll
        for (int i = 0; i < C::TOK / RPI; ++i) {
          const int t = i * RPI + rsub, at = s * C::TOK + t;
          const int slot = at < n ? slots[at] : -1;
          cp_async16_or_zero(dst + t * C::RS, src + (int64_t)max(slot, 0) * slot_bytes + cc,
                             slot >= 0);
        }
      }
      cp_async_commit();
    };
    const float qscale = p.a.sm_scale * kLog2e;
    const uint32_t qs = smem_u32(smem) + p.slots_at + kSegment * 4;
    const int k_row = (lane & 7) + ((lane >> 3) & 1) * 8, k_col = (lane >> 4) * 8;
    const int v_row = (lane & 7) + (lane >> 4) * 8, v_col = ((lane >> 3) & 1) * 8;
    issue(0, 0);
    issue(1, 1);
    int buf = 0;   // of K; V is in the next one
    for (int s = wid, h = 0; s < stages; s += kWarps, h += 2, buf = next2(buf)) {
      issue(h + 2, next2(buf));
      cp_async_wait<2>();
      __syncwarp();
      const uint32_t kb = ring + buf * C::STAGE, vb = ring + next1(buf) * C::STAGE;
      float sc[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t r[4];
        ldmatrix_x4(kb + k_row * C::RS + (k * 16 + k_col) * 2, r);
        if constexpr (C::Q_SHARED) {
          uint32_t b[4];   // two tiles of heads
          ldmatrix_x4(qs + v_row * C::RS + (k * 16 + v_col) * 2, b);
          mma_bf16(sc[0], r[0], r[1], r[2], r[3], b[0], b[1]);
          mma_bf16(sc[1], r[0], r[1], r[2], r[3], b[2], b[3]);
        } else {
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma_bf16(sc[t], r[0], r[1], r[2], r[3], qb[t][k][0], qb[t][k][1]);
        }
      }
      __syncwarp();   // K is used up: its place takes the next V
      issue(h + 3, buf);
      const int at = s * C::TOK + gid;
      const bool ok0 = at < n && slots[at] >= 0, ok1 = at + 8 < n && slots[at + 8] >= 0;
      uint32_t w[NT][3][2];
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
          sc[t][e] = exp2f(sc[t][e] - u) * kWeightScale;
          sc[t][2 + e] = exp2f(sc[t][2 + e] - u) * kWeightScale;
          l[t][e] = l[t][e] * al + sc[t][e] + sc[t][2 + e];
          if (__any_sync(0xffffffffu, al != 1.f)) {
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              acc[t][i][e] *= al;
              acc[t][i][2 + e] *= al;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 3; ++j) {   // the rest of each weight: its next part is split off
          float a[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] = j < 2 ? head_part(sc[t][e]) : sc[t][e];
            sc[t][e] -= a[e];
          }
          w[t][j][0] = movmatrix_trans(pack2_cut(a[0], a[1]));
          w[t][j][1] = movmatrix_trans(pack2_cut(a[2], a[3]));
        }
      }
      cp_async_wait<2>();
      __syncwarp();
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        uint32_t r[4];
        ldmatrix_x4_trans(vb + v_row * C::RS + (i * 16 + v_col) * 2, r);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float z[4] = {};   // the least parts first
#pragma unroll
          for (int j = 2; j >= 0; --j) mma_bf16(z, r[0], r[1], r[2], r[3], w[t][j][0], w[t][j][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[t][i][e] += z[e];
        }
      }
      __syncwarp();   // the buffer may be filled again
    }
    cp_async_wait<0>();
  }

  // m (base 2), l and unnormalised o of this warp: sm/sl [kWarps][G], so [kWarps][G][D]
  __device__ __forceinline__ void end(int G, float* sm, float* sl, float* so) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
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
  }
};

// The fp32 form: a warp takes every 4th group of TB tokens, lanes over the dimensions (D / 32
// consecutive ones each), GM >= G query heads. Groups stream through a ring in shared memory; a lane
// reads only what it copied itself. The V = GM * TB scores of a group are summed over the lanes
// together (sum_values), so each lane ends with one score, of head h = its place / TB, takes one
// exponential, and hands its weight to the others through shared memory.
template <int D, int GM>
struct AttendF32 {
  using C = Cfg<float, D, GM>;
  static constexpr int E = D / 32, TB = C::TB, V = GM * TB, SPAN = 32 / V;   // lanes per score
  float q[GM][E], acc[GM][E], m, l;   // m, l: of this lane's head (l: of its token alone)

  __device__ __forceinline__ void begin(const Params& p, char*, int64_t n, int g) {
    const float scale = p.a.sm_scale * kLog2e;
    const float* src = (const float*)p.a.q + (n * p.a.num_q_heads + (int64_t)g * p.G) * D +
                       (threadIdx.x & 31) * E;
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int h = 0; h < GM; ++h)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        q[h][e] = h < p.G ? src[h * D + e] * scale : 0.f;
        acc[h][e] = 0.f;
      }
  }

  __device__ __forceinline__ void tokens(const Params& p, char* smem, int g, const int* slots,
                                         int n) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int64_t base = (int64_t)g * D + lane * E, step = (int64_t)p.a.num_kv_heads * D;
    float* ring = (float*)(smem + wid * C::STAGES * C::STAGE) + lane * E;
    float* weights = (float*)(smem + C::WEIGHTS) + wid * 64;   // then what the heads are scaled by
    const int groups = (n + TB - 1) / TB;
    auto at = [&](int st, int b, int v) { return ring + (st * 2 * TB + 2 * b + v) * D; };
    auto issue = [&](int s, int st) {
      if (s < groups) {
#pragma unroll
        for (int b = 0; b < TB; ++b) {
          const int slot = s * TB + b < n ? slots[s * TB + b] : -1;
          const int64_t off = (int64_t)max(slot, 0) * step + base;
          cp_async_or_zero<4 * E>(smem_u32(at(st, b, 0)), (const float*)p.a.k_pool + off, slot >= 0);
          cp_async_or_zero<4 * E>(smem_u32(at(st, b, 1)), (const float*)p.a.v_pool + off, slot >= 0);
        }
      }
      cp_async_commit();
    };
    int head = 0;
#pragma unroll
    for (; head < C::STAGES - 1; ++head) issue(wid + head * kWarps, head);
    int st = 0;
    for (int s = wid; s < groups; s += kWarps) {
      issue(s + (C::STAGES - 1) * kWarps, st == 0 ? C::STAGES - 1 : st - 1);
      cp_async_wait<C::STAGES - 1>();
      float sc[V];
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        float k[E];
        load_e(at(st, b, 0), k);
#pragma unroll
        for (int h = 0; h < GM; ++h) {
          float x = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) x = fmaf(q[h][e], k[e], x);
          sc[h * TB + b] = x;
        }
      }
      const int mine = s * TB + (lane / SPAN) % TB;
      float x = sum_values<V>(sc);
      x = mine < n && slots[mine] >= 0 ? x : -INFINITY;
      float mx = x;
#pragma unroll
      for (int o = SPAN; o < SPAN * TB; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      // the running maximum moves only when it grows by more than 2^8
      const float top = fmaxf(m, mx);
      const bool grow = top > m + 8.f;
      const float al = grow && m != -INFINITY ? exp2f(m - top) : 1.f;
      if (grow) m = top;
      // 0 for a score of -inf, NaN for one
      const float w = exp2f(x - (m == -INFINITY ? 0.f : m)) * kWeightScale;
      l = l * al + w;
      __syncwarp();   // the last group's weights are used up
      if (lane % SPAN == 0) weights[lane / SPAN] = w;
      const bool rescale = __any_sync(0xffffffffu, al != 1.f);
      if (rescale && lane % (SPAN * TB) == 0) weights[32 + lane / (SPAN * TB)] = al;
      __syncwarp();
      if (rescale) {
#pragma unroll
        for (int h = 0; h < GM; ++h)
#pragma unroll
          for (int e = 0; e < E; ++e) acc[h][e] *= weights[32 + h];
      }
      float v[TB][E];
#pragma unroll
      for (int b = 0; b < TB; ++b) load_e(at(st, b, 1), v[b]);
#pragma unroll
      for (int h = 0; h < GM; ++h) {
        float wt[TB];
        if constexpr (TB == 4)
          *(float4*)wt = *(const float4*)(weights + h * TB);
        else
          *(float2*)wt = *(const float2*)(weights + h * TB);
#pragma unroll
        for (int b = 0; b < TB; ++b)
#pragma unroll
          for (int e = 0; e < E; ++e) acc[h][e] = fmaf(wt[b], v[b][e], acc[h][e]);
      }
      st = st == C::STAGES - 1 ? 0 : st + 1;
    }
    cp_async_wait<0>();
  }

  static __device__ __forceinline__ void load_e(const float* p, float (&v)[E]) {
    if constexpr (E == 4)
      *(float4*)v = *(const float4*)p;
    else
      *(float2*)v = *(const float2*)p;
  }

  __device__ __forceinline__ void end(int G, float* sm, float* sl, float* so) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    float sum = l;
#pragma unroll
    for (int o = SPAN; o < SPAN * TB; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int mine = lane / (SPAN * TB);
    if (lane % (SPAN * TB) == 0 && mine < G) {
      sm[wid * G + mine] = m;
      sl[wid * G + mine] = sum;
    }
#pragma unroll
    for (int h = 0; h < GM; ++h) {
      if (h >= G) break;
#pragma unroll
      for (int e = 0; e < E; ++e) so[(wid * G + h) * D + lane * E + e] = acc[h][e];
    }
  }
};

// Joins `count` states (maxima m(c), sums l(c), unnormalised elements o(c)) in their order. An
// empty state is m = -inf and zeros.
template <typename M, typename L, typename O>
__device__ __forceinline__ void join(int count, M m, L l, O o, float& mx, float& den, float& num) {
  mx = -INFINITY;
  for (int c = 0; c < count; ++c) mx = fmaxf(mx, m(c));
  den = num = 0.f;
  for (int c = 0; c < count; ++c) {
    const float mc = m(c);
    const float k = mc == -INFINITY ? 1.f : exp2f(mc - mx);
    den = fmaf(l(c), k, den);
    num = fmaf(o(c), k, num);
  }
}

// (fp32 is held to the registers of four CTAs per SM, 16 heads of 128 to those of two, in bf16 three)
template <typename T, int D, int GM>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? (D * GM > 1024 ? 3 : 0) : D * GM > 1024 ? 2 : 4)
    sparse_decode_kernel(Params p) {
  using C = Cfg<T, D, GM>;
  extern __shared__ __align__(128) char smem[];
  __shared__ SelectShared sh;
  __shared__ float sm[(kWarps + 1) * GM], sl[(kWarps + 1) * GM];
  const rc_sparse_decode_args& a = p.a;
  const cg::cluster_group cl = cg::this_cluster();
  const int P = p.cluster, G = p.G;
  const int tid = threadIdx.x, wid = tid >> 5;
  const int64_t unit = blockIdx.x / P;
  const int rank = blockIdx.x - (int)unit * P;
  const int64_t n = unit / a.num_kv_heads;
  const int g = (int)(unit - n * a.num_kv_heads);
  const int L = row_len(p, n, rank == 0 && tid == 0 && g == 0);
  const int shift = __ffs(a.block) - 1;
  const int have = (L + a.block - 1) >> shift;
  const int take = min(have, a.top_blocks);
  int* slots = (int*)(smem + p.slots_at);
  int* list = (int*)(smem + p.list_at);
  const bool choose = take < have;   // else every block is taken and none is scored
  if (choose) {
    const int f0 = min(a.sink_blocks, have), f1 = max(f0, have - a.recent_blocks);
    const int m = f1 - f0, k = take - (have - m);   // k of m blocks are taken by their scores
    for (int i = tid; i < f0; i += kThreads) list[i] = i;
    for (int i = tid; i < have - f1; i += kThreads) list[f0 + k + i] = f1 + i;
    if (k > 0) {
      const bool own = p.nb <= kSmemBlocks;
      unsigned long long* r64_s = (unsigned long long*)smem;
      float* score_s = (float*)(smem + p.score_at);
      if (tid == 0) {
        sh.lo = 0xffffffffu;
        sh.hi = sh.tmax = 0;
      }
      if (P > 1) cl.sync(); else __syncthreads();   // every CTA runs and has its words set
      ScoreSink sink{own ? score_s : p.w.score + unit * p.nb, own, P, f0, f1};
      if constexpr (C::kBf16)
        score_tiles<D, GM / 8>(p, n, g, rank * kWarps + wid, P * kWarps, sink);
      else
        score_blocks_f32<D, GM>(p, n, g, rank * kWarps + wid, P * kWarps, sink);
      const uint32_t lo = __reduce_min_sync(0xffffffffu, sink.lo);
      const uint32_t hi = __reduce_max_sync(0xffffffffu, sink.hi);
      const uint32_t tb = __reduce_max_sync(0xffffffffu, __float_as_uint(sink.tmax) & 0x7fffffffu);
      for (int r = tid & 31; r < P; r += 32) {   // a lane tells one CTA
        SelectShared* to = P > 1 ? cl.map_shared_rank(&sh, r) : &sh;
        atomicMin(&to->lo, lo);
        atomicMax(&to->hi, hi);
        atomicMax(&to->tmax, tb);
      }
      if (P > 1) cl.sync(); else __syncthreads();
      int* hist = (int*)(smem + p.hist_at);
      if (own)
        select_blocks<T, D, true>(p, sh, hist, n, g, f0, m, k, score_s, r64_s, list + f0);
      else
        select_blocks<T, D, false>(p, sh, hist, n, g, f0, m, k, p.w.score + unit * p.nb,
                                   p.w.rank + unit * p.nb, list + f0);
    } else {
      __syncthreads();
    }
  } else {
    for (int i = tid; i < take; i += kThreads) list[i] = i;
    __syncthreads();
  }
  if (a.selected && rank == 0)
    for (int i = tid; i < a.top_blocks; i += kThreads)
      a.selected[unit * a.top_blocks + i] = i < take ? list[i] : -1;

  // the newest block is selected and comes last, so it alone may be short: the selected tokens
  // are the first `count` of the listed blocks
  const int count = L - ((have - take) << shift);
  const int share = ((count + P - 1) / P + 15) & ~15;
  const int t0 = min(count, rank * share), t1 = min(count, t0 + share);
  std::conditional_t<C::kBf16, AttendMma<D, (GM + 7) / 8>, AttendF32<D, GM>> at;
  at.begin(p, smem, n, g);
  for (int seg = t0; seg < t1; seg += kSegment) {
    const int len = min(kSegment, t1 - seg);
    const int32_t* rt = a.req_to_token + (int64_t)a.req_idx[n] * a.max_ctx;
    for (int i = tid; i < len; i += kThreads) {
      const int t = seg + i;
      int s = rt[(list[t >> shift] << shift) + (t & (a.block - 1))];
      if (s < 0 || s >= a.num_slots) {
        set_status(p.status, kStatusSlotRange);
        s = -1;
      }
      slots[i] = s;
    }
    __syncthreads();
    at.tokens(p, smem, g, slots, len);
    __syncthreads();
  }
  float* so = (float*)smem;
  at.end(G, sm, sl, so);
  __syncthreads();
  const int64_t o0 = (n * a.num_q_heads + (int64_t)g * G) * D, l0 = n * a.num_q_heads + (int64_t)g * G;
  if (P == 1) {
    for (int x = tid; x < G * D; x += kThreads) {
      const int h = x / D;
      float mx, den, num;
      join(kWarps, [&](int c) { return sm[c * G + h]; }, [&](int c) { return sl[c * G + h]; },
           [&](int c) { return so[c * G * D + x]; }, mx, den, num);
      ((T*)a.o)[o0 + x] = Elem<T>::from_f(den == 0.f ? 0.f : num / den);
      if (a.lse && x % D == 0) a.lse[l0 + h] = den == 0.f ? -INFINITY : log_sum(mx, den);
    }
    return;
  }
  // this CTA's state, then its share of the outputs from all CTAs' states
  float* mo = so + kWarps * G * D;
  float *mm = sm + kWarps * G, *ml = sl + kWarps * G;
  for (int x = tid; x < G * D; x += kThreads) {
    const int h = x / D;
    float mx, den, num;
    join(kWarps, [&](int c) { return sm[c * G + h]; }, [&](int c) { return sl[c * G + h]; },
         [&](int c) { return so[c * G * D + x]; }, mx, den, num);
    mo[x] = num;
    if (x % D == 0) {
      mm[h] = mx;
      ml[h] = den;
    }
  }
  cl.sync();
  const int each = (G * D + P - 1) / P;
  for (int x = rank * each + tid; x < min(G * D, (rank + 1) * each); x += kThreads) {
    const int h = x / D;
    float mx, den, num;
    join(P, [&](int c) { return cl.map_shared_rank(mm, c)[h]; },
         [&](int c) { return cl.map_shared_rank(ml, c)[h]; },
         [&](int c) { return cl.map_shared_rank(mo, c)[x]; }, mx, den, num);
    ((T*)a.o)[o0 + x] = Elem<T>::from_f(den == 0.f ? 0.f : num / den);
    if (a.lse && x % D == 0) a.lse[l0 + h] = den == 0.f ? -INFINITY : log_sum(mx, den);
  }
  cl.sync();   // no CTA leaves while another reads its shared memory
}

// ---------------------------------------------------------------- host side
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
  RC_CHECK_ARG(a->top_blocks > 0 && a->top_blocks <= kMaxTop && a->sink_blocks >= 0 &&
                   a->recent_blocks >= 1 &&
                   (int64_t)a->sink_blocks + a->recent_blocks <= a->top_blocks,
               "%s: top_blocks (at most %d) must hold the sink blocks and at least one recent block",
               fn, kMaxTop);
  RC_CHECK_ARG((int64_t)a->num_rows * a->num_q_heads < (1ll << 28), "%s: too many rows", fn);
  return RC_OK;
}

Params params_of(const rc_sparse_decode_args* a) {
  Params p{};
  p.a = *a;
  p.G = a->num_q_heads / a->num_kv_heads;
  p.nb = std::max(1, (a->max_seq_len + a->block - 1) / a->block);
  return p;
}

Workspace carve(void* base, const Params& p, size_t* total) {
  const size_t cells = p.nb > kSmemBlocks ? (size_t)p.a.num_rows * p.a.num_kv_heads * p.nb : 0;
  Workspace w{};
  char* b = (char*)base;
  w.rank = (unsigned long long*)b;
  w.score = (float*)(b + align256(cells * 8));
  *total = align256(cells * 8) + align256(cells * 4);
  return w;
}

// What fits on the GPU at once: clusters of 2^i CTAs when shared memory lets c CTAs on an SM
// (clusters stay within a group of SMs, so there are fewer than the SMs' room divided by 2^i: of the 608
// places for bf16 heads of 128, 152 units take 39 us with 4 CTAs each and 27 with 2, 36 units 29 with 16
// and 15 with 8; contexts of 8192, 16 blocks of 64 read).
constexpr int kMaxPerSm = 8;
struct Room {
  int per_sm;               // CTAs per SM by registers and threads, at most kMaxPerSm
  int sm_bytes, cta_bytes;  // shared memory of an SM; what a CTA takes beside its dynamic part
  int clusters[kMaxPerSm + 1][5];
  int of(int smem, int i) const {
    return clusters[std::min(per_sm, std::max(1, sm_bytes / (smem + cta_bytes)))][i];
  }
};

cudaLaunchConfig_t launch_config(int64_t ctas, int smem, int cluster, cudaLaunchAttribute* at) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  at->id = cudaLaunchAttributeClusterDimension;
  at->val.clusterDim.x = cluster;
  at->val.clusterDim.y = at->val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

template <typename T, int D, int GM>
cudaError_t room_of(Room& m) {
  const auto kernel = sparse_decode_kernel<T, D, GM>;
  const int most = Cfg<T, D, GM>::MOST;
  cudaFuncAttributes fa = {};
  int dev = 0, reserved = 0;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kernel);
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&m.sm_bytes, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev);
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&m.per_sm, kernel, kThreads, 0);
  m.per_sm = std::min(std::max(m.per_sm, 1), kMaxPerSm);
  m.cta_bytes = (int)fa.sharedSizeBytes + reserved;
  for (int c = 1; c <= m.per_sm && e == cudaSuccess; ++c) {
    const int smem = std::min(most, (m.sm_bytes / c - m.cta_bytes) / 128 * 128);
    for (int i = 0; i < 5 && e == cudaSuccess; ++i) {
      cudaLaunchAttribute at;
      const cudaLaunchConfig_t cfg = launch_config(1 << i, smem, 1 << i, &at);
      e = cudaOccupancyMaxActiveClusters(&m.clusters[c][i], kernel, &cfg);
    }
  }
  return e;
}

template <typename T, int D, int GM>
cudaError_t launch_t(Params p, cudaStream_t s) {
  static PerDevice<Room> setup;
  const Room* room = nullptr;
  cudaError_t e = setup.get(room_of<T, D, GM>, &room);
  if (e != cudaSuccess) return e;
  const int smem = Cfg<T, D, GM>::layout(p);
  // CTAs per unit (us, contexts of 8192 in blocks of 64). Few units are split while all clusters fit
  // at once and each CTA has two stages for every warp: beyond that a split only adds joins (bf16,
  // 32+8 heads of 128, 16 blocks read: 40 units 16.5 in one wave, 31.0 with twice the CTAs, 96 units
  // 20.4 and 33.3, 320 units 50.6 and 67.5; fp32, 8+8 heads, 40 units 17.0 and 32.8). More units than
  // fit whole are split where a CTA would read over 2048 tokens, which shortens the last wave (640
  // units of 64 blocks: bf16 273 split, 315 whole; fp32 475 and 550); fewer are not (320 units of 64
  // blocks: 141 whole, 180 split).
  const int64_t units = (int64_t)p.a.num_rows * p.a.num_kv_heads;
  const int64_t tokens = (int64_t)std::min(p.nb, p.a.top_blocks) * p.a.block;
  p.cluster = 1;
  for (int i = 1; 2 * p.cluster <= kMaxCluster && tokens >= 128 * p.cluster &&
                  2 * p.cluster * units < (1ll << 31) &&
                  (units <= room->of(smem, i) ||
                   (units > room->of(smem, 0) && tokens > 2048 * p.cluster));
       ++i)
    p.cluster *= 2;
  cudaLaunchAttribute at;
  cudaLaunchConfig_t cfg = launch_config(units * p.cluster, smem, p.cluster, &at);
  cfg.stream = s;
  e = cudaLaunchKernelEx(&cfg, sparse_decode_kernel<T, D, GM>, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <int D>
cudaError_t launch_d(const Params& p, cudaStream_t s) {
  if (p.a.dtype == RC_DTYPE_BF16)
    return p.G <= 8 ? launch_t<__nv_bfloat16, D, 8>(p, s) : launch_t<__nv_bfloat16, D, 16>(p, s);
  if (p.G <= 1) return launch_t<float, D, 1>(p, s);
  if (p.G <= 4) return launch_t<float, D, 4>(p, s);
  if (p.G <= 8) return launch_t<float, D, 8>(p, s);
  return launch_t<float, D, 16>(p, s);
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
                   a->bounds && a->o,
               "%s: NULL pointer", fn);
  const uintptr_t al = (uintptr_t)a->q | (uintptr_t)a->k_pool | (uintptr_t)a->v_pool |
                       (uintptr_t)a->bounds | (uintptr_t)a->o | (uintptr_t)workspace;
  RC_CHECK_ARG((al & 15) == 0, "%s: tensors and workspace must be 16-byte aligned", fn);
  rc::Params p = rc::params_of(a);
  size_t need = 0;
  p.w = rc::carve(workspace, p, &need);
  RC_CHECK_ARG(need == 0 || (workspace && workspace_bytes >= need),
               "%s: workspace %zu bytes < %zu needed", fn, workspace ? workspace_bytes : 0, need);
  p.status = rc::device_status_ptr();
  if (!p.status) return rc::fail(RC_ERR_CUDA, "%s: no device status word", fn);
  const cudaError_t e = a->head_dim == 128 ? rc::launch_d<128>(p, (cudaStream_t)stream)
                                           : rc::launch_d<64>(p, (cudaStream_t)stream);
  if (e != cudaSuccess)
    return rc::fail(RC_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return rc::check_launch(fn);
}
