// Appending keys and values to the paged cache, the keys normalised and rotated on the way, and
// the bounds of cached keys block by block that sparse_decode.cu selects blocks with.
//
// Work items are (request, block of positions the new tokens touch, group of KV heads), so one CTA
// owns every new key of a (block, head) and reduces its bounds without atomics: a block that the
// new tokens begin gets their bounds, a block that cached tokens began takes the minimum and
// maximum with what it holds (which makes a repeated append of the same tokens change nothing).
// CTAs walk the items grid-stride; requests are taken in windows of kWindow, whose item offsets
// each CTA sums up in shared memory, so neither their number nor their lengths need to be known on
// the host.
#include <algorithm>

#include "host_common.h"
#include "norm_rope.cuh"
#include "warp_mma.cuh"

namespace rc {
namespace {

constexpr int kThreads = 256;
constexpr int kWindow = 1024;   // requests whose item offsets a CTA holds at a time

// off[k] = items of the window's requests before k (off[n] = all), each of n <= kWindow requests
// having count(k) items. All threads of the CTA call it.
template <typename F>
__device__ void window_offsets(int* off, int* warp_sums, int n, F count) {
  constexpr int PER = kWindow / kThreads;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int c[PER], sum = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int k = threadIdx.x * PER + j;
    c[j] = k < n ? count(k) : 0;
    sum += c[j];
  }
  int v = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();   // the last window's readers are done with off and warp_sums
  if (lane == 31) warp_sums[wid] = v;
  __syncthreads();
  int base = v - sum;
  for (int w = 0; w < wid; ++w) base += warp_sums[w];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    off[threadIdx.x * PER + j] = base;
    base += c[j];
  }
  if (threadIdx.x == kThreads - 1) off[kWindow] = base;
  __syncthreads();
}
// the request k of the window with off[k] <= item < off[k + 1]
__device__ __forceinline__ int find_request(const int* off, int n, int item) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= item) lo = mid; else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------- append
// Request b's new tokens: positions P .. P + S - 1, rows t0 .. t0 + S - 1 of k and v. S = 0 for a
// request with bad data (recorded once, by `report`).
struct Span {
  int t0, P, S, row;
};
__device__ __forceinline__ Span span_of(const rc_kv_append_args& a, int b, int* status,
                                        bool report) {
  Span s;
  s.t0 = a.qo_indptr[b];
  s.S = a.qo_indptr[b + 1] - s.t0;
  s.P = a.prefix_len[b];
  s.row = a.bounds ? a.req_idx[b] : 0;
  bool ok = s.t0 >= 0 && s.S >= 0 && (int64_t)s.t0 + s.S <= a.num_tokens && s.P >= 0 &&
            (int64_t)s.P + s.S <= 0x7fffffff;
  if (ok && s.S > 0) {
    const int64_t last = (int64_t)s.P + s.S - 1;
    if (a.rotary_dim && last >= a.max_position) ok = false;
    if (a.bounds && (s.row < 0 || s.row >= a.max_reqs || last / a.block >= a.max_blocks)) ok = false;
  }
  if (!ok) {
    if (report) set_status(status, kStatusPosRange);
    s.S = 0;
  }
  return s;
}

// Least and greatest elements of 16-byte chunks, NaN kept: pairs of bf16, or single fp32.
template <typename T>
struct Extremes;
template <>
struct Extremes<__nv_bfloat16> {
  static constexpr uint32_t kLo = 0x7f807f80u, kHi = 0xff80ff80u;   // inf, -inf
  static __device__ __forceinline__ uint32_t lo(uint32_t a, uint32_t b) { return min_nan_bf16x2(a, b); }
  static __device__ __forceinline__ uint32_t hi(uint32_t a, uint32_t b) { return max_nan_bf16x2(a, b); }
};
template <>
struct Extremes<float> {
  static constexpr uint32_t kLo = 0x7f800000u, kHi = 0xff800000u;
  static __device__ __forceinline__ uint32_t lo(uint32_t a, uint32_t b) {
    return __float_as_uint(min_nan(__uint_as_float(a), __uint_as_float(b)));
  }
  static __device__ __forceinline__ uint32_t hi(uint32_t a, uint32_t b) {
    return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
  }
};
template <typename T>
__device__ __forceinline__ void lower(uint4& a, const uint4& b) {
  a = make_uint4(Extremes<T>::lo(a.x, b.x), Extremes<T>::lo(a.y, b.y), Extremes<T>::lo(a.z, b.z),
                 Extremes<T>::lo(a.w, b.w));
}
template <typename T>
__device__ __forceinline__ void raise(uint4& a, const uint4& b) {
  a = make_uint4(Extremes<T>::hi(a.x, b.x), Extremes<T>::hi(a.y, b.y), Extremes<T>::hi(a.z, b.z),
                 Extremes<T>::hi(a.w, b.w));
}
__device__ __forceinline__ uint4 splat(uint32_t x) { return make_uint4(x, x, x, x); }

// TOK tokens of a thread are in flight together.
template <typename T, int L, int TOK>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(rc_kv_append_args a, int heads_per_cta,
                                                             int head_groups, int* status) {
  constexpr int ROWS = kThreads / L;   // (token, head) rows a pass of the CTA covers
  constexpr int N = Raw<T>::N;
  __shared__ int off[kWindow + 1];
  __shared__ int warp_sums[kThreads / 32];
  __shared__ uint4 red[4 * N][kThreads];   // extremes of 16 elements per thread
  const int d = a.head_dim, r = a.rotary_dim;
  const bool inter = a.interleaved != 0;
  const int i = threadIdx.x % L, row_in = threadIdx.x / L;
  const int hl = row_in % heads_per_cta, w = row_in / heads_per_cta;
  const int W = ROWS / heads_per_cta;   // tokens a pass covers; threads past W * heads idle
  const LaneChunks lc = lane_chunks(i, d, r, inter);
  const T* kw = (const T*)a.k_weight;

  for (int b0 = 0; b0 < a.num_reqs; b0 += kWindow) {
    const int nreq = min(kWindow, a.num_reqs - b0);
    window_offsets(off, warp_sums, nreq, [&](int k) {
      const Span s = span_of(a, b0 + k, status, blockIdx.x == 0);
      return s.S ? (s.P + s.S - 1) / a.block - s.P / a.block + 1 : 0;
    });
    const int64_t items = (int64_t)off[kWindow] * head_groups;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
      const int job = (int)(it / head_groups), hg = (int)(it - (int64_t)job * head_groups);
      const int k = find_request(off, nreq, job);
      const Span s = span_of(a, b0 + k, status, false);
      const int blk = s.P / a.block + (job - off[k]);
      const int p0 = max(s.P, blk * a.block);
      const int p1 = (int)min((int64_t)s.P + s.S, (int64_t)(blk + 1) * a.block);
      const int h = hg * heads_per_cta + hl;
      const bool mine = h < a.num_kv_heads && w < W;
      const bool m0 = mine && lc.c0 >= 0, m1 = mine && lc.c1 >= 0;
      T* cell = (T*)a.bounds +
                ((((int64_t)s.row * a.max_blocks + blk) * a.num_kv_heads + h) * 2) * d;
      Raw<T> lo0, lo1, hi0, hi1;
#pragma unroll
      for (int c = 0; c < N; ++c) {
        lo0.v[c] = lo1.v[c] = splat(Extremes<T>::kLo);
        hi0.v[c] = hi1.v[c] = splat(Extremes<T>::kHi);
      }
      if (a.bounds && w == 0 && blk * a.block < s.P) {   // cached tokens began the block
        if (m0) {
          lo0.load(cell + lc.c0 * 8);
          hi0.load(cell + d + lc.c0 * 8);
        }
        if (m1) {
          lo1.load(cell + lc.c1 * 8);
          hi1.load(cell + d + lc.c1 * 8);
        }
      }
      for (int p = p0; p < p1; p += W * TOK) {   // the same count for every thread: shuffles inside
        Raw<T> x0[TOK], x1[TOK], y0[TOK], y1[TOK];
        LaneAngles ang[TOK];
        int slot[TOK];
#pragma unroll
        for (int u = 0; u < TOK; ++u) {
          const int pos = p + u * W + w;
          const int64_t t = s.t0 + (int64_t)(pos - s.P);
          const bool in = pos < p1;
          slot[u] = mine && in ? a.out_loc[t] : 0;
          const T* ks = (const T*)a.k + t * a.k_token_stride + (int64_t)h * a.k_head_stride;
          const T* vs = (const T*)a.v + t * a.v_token_stride + (int64_t)h * a.v_head_stride;
          x0[u].clear();
          x1[u].clear();
          if (m0 && in) x0[u].load(ks + lc.c0 * 8);
          if (m1 && in) x1[u].load(ks + lc.c1 * 8);
          if (m0 && in) y0[u].load(vs + lc.c0 * 8);
          if (m1 && in) y1[u].load(vs + lc.c1 * 8);
          if (lc.rot && mine && in) load_angles(a.rope + (int64_t)pos * r, i, r, ang[u]);
        }
#pragma unroll
        for (int u = 0; u < TOK; ++u) {
          const bool in = p + u * W + w < p1;
          bool live = mine && in;
          if (live && (slot[u] < 0 || slot[u] >= a.num_slots)) {
            if (i == 0) set_status(status, kStatusSlotRange);
            live = false;
          }
          if (kw || r) {
            float x[8], y[8];
            x0[u].get(x);
            x1[u].get(y);
            if (kw) {
              const float inv = norm_scale<L>(x, y, d, a.eps);
              if (m0) scale8(x, inv, kw + lc.c0 * 8);
              if (m1) scale8(y, inv, kw + lc.c1 * 8);
            }
            if (lc.rot) rotate_pairs(x, y, inter, ang[u]);
            x0[u].set(x);
            x1[u].set(y);
          }
          const int64_t dst = ((int64_t)slot[u] * a.num_kv_heads + h) * d;
          if (live && lc.c0 >= 0) {
            x0[u].store((T*)a.k_pool + dst + lc.c0 * 8);
            y0[u].store((T*)a.v_pool + dst + lc.c0 * 8);
          }
          if (live && lc.c1 >= 0) {
            x1[u].store((T*)a.k_pool + dst + lc.c1 * 8);
            y1[u].store((T*)a.v_pool + dst + lc.c1 * 8);
          }
          if (a.bounds && live) {   // the extremes of the stored (rounded) keys
#pragma unroll
            for (int c = 0; c < N; ++c) {
              lower<T>(lo0.v[c], x0[u].v[c]);
              raise<T>(hi0.v[c], x0[u].v[c]);
              lower<T>(lo1.v[c], x1[u].v[c]);
              raise<T>(hi1.v[c], x1[u].v[c]);
            }
          }
        }
      }
      if (!a.bounds) continue;
      if (W > 1 && p1 - p0 > 1) {   // join the token lanes (uniform over the CTA)
#pragma unroll
        for (int c = 0; c < N; ++c) {
          red[c][threadIdx.x] = lo0.v[c];
          red[N + c][threadIdx.x] = lo1.v[c];
          red[2 * N + c][threadIdx.x] = hi0.v[c];
          red[3 * N + c][threadIdx.x] = hi1.v[c];
        }
        __syncthreads();
        if (w == 0) {
          for (int u = 1; u < W && p0 + u < p1; ++u) {
            const int o = threadIdx.x + u * heads_per_cta * L;
#pragma unroll
            for (int c = 0; c < N; ++c) {
              lower<T>(lo0.v[c], red[c][o]);
              lower<T>(lo1.v[c], red[N + c][o]);
              raise<T>(hi0.v[c], red[2 * N + c][o]);
              raise<T>(hi1.v[c], red[3 * N + c][o]);
            }
          }
        }
        __syncthreads();
      }
      if (w == 0 && m0) {
        lo0.store(cell + lc.c0 * 8);
        hi0.store(cell + d + lc.c0 * 8);
      }
      if (w == 0 && m1) {
        lo1.store(cell + lc.c1 * 8);
        hi1.store(cell + d + lc.c1 * 8);
      }
    }
  }
}

// ---------------------------------------------------------------- bounds of cached keys
// Work items are (layer, row, block, column group of 16-byte chunks); a thread keeps the extremes
// of one chunk over every W-th token of the block, kFly of them in flight.
constexpr int kFly = 8;

template <typename T>
__global__ void __launch_bounds__(kThreads) kv_block_bounds_kernel(rc_kv_block_bounds_args a,
                                                                   int chunks_per_cta, int col_groups,
                                                                   int* status) {
  constexpr int V = 16 / (int)sizeof(T);   // elements of a chunk
  __shared__ int off[kWindow + 1];
  __shared__ int warp_sums[kThreads / 32];
  __shared__ uint4 red[2][kThreads];
  const int d = a.head_dim;
  const int chunks = a.num_kv_heads * d / V;
  const int cl = threadIdx.x % chunks_per_cta, w = threadIdx.x / chunks_per_cta;
  const int W = kThreads / chunks_per_cta;
  for (int b0 = 0; b0 < a.num_rows; b0 += kWindow) {
    const int nreq = min(kWindow, a.num_rows - b0);
    window_offsets(off, warp_sums, nreq, [&](int k) {
      const int L = a.seq_len[b0 + k], row = a.req_idx[b0 + k];
      if (L < 0 || L > a.max_ctx || row < 0 || row >= a.max_reqs ||
          (L - 1) / a.block >= a.max_blocks) {
        if (blockIdx.x == 0) set_status(status, kStatusPosRange);
        return 0;
      }
      return (L + a.block - 1) / a.block;
    });
    const int64_t per_layer = (int64_t)off[kWindow] * col_groups;
    const int64_t items = per_layer * a.num_layers;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
      const int64_t layer = it / per_layer;
      const int64_t rest = it - layer * per_layer;
      const int job = (int)(rest / col_groups), cg = (int)(rest - (int64_t)job * col_groups);
      const int k = find_request(off, nreq, job);
      const int L = a.seq_len[b0 + k], row = a.req_idx[b0 + k];
      const int blk = job - off[k];
      const int p0 = blk * a.block, p1 = (int)min((int64_t)L, (int64_t)p0 + a.block);
      const int c = cg * chunks_per_cta + cl;
      const bool mine = c < chunks && w < W;
      const int32_t* rt = a.req_to_token + (int64_t)row * a.max_ctx;
      const uint4* kp = (const uint4*)((const T*)a.k_pool +
                                       layer * a.num_slots * a.num_kv_heads * d) + c;
      uint4 lo = splat(Extremes<T>::kLo), hi = splat(Extremes<T>::kHi);
      for (int p = p0 + w; mine && p < p1; p += W * kFly) {
        int slot[kFly];
        uint4 v[kFly];
#pragma unroll
        for (int u = 0; u < kFly; ++u) slot[u] = p + u * W < p1 ? rt[p + u * W] : -2;
#pragma unroll
        for (int u = 0; u < kFly; ++u) {
          if (slot[u] == -2 && p + u * W >= p1) continue;
          if (slot[u] < 0 || slot[u] >= a.num_slots) {
            if (cl == 0) set_status(status, kStatusSlotRange);
            slot[u] = -2;
          } else {
            v[u] = kp[(int64_t)slot[u] * chunks];
          }
        }
#pragma unroll
        for (int u = 0; u < kFly; ++u) {
          if (slot[u] != -2) {
            lower<T>(lo, v[u]);
            raise<T>(hi, v[u]);
          }
        }
      }
      if (W > 1) {
        red[0][threadIdx.x] = lo;
        red[1][threadIdx.x] = hi;
        __syncthreads();
        if (w == 0) {
          for (int u = 1; u < W; ++u) {
            const int o = threadIdx.x + u * chunks_per_cta;
            lower<T>(lo, red[0][o]);
            raise<T>(hi, red[1][o]);
          }
        }
        __syncthreads();
      }
      if (w == 0 && mine) {
        const int h = c * V / d, e0 = c * V - h * d;
        T* cell = (T*)a.bounds +
                  ((((layer * a.max_reqs + row) * a.max_blocks + blk) * a.num_kv_heads + h) * 2) * d;
        *(uint4*)(cell + e0) = lo;
        *(uint4*)(cell + d + e0) = hi;
      }
    }
  }
}

bool block_ok(int block) { return block == 16 || block == 32 || block == 64 || block == 128; }

template <typename T, int L>
void launch_append(const rc_kv_append_args& a, int sms, int* st, cudaStream_t s) {
  // single tokens: every thread a head; prompts: 8 tokens of a block beside one another
  const bool prompts = a.num_tokens >= 16 * (int64_t)a.num_reqs;
  const int hpc = std::min(a.num_kv_heads, prompts ? std::max(1, kThreads / L / 8) : kThreads / L);
  const int hg = (a.num_kv_heads + hpc - 1) / hpc;
  // blocks the tokens can touch: each request begins and ends inside at most two more
  const int64_t most = (a.num_tokens / a.block + 2 * (int64_t)a.num_reqs) * hg;
  const int grid = (int)std::min<int64_t>(std::max<int64_t>(most, 1), (int64_t)sms * 4);
  if (prompts)
    kv_append_kernel<T, L, 2><<<grid, kThreads, 0, s>>>(a, hpc, hg, st);
  else
    kv_append_kernel<T, L, 1><<<grid, kThreads, 0, s>>>(a, hpc, hg, st);
}

template <typename T>
void launch_append(const rc_kv_append_args& a, int sms, int* st, cudaStream_t s) {
  switch (head_lanes(a.head_dim)) {
    case 4: launch_append<T, 4>(a, sms, st, s); break;
    case 8: launch_append<T, 8>(a, sms, st, s); break;
    default: launch_append<T, 16>(a, sms, st, s); break;
  }
}

}  // namespace
}  // namespace rc

extern "C" int rc_kv_append(const rc_kv_append_args* a, void* stream) {
  static const char* fn = "rc_kv_append";
  RC_CHECK_ARG(a != nullptr, "%s: args is NULL", fn);
  RC_CHECK_ARG(a->dtype == RC_DTYPE_BF16 || a->dtype == RC_DTYPE_F32, "%s: dtype %d", fn, a->dtype);
  RC_CHECK_ARG(a->num_reqs >= 0 && a->num_tokens >= 0 && a->num_tokens <= 0x7fffffff &&
                   a->num_kv_heads > 0 && a->num_kv_heads <= 65536 && a->num_slots > 0,
               "%s: bad sizes", fn);
  const int c = rc::check_norm_rope(fn, a->head_dim, a->rotary_dim, a->max_position, a->rope, a->eps,
                                    a->k_weight != nullptr);
  if (c != RC_OK) return c;
  RC_CHECK_ARG(rc::block_ok(a->block), "%s: block %d (16, 32, 64 or 128)", fn, a->block);
  RC_CHECK_ARG(!a->bounds || (a->req_idx && a->max_reqs > 0 && a->max_blocks > 0),
               "%s: bounds without rows, blocks or req_idx", fn);
  if (a->num_reqs == 0 || a->num_tokens == 0) return RC_OK;
  RC_CHECK_ARG(a->k && a->v && a->out_loc && a->qo_indptr && a->prefix_len && a->k_pool && a->v_pool,
               "%s: NULL pointer", fn);
  const uintptr_t ptrs = (uintptr_t)a->k | (uintptr_t)a->v | (uintptr_t)a->k_pool |
                         (uintptr_t)a->v_pool | (uintptr_t)a->k_weight | (uintptr_t)a->bounds;
  const int64_t strides =
      a->k_token_stride | a->k_head_stride | a->v_token_stride | a->v_head_stride;
  const int es = a->dtype == RC_DTYPE_BF16 ? 2 : 4;
  RC_CHECK_ARG((ptrs & 15) == 0 && (strides * es & 15) == 0,
               "%s: pointers and strides must be multiples of 16 bytes", fn);
  int* st = rc::device_status_ptr();
  if (!st) return rc::fail(RC_ERR_CUDA, "%s: no device status word", fn);
  int sms = 0;
  const int e = rc::sm_count(fn, &sms);
  if (e != RC_OK) return e;
  if (a->dtype == RC_DTYPE_BF16)
    rc::launch_append<__nv_bfloat16>(*a, sms, st, (cudaStream_t)stream);
  else
    rc::launch_append<float>(*a, sms, st, (cudaStream_t)stream);
  rc::count_launches(1);
  return rc::check_launch(fn);
}

extern "C" int rc_kv_block_bounds(const rc_kv_block_bounds_args* a, void* stream) {
  static const char* fn = "rc_kv_block_bounds";
  RC_CHECK_ARG(a != nullptr, "%s: args is NULL", fn);
  RC_CHECK_ARG(a->dtype == RC_DTYPE_BF16 || a->dtype == RC_DTYPE_F32, "%s: dtype %d", fn, a->dtype);
  RC_CHECK_ARG(a->num_layers > 0 && a->num_rows >= 0 && a->num_kv_heads > 0 &&
                   a->num_kv_heads <= 65536 && a->num_slots > 0 && a->max_reqs > 0 &&
                   a->max_ctx > 0 && a->max_ctx <= (1 << 24) && a->max_blocks > 0,
               "%s: bad sizes", fn);
  RC_CHECK_ARG(a->head_dim >= 8 && a->head_dim <= rc::kNormRopeMaxDim && a->head_dim % 8 == 0,
               "%s: head_dim %d (a multiple of 8 up to %d)", fn, a->head_dim, rc::kNormRopeMaxDim);
  RC_CHECK_ARG(rc::block_ok(a->block), "%s: block %d (16, 32, 64 or 128)", fn, a->block);
  if (a->num_rows == 0) return RC_OK;
  RC_CHECK_ARG(a->seq_len && a->req_idx && a->req_to_token && a->k_pool && a->bounds,
               "%s: NULL pointer", fn);
  RC_CHECK_ARG((((uintptr_t)a->k_pool | (uintptr_t)a->bounds) & 15) == 0,
               "%s: k_pool and bounds must be 16-byte aligned", fn);
  int* st = rc::device_status_ptr();
  if (!st) return rc::fail(RC_ERR_CUDA, "%s: no device status word", fn);
  int sms = 0;
  const int e = rc::sm_count(fn, &sms);
  if (e != RC_OK) return e;
  const int chunks = a->num_kv_heads * a->head_dim * (a->dtype == RC_DTYPE_BF16 ? 2 : 4) / 16;
  const int cpc = std::min(chunks, rc::kThreads);
  const int cg = (chunks + cpc - 1) / cpc;
  const int64_t most = (int64_t)a->num_layers * a->num_rows * a->max_blocks * cg;
  const int grid = (int)std::min<int64_t>(most, (int64_t)sms * 8);
  cudaStream_t s = (cudaStream_t)stream;
  if (a->dtype == RC_DTYPE_BF16)
    rc::kv_block_bounds_kernel<__nv_bfloat16><<<grid, rc::kThreads, 0, s>>>(*a, cpc, cg, st);
  else
    rc::kv_block_bounds_kernel<float><<<grid, rc::kThreads, 0, s>>>(*a, cpc, cg, st);
  rc::count_launches(1);
  return rc::check_launch(fn);
}
