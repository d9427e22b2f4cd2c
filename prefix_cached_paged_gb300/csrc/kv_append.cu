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
__device__ __forceinline__ int find_request(const int* off, int item) {
  int lo = 0, hi = kWindow;
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

template <typename T, int L>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(rc_kv_append_args a, int heads_per_cta,
                                                             int head_groups, int* status) {
  constexpr int ROWS = kThreads / L;   // (token, head) rows a pass of the CTA covers
  __shared__ int off[kWindow + 1];
  __shared__ int warp_sums[kThreads / 32];
  __shared__ float red[kThreads * 32];   // lo and hi of 16 elements per thread
  const int d = a.head_dim, r = a.rotary_dim;
  const bool inter = a.interleaved != 0;
  const int i = threadIdx.x % L, row_in = threadIdx.x / L;
  const int hl = row_in % heads_per_cta, w = row_in / heads_per_cta;
  const int W = ROWS / heads_per_cta;   // tokens a pass covers; threads past W * heads idle
  const LaneChunks lc = lane_chunks(i, d, r, inter);
  const T* kw = (const T*)a.k_weight;
  float g0[8], g1[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) g0[e] = g1[e] = 1.f;
  if (kw && lc.c0 >= 0) load8(kw + lc.c0 * 8, g0);
  if (kw && lc.c1 >= 0) load8(kw + lc.c1 * 8, g1);

  for (int b0 = 0; b0 < a.num_reqs; b0 += kWindow) {
    window_offsets(off, warp_sums, min(kWindow, a.num_reqs - b0), [&](int k) {
      const Span s = span_of(a, b0 + k, status, blockIdx.x == 0);
      return s.S ? (s.P + s.S - 1) / a.block - s.P / a.block + 1 : 0;
    });
    const int64_t items = (int64_t)off[kWindow] * head_groups;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
      const int job = (int)(it / head_groups), hg = (int)(it - (int64_t)job * head_groups);
      const int k = find_request(off, job);
      const Span s = span_of(a, b0 + k, status, false);
      const int blk = s.P / a.block + (job - off[k]);
      const int p0 = max(s.P, blk * a.block);
      const int p1 = (int)min((int64_t)s.P + s.S, (int64_t)(blk + 1) * a.block);
      const int h = hg * heads_per_cta + hl;
      const bool mine = h < a.num_kv_heads && w < W;
      float lo[16], hi[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) { lo[e] = INFINITY; hi[e] = -INFINITY; }
      for (int p = p0; p < p1; p += W) {   // the same count for every thread: shuffles inside
        const int pos = p + w;
        const int64_t t = s.t0 + (pos - s.P);
        bool live = mine && pos < p1;
        int64_t dst = 0;
        if (live) {
          const int sl = a.out_loc[t];
          if (sl < 0 || sl >= a.num_slots) {
            if (i == 0) set_status(status, kStatusSlotRange);
            live = false;
          } else {
            dst = ((int64_t)sl * a.num_kv_heads + h) * d;
          }
        }
        const bool v0 = live && lc.c0 >= 0, v1 = live && lc.c1 >= 0;
        const T* ks = (const T*)a.k + t * a.k_token_stride + (int64_t)h * a.k_head_stride;
        const T* vs = (const T*)a.v + t * a.v_token_stride + (int64_t)h * a.v_head_stride;
        float x[8] = {}, y[8] = {};
        if (v0) load8(ks + lc.c0 * 8, x);
        if (v1) load8(ks + lc.c1 * 8, y);
        if (v0) copy8((T*)a.v_pool + dst + lc.c0 * 8, vs + lc.c0 * 8);
        if (v1) copy8((T*)a.v_pool + dst + lc.c1 * 8, vs + lc.c1 * 8);
        if (kw) {
          const float inv = norm_scale<L>(x, y, d, a.eps);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] *= inv * g0[e];
            y[e] *= inv * g1[e];
          }
        }
        if (r && live && lc.rot) {
          LaneAngles ang;
          load_angles(a.rope + (int64_t)pos * r, i, r, ang);
          rotate_pairs(x, y, inter, ang);
        }
        if (v0) store8((T*)a.k_pool + dst + lc.c0 * 8, x);
        if (v1) store8((T*)a.k_pool + dst + lc.c1 * 8, y);
        if (a.bounds && live) {
          // the bounds are those of the stored (rounded) keys
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float xr = Elem<T>::to_f(Elem<T>::from_f(x[e]));
            const float yr = Elem<T>::to_f(Elem<T>::from_f(y[e]));
            lo[e] = min_nan(lo[e], xr);
            hi[e] = max_nan(hi[e], xr);
            lo[8 + e] = min_nan(lo[8 + e], yr);
            hi[8 + e] = max_nan(hi[8 + e], yr);
          }
        }
      }
      if (!a.bounds) continue;
      if (W > 1 && p1 - p0 > 1) {   // join the token lanes (uniform over the CTA)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          red[e * kThreads + threadIdx.x] = lo[e];
          red[(16 + e) * kThreads + threadIdx.x] = hi[e];
        }
        __syncthreads();
        if (w == 0) {
          for (int u = 1; u < W && p0 + u < p1; ++u) {
            const int o = threadIdx.x + u * heads_per_cta * L;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              lo[e] = min_nan(lo[e], red[e * kThreads + o]);
              hi[e] = max_nan(hi[e], red[(16 + e) * kThreads + o]);
            }
          }
        }
        __syncthreads();
      }
      if (w == 0 && mine) {
        T* cell = (T*)a.bounds +
                  ((((int64_t)s.row * a.max_blocks + blk) * a.num_kv_heads + h) * 2) * d;
        const bool began = blk * a.block >= s.P;   // no cached token lies in this block
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int cc = c ? lc.c1 : lc.c0;
          if (cc < 0) continue;
          if (!began) {
            float v[8];
            load8(cell + cc * 8, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) lo[c * 8 + e] = min_nan(lo[c * 8 + e], v[e]);
            load8(cell + d + cc * 8, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) hi[c * 8 + e] = max_nan(hi[c * 8 + e], v[e]);
          }
          store8(cell + cc * 8, lo + c * 8);
          store8(cell + d + cc * 8, hi + c * 8);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- bounds of cached keys
// Work items are (layer, row, block, column group of 16-byte chunks); a thread keeps the bounds of
// one chunk over every W-th token of the block.
template <typename T>
__global__ void __launch_bounds__(kThreads) kv_block_bounds_kernel(rc_kv_block_bounds_args a,
                                                                   int chunks_per_cta, int col_groups,
                                                                   int* status) {
  constexpr int V = 8;   // elements of a chunk
  __shared__ int off[kWindow + 1];
  __shared__ int warp_sums[kThreads / 32];
  __shared__ float red[kThreads * 2 * V];
  const int d = a.head_dim;
  const int chunks = a.num_kv_heads * d / V;
  const int cl = threadIdx.x % chunks_per_cta, w = threadIdx.x / chunks_per_cta;
  const int W = kThreads / chunks_per_cta;
  for (int b0 = 0; b0 < a.num_rows; b0 += kWindow) {
    window_offsets(off, warp_sums, min(kWindow, a.num_rows - b0), [&](int k) {
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
      const int k = find_request(off, job);
      const int L = a.seq_len[b0 + k], row = a.req_idx[b0 + k];
      const int blk = job - off[k];
      const int p0 = blk * a.block, p1 = (int)min((int64_t)L, (int64_t)p0 + a.block);
      const int c = cg * chunks_per_cta + cl;
      const bool mine = c < chunks && w < W;
      const int32_t* rt = a.req_to_token + (int64_t)row * a.max_ctx;
      const T* kp = (const T*)a.k_pool + layer * a.num_slots * a.num_kv_heads * d;
      float lo[V], hi[V];
#pragma unroll
      for (int e = 0; e < V; ++e) { lo[e] = INFINITY; hi[e] = -INFINITY; }
      for (int p = p0 + w; mine && p < p1; p += W) {
        const int sl = rt[p];
        if (sl < 0 || sl >= a.num_slots) {
          if (cl == 0) set_status(status, kStatusSlotRange);
          continue;
        }
        float v[V];
        load8(kp + (int64_t)sl * a.num_kv_heads * d + c * V, v);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          lo[e] = min_nan(lo[e], v[e]);
          hi[e] = max_nan(hi[e], v[e]);
        }
      }
      if (W > 1) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          red[e * kThreads + threadIdx.x] = lo[e];
          red[(V + e) * kThreads + threadIdx.x] = hi[e];
        }
        __syncthreads();
        if (w == 0) {
          for (int u = 1; u < W; ++u) {
            const int o = threadIdx.x + u * chunks_per_cta;
#pragma unroll
            for (int e = 0; e < V; ++e) {
              lo[e] = min_nan(lo[e], red[e * kThreads + o]);
              hi[e] = max_nan(hi[e], red[(V + e) * kThreads + o]);
            }
          }
        }
        __syncthreads();
      }
      if (w == 0 && mine) {
        const int h = c * V / d, e0 = c * V - h * d;
        T* cell = (T*)a.bounds +
                  ((((layer * a.max_reqs + row) * a.max_blocks + blk) * a.num_kv_heads + h) * 2) * d;
        store8(cell + e0, lo);
        store8(cell + d + e0, hi);
      }
    }
  }
}

bool block_ok(int block) { return block == 16 || block == 32 || block == 64 || block == 128; }

int sm_count(int* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return fail(RC_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
  return RC_OK;
}

template <typename T>
void launch_append(const rc_kv_append_args& a, int sms, int* st, cudaStream_t s) {
  const int L = head_lanes(a.head_dim);
  const int hpc = std::min(a.num_kv_heads, kThreads / L);
  const int hg = (a.num_kv_heads + hpc - 1) / hpc;
  // blocks the tokens can touch: each request begins and ends inside at most two more
  const int64_t most = (a.num_tokens / a.block + 2 * (int64_t)a.num_reqs) * hg;
  const int grid = (int)std::min<int64_t>(std::max<int64_t>(most, 1), (int64_t)sms * 4);
  switch (L) {
    case 4: kv_append_kernel<T, 4><<<grid, kThreads, 0, s>>>(a, hpc, hg, st); break;
    case 8: kv_append_kernel<T, 8><<<grid, kThreads, 0, s>>>(a, hpc, hg, st); break;
    default: kv_append_kernel<T, 16><<<grid, kThreads, 0, s>>>(a, hpc, hg, st); break;
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
  const int e = rc::sm_count(&sms);
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
  const int e = rc::sm_count(&sms);
  if (e != RC_OK) return e;
  const int chunks = a->num_kv_heads * a->head_dim / 8;
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
