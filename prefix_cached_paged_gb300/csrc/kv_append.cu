// Appending keys and values to the paged cache, the keys normalised and rotated on the way, and
// the bounds of cached keys block by block that sparse_decode.cu selects blocks with.
//
// Work items are (request, block of positions the new tokens touch, a few KV heads), one warp each,
// so a warp owns every new key of a (block, head) and reduces its bounds without atomics: a block
// that the new tokens begin gets their bounds, a block that cached tokens began takes the minimum
// and maximum with what it holds (which makes a repeated append of the same tokens change nothing).
// Requests are taken in windows of kWindow, whose item offsets each CTA sums up in shared memory, so
// neither their number nor their lengths need to be known on the host; the warps of the resident
// CTAs then take the items one by one.
//
// Both kernels are bound by HBM. Measured (bf16, heads of 128, inputs beyond L2):
//   append, 80 requests x 200 tokens x 32 heads, with bounds: 94 us, 5.7 TB/s, 85 % of the copy rate
//     (half of it writes of 256-byte rows to scattered slots). A CTA per block with the tokens in
//     turn took 208 us, warps with a fixed share of the items 121 (blocks hold 36 or 64 tokens),
//     angles loaded as they are needed 98, angles copied past L1 180: every head reads them.
//   append, 256 requests x 1 token x 8 heads: 8 us, launch and dependent loads.
//   bounds, 256 contexts of 128 .. 16384 tokens, 8 heads: 262 us, 6.53 TB/s, 97 % of the copy rate.
//     With the keys loaded into registers 316 us (64 KB in flight per SM instead of 192), joined by
//     a CTA 336; two ring stages 267, four 308 (one CTA less per SM).
#include <algorithm>

#include "host_common.h"
#include "norm_rope.cuh"
#include "warp_mma.cuh"

namespace rc {
namespace {

constexpr int kThreads = 256;
constexpr int kRun = 4;         // items a CTA takes beside one another
constexpr int kWindow = 1024;   // requests whose item offsets a CTA holds at a time
// Tokens of a call: a window's items can then be counted in 32 bits whatever the offsets hold (each
// request passed on is within the tokens, so has at most kMaxAppend / 16 + 1 items).
constexpr int kMaxAppend = 1 << 24;

// off[k] = items of the window's requests before k (off[n] = all), each of n <= kWindow requests
// having count(k) items; none taken yet. All threads of the CTA call it.
template <typename F>
__device__ void window_offsets(int* off, int* warp_sums, int* taken, int n, F count) {
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
  if (threadIdx.x == 0) *taken = 0;
  __syncthreads();
}
// The warp's next item of the window. A CTA has runs of kRun neighbouring items (the heads of a block:
// its warps share the block's angles and write neighbouring rows) where there are plenty of items,
// else single ones, spread over the SMs (2 000 tokens of 2 heads 24 us so, 33 in runs of 4). Its
// warps take them as they come free, since blocks hold unlike numbers of tokens.
__device__ __forceinline__ int64_t next_item(int* taken, int64_t items) {
  int k = 0;
  if ((threadIdx.x & 31) == 0) k = atomicAdd(taken, 1);
  k = __shfl_sync(0xffffffffu, k, 0);
  return items < (int64_t)gridDim.x * kRun * 4
             ? (int64_t)k * gridDim.x + blockIdx.x
             : ((int64_t)(k / kRun) * gridDim.x + blockIdx.x) * kRun + k % kRun;
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
  if (s.S == 0) return s;   // nothing to do, whatever the rest says (a padded batch)
  bool ok = s.t0 >= 0 && s.S >= 0 && (int64_t)s.t0 + s.S <= a.num_tokens && s.P >= 0 &&
            (int64_t)s.P + s.S <= 0x7fffffff;
  if (ok) {
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
  static constexpr uint32_t kLo = 0x7f807f80u, kHi = 0xff80ff80u;        // inf, -inf
  static constexpr uint32_t kMost = 0x7f7f7f7fu, kLeast = 0xff7fff7fu;   // finite
  static __device__ __forceinline__ uint32_t lo(uint32_t a, uint32_t b) { return min_nan_bf16x2(a, b); }
  static __device__ __forceinline__ uint32_t hi(uint32_t a, uint32_t b) { return max_nan_bf16x2(a, b); }
};
template <>
struct Extremes<float> {
  static constexpr uint32_t kLo = 0x7f800000u, kHi = 0xff800000u;
  static constexpr uint32_t kMost = 0x7f7fffffu, kLeast = 0xff7fffffu;
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
__device__ __forceinline__ uint4 shfl_xor4(const uint4& v, int o) {
  return make_uint4(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o),
                    __shfl_xor_sync(0xffffffffu, v.z, o), __shfl_xor_sync(0xffffffffu, v.w, o));
}
__device__ __forceinline__ uint4 splat(uint32_t x) { return make_uint4(x, x, x, x); }
// Extremes of no key at all (every slot outside the pool; any key would make them meet) become the
// largest and the lowest finite number: infinities would give NaN with a query element of 0, which
// ranks a block first, and these rank it last.
template <typename T>
__device__ __forceinline__ void settle(uint4& lo, uint4& hi) {
  if (lo.x == Extremes<T>::kLo && hi.x == Extremes<T>::kHi) {
    lo = splat(Extremes<T>::kMost);
    hi = splat(Extremes<T>::kLeast);
  }
}

// Each warp streams its tokens through a ring of a few groups in shared memory by 16-byte
// asynchronous copies. A lane reads only what it copied itself, so the ring needs no barrier, and
// the bytes in flight cost no registers.
constexpr int kAppendStages = 2, kBoundsStages = 3;
constexpr int kWarps = kThreads / 32;

// What a lane keeps of a token in the ring: 16-byte chunks of K (2 N) and V (2 N), four of its
// angles, and the token's slot.
template <typename T>
constexpr int kTokenBytes = (4 * Raw<T>::N + 4) * 512 + 128;
template <typename T>
constexpr int append_smem() { return kWarps * kAppendStages * kTokenBytes<T>; }

// A warp's lanes are 32 / L rows: `heads` KV heads beside one another (a power of two), the other
// rows later tokens of the block; one token of each row is a group. kShare: an item is a whole CTA's,
// its warps taking groups in turn and joining their extremes at the end.
template <typename T, int L, bool kShare>
__global__ void __launch_bounds__(kThreads, 3)
    kv_append_kernel(rc_kv_append_args a, int heads, int* status) {
  constexpr int N = Raw<T>::N;
  extern __shared__ __align__(128) char ring[];
  __shared__ int off[kWindow + 1];
  __shared__ int warp_sums[kWarps], taken;
  const int d = a.head_dim, r = a.rotary_dim;
  const bool inter = a.interleaved != 0;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int i = lane % L, row_in = lane / L;
  const int hl = row_in & (heads - 1), w = row_in / heads;
  // this row has every W-th token, from its w0-th on
  const int W = 32 / L / heads * (kShare ? kWarps : 1);
  const int w0 = kShare ? wid * (32 / L / heads) + w : w;
  const int head_groups = (a.num_kv_heads + heads - 1) / heads;
  const LaneChunks lc = lane_chunks(i, d, r, inter);
  const T* kw = (const T*)a.k_weight;
  // chunk c (K, V, angles) of the token in stage st of this lane, and the token's slot
  char* warp_ring = ring + wid * (kAppendStages * kTokenBytes<T>);
  auto cell_of = [&](int st, int c) {
    return warp_ring + st * kTokenBytes<T> + c * 512 + lane * 16;
  };
  auto slot_of = [&](int st) {
    return (int*)(warp_ring + (st + 1) * kTokenBytes<T> - 128 + lane * 4);
  };

  for (int b0 = 0; b0 < a.num_reqs; b0 += kWindow) {
    const int nreq = min(kWindow, a.num_reqs - b0);
    window_offsets(off, warp_sums, &taken, nreq, [&](int k) {
      const Span s = span_of(a, b0 + k, status, blockIdx.x == 0);
      return s.S ? (s.P + s.S - 1) / a.block - s.P / a.block + 1 : 0;
    });
    const int64_t items = (int64_t)off[kWindow] * head_groups;
    int64_t it = kShare ? blockIdx.x : next_item(&taken, items);
    for (; it < items; it = kShare ? it + gridDim.x : next_item(&taken, items)) {
      const int job = (int)(it / head_groups), hg = (int)(it - (int64_t)job * head_groups);
      const int k = find_request(off, nreq, job);
      const Span s = span_of(a, b0 + k, status, false);
      const int blk = s.P / a.block + (job - off[k]);
      const int p0 = max(s.P, blk * a.block);
      const int n = (int)(min((int64_t)s.P + s.S, (int64_t)(blk + 1) * a.block) - p0);
      const int64_t tok0 = (int64_t)s.t0 + (p0 - s.P);
      const int h = hg * heads + hl;
      const bool mine = h < a.num_kv_heads;
      const bool m0 = mine && lc.c0 >= 0, m1 = mine && lc.c1 >= 0;
      const T* ksrc = (const T*)a.k + tok0 * a.k_token_stride + (int64_t)h * a.k_head_stride;
      const T* vsrc = (const T*)a.v + tok0 * a.v_token_stride + (int64_t)h * a.v_head_stride;
      const int groups = (n + W - 1) / W;
      auto issue = [&](int gr) {
        const int at = gr * W + w0;
        if (gr < groups && mine && at < n) {
          const int st = gr % kAppendStages;
          cp_async4(smem_u32(slot_of(st)), a.out_loc + tok0 + at);
          if (lc.rot) {
            const float* row = a.rope + (int64_t)(p0 + at) * r + 8 * i;
            cp_async16_l1(smem_u32(cell_of(st, 4 * N)), row);
            cp_async16_l1(smem_u32(cell_of(st, 4 * N + 1)), row + 4);
            cp_async16_l1(smem_u32(cell_of(st, 4 * N + 2)), row + (r >> 1));
            cp_async16_l1(smem_u32(cell_of(st, 4 * N + 3)), row + (r >> 1) + 4);
          }
          const T* ks = ksrc + at * a.k_token_stride;
          const T* vs = vsrc + at * a.v_token_stride;
#pragma unroll
          for (int c = 0; c < N; ++c) {
            if (m0) {
              cp_async16(smem_u32(cell_of(st, c)), (const uint4*)(ks + lc.c0 * 8) + c);
              cp_async16(smem_u32(cell_of(st, 2 * N + c)), (const uint4*)(vs + lc.c0 * 8) + c);
            }
            if (m1) {
              cp_async16(smem_u32(cell_of(st, N + c)), (const uint4*)(ks + lc.c1 * 8) + c);
              cp_async16(smem_u32(cell_of(st, 3 * N + c)), (const uint4*)(vs + lc.c1 * 8) + c);
            }
          }
        }
        cp_async_commit();
      };
#pragma unroll
      for (int gr = 0; gr < kAppendStages - 1; ++gr) issue(gr);
      T* cell = (T*)a.bounds +
                ((((int64_t)s.row * a.max_blocks + blk) * a.num_kv_heads + h) * 2) * d;
      Raw<T> lo0, lo1, hi0, hi1;
#pragma unroll
      for (int c = 0; c < N; ++c) {
        lo0.v[c] = lo1.v[c] = splat(Extremes<T>::kLo);
        hi0.v[c] = hi1.v[c] = splat(Extremes<T>::kHi);
      }
      if (a.bounds && w0 == 0 && blk * a.block < s.P) {   // cached tokens began the block
        if (m0) {
          lo0.load(cell + lc.c0 * 8);
          hi0.load(cell + d + lc.c0 * 8);
        }
        if (m1) {
          lo1.load(cell + lc.c1 * 8);
          hi1.load(cell + d + lc.c1 * 8);
        }
      }
      for (int gr = 0; gr < groups; ++gr) {   // the same count for every lane: shuffles inside
        issue(gr + kAppendStages - 1);
        const int st = gr % kAppendStages;
        cp_async_wait<kAppendStages - 1>();
        bool live = mine && gr * W + w0 < n;
        const int slot = live ? *slot_of(st) : 0;
        if (live && (slot < 0 || slot >= a.num_slots)) {
          if (i == 0) set_status(status, kStatusSlotRange);
          live = false;
        }
        Raw<T> x0, x1;
        x0.clear();
        x1.clear();
#pragma unroll
        for (int c = 0; c < N; ++c) {
          if (m0 && live) x0.v[c] = *(const uint4*)cell_of(st, c);
          if (m1 && live) x1.v[c] = *(const uint4*)cell_of(st, N + c);
        }
        const int64_t dst = ((int64_t)slot * a.num_kv_heads + h) * d;
#pragma unroll
        for (int c = 0; c < N; ++c) {
          if (m0 && live)
            ((uint4*)((T*)a.v_pool + dst + lc.c0 * 8))[c] = *(const uint4*)cell_of(st, 2 * N + c);
          if (m1 && live)
            ((uint4*)((T*)a.v_pool + dst + lc.c1 * 8))[c] = *(const uint4*)cell_of(st, 3 * N + c);
        }
        if (kw || r) {
          ScalarRow row;
          row.get(x0, x1);
          if (kw) row.scale(row.template norm_scale<L>(d, a.eps), kw, lc);
          if (lc.rot) {
            float cs[8], sn[8];
            *(float4*)cs = *(const float4*)cell_of(st, 4 * N);
            *(float4*)(cs + 4) = *(const float4*)cell_of(st, 4 * N + 1);
            *(float4*)sn = *(const float4*)cell_of(st, 4 * N + 2);
            *(float4*)(sn + 4) = *(const float4*)cell_of(st, 4 * N + 3);
            row.rotate(cs, sn, inter);
          }
          row.set(x0, x1);
        }
        if (m0 && live) x0.store((T*)a.k_pool + dst + lc.c0 * 8);
        if (m1 && live) x1.store((T*)a.k_pool + dst + lc.c1 * 8);
        if (a.bounds && live) {   // the extremes of the stored (rounded) keys
#pragma unroll
          for (int c = 0; c < N; ++c) {
            lower<T>(lo0.v[c], x0.v[c]);
            raise<T>(hi0.v[c], x0.v[c]);
            lower<T>(lo1.v[c], x1.v[c]);
            raise<T>(hi1.v[c], x1.v[c]);
          }
        }
      }
      cp_async_wait<0>();
      if (!a.bounds) continue;
      for (int o = L * heads; o < 32; o <<= 1) {   // join the token rows
#pragma unroll
        for (int c = 0; c < N; ++c) {
          lower<T>(lo0.v[c], shfl_xor4(lo0.v[c], o));
          lower<T>(lo1.v[c], shfl_xor4(lo1.v[c], o));
          raise<T>(hi0.v[c], shfl_xor4(hi0.v[c], o));
          raise<T>(hi1.v[c], shfl_xor4(hi1.v[c], o));
        }
      }
      if (kShare) {   // join the warps, through their rings
#pragma unroll
        for (int c = 0; c < N; ++c) {
          *(uint4*)cell_of(0, c) = lo0.v[c];
          *(uint4*)cell_of(0, N + c) = lo1.v[c];
          *(uint4*)cell_of(0, 2 * N + c) = hi0.v[c];
          *(uint4*)cell_of(0, 3 * N + c) = hi1.v[c];
        }
        __syncthreads();
        for (int v = 1; v < kWarps && wid == 0; ++v) {
          const char* theirs = cell_of(0, 0) + v * (kAppendStages * kTokenBytes<T>);
#pragma unroll
          for (int c = 0; c < N; ++c) {
            lower<T>(lo0.v[c], *(const uint4*)(theirs + c * 512));
            lower<T>(lo1.v[c], *(const uint4*)(theirs + (N + c) * 512));
            raise<T>(hi0.v[c], *(const uint4*)(theirs + (2 * N + c) * 512));
            raise<T>(hi1.v[c], *(const uint4*)(theirs + (3 * N + c) * 512));
          }
        }
        __syncthreads();
      }
#pragma unroll
      for (int c = 0; c < N; ++c) {
        settle<T>(lo0.v[c], hi0.v[c]);
        settle<T>(lo1.v[c], hi1.v[c]);
      }
      if (w0 == 0 && m0) {
        lo0.store(cell + lc.c0 * 8);
        hi0.store(cell + d + lc.c0 * 8);
      }
      if (w0 == 0 && m1) {
        lo1.store(cell + lc.c1 * 8);
        hi1.store(cell + d + lc.c1 * 8);
      }
    }
  }
}

// ---------------------------------------------------------------- bounds of cached keys
// Work items are (layer, row, block, group of at most 32 16-byte chunks of a token's keys), one warp
// each: `cols` chunks (a power of two) beside one another, the other lanes later tokens of the
// block. A group is kFly tokens of each, or fewer where the keys are narrower than 8 chunks: the
// block's slots are loaded 32 at a time, coalesced, and handed to the lanes by shuffles, so a group
// has at most 32 tokens.
constexpr int kFly = 8;
constexpr int kBoundsSmem = kWarps * kBoundsStages * kFly * 512;

template <typename T>
__global__ void __launch_bounds__(kThreads) kv_block_bounds_kernel(rc_kv_block_bounds_args a, int cols,
                                                                   int* status) {
  constexpr int V = 16 / (int)sizeof(T);   // elements of a chunk
  extern __shared__ __align__(128) char ring[];
  __shared__ int off[kWindow + 1];
  __shared__ int warp_sums[kWarps], taken;
  const int d = a.head_dim;
  const int chunks = a.num_kv_heads * d / V;
  const int col_groups = (chunks + cols - 1) / cols;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int cl = lane & (cols - 1), w = lane / cols, W = 32 / cols;
  const int fly = min(kFly, cols), group = W * fly;
  char* mine_ring = ring + wid * (kBoundsStages * kFly * 512) + lane * 16;
  for (int b0 = 0; b0 < a.num_rows; b0 += kWindow) {
    const int nreq = min(kWindow, a.num_rows - b0);
    window_offsets(off, warp_sums, &taken, nreq, [&](int k) {
      const int L = a.seq_len[b0 + k], row = a.req_idx[b0 + k];
      if (L == 0) return 0;
      if (L < 0 || L > a.max_ctx || row < 0 || row >= a.max_reqs ||
          (L - 1) / a.block >= a.max_blocks) {
        if (blockIdx.x == 0) set_status(status, kStatusPosRange);
        return 0;
      }
      return (L + a.block - 1) / a.block;
    });
    const int64_t per_layer = (int64_t)off[kWindow] * col_groups;
    const int64_t items = per_layer * a.num_layers;
    for (int64_t it = next_item(&taken, items); it < items; it = next_item(&taken, items)) {
      const int64_t layer = it / per_layer;
      const int64_t rest = it - layer * per_layer;
      const int job = (int)(rest / col_groups), cg = (int)(rest - (int64_t)job * col_groups);
      const int k = find_request(off, nreq, job);
      const int L = a.seq_len[b0 + k], row = a.req_idx[b0 + k];
      const int blk = job - off[k];
      const int p0 = blk * a.block, n = (int)min((int64_t)a.block, (int64_t)L - p0);
      const int c = cg * cols + cl;
      const bool mine = c < chunks;
      const int32_t* rt = a.req_to_token + (int64_t)row * a.max_ctx + p0;
      const char* kp = (const char*)a.k_pool +
                       ((layer * a.num_slots * chunks) + (mine ? c : 0)) * 16;
      int slots = -1;   // of tokens 32 j + lane, -1: nothing to read
      uint32_t have = 0;   // bit u of group gr at gr % kBoundsStages * kFly: this lane copied a token
      const int groups = (n + group - 1) / group;
      auto issue = [&](int gr) {
        if (gr < groups) {
          if (gr * group % 32 == 0) {
            const int t = gr * group + lane;
            slots = t < n ? rt[t] : -1;
            if (t < n && (slots < 0 || slots >= a.num_slots)) {
              set_status(status, kStatusSlotRange);
              slots = -1;
            }
          }
          const int st = gr % kBoundsStages;
#pragma unroll
          for (int u = 0; u < kFly; ++u) {
            const int at = (gr * fly + u) * W + w;
            const int slot = __shfl_sync(0xffffffffu, slots, at & 31);
            const uint32_t bit = 1u << (st * kFly + u);
            if (u < fly && mine && at < n && slot >= 0) {
              cp_async16(smem_u32(mine_ring + (st * kFly + u) * 512), kp + (int64_t)slot * chunks * 16);
              have |= bit;
            } else {
              have &= ~bit;
            }
          }
        }
        cp_async_commit();
      };
#pragma unroll
      for (int gr = 0; gr < kBoundsStages - 1; ++gr) issue(gr);
      uint4 lo = splat(Extremes<T>::kLo), hi = splat(Extremes<T>::kHi);
      for (int gr = 0; gr < groups; ++gr) {
        issue(gr + kBoundsStages - 1);
        cp_async_wait<kBoundsStages - 1>();
        const int st = gr % kBoundsStages;
#pragma unroll
        for (int u = 0; u < kFly; ++u) {
          if (have >> (st * kFly + u) & 1) {
            const uint4 v = *(const uint4*)(mine_ring + (st * kFly + u) * 512);
            lower<T>(lo, v);
            raise<T>(hi, v);
          }
        }
      }
      cp_async_wait<0>();
      for (int o = cols; o < 32; o <<= 1) {   // join the token lanes
        lower<T>(lo, shfl_xor4(lo, o));
        raise<T>(hi, shfl_xor4(hi, o));
      }
      if (w == 0 && mine) {
        const int h = c * V / d, e0 = c * V - h * d;
        T* cell = (T*)a.bounds +
                  ((((layer * a.max_reqs + row) * a.max_blocks + blk) * a.num_kv_heads + h) * 2) * d;
        settle<T>(lo, hi);
        *(uint4*)(cell + e0) = lo;
        *(uint4*)(cell + d + e0) = hi;
      }
    }
  }
}

// Launches a grid of as many CTAs as are resident at once, or fewer where there is less to do.
template <typename K, typename A>
int launch_resident(const char* fn, K kernel, PerDevice<int>& setup, int64_t items, const A& a,
                    int width, int smem, int* st, cudaStream_t s) {
  const int* resident = nullptr;
  const cudaError_t e = setup.get(
      [&](int& n) {
        int dev = 0, sms = 0, per = 0;
        cudaError_t r = cudaGetDevice(&dev);
        if (r == cudaSuccess) r = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (r == cudaSuccess)
          r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (r == cudaSuccess)
          r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kThreads, smem);
        n = std::max(1, sms * per);
        return r;
      },
      &resident);
  if (e != cudaSuccess) return fail(RC_ERR_CUDA, "%s: setup: %s", fn, cudaGetErrorString(e));
  kernel<<<(unsigned)std::min<int64_t>(std::max<int64_t>(items, 1), *resident), kThreads, smem, s>>>(
      a, width, st);
  count_launches(1);
  return check_launch(fn);
}

bool block_ok(int block) { return block == 16 || block == 32 || block == 64 || block == 128; }

int pow2_at_least(int x) {
  int p = 1;
  while (p < x) p *= 2;
  return p;
}

template <typename T, int L>
int launch_append(const char* fn, const rc_kv_append_args& args, int* st, cudaStream_t s) {
  rc_kv_append_args a = args;
  int sms = 0;
  const int e = sm_count(fn, &sms);
  if (e != RC_OK) return e;
  // Single tokens: every row of a warp a head; prompts: one head, tokens of its block beside one
  // another. 80 x 200 tokens: 93 us so, 110 with the heads beside one another; 256 x 1 tokens of 8
  // heads, waited for: 27 us with the heads, 32 with the tokens beside one another.
  const bool prompts = a.num_tokens >= 16 * (int64_t)a.num_reqs;
  const int heads = std::min(pow2_at_least(a.num_kv_heads), prompts ? std::max(1, 8 / L) : 32 / L);
  const int groups = (a.num_kv_heads + heads - 1) / heads;
  // Few items: without bounds an item is any run of tokens, so it is made a short one (2 000 fp32
  // tokens of 2 heads: 11 us so, 24 with 64 tokens each); with bounds the warps of a CTA share a block
  // (8 requests x 300 .. 600 tokens, 2 heads: 10.5 us so, 16.6 with a warp each and two tokens in
  // flight; 5 x 1 .. 46 tokens in blocks of 128: 9.1 against 14.4; 40 x 200 tokens of 8 heads, near the
  // rule's border: 23.9 against 22.7).
  const bool few = prompts && a.num_tokens / a.block * groups < (int64_t)sms * kWarps * 2;
  if (few && !a.bounds) a.block = 16;
  // blocks the tokens can touch: each request begins and ends inside at most two more
  const int64_t items = (a.num_tokens / a.block + 2 * (int64_t)a.num_reqs) * groups;
  static PerDevice<int> alone, shared;
  if (few && a.bounds)
    return launch_resident(fn, kv_append_kernel<T, L, true>, shared, items, a, heads,
                           append_smem<T>(), st, s);
  return launch_resident(fn, kv_append_kernel<T, L, false>, alone, items, a, heads, append_smem<T>(),
                         st, s);
}

template <typename T>
int launch_append(const char* fn, const rc_kv_append_args& a, int* st, cudaStream_t s) {
  switch (head_lanes(a.head_dim)) {
    case 4: return launch_append<T, 4>(fn, a, st, s);
    case 8: return launch_append<T, 8>(fn, a, st, s);
    default: return launch_append<T, 16>(fn, a, st, s);
  }
}

template <typename T>
int launch_bounds(const char* fn, const rc_kv_block_bounds_args& a, int* st, cudaStream_t s) {
  const int chunks = a.num_kv_heads * a.head_dim * (int)sizeof(T) / 16;
  const int cols = std::min(32, pow2_at_least(chunks));
  const int64_t items = (int64_t)a.num_layers * a.num_rows * a.max_blocks *
                        ((chunks + cols - 1) / cols);
  static PerDevice<int> setup;
  return launch_resident(fn, kv_block_bounds_kernel<T>, setup, items, a, cols, kBoundsSmem, st,
                         s);
}

}  // namespace
}  // namespace rc

extern "C" int rc_kv_append(const rc_kv_append_args* a, void* stream) {
  static const char* fn = "rc_kv_append";
  RC_CHECK_ARG(a != nullptr, "%s: args is NULL", fn);
  RC_CHECK_ARG(a->dtype == RC_DTYPE_BF16 || a->dtype == RC_DTYPE_F32, "%s: dtype %d", fn, a->dtype);
  RC_CHECK_ARG(a->num_reqs >= 0 && a->num_tokens >= 0 && a->num_tokens <= rc::kMaxAppend &&
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
  return a->dtype == RC_DTYPE_BF16
             ? rc::launch_append<__nv_bfloat16>(fn, *a, st, (cudaStream_t)stream)
             : rc::launch_append<float>(fn, *a, st, (cudaStream_t)stream);
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
  return a->dtype == RC_DTYPE_BF16
             ? rc::launch_bounds<__nv_bfloat16>(fn, *a, st, (cudaStream_t)stream)
             : rc::launch_bounds<float>(fn, *a, st, (cudaStream_t)stream);
}
