// Writes keys and values into a cache held in 4 bits (format: kv4.cuh) and reads them back.
//
// Both are bound by HBM: a head of 128 in bf16 is 256 bytes on one side and 80 on the other. One warp
// per (token, K or V) where tokens are many and wide, else the chunks of all tokens in a line. A lane
// takes 8 neighbouring elements, a chunk (one 16- or two 16-byte accesses on the wide side, one 32-bit
// word of codes on the other), the four lanes of a group find its extremes by two shuffles, and a warp
// keeps several chunks of 32 lanes in flight.
#include <algorithm>

#include "host_common.h"
#include "kv4.cuh"
#include "norm_rope.cuh"
#include "views.h"

namespace rc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 4;       // chunks of a warp in flight while it writes the cache
constexpr int kReadAhead = 8;   // and while it reads it, 32 bits of codes each

template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const void* p) { r = __ldcs((const uint4*)p); }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = bf16lo(r.x), x[1] = bf16hi(r.x), x[2] = bf16lo(r.y), x[3] = bf16hi(r.y);
    x[4] = bf16lo(r.z), x[5] = bf16hi(r.z), x[6] = bf16lo(r.w), x[7] = bf16hi(r.w);
  }
  // least and greatest of the four lanes' elements; a NaN stays
  __device__ __forceinline__ void extremes(float& lo, float& hi) const {
    uint32_t a = min_nan_bf16x2(min_nan_bf16x2(r.x, r.y), min_nan_bf16x2(r.z, r.w));
    uint32_t b = max_nan_bf16x2(max_nan_bf16x2(r.x, r.y), max_nan_bf16x2(r.z, r.w));
    // least and negated greatest side by side, so that a minimum finds both
    b ^= 0x80008000u;
    uint32_t m = min_nan_bf16x2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
    m = min_nan_bf16x2(m, __shfl_xor_sync(~0u, m, 1));
    m = min_nan_bf16x2(m, __shfl_xor_sync(~0u, m, 2));
    lo = bf16lo(m), hi = -bf16hi(m);
  }
  static __device__ __forceinline__ void store(void* p, const float* x) {
    *(uint4*)p = make_uint4(pack2_bf16(x[0], x[1]), pack2_bf16(x[2], x[3]),
                            pack2_bf16(x[4], x[5]), pack2_bf16(x[6], x[7]));
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p) {
    a = __ldcs((const float4*)p), b = __ldcs((const float4*)p + 1);
  }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  __device__ __forceinline__ void extremes(float& lo, float& hi) const {
    lo = min_nan(min_nan(min_nan(a.x, a.y), min_nan(a.z, a.w)),
                 min_nan(min_nan(b.x, b.y), min_nan(b.z, b.w)));
    hi = max_nan(max_nan(max_nan(a.x, a.y), max_nan(a.z, a.w)),
                 max_nan(max_nan(b.x, b.y), max_nan(b.z, b.w)));
#pragma unroll
    for (int s = 1; s < 4; s *= 2) {
      lo = min_nan(lo, __shfl_xor_sync(~0u, lo, s));
      hi = max_nan(hi, __shfl_xor_sync(~0u, hi, s));
    }
  }
  static __device__ __forceinline__ void store(void* p, const float* x) {
    ((float4*)p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    ((float4*)p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// Where a lane's chunk of eight elements (of codes: its word) lies in a token's heads. Chunks that are 32
// apart are a whole number of heads apart where a head's chunks divide a warp: distances are then
// constants and one stride.
template <int NG>
struct Chunks {
  static constexpr int C = 4 * NG, RB = kv4_row_bytes(32 * NG);
  static constexpr bool EVEN = 32 % C == 0;
  // the head and the chunk of it of number c0 + 32 u + lane, c0 a multiple of 32
  static __device__ __forceinline__ int head(int c0, int u, int lane) {
    return EVEN ? c0 / C + u * (32 / C) + lane / C : (c0 + 32 * u + lane) / C;
  }
  static __device__ __forceinline__ int of_head(int c0, int u, int lane) {
    return EVEN ? lane % C : (c0 + 32 * u + lane) % C;
  }
};

// FULL: all of the kAhead chunks exist.
template <typename T, int NG, bool FULL>
__device__ __forceinline__ void append_chunks(const T* x, int64_t hs, char* row, int c0, int chunks,
                                              int lane) {
  using K = Chunks<NG>;
  Eight<T> e[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    if (!FULL) e[u] = Eight<T>();
    if (FULL || c0 + 32 * u + lane < chunks)
      e[u].load(x + K::head(c0, u, lane) * hs + K::of_head(c0, u, lane) * 8);
  }
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    float v[8], lo, hi;
    e[u].get(v);
    e[u].extremes(lo, hi);
    const Kv4Group g = kv4_group<sizeof(T) == 4>(lo, hi);
    const uint32_t w = kv4_codes(g, v);
    if (!FULL && c0 + 32 * u + lane >= chunks) continue;   // a group's lanes are all in or out
    const int c = K::of_head(c0, u, lane), j = c / 4, q = c % 4;
    uint32_t* head = (uint32_t*)(row + K::head(c0, u, lane) * K::RB);
    head[q * NG + j] = w;
    if (q == 0) head[K::C + j] = g.pair;
  }
}

template <typename T, int NG>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(rc_kv4_append_args a, int* status) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * kWarps;
  int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  // a token's slot is on its way before it is needed, the first before the number of tokens is known
  int next = i < 2 * a.num_tokens ? a.out_loc[i >> 1] : 0;
  const int64_t items = 2 * min(max((int64_t)a.qo_indptr[a.num_reqs], (int64_t)0), a.num_tokens);
  const int chunks = a.num_kv_heads * Chunks<NG>::C;
  for (; i < items; i += warps) {
    const int64_t t = i >> 1;
    const bool is_v = i & 1;
    const int slot = next;
    if (i + warps < items) next = a.out_loc[(i + warps) >> 1];
    if (slot < 0 || slot >= a.num_slots) {
      if (lane == 0) set_status(status, kStatusSlotRange);
      continue;
    }
    const T* x = is_v ? (const T*)a.v + t * a.v_token_stride : (const T*)a.k + t * a.k_token_stride;
    const int64_t hs = is_v ? a.v_head_stride : a.k_head_stride;
    char* row = (char*)(is_v ? a.v_pool : a.k_pool) + (int64_t)slot * a.num_kv_heads * Chunks<NG>::RB;
    int c0 = 0;
    for (; c0 + 32 * kAhead <= chunks; c0 += 32 * kAhead)
      append_chunks<T, NG, true>(x, hs, row, c0, chunks, lane);
    if (c0 < chunks) append_chunks<T, NG, false>(x, hs, row, c0, chunks, lane);
  }
}

template <typename T, int NG, bool FULL>
__device__ __forceinline__ void read_chunks(const char* row, T* out, int64_t hs, int c0, int chunks,
                                            int lane) {
  using K = Chunks<NG>;
  uint32_t w[kReadAhead], p[kReadAhead];
#pragma unroll
  for (int u = 0; u < kReadAhead; ++u) {
    if (!FULL && c0 + 32 * u + lane >= chunks) continue;
    const uint32_t* head = (const uint32_t*)(row + K::head(c0, u, lane) * K::RB);
    const int c = K::of_head(c0, u, lane);
    w[u] = head[c];
    p[u] = head[K::C + c % NG];
  }
#pragma unroll
  for (int u = 0; u < kReadAhead; ++u) {
    if (!FULL && c0 + 32 * u + lane >= chunks) continue;
    const float s = bf16lo(p[u]), m = bf16hi(p[u]);
    const int c = K::of_head(c0, u, lane);
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = fmaf((float)(w[u] >> 4 * k & 15u), s, m);
    Eight<T>::store(out + K::head(c0, u, lane) * hs + c % NG * 32 + c / NG * 8, v);
  }
}

template <typename T, int NG>
__global__ void __launch_bounds__(kThreads) kv4_read_kernel(rc_kv4_read_args a, int* status) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * kWarps;
  const int64_t items = 2 * a.num_tokens;
  const int chunks = a.num_kv_heads * Chunks<NG>::C;
  int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  int next = i < items ? a.slots[i >> 1] : 0;   // as in kv4_append_kernel
  for (; i < items; i += warps) {
    const int64_t t = i >> 1;
    const bool is_v = i & 1;
    const int slot = next;
    if (i + warps < items) next = a.slots[(i + warps) >> 1];
    const int64_t to = a.out_loc ? a.out_loc[t] : t;
    if (slot < 0 || slot >= a.num_slots || to < 0 || to >= a.out_rows) {
      if (lane == 0) set_status(status, kStatusSlotRange);
      continue;
    }
    const char* row = (const char*)(is_v ? a.v_pool : a.k_pool) +
                      (int64_t)slot * a.num_kv_heads * Chunks<NG>::RB;
    T* out = is_v ? (T*)a.v_out + to * a.v_token_stride : (T*)a.k_out + to * a.k_token_stride;
    const int64_t hs = is_v ? a.v_head_stride : a.k_head_stride;
    int c0 = 0;
    for (; c0 + 32 * kReadAhead <= chunks; c0 += 32 * kReadAhead)
      read_chunks<T, NG, true>(row, out, hs, c0, chunks, lane);
    if (c0 < chunks) read_chunks<T, NG, false>(row, out, hs, c0, chunks, lane);
  }
}

// ---- few KV heads: the chunks of all tokens as one line, so that no lane is idle where a token has less
// than a warp of them, and a warp has as many in flight as with many heads. blockIdx.y: K, V. For tokens of
// up to kFlat chunks (bf16, a warp per token -> this way; writes with the same tokens read back): 149 682
// tokens of one head of 128 read in 76 -> 25 us, 324 800 of one head of 64 written in 325 -> 60, 24 000 of
// four heads of 128 (64 chunks) read in 22 -> 17. More chunks lose, as each lane finds its own slot: eight
// heads of 128 written in 38 -> 48, 32 heads in 116 -> 166.
constexpr int kFlat = 64;
// n / chunks: by is 2^36 / chunks rounded up. Exact for n * chunks <= 2^36: 2^24 tokens at most of up to 64
// chunks, or n within the lanes of the GPU (under 2^18) and chunks within n.
__device__ __forceinline__ uint32_t token_of(uint32_t n, uint64_t by) { return (uint32_t)(n * by >> 36); }

template <typename T, int NG>
__global__ void __launch_bounds__(kThreads) kv4_append_flat_kernel(rc_kv4_append_args a, uint64_t by,
                                                                   int each, int* status) {
  constexpr int C = Chunks<NG>::C, RB = Chunks<NG>::RB;
  const bool is_v = blockIdx.y;
  const uint32_t chunks = a.num_kv_heads * C;
  const uint32_t n =
      (uint32_t)min(max((int64_t)a.qo_indptr[a.num_reqs], (int64_t)0), a.num_tokens) * chunks;
  const T* x = (const T*)(is_v ? a.v : a.k);
  const int64_t ts = is_v ? a.v_token_stride : a.k_token_stride;
  const int64_t hs = is_v ? a.v_head_stride : a.k_head_stride;
  char* pool = (char*)(is_v ? a.v_pool : a.k_pool);
  for (uint32_t i0 = (blockIdx.x * kThreads + (threadIdx.x & ~31u)) * each; i0 < n;
       i0 += gridDim.x * kThreads * each) {
    Eight<T> e[kAhead];
    int slot[kAhead];
    uint32_t c[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const uint32_t i = i0 + 32 * u + (threadIdx.x & 31);
      e[u] = Eight<T>();
      slot[u] = -1, c[u] = 0;
      if (u < each && i < n) {
        const uint32_t t = token_of(i, by);
        c[u] = i - t * chunks;
        slot[u] = a.out_loc[t];
        e[u].load(x + t * ts + c[u] / C * hs + c[u] % C * 8);
        if ((slot[u] < 0 || slot[u] >= a.num_slots) && c[u] == 0) set_status(status, kStatusSlotRange);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      float v[8], lo, hi;
      e[u].get(v);
      e[u].extremes(lo, hi);   // a group's four lanes are of one token
      const Kv4Group g = kv4_group<sizeof(T) == 4>(lo, hi);
      const uint32_t w = kv4_codes(g, v);
      if (slot[u] < 0 || slot[u] >= a.num_slots) continue;
      const int k = c[u] % C, j = k / 4, q = k % 4;
      uint32_t* head = (uint32_t*)(pool + ((int64_t)slot[u] * a.num_kv_heads + c[u] / C) * RB);
      head[q * NG + j] = w;
      if (q == 0) head[C + j] = g.pair;
    }
  }
}

template <typename T, int NG>
__global__ void __launch_bounds__(kThreads) kv4_read_flat_kernel(rc_kv4_read_args a, uint64_t by,
                                                                 int each, int* status) {
  constexpr int C = Chunks<NG>::C, RB = Chunks<NG>::RB;
  const bool is_v = blockIdx.y;
  const uint32_t chunks = a.num_kv_heads * C, n = (uint32_t)a.num_tokens * chunks;
  const char* pool = (const char*)(is_v ? a.v_pool : a.k_pool);
  T* out = (T*)(is_v ? a.v_out : a.k_out);
  const int64_t ts = is_v ? a.v_token_stride : a.k_token_stride;
  const int64_t hs = is_v ? a.v_head_stride : a.k_head_stride;
  for (uint32_t i0 = (blockIdx.x * kThreads + (threadIdx.x & ~31u)) * each; i0 < n;
       i0 += gridDim.x * kThreads * each) {
    uint32_t w[kReadAhead], p[kReadAhead], c[kReadAhead];
    int64_t to[kReadAhead];
#pragma unroll
    for (int u = 0; u < kReadAhead; ++u) {
      const uint32_t i = i0 + 32 * u + (threadIdx.x & 31);
      to[u] = -1;
      if (u < each && i < n) {
        const uint32_t t = token_of(i, by);
        c[u] = i - t * chunks;
        const int slot = a.slots[t];
        to[u] = a.out_loc ? a.out_loc[t] : t;
        if (slot < 0 || slot >= a.num_slots || to[u] < 0 || to[u] >= a.out_rows) {
          to[u] = -1;
          if (c[u] == 0) set_status(status, kStatusSlotRange);
        } else {
          const uint32_t* head =
              (const uint32_t*)(pool + ((int64_t)slot * a.num_kv_heads + c[u] / C) * RB);
          w[u] = head[c[u] % C];
          p[u] = head[C + c[u] % C % NG];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kReadAhead; ++u) {
      if (to[u] < 0) continue;
      const float s = bf16lo(p[u]), m = bf16hi(p[u]);
      const int k = c[u] % C;
      float v[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = fmaf((float)(w[u] >> 4 * x & 15u), s, m);
      Eight<T>::store(out + to[u] * ts + c[u] / C * hs + k % NG * 32 + k / NG * 8, v);
    }
  }
}
// A lane takes up to `ahead` chunks in a go, fewer where the GPU's lanes then have none. Also for few tokens
// of many heads, whose chunks all find a lane of their own (two to four of 32 heads of 256 written and read
// back in 12.6 -> 8.2 us; up to four times as many chunks: 16 heads of fp32 14.4 -> 15.6).
struct Flat {
  uint64_t by;
  int each;
  dim3 grid;   // CTAs for each of K and V
  bool fits;
  Flat(int64_t tokens, int64_t chunks, int ahead, int sms) {
    const int64_t n = tokens * chunks, most = (int64_t)sms * 4, lanes = most * kThreads;
    fits = chunks <= kFlat || n <= lanes;
    by = ((1ull << 36) + chunks - 1) / chunks;
    each = (int)std::min<int64_t>(ahead, (n + lanes - 1) / lanes);
    grid = dim3((unsigned)std::min(most, (n + kThreads * each - 1) / (kThreads * each)), 2);
  }
};

// Two warps of work per token; more CTAs than fit at once even out the tokens (reading 24 000 tokens of 32
// heads: 4 for each SM 88.7 us, 8 90.6, 16 85.2; 82.3 since slots are loaded a token ahead).
unsigned grid_of(int64_t tokens, int sms) {
  return (unsigned)std::min<int64_t>((2 * tokens + kWarps - 1) / kWarps, (int64_t)sms * 16);
}

template <typename T, int NG>
void launch_append(const rc_kv4_append_args& a, int sms, int* st, cudaStream_t s) {
  const int64_t chunks = (int64_t)a.num_kv_heads * Chunks<NG>::C;
  const Flat f(a.num_tokens, chunks, kAhead, sms);
  if (f.fits)
    kv4_append_flat_kernel<T, NG><<<f.grid, kThreads, 0, s>>>(a, f.by, f.each, st);
  else
    kv4_append_kernel<T, NG><<<grid_of(a.num_tokens, sms), kThreads, 0, s>>>(a, st);
}
template <typename T, int NG>
void launch_read(const rc_kv4_read_args& a, int sms, int* st, cudaStream_t s) {
  const int64_t chunks = (int64_t)a.num_kv_heads * Chunks<NG>::C;
  const Flat f(a.num_tokens, chunks, kReadAhead, sms);
  if (f.fits)
    kv4_read_flat_kernel<T, NG><<<f.grid, kThreads, 0, s>>>(a, f.by, f.each, st);
  else
    kv4_read_kernel<T, NG><<<grid_of(a.num_tokens, sms), kThreads, 0, s>>>(a, st);
}
template <typename T>
void launch_append(const rc_kv4_append_args& a, int sms, int* st, cudaStream_t s) {
  switch (a.head_dim / 64) {
    case 1: launch_append<T, 2>(a, sms, st, s); break;
    case 2: launch_append<T, 4>(a, sms, st, s); break;
    case 3: launch_append<T, 6>(a, sms, st, s); break;
    default: launch_append<T, 8>(a, sms, st, s); break;
  }
}
template <typename T>
void launch_read(const rc_kv4_read_args& a, int sms, int* st, cudaStream_t s) {
  switch (a.head_dim / 64) {
    case 1: launch_read<T, 2>(a, sms, st, s); break;
    case 2: launch_read<T, 4>(a, sms, st, s); break;
    case 3: launch_read<T, 6>(a, sms, st, s); break;
    default: launch_read<T, 8>(a, sms, st, s); break;
  }
}

int check_sizes(const char* fn, int dtype, int heads, int d, int64_t tokens, int64_t slots) {
  RC_CHECK_ARG(dtype == RC_DTYPE_BF16 || dtype == RC_DTYPE_F32, "%s: dtype %d", fn, dtype);
  RC_CHECK_ARG(d >= 64 && d <= kKv4MaxDim && d % 64 == 0, "%s: head_dim %d (64, 128, 192 or 256)", fn,
               d);
  RC_CHECK_ARG(heads > 0 && heads <= 65536 && tokens >= 0 && tokens <= (1 << 24) && slots > 0,
               "%s: bad sizes", fn);
  return RC_OK;
}

}  // namespace
}  // namespace rc

extern "C" int rc_kv4_append(const rc_kv4_append_args* a, void* stream) {
  static const char* fn = "rc_kv4_append";
  RC_CHECK_ARG(a != nullptr, "%s: args is NULL", fn);
  const int c = rc::check_sizes(fn, a->dtype, a->num_kv_heads, a->head_dim, a->num_tokens,
                                a->num_slots);
  if (c != RC_OK) return c;
  RC_CHECK_ARG(a->num_reqs >= 0, "%s: bad sizes", fn);
  if (a->num_tokens == 0 || a->num_reqs == 0) return RC_OK;
  RC_CHECK_ARG(a->k && a->v && a->out_loc && a->qo_indptr && a->k_pool && a->v_pool,
               "%s: NULL pointer", fn);
  const int es = a->dtype == RC_DTYPE_BF16 ? 2 : 4;
  const int64_t strides = a->k_token_stride | a->k_head_stride | a->v_token_stride | a->v_head_stride;
  RC_CHECK_ARG((((uintptr_t)a->k | (uintptr_t)a->v) & 15) == 0 && (strides * es & 15) == 0,
               "%s: k, v and strides must be multiples of 16 bytes", fn);
  RC_CHECK_ARG((((uintptr_t)a->k_pool | (uintptr_t)a->v_pool) & (rc::kv4_align(a->head_dim) - 1)) == 0,
               "%s: planes must be multiples of %d bytes", fn, rc::kv4_align(a->head_dim));
  const int64_t T = a->num_tokens, h = a->num_kv_heads, w = (int64_t)a->head_dim * es;
  const int64_t plane = a->num_slots * h * rc::kv4_row_bytes(a->head_dim);
  const rc::RowsView k{a->k, a->k_token_stride * es, a->k_head_stride * es, T, h, w};
  const rc::RowsView v{a->v, a->v_token_stride * es, a->v_head_stride * es, T, h, w};
  const rc::RowsView kp{a->k_pool, 0, 0, 1, 1, plane}, vp{a->v_pool, 0, 0, 1, 1, plane};
  RC_CHECK_ARG(!rc::views_overlap(kp, vp) && !rc::views_overlap(kp, k) && !rc::views_overlap(kp, v) &&
                   !rc::views_overlap(vp, k) && !rc::views_overlap(vp, v),
               "%s: a plane overlaps the other or an input", fn);
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

extern "C" int rc_kv4_read(const rc_kv4_read_args* a, void* stream) {
  static const char* fn = "rc_kv4_read";
  RC_CHECK_ARG(a != nullptr, "%s: args is NULL", fn);
  const int c = rc::check_sizes(fn, a->dtype, a->num_kv_heads, a->head_dim, a->num_tokens,
                                a->num_slots);
  if (c != RC_OK) return c;
  RC_CHECK_ARG(a->out_rows >= 0 && a->out_rows <= INT32_MAX &&
                   (a->out_loc || a->out_rows >= a->num_tokens),
               "%s: bad sizes", fn);
  if (a->num_tokens == 0) return RC_OK;
  RC_CHECK_ARG(a->k_pool && a->v_pool && a->slots && a->k_out && a->v_out, "%s: NULL pointer", fn);
  const int es = a->dtype == RC_DTYPE_BF16 ? 2 : 4;
  const int64_t strides = a->k_token_stride | a->k_head_stride | a->v_token_stride | a->v_head_stride;
  RC_CHECK_ARG((((uintptr_t)a->k_out | (uintptr_t)a->v_out) & 15) == 0 && (strides * es & 15) == 0,
               "%s: outputs and strides must be multiples of 16 bytes", fn);
  RC_CHECK_ARG((((uintptr_t)a->k_pool | (uintptr_t)a->v_pool) & (rc::kv4_align(a->head_dim) - 1)) == 0,
               "%s: planes must be multiples of %d bytes", fn, rc::kv4_align(a->head_dim));
  const int64_t R = a->out_rows, h = a->num_kv_heads, w = (int64_t)a->head_dim * es;
  const int64_t plane = a->num_slots * h * rc::kv4_row_bytes(a->head_dim);
  const rc::RowsView k{a->k_out, a->k_token_stride * es, a->k_head_stride * es, R, h, w};
  const rc::RowsView v{a->v_out, a->v_token_stride * es, a->v_head_stride * es, R, h, w};
  const rc::RowsView kp{a->k_pool, 0, 0, 1, 1, plane}, vp{a->v_pool, 0, 0, 1, 1, plane};
  RC_CHECK_ARG(!rc::rows_overlap(k) && !rc::rows_overlap(v) && !rc::views_overlap(k, v) &&
                   !rc::views_overlap(kp, k) && !rc::views_overlap(kp, v) &&
                   !rc::views_overlap(vp, k) && !rc::views_overlap(vp, v),
               "%s: an output overlaps itself, the other or a plane", fn);
  int* st = rc::device_status_ptr();
  if (!st) return rc::fail(RC_ERR_CUDA, "%s: no device status word", fn);
  int sms = 0;
  const int e = rc::sm_count(fn, &sms);
  if (e != RC_OK) return e;
  if (a->dtype == RC_DTYPE_BF16)
    rc::launch_read<__nv_bfloat16>(*a, sms, st, (cudaStream_t)stream);
  else
    rc::launch_read<float>(*a, sms, st, (cudaStream_t)stream);
  rc::count_launches(1);
  return rc::check_launch(fn);
}
