// Decode attention over the blocks of positions that a cheap score selects for each query row and
// KV head.
//
// A block's box (lo_d, hi_d: the least and greatest of its keys in each dimension) bounds q.k from
// above by s = sum_d (q_d >= 0 ? q_d hi_d : q_d lo_d); the largest s over the query heads of a KV head
// ranks the block. Three kernels:
//   score:  every (row, KV head, block) gets its rank as an ordered 64-bit integer;
//   select: one CTA per (row, KV head) finds the top_blocks-th largest and writes the chosen block
//           numbers in ascending order;
//   attend: one CTA per (row, KV head, part of the selected tokens), softmax in fp32 with running
//           maximum and sum; partial states are joined by the merge kernel.
#include <algorithm>
#include <cmath>

#include "host_common.h"
#include "norm_rope.cuh"

namespace rc {
namespace {

constexpr int kPart = 256;      // selected tokens per attention CTA
constexpr int kMaxGroup = 16;   // query heads per KV head

struct Workspace {
  unsigned long long* rank;   // [rows * Hkv * nb]
  int* sel;                   // [rows * Hkv * top]
  float* plse;                // [rows * Hkv * parts * G], base 2
  float* po;                  // [rows * Hkv * parts * G * D]
};
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Params {
  rc_sparse_decode_args a;
  Workspace w;
  int nb;      // blocks of max_seq_len
  int parts;   // attention CTAs per (row, KV head)
  int G;
  int* status;
};

Workspace carve(void* base, const Params& p, size_t* total) {
  const int64_t units = (int64_t)p.a.num_rows * p.a.num_kv_heads;
  Workspace w{};
  char* b = (char*)base;
  size_t o = 0;
  w.rank = (unsigned long long*)(b + o);
  o += align256((size_t)units * p.nb * 8);
  w.sel = (int*)(b + o);
  o += align256((size_t)units * p.a.top_blocks * 4);
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

// Larger score <=> larger integer; the forced blocks rank above every score.
__device__ __forceinline__ unsigned long long order64(double s) {
  if (!(s < 1.7976931348623157e308)) s = 1.7976931348623157e308;   // NaN, +inf
  if (s < -1.7976931348623157e308) s = -1.7976931348623157e308;
  if (s == 0.0) s = 0.0;                                            // -0 ranks as 0
  const long long b = __double_as_longlong(s);
  return (unsigned long long)(b < 0 ? ~b : (b | (1ll << 63)));
}
constexpr unsigned long long kForced = ~0ull;

// One warp per (row, KV head, block).
template <typename T>
__global__ void __launch_bounds__(256) sparse_score_kernel(Params p) {
  const rc_sparse_decode_args& a = p.a;
  const int lane = threadIdx.x & 31;
  const int64_t unit = blockIdx.x;
  const int64_t n = unit / a.num_kv_heads;
  const int g = (int)(unit - n * a.num_kv_heads);
  const int L = row_len(p, n, blockIdx.y == 0 && threadIdx.x == 0 && g == 0);
  const int have = (L + a.block - 1) / a.block;
  const int d = a.head_dim;
  for (int b = blockIdx.y * 8 + (threadIdx.x >> 5); b < have; b += gridDim.y * 8) {
    unsigned long long rank = 0;
    if (b < a.sink_blocks || b >= have - a.recent_blocks) {
      rank = kForced;
    } else {
      const T* box = (const T*)a.bounds +
                     ((((int64_t)a.req_idx[n] * a.max_blocks + b) * a.num_kv_heads + g) * 2) * d;
      for (int h = 0; h < p.G; ++h) {
        const T* q = (const T*)a.q + (n * a.num_q_heads + (int64_t)g * p.G + h) * d;
        double s = 0.0;
        for (int e = lane; e < d; e += 32) {
          const double qe = Elem<T>::to_f(q[e]);
          s += qe * (double)Elem<T>::to_f(qe >= 0.0 ? box[d + e] : box[e]);
        }
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        rank = max(rank, order64(s));
      }
    }
    if (lane == 0) p.w.rank[unit * p.nb + b] = rank;
  }
}

// One CTA per (row, KV head): the largest threshold that at least `top` ranks reach, bit by bit;
// blocks above it are chosen, and of those that equal it the lowest-numbered.
__global__ void __launch_bounds__(256) sparse_select_kernel(Params p) {
  const rc_sparse_decode_args& a = p.a;
  __shared__ int total;
  __shared__ int wsum[2][8];
  const int64_t unit = blockIdx.x;
  const int64_t n = unit / a.num_kv_heads;
  const int L = row_len(p, n, false);
  const int have = (L + a.block - 1) / a.block;
  const int take = min(have, a.top_blocks);
  int* out = p.w.sel + unit * a.top_blocks;
  int* user = a.selected ? a.selected + unit * a.top_blocks : nullptr;
  const unsigned long long* rank = p.w.rank + unit * p.nb;
  for (int i = take + threadIdx.x; i < a.top_blocks; i += 256) {
    out[i] = -1;
    if (user) user[i] = -1;
  }
  if (take == 0) return;
  unsigned long long thr = 0;
  int above = 0;   // ranks > thr
  if (take < have) {
    for (int bit = 63; bit >= 0; --bit) {
      const unsigned long long t = thr | (1ull << bit);
      int c = 0;
      for (int b = threadIdx.x; b < have; b += 256) c += rank[b] >= t;
      if (threadIdx.x == 0) total = 0;
      __syncthreads();
      atomicAdd(&total, c);
      __syncthreads();
      if (total >= take) thr = t;
      __syncthreads();
    }
    int c = 0;
    for (int b = threadIdx.x; b < have; b += 256) c += rank[b] > thr;
    if (threadIdx.x == 0) total = 0;
    __syncthreads();
    atomicAdd(&total, c);
    __syncthreads();
    above = total;
  }
  const int equal_take = take < have ? take - above : have;
  // compaction in block order: running counts of chosen and of equal blocks
  int done = 0, eq_done = 0;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  for (int b0 = 0; b0 < have; b0 += 256) {
    const int b = b0 + threadIdx.x;
    const unsigned long long rk = b < have ? rank[b] : 0;
    const bool eq = b < have && rk == thr && take < have;
    const unsigned me = __ballot_sync(0xffffffffu, eq);
    __syncthreads();
    if (lane == 0) wsum[0][wid] = __popc(me);
    __syncthreads();
    int ebase = eq_done;
    for (int w = 0; w < wid; ++w) ebase += wsum[0][w];
    const bool pick = b < have && (take == have || rk > thr ||
                                   (eq && ebase + __popc(me & ((1u << lane) - 1)) < equal_take));
    const unsigned mp = __ballot_sync(0xffffffffu, pick);
    if (lane == 0) wsum[1][wid] = __popc(mp);
    __syncthreads();
    int base = done;
    for (int w = 0; w < wid; ++w) base += wsum[1][w];
    if (pick) {
      const int at = base + __popc(mp & ((1u << lane) - 1));
      out[at] = b;
      if (user) user[at] = b;
    }
    for (int w = 0; w < 8; ++w) {
      done += wsum[1][w];
      eq_done += wsum[0][w];
    }
  }
}

// One CTA of 4 warps per (row, KV head, part): warp w takes every 4th token of the part.
template <typename T, int D, int G>
__global__ void __launch_bounds__(128) sparse_attend_kernel(Params p) {
  constexpr int E = D / 32;
  const rc_sparse_decode_args& a = p.a;
  __shared__ float q_s[G][D];
  __shared__ float sm[4][G], sl[4][G], so[4][G][D];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int64_t unit = blockIdx.x;
  const int part = blockIdx.y;
  const int64_t n = unit / a.num_kv_heads;
  const int g = (int)(unit - n * a.num_kv_heads);
  const int L = row_len(p, n, false);
  const int Gr = p.G;
  const int have = (L + a.block - 1) / a.block;
  const int take = min(have, a.top_blocks);
  const int t0 = part * kPart, t1 = min(take * a.block, t0 + kPart);
  const int* sel = p.w.sel + unit * a.top_blocks;
  const int32_t* rt = a.req_to_token + (int64_t)(L ? a.req_idx[n] : 0) * a.max_ctx;
  const float scale = a.sm_scale * kLog2e;
  for (int e = threadIdx.x; e < Gr * D; e += 128)
    (&q_s[0][0])[e] =
        Elem<T>::to_f(((const T*)a.q)[(n * a.num_q_heads + (int64_t)g * Gr) * D + e]) * scale;
  __syncthreads();
  float m[G], l[G], acc[G][E];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[h][e] = 0.f;
  }
  for (int t = t0 + wid; t < t1; t += 4) {
    const int pos = sel[t / a.block] * a.block + t % a.block;
    if (pos >= L) continue;
    const int slot = rt[pos];
    if (slot < 0 || slot >= a.num_slots) {
      if (lane == 0) set_status(p.status, kStatusSlotRange);
      continue;
    }
    const int64_t r = ((int64_t)slot * a.num_kv_heads + g) * D;
    float k[E], v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      k[e] = Elem<T>::to_f(((const T*)a.k_pool)[r + e * 32 + lane]);
      v[e] = Elem<T>::to_f(((const T*)a.v_pool)[r + e * 32 + lane]);
    }
#pragma unroll
    for (int h = 0; h < G; ++h) {
      if (h >= Gr) break;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(q_s[h][e * 32 + lane], k[e], s);
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
  for (int h = 0; h < G; ++h) {
    if (lane == 0) {
      sm[wid][h] = m[h];
      sl[wid][h] = l[h];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) so[wid][h][e * 32 + lane] = acc[h][e];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < Gr * D; x += 128) {
    const int h = x / D, e = x - h * D;
    float M = fmaxf(fmaxf(sm[0][h], sm[1][h]), fmaxf(sm[2][h], sm[3][h]));
    float den = 0.f, num = 0.f;
    for (int w = 0; w < 4; ++w) {
      const float c = sm[w][h] == -INFINITY ? 1.f : exp2f(sm[w][h] - M);
      den = fmaf(sl[w][h], c, den);
      num = fmaf(so[w][h][e], c, num);
    }
    const int64_t pi = (unit * p.parts + part) * Gr + h;
    p.w.po[pi * D + e] = den == 0.f ? 0.f : num / den;
    if (e == 0) p.w.plse[pi] = den == 0.f ? -INFINITY : M + log2f(den);
  }
}

template <typename T>
__global__ void sparse_merge_kernel(Params p) {
  const rc_sparse_decode_args& a = p.a;
  const int64_t x = blockIdx.x;   // row * Hq + query head
  const int64_t n = x / a.num_q_heads;
  const int hq = (int)(x - n * a.num_q_heads);
  const int g = hq / p.G, h = hq - g * p.G;
  const int D = a.head_dim, e = threadIdx.x;
  const int64_t unit = n * a.num_kv_heads + g;
  float M = -INFINITY;
  for (int c = 0; c < p.parts; ++c) M = fmaxf(M, p.w.plse[(unit * p.parts + c) * p.G + h]);
  float num = 0.f, den = 0.f;
  for (int c = 0; c < p.parts; ++c) {
    const int64_t pi = (unit * p.parts + c) * p.G + h;
    const float pl = p.w.plse[pi];
    const float w = pl == -INFINITY ? 0.f : exp2f(pl - M);
    den += w;
    num = fmaf(w, p.w.po[pi * D + e], num);
  }
  ((T*)a.o)[x * D + e] = Elem<T>::from_f(den == 0.f ? 0.f : num / den);
  if (a.lse && e == 0) a.lse[x] = den == 0.f ? -INFINITY : (M + log2f(den)) * kLn2;
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
  RC_CHECK_ARG((int64_t)a->num_rows * a->num_q_heads < (1ll << 31), "%s: too many rows", fn);
  return RC_OK;
}

Params params_of(const rc_sparse_decode_args* a) {
  Params p{};
  p.a = *a;
  p.G = a->num_q_heads / a->num_kv_heads;
  p.nb = std::max(1, (a->max_seq_len + a->block - 1) / a->block);
  const int64_t tokens = (int64_t)std::min(p.nb, a->top_blocks) * a->block;
  p.parts = (int)((tokens + kPart - 1) / kPart);
  return p;
}

template <typename T, int D>
void launch_attend(const Params& p, dim3 grid, cudaStream_t s) {
  if (p.G <= 1) sparse_attend_kernel<T, D, 1><<<grid, 128, 0, s>>>(p);
  else if (p.G <= 2) sparse_attend_kernel<T, D, 2><<<grid, 128, 0, s>>>(p);
  else if (p.G <= 4) sparse_attend_kernel<T, D, 4><<<grid, 128, 0, s>>>(p);
  else if (p.G <= 8) sparse_attend_kernel<T, D, 8><<<grid, 128, 0, s>>>(p);
  else sparse_attend_kernel<T, D, 16><<<grid, 128, 0, s>>>(p);
}

template <typename T>
int launch(const Params& p, cudaStream_t s) {
  const unsigned units = (unsigned)(p.a.num_rows * p.a.num_kv_heads);
  sparse_score_kernel<T><<<dim3(units, std::min((p.nb + 7) / 8, 64)), 256, 0, s>>>(p);
  sparse_select_kernel<<<units, 256, 0, s>>>(p);
  const dim3 grid(units, p.parts);
  if (p.a.head_dim == 128) launch_attend<T, 128>(p, grid, s);
  else launch_attend<T, 64>(p, grid, s);
  sparse_merge_kernel<T><<<p.a.num_rows * p.a.num_q_heads, p.a.head_dim, 0, s>>>(p);
  count_launches(4);
  return check_launch("rc_sparse_decode_attention");
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
  RC_CHECK_ARG(p.parts <= 65535, "%s: top_blocks %d of %d tokens are too many", fn, a->top_blocks,
               a->block);
  size_t need = 0;
  p.w = rc::carve(workspace, p, &need);
  RC_CHECK_ARG(workspace_bytes >= need, "%s: workspace %zu bytes < %zu needed", fn, workspace_bytes,
               need);
  p.status = rc::device_status_ptr();
  if (!p.status) return rc::fail(RC_ERR_CUDA, "%s: no device status word", fn);
  return a->dtype == RC_DTYPE_BF16 ? rc::launch<__nv_bfloat16>(p, (cudaStream_t)stream)
                                   : rc::launch<float>(p, (cudaStream_t)stream);
}
