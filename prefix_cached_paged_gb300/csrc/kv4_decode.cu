// Decode attention over the cache held in 4 bits (format: kv4.cuh).
//
// One CTA per (query row, KV head); its warps take the row's tokens in turn, a lane holding d / 32
// elements of all the head's queries, and keep running maxima and sums that are joined at the end.
#include <algorithm>
#include <cmath>

#include "host_common.h"
#include "kv4.cuh"

namespace rc {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxGroup = 16;

struct Params {
  rc_kv4_decode_args a;
  int G;
  int* status;
};

template <int D>
__device__ __forceinline__ void token_values(const char* head, int lane, float* x) {
  constexpr int E = D / 32, NG = D / 32, RB = kv4_row_bytes(D);
  (void)RB;
  const int w = lane * E / 8, n = lane * E % 8;
  const uint32_t c = ((const uint32_t*)head)[w] >> 4 * n, p = ((const uint32_t*)head)[D / 8 + w % NG];
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = fmaf((float)(c >> 4 * e & 15u), bf16lo(p), bf16hi(p));
}

template <typename T, int D, int GM>
__global__ void __launch_bounds__(kThreads) kv4_decode_kernel(Params p) {
  constexpr int E = D / 32, NG = D / 32, RB = kv4_row_bytes(D);
  __shared__ float so[kWarps][GM][D], sm[kWarps][GM], sl[kWarps][GM];
  const auto& a = p.a;
  const int G = p.G, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = blockIdx.x / a.num_kv_heads, h = blockIdx.x % a.num_kv_heads;
  int len = a.seq_len[n];
  const int req = a.req_idx[n];
  if (len != 0 && (len < 0 || len > a.max_seq_len || req < 0 || req >= a.max_reqs)) {
    if (threadIdx.x == 0) set_status(p.status, kStatusPosRange);
    len = 0;
  }
  // the lane's elements: 32 j + 8 t + n0 ..
  const int w = lane * E / 8;
  const int d0 = 32 * (w % NG) + 8 * (w / NG) + lane * E % 8;
  float q[GM][E], o[GM][E] = {}, m[GM], l[GM] = {};
  const T* qr = (const T*)a.q + ((int64_t)n * a.num_q_heads + (int64_t)h * G) * D + d0;
#pragma unroll
  for (int g = 0; g < GM; ++g) {
    m[g] = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e)
      q[g][e] = g < G ? Elem<T>::to_f(qr[g * D + e]) * a.sm_scale * kLog2e : 0.f;
  }
  const int32_t* row = a.req_to_token + (int64_t)(len ? req : 0) * a.max_ctx;
  for (int t = warp; t < len; t += kWarps) {
    const int slot = row[t];
    if (slot < 0 || slot >= a.num_slots) {
      if (lane == 0) set_status(p.status, kStatusSlotRange);
      continue;
    }
    const int64_t at = ((int64_t)slot * a.num_kv_heads + h) * RB;
    float k[E], v[E];
    token_values<D>((const char*)a.k_pool + at, lane, k);
    token_values<D>((const char*)a.v_pool + at, lane, v);
#pragma unroll
    for (int g = 0; g < GM; ++g) {
      if (g >= G) break;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(q[g][e], k[e], s);
#pragma unroll
      for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
      const float mx = fmaxf(m[g], s), c = m[g] == -INFINITY ? 0.f : exp2f(m[g] - mx);
      const float w = exp2f(s - mx);
      m[g] = mx;
      l[g] = l[g] * c + w;
#pragma unroll
      for (int e = 0; e < E; ++e) o[g][e] = fmaf(w, v[e], o[g][e] * c);
    }
  }
#pragma unroll
  for (int g = 0; g < GM; ++g) {
    if (lane == 0) sm[warp][g] = m[g], sl[warp][g] = l[g];
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][g][d0 + e] = o[g][e];
  }
  __syncthreads();
  const int64_t o0 = ((int64_t)n * a.num_q_heads + (int64_t)h * G) * D;
  for (int x = threadIdx.x; x < G * D; x += kThreads) {
    const int g = x / D;
    float mx = -INFINITY, den = 0.f, num = 0.f;
    for (int c = 0; c < kWarps; ++c) mx = fmaxf(mx, sm[c][g]);
    for (int c = 0; c < kWarps; ++c) {
      const float f = sm[c][g] == -INFINITY ? (sl[c][g] == 0.f ? 0.f : 1.f) : exp2f(sm[c][g] - mx);
      den += f * sl[c][g];
      num += f * so[c][g][x % D];
    }
    ((T*)a.o)[o0 + x] = Elem<T>::from_f(den == 0.f ? 0.f : num / den);
    if (a.lse && x % D == 0)
      a.lse[(int64_t)n * a.num_q_heads + (int64_t)h * G + g] =
          den == 0.f ? -INFINITY : kLn2 * (mx + log2f(den));
  }
}

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

template <typename T, int D>
void launch(const Params& p, cudaStream_t s) {
  const unsigned grid = (unsigned)(p.a.num_rows * p.a.num_kv_heads);
  if (p.G <= 4)
    kv4_decode_kernel<T, D, 4><<<grid, kThreads, 0, s>>>(p);
  else
    kv4_decode_kernel<T, D, 16><<<grid, kThreads, 0, s>>>(p);
  count_launches(1);
}

}  // namespace
}  // namespace rc

extern "C" int rc_kv4_decode_workspace_bytes(const rc_kv4_decode_args* a, size_t* out_bytes) {
  const int v = rc::validate(a, "rc_kv4_decode_workspace_bytes");
  if (v != RC_OK) return v;
  RC_CHECK_ARG(out_bytes != nullptr, "rc_kv4_decode_workspace_bytes: out_bytes is NULL");
  *out_bytes = 0;
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
  size_t need = 0;
  rc_kv4_decode_workspace_bytes(a, &need);
  RC_CHECK_ARG(need == 0 || (workspace && workspace_bytes >= need),
               "%s: workspace %zu bytes < %zu needed", fn, workspace ? workspace_bytes : 0, need);
  rc::Params p{*a, a->num_q_heads / a->num_kv_heads, rc::device_status_ptr()};
  if (!p.status) return rc::fail(RC_ERR_CUDA, "%s: no device status word", fn);
  const cudaStream_t s = (cudaStream_t)stream;
  if (a->dtype == RC_DTYPE_BF16)
    a->head_dim == 128 ? rc::launch<__nv_bfloat16, 128>(p, s) : rc::launch<__nv_bfloat16, 64>(p, s);
  else
    a->head_dim == 128 ? rc::launch<float, 128>(p, s) : rc::launch<float, 64>(p, s);
  return rc::check_launch(fn);
}
