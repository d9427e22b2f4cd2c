// Norms of queries and keys for each head with the position rotation in the same pass:
//   y = x * rsqrt(mean(x^2) + eps) * w   per head row,   then (a, b) -> (a cos - b sin, b cos + a sin)
// in fp32, rounded once at the store.
//
// One group of L lanes per (token, head) row (norm_rope.cuh). A CTA works on heads of one token, so
// the token's cosines and sines are loaded once per lane and serve every head the lane works on;
// the loads of kBatch heads are in flight together.
#include <algorithm>
#include <cmath>

#include "host_common.h"
#include "norm_rope.cuh"

namespace rc {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 2;   // heads a lane group holds at a time

// splits CTAs per token, each with every splits-th group of kBatch * kThreads / L heads
template <typename T, int L, int NB>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(rc_qk_norm_rope_args a, int splits,
                                                                int* status) {
  constexpr int ROWS = kThreads / L;
  const int64_t t = blockIdx.x / splits;
  const int split = blockIdx.x - (int)t * splits;
  const int i = threadIdx.x % L;
  const int r = a.rotary_dim;
  const bool inter = a.interleaved != 0;
  const LaneChunks lc = lane_chunks(i, a.head_dim, r, inter);
  const int pos = r ? a.positions[t] : 0;
  const int rows = a.num_q_heads + a.num_kv_heads;
  LaneAngles ang;
  bool have_angles = false;
  for (int h0 = split * ROWS * NB + threadIdx.x / L; h0 - (int)threadIdx.x / L < rows;
       h0 += splits * ROWS * NB) {
    Raw<T> x[NB], y[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int h = h0 + b * ROWS;
      const bool is_q = h < a.num_q_heads;
      const int64_t hh = is_q ? h : h - a.num_q_heads;
      const T* src = is_q ? (const T*)a.q + t * a.q_token_stride + hh * a.q_head_stride
                          : (const T*)a.k + t * a.k_token_stride + hh * a.k_head_stride;
      x[b].clear();
      y[b].clear();
      if (h < rows && lc.c0 >= 0) x[b].load(src + lc.c0 * 8);
      if (h < rows && lc.c1 >= 0) y[b].load(src + lc.c1 * 8);
    }
    if (r && !have_angles) {
      if (pos < 0 || pos >= a.max_position) {   // the same for the whole CTA
        if (threadIdx.x == 0) set_status(status, kStatusPosRange);
        return;
      }
      if (lc.rot) load_angles(a.rope + (int64_t)pos * r, i, r, ang);
      have_angles = true;
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int h = h0 + b * ROWS;
      const bool is_q = h < a.num_q_heads;
      const int64_t hh = is_q ? h : h - a.num_q_heads;
      T* dst = is_q ? (T*)a.q_out + t * a.q_out_token_stride + hh * a.q_out_head_stride
                    : (T*)a.k_out + t * a.k_out_token_stride + hh * a.k_out_head_stride;
      const T* w = (const T*)(is_q ? a.q_weight : a.k_weight);
      const bool v0 = h < rows && lc.c0 >= 0, v1 = h < rows && lc.c1 >= 0;
      float u[8], v[8];
      x[b].get(u);
      y[b].get(v);
      const float inv = norm_scale<L>(u, v, a.head_dim, a.eps);
      if (w && v0) scale8(u, inv, w + lc.c0 * 8);
      if (w && v1) scale8(v, inv, w + lc.c1 * 8);
      if (lc.rot) rotate_pairs(u, v, inter, ang);
      if (v0) store8(dst + lc.c0 * 8, u);
      if (v1) store8(dst + lc.c1 * 8, v);
    }
  }
}

template <typename T, int L>
void launch_l(const rc_qk_norm_rope_args& a, int sms, int* st, cudaStream_t s) {
  // with few tokens the heads of one go to several CTAs, one batch of one head each
  const int rows = a.num_q_heads + a.num_kv_heads;
  const int groups = (rows + kThreads / L - 1) / (kThreads / L);
  if (a.num_tokens * groups <= (int64_t)sms * 8)
    qk_norm_rope_kernel<T, L, 1><<<(unsigned)(a.num_tokens * groups), kThreads, 0, s>>>(a, groups, st);
  else
    qk_norm_rope_kernel<T, L, kBatch><<<(unsigned)a.num_tokens, kThreads, 0, s>>>(a, 1, st);
}

template <typename T>
void launch(const rc_qk_norm_rope_args& a, int sms, int* st, cudaStream_t s) {
  switch (head_lanes(a.head_dim)) {
    case 4: launch_l<T, 4>(a, sms, st, s); break;
    case 8: launch_l<T, 8>(a, sms, st, s); break;
    default: launch_l<T, 16>(a, sms, st, s); break;
  }
}

}  // namespace

int check_norm_rope(const char* fn, int head_dim, int rotary_dim, int64_t max_position,
                    const float* rope, float eps, bool any_weight) {
  RC_CHECK_ARG(head_dim >= 8 && head_dim <= kNormRopeMaxDim && head_dim % 8 == 0,
               "%s: head_dim %d (a multiple of 8 up to %d)", fn, head_dim, kNormRopeMaxDim);
  RC_CHECK_ARG(rotary_dim >= 0 && rotary_dim <= head_dim && rotary_dim % 16 == 0,
               "%s: rotary_dim %d (a multiple of 16 up to head_dim)", fn, rotary_dim);
  RC_CHECK_ARG(rotary_dim == 0 || (rope && ((uintptr_t)rope & 15) == 0 && max_position > 0),
               "%s: the rotation needs a 16-byte aligned table with at least one position", fn);
  RC_CHECK_ARG(!any_weight || (eps >= 0.f && std::isfinite(eps)), "%s: eps must be finite and >= 0",
               fn);
  return RC_OK;
}

int sm_count(const char* fn, int* out) {
  static PerDevice<int> sms;
  const int* v = nullptr;
  const cudaError_t e = sms.get(
      [](int& n) {
        int dev = 0;
        const cudaError_t r = cudaGetDevice(&dev);
        return r == cudaSuccess ? cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) : r;
      },
      &v);
  if (e != cudaSuccess) return fail(RC_ERR_CUDA, "%s: device query: %s", fn, cudaGetErrorString(e));
  *out = *v;
  return RC_OK;
}

}  // namespace rc

extern "C" int rc_qk_norm_rope(const rc_qk_norm_rope_args* a, void* stream) {
  static const char* fn = "rc_qk_norm_rope";
  RC_CHECK_ARG(a != nullptr, "%s: args is NULL", fn);
  RC_CHECK_ARG(a->dtype == RC_DTYPE_BF16 || a->dtype == RC_DTYPE_F32, "%s: dtype %d", fn, a->dtype);
  RC_CHECK_ARG(a->num_tokens >= 0 && a->num_tokens <= 0x7fffffff && a->num_q_heads >= 0 &&
                   a->num_kv_heads >= 0 && a->num_q_heads <= 65536 && a->num_kv_heads <= 65536,
               "%s: bad sizes", fn);
  const int c = rc::check_norm_rope(fn, a->head_dim, a->rotary_dim, a->max_position, a->rope, a->eps,
                                    a->q_weight || a->k_weight);
  if (c != RC_OK) return c;
  if (a->num_tokens == 0 || a->num_q_heads + a->num_kv_heads == 0) return RC_OK;
  RC_CHECK_ARG(a->num_q_heads == 0 || (a->q && a->q_out), "%s: q or q_out is NULL", fn);
  RC_CHECK_ARG(a->num_kv_heads == 0 || (a->k && a->k_out), "%s: k or k_out is NULL", fn);
  RC_CHECK_ARG(a->rotary_dim == 0 || a->positions, "%s: positions is NULL", fn);
  const uintptr_t ptrs = (uintptr_t)a->q | (uintptr_t)a->k | (uintptr_t)a->q_out |
                         (uintptr_t)a->k_out | (uintptr_t)a->q_weight | (uintptr_t)a->k_weight;
  const int64_t strides = a->q_token_stride | a->q_head_stride | a->k_token_stride |
                          a->k_head_stride | a->q_out_token_stride | a->q_out_head_stride |
                          a->k_out_token_stride | a->k_out_head_stride;
  const int es = a->dtype == RC_DTYPE_BF16 ? 2 : 4;
  RC_CHECK_ARG((ptrs & 15) == 0 && (strides * es & 15) == 0,
               "%s: pointers and strides must be multiples of 16 bytes", fn);
  int* st = rc::device_status_ptr();
  if (!st) return rc::fail(RC_ERR_CUDA, "%s: no device status word", fn);
  int sms = 0;
  const int e = rc::sm_count(fn, &sms);
  if (e != RC_OK) return e;
  if (a->dtype == RC_DTYPE_BF16)
    rc::launch<__nv_bfloat16>(*a, sms, st, (cudaStream_t)stream);
  else
    rc::launch<float>(*a, sms, st, (cudaStream_t)stream);
  rc::count_launches(1);
  return rc::check_launch(fn);
}
