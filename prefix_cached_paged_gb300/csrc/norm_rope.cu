// Norms of queries and keys for each head with the position rotation in the same pass:
//   y = x * rsqrt(mean(x^2) + eps) * w   per head row,   then (a, b) -> (a cos - b sin, b cos + a sin)
// in fp32, rounded once at the store.
//
// Bound by HBM: every element is read and written once, the table row once per token. A warp works
// on the heads of one token, 32 / L head rows (norm_rope.cuh) at a time, so the token's cosines and
// sines are loaded once per lane and serve every head. Rows stream through a ring in shared memory
// by 16-byte asynchronous copies; a lane reads only what it copied itself, so the ring needs no
// barrier, and the arithmetic runs on packed fp32 pairs.
//
// Measured, 16 000 tokens of 32 + 32 heads of 128, bf16, sliced from a fused projection: 84 us,
// 6.29 TB/s, 94 % of the copy rate (issue slots 68 % busy, DRAM 74 % of its nominal peak). On the way:
// one CTA per token and scalar arithmetic 94 us (267 warp instructions per 4 rows, a third of them
// per-CTA set-up); four rows per lane in registers 152 us (115 registers, too few warps); one head
// group per warp, the angles loaded anew for each, 121 us; three ring stages instead of four 87 us.
#include <algorithm>
#include <cmath>

#include "host_common.h"
#include "norm_rope.cuh"
#include "views.h"

namespace rc {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kStages = 4;   // row groups of a warp in flight

// splits warps per token, each with consecutive groups of 32 / L heads (queries, then keys)
template <typename T, int L>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(rc_qk_norm_rope_args a, int splits,
                                                                int* status) {
  constexpr int ROWS = 32 / L, N = Raw<T>::N;
  __shared__ uint4 ring[kWarps][kStages][2 * N][32];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int64_t gw = (int64_t)blockIdx.x * kWarps + wid;
  const int64_t t = gw / splits;
  if (t >= a.num_tokens) return;
  const int i = lane % L, r = a.rotary_dim;
  const bool inter = a.interleaved != 0;
  const LaneChunks lc = lane_chunks(i, a.head_dim, r, inter);
  const int rows = a.num_q_heads + a.num_kv_heads;
  const int groups = (rows + ROWS - 1) / ROWS, per = (groups + splits - 1) / splits;
  const int g0 = (int)(gw - t * splits) * per, g1 = min(groups, g0 + per);
  const T* q = (const T*)a.q + t * a.q_token_stride;
  const T* k = (const T*)a.k + t * a.k_token_stride;
  T* qo = (T*)a.q_out + t * a.q_out_token_stride;
  T* ko = (T*)a.k_out + t * a.k_out_token_stride;
  auto issue = [&](int g) {
    const int h = g * ROWS + lane / L;
    if (g < g1 && h < rows) {
      const T* src = h < a.num_q_heads ? q + h * a.q_head_stride
                                       : k + (h - a.num_q_heads) * a.k_head_stride;
      uint4(*st)[32] = ring[wid][g % kStages];
#pragma unroll
      for (int c = 0; c < N; ++c) {
        if (lc.c0 >= 0) cp_async16(smem_u32(&st[c][lane]), (const uint4*)(src + lc.c0 * 8) + c);
        if (lc.c1 >= 0) cp_async16(smem_u32(&st[N + c][lane]), (const uint4*)(src + lc.c1 * 8) + c);
      }
    }
    cp_async_commit();
  };
  const int pos = r ? a.positions[t] : 0;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue(g0 + s);
  LaneAngles ang;
  if (r) {
    if (pos < 0 || pos >= a.max_position) {   // the same for the whole warp
      if (lane == 0) set_status(status, kStatusPosRange);
      cp_async_wait<0>();
      return;
    }
    if (lc.rot) ang.load(a.rope + (int64_t)pos * r, i, r);
  }
  LaneRow w;
  int part = -1;   // whose weights w holds: 0 queries', 1 keys'
  for (int g = g0; g < g1; ++g) {
    issue(g + kStages - 1);
    cp_async_wait<kStages - 1>();
    const int h = g * ROWS + lane / L;
    const int mine = h < a.num_q_heads ? 0 : 1;
    const bool v0 = h < rows && lc.c0 >= 0, v1 = h < rows && lc.c1 >= 0;
    const T* weights = (const T*)(mine ? a.k_weight : a.q_weight);
    if (mine != part && weights) load_weights(weights, lc, w);
    part = mine;
    Raw<T> x, y;
    x.clear();
    y.clear();
    uint4(*st)[32] = ring[wid][g % kStages];
#pragma unroll
    for (int c = 0; c < N; ++c) {
      if (v0) x.v[c] = st[c][lane];
      if (v1) y.v[c] = st[N + c][lane];
    }
    LaneRow row;
    x.get(row.x);
    y.get(row.y);
    const float inv = row.template norm_scale<L>(a.head_dim, a.eps);
    if (weights) row.scale(inv, w);
    if (lc.rot) row.rotate(ang, inter);
    x.set(row.x);
    y.set(row.y);
    T* dst = mine ? ko + (h - a.num_q_heads) * a.k_out_head_stride : qo + h * a.q_out_head_stride;
    if (v0) x.store(dst + lc.c0 * 8);
    if (v1) y.store(dst + lc.c1 * 8);
  }
  cp_async_wait<0>();
}

template <typename T, int L>
void launch_l(const rc_qk_norm_rope_args& a, int sms, int* st, cudaStream_t s) {
  // One warp per token where there are tokens enough; with fewer, their heads go to more warps, down
  // to one group of heads each. 16 000 tokens: 84 us with one warp each, 90 with two, 104 with four;
  // 8 tokens of 40 heads: 3.7 us with ten warps each, 6.3 with a CTA of four.
  const int groups = (a.num_q_heads + a.num_kv_heads + 32 / L - 1) / (32 / L);
  int splits = 1;
  while (splits < groups && a.num_tokens * splits < (int64_t)sms * kWarps * 16) splits *= 2;
  splits = std::min(splits, groups);
  const int64_t ctas = (a.num_tokens * splits + kWarps - 1) / kWarps;
  qk_norm_rope_kernel<T, L><<<(unsigned)ctas, kThreads, 0, s>>>(a, splits, st);
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

namespace {
bool same_rows(const RowsView& a, const RowsView& b) {
  return a.p == b.p && (a.tokens == 1 || a.token_stride == b.token_stride) &&
         (a.heads == 1 || a.head_stride == b.head_stride);
}
// Rows are read up to three groups of heads ahead of what is written, by other warps too: an output
// is its input, row for row, or shares nothing with any input and the other output.
bool outputs_clear(const rc_qk_norm_rope_args& a, int es) {
  const int64_t T = a.num_tokens, w = (int64_t)a.head_dim * es;
  const int64_t hq = a.num_q_heads, hk = a.num_kv_heads;
  const RowsView q{a.q, a.q_token_stride * es, a.q_head_stride * es, T, hq, w};
  const RowsView k{a.k, a.k_token_stride * es, a.k_head_stride * es, T, hk, w};
  const RowsView qo{a.q_out, a.q_out_token_stride * es, a.q_out_head_stride * es, T, hq, w};
  const RowsView ko{a.k_out, a.k_out_token_stride * es, a.k_out_head_stride * es, T, hk, w};
  const bool q_in_place = hq == 0 || same_rows(q, qo), k_in_place = hk == 0 || same_rows(k, ko);
  if ((hq && rows_overlap(qo)) || (hk && rows_overlap(ko))) return false;
  if (!q_in_place && views_overlap(qo, q)) return false;
  if (!k_in_place && views_overlap(ko, k)) return false;
  if (hq == 0 || hk == 0) return true;
  if (views_overlap(qo, ko)) return false;
  return (k_in_place || !views_overlap(qo, k)) && (q_in_place || !views_overlap(ko, q));
}
}  // namespace

}  // namespace rc

extern "C" int rc_qk_norm_rope(const rc_qk_norm_rope_args* a, void* stream) {
  static const char* fn = "rc_qk_norm_rope";
  RC_CHECK_ARG(a != nullptr, "%s: args is NULL", fn);
  RC_CHECK_ARG(a->dtype == RC_DTYPE_BF16 || a->dtype == RC_DTYPE_F32, "%s: dtype %d", fn, a->dtype);
  RC_CHECK_ARG(a->num_tokens >= 0 && a->num_tokens <= (1 << 24) && a->num_q_heads >= 0 &&
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
  RC_CHECK_ARG(rc::outputs_clear(*a, es),
               "%s: an output overlaps an input it is not the same rows of, the other output or "
               "itself", fn);
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
