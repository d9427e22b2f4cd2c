// rc_kv4_decode_attention: checks, sizes and the bf16 kernels of kv4_decode.cuh.
#include "kv4_decode.cuh"

namespace rc {
namespace kv4 {

template cudaError_t launch<__nv_bfloat16>(const Params&, cudaStream_t);

namespace {

// Whether two ranges of bytes meet.
bool meet(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + (uint64_t)nb && y < x + (uint64_t)na;
}

int validate(const rc_kv4_decode_args* a, const char* fn) {
  RC_CHECK_ARG(a != nullptr, "%s: args is NULL", fn);
  RC_CHECK_ARG(a->dtype == RC_DTYPE_BF16 || a->dtype == RC_DTYPE_F32, "%s: dtype %d", fn, a->dtype);
  RC_CHECK_ARG(a->num_rows >= 0 && a->num_q_heads > 0 && a->num_kv_heads > 0 &&
                   a->num_kv_heads <= 65536 && a->num_q_heads % a->num_kv_heads == 0,
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

// What the configuration of the kernel that runs these sizes says.
template <typename F>
int by_kernel(const rc_kv4_decode_args& a, F f) {
  const bool many = a.num_q_heads / a.num_kv_heads > 8, wide = a.head_dim == 128;
  if (a.dtype == RC_DTYPE_F32)
    return many ? wide ? f(Cfg<float, 128, 2>()) : f(Cfg<float, 64, 2>())
                : wide ? f(Cfg<float, 128, 1>()) : f(Cfg<float, 64, 1>());
  return many ? wide ? f(Cfg<__nv_bfloat16, 128, 2>()) : f(Cfg<__nv_bfloat16, 64, 2>())
              : wide ? f(Cfg<__nv_bfloat16, 128, 1>()) : f(Cfg<__nv_bfloat16, 64, 1>());
}

Params params_of(const rc_kv4_decode_args* a) {
  Params p{};
  p.a = *a;
  p.G = a->num_q_heads / a->num_kv_heads;
  const int warps = by_kernel(*a, [](auto c) { return decltype(c)::WARPS; });
  for (int h = 1; h <= warps; ++h)
    if (a->num_kv_heads % h == 0) p.HG = h;
  p.TS = warps / p.HG;
  p.stride = a->num_kv_heads * kv4_row_bytes(a->head_dim);
  p.tokens = 16 * p.TS * by_kernel(*a, [](auto c) { return decltype(c)::U; });
  while (1 << p.log_tokens < p.tokens) ++p.log_tokens;   // 8 and 4 by any number of heads, rounded down, are powers of two
  p.groups = a->num_kv_heads / p.HG;
  return p;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }
Workspace carve(void* base, const Params& p, size_t* total) {
  const size_t c = (size_t)most_ctas(p), heads = c * 2 * p.HG * p.G;
  Workspace w{};
  char* b = (char*)base;
  size_t at = 0;
  w.range = (Range*)b;
  at += align256(c * sizeof(Range));
  w.ml = (float*)(b + at);
  at += align256(heads * 8);
  w.o = (float*)(b + at);
  at += align256(heads * p.a.head_dim * 4);
  *total = at;
  return w;
}

}  // namespace
}  // namespace kv4
}  // namespace rc

extern "C" int rc_kv4_decode_workspace_bytes(const rc_kv4_decode_args* a, size_t* out_bytes) {
  const int v = rc::kv4::validate(a, "rc_kv4_decode_workspace_bytes");
  if (v != RC_OK) return v;
  RC_CHECK_ARG(out_bytes != nullptr, "rc_kv4_decode_workspace_bytes: out_bytes is NULL");
  const rc::kv4::Params p = rc::kv4::params_of(a);
  rc::kv4::carve(nullptr, p, out_bytes);
  return RC_OK;
}

extern "C" int rc_kv4_decode_attention(const rc_kv4_decode_args* a, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  static const char* fn = "rc_kv4_decode_attention";
  const int v = rc::kv4::validate(a, fn);
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
  rc::kv4::Params p = rc::kv4::params_of(a);
  size_t need = 0;
  p.w = rc::kv4::carve(workspace, p, &need);
  RC_CHECK_ARG(workspace && workspace_bytes >= need, "%s: workspace %zu bytes < %zu needed", fn,
               workspace ? workspace_bytes : 0, need);
  // pairs that several CTAs share read q and the cache while others write o
  const int64_t outs = (int64_t)a->num_rows * a->num_q_heads * a->head_dim *
                       (a->dtype == RC_DTYPE_BF16 ? 2 : 4);
  const int64_t plane = a->num_slots * p.stride;
  RC_CHECK_ARG(!rc::kv4::meet(a->o, outs, a->q, outs) && !rc::kv4::meet(a->o, outs, a->k_pool, plane) &&
                   !rc::kv4::meet(a->o, outs, a->v_pool, plane) &&
                   !rc::kv4::meet(a->o, outs, workspace, (int64_t)need),
               "%s: o overlaps q, a plane or the workspace", fn);
  p.wait_ns = rc::wait_limit_ns();
  p.status = rc::device_status_ptr();
  if (!p.status) return rc::fail(RC_ERR_CUDA, "%s: no device status word", fn);
  const cudaError_t e = a->dtype == RC_DTYPE_BF16
                            ? rc::kv4::launch<__nv_bfloat16>(p, (cudaStream_t)stream)
                            : rc::kv4::launch<float>(p, (cudaStream_t)stream);
  if (e != cudaSuccess)
    return rc::fail(RC_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return rc::check_launch(fn);
}
