#include "views.h"

#include <algorithm>

namespace rc {
namespace {

using i128 = __int128;   // strides are a caller's: products of any of them stay exact

struct Rows {
  i128 p, ts, hs, T, H, w;
  explicit Rows(const RowsView& v)
      : p((i128)(uintptr_t)v.p), ts(v.tokens > 1 ? v.token_stride : 0),
        hs(v.heads > 1 ? v.head_stride : 0), T(v.tokens), H(v.heads), w(v.width) {}
  i128 low() const { return p + std::min<i128>(0, (T - 1) * ts) + std::min<i128>(0, (H - 1) * hs); }
  i128 high() const {
    return p + std::max<i128>(0, (T - 1) * ts) + std::max<i128>(0, (H - 1) * hs) + w;
  }
  i128 span() const { return (H - 1) * hs + w; }   // of a token's rows, hs >= 0
};

// Whether rows of w bytes, x apart for tokens of the same number, meet for any two of T tokens.
bool meet(i128 x, i128 ts, i128 T, i128 w) {
  if (ts < 0) ts = -ts;   // the same set of differences
  i128 dt = 0;
  if (ts > 0) {   // the two multiples of ts nearest to -x
    dt = -x / ts;
    if (dt * ts > -x) --dt;
  }
  for (int i = 0; i < 2; ++i) {
    const i128 d = x + std::min(std::max(dt + i, -(T - 1)), T - 1) * ts;
    if (d > -w && d < w) return true;
  }
  return false;
}

}  // namespace

bool views_overlap(const RowsView& va, const RowsView& vb) {
  const Rows a(va), b(vb);
  if (a.T <= 0 || a.H <= 0 || b.H <= 0) return false;
  if (a.high() <= b.low() || b.high() <= a.low()) return false;
  if (a.ts != b.ts) return true;
  const i128 x = b.p - a.p;
  if (a.ts > 0 && a.hs >= 0 && b.hs >= 0) {   // slices of one row, the usual case
    const i128 r = (x % a.ts + a.ts) % a.ts;
    if (r >= a.span() && r + b.span() <= a.ts) return false;
  }
  const i128 hs = a.H > 1 ? a.hs : b.hs;
  if (b.H == 1 || b.hs == hs) {
    for (i128 dh = -(a.H - 1); dh <= b.H - 1; ++dh)
      if (meet(x + dh * hs, a.ts, a.T, a.w)) return true;
    return false;
  }
  if (a.H * b.H > 4096) return true;
  for (i128 i = 0; i < a.H; ++i)
    for (i128 j = 0; j < b.H; ++j)
      if (meet(x + j * b.hs - i * a.hs, a.ts, a.T, a.w)) return true;
  return false;
}

bool rows_overlap(const RowsView& va) {
  const Rows a(va);
  if (a.T > 1 && a.ts < a.w && a.ts > -a.w) return true;
  if (a.H <= 1) return false;
  if (a.hs >= a.w && (a.T <= 1 || a.ts >= a.span())) return false;                      // tokens first
  if (a.hs >= a.w && a.ts >= a.w && a.hs >= (a.T - 1) * a.ts + a.w) return false;   // heads first
  for (i128 dh = 1; dh < a.H; ++dh)
    if (meet(dh * a.hs, a.ts, a.T, a.w)) return true;
  return false;
}

}  // namespace rc
