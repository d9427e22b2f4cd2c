// Whether strided tensors of a call share memory (host side).
#pragma once
#include <cstdint>

namespace rc {

// The rows of a [tokens, heads, width] tensor, all in bytes.
struct RowsView {
  const void* p;
  int64_t token_stride, head_stride;
  int64_t tokens, heads, width;
};
// False only if no byte of a is one of b's. Both have as many tokens. Views with unlike token strides
// are told apart by the ranges of their addresses alone.
bool views_overlap(const RowsView& a, const RowsView& b);
// Whether two rows of a view share a byte.
bool rows_overlap(const RowsView& a);

}  // namespace rc
