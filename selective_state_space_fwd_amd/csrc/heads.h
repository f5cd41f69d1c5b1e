// Argument checks of strided [batch, seqlen, heads, dim] arrays, shared by the C-ABI entry points of
// linear attention and of the queries' and keys' norm (host only).
#pragma once
#include <stdint.h>

#include "linattn_launch.h"
#include "strided.h"

namespace ssm_api {

// `strides` (batch, step, head; NULL: contiguous) of p as `rows`, and the bytes from its first to
// past its last element. The contiguous size in bytes fits int64.
inline int check_heads(const void* p, const int64_t* strides, int64_t batch, int64_t seqlen, int64_t heads,
                       int64_t dim, int64_t esz, ssm::HeadRows* rows, int64_t* bytes) {
  const int64_t size[3] = {batch, seqlen, heads};
  int64_t st[3] = {seqlen * heads * dim, heads * dim, dim};
  *rows = ssm::HeadRows{p, st[0], st[1], st[2]};
  *bytes = 0;
  if (batch == 0 || seqlen == 0 || heads == 0 || dim == 0) return SSM_OK;
  int64_t last = dim - 1;
  for (int i = 0; i < 3; ++i) {
    if (size[i] == 1) continue;  // the only index of its axis: the stride is never used
    if (strides) st[i] = strides[i];
    int64_t reach;
    if (st[i] < 0) return SSM_ERR_INVALID_ARG;
    if (!mul_ok(size[i] - 1, st[i], &reach) || reach > INT64_MAX - last) return SSM_ERR_UNSUPPORTED;
    last += reach;
  }
  if (last == INT64_MAX || !mul_ok(last + 1, esz, bytes)) return SSM_ERR_UNSUPPORTED;
  *rows = ssm::HeadRows{p, st[0], st[1], st[2]};
  return SSM_OK;
}

inline int io_bytes(uint32_t flags) {
  const uint32_t io = flags & SSM_IO_MASK;
  return io == SSM_IO_BF16 ? 2 : io == SSM_IO_F32 ? 4 : 0;
}

// The product of non-negative sizes, or -1 where it passes int64.
inline int64_t product(std::initializer_list<int64_t> sizes) {
  int64_t n = 1;
  for (int64_t s : sizes) {
    if (s == 0) return 0;
  }
  for (int64_t s : sizes)
    if (!mul_ok(n, s, &n)) return -1;
  return n;
}

}  // namespace ssm_api
