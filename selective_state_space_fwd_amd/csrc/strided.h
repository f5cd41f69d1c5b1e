// Argument checks of strided [batch, dim, seqlen] arrays, shared by the C-ABI entry points of
// the operators around the scan (host only).
#pragma once
#include <stdint.h>

#include "api_util.h"
#include "block_launch.h"
#include "ssm_scan.h"

namespace ssm_api {

// Several arguments' byte ranges, of which the outputs must overlap nothing.
struct Ranges {
  static constexpr int kMost = 20;
  Range r[kMost];
  bool out[kMost];
  int n = 0;
  void add(const void* p, int64_t bytes, bool output) {
    if (!p || bytes <= 0 || n >= kMost) return;
    r[n] = span(p, bytes);
    out[n++] = output;
  }
  bool clash() const {
    for (int i = 0; i < n; ++i)
      for (int j = i + 1; j < n; ++j)
        if ((out[i] || out[j]) && overlaps(r[i], r[j])) return true;
    return false;
  }
};

// Bytes from the first to past the last element, its strides and its order. SSM_OK or an error.
struct StridedArray {
  ssm::Strides s{};
  ssm::Order order = ssm::Order::Time;
  int64_t bytes = 0;
};

// strides NULL: contiguous. `output`: no two elements may share an address. Sizes are >= 0 and
// the contiguous size in bytes fits int64.
inline int check_strided(const int64_t* strides, int64_t batch, int64_t dim, int64_t seqlen,
                         int64_t esz, bool output, StridedArray* a) {
  const int64_t size[3] = {batch, dim, seqlen};
  int64_t st[3] = {dim * seqlen, seqlen, 1};
  if (strides)
    for (int i = 0; i < 3; ++i) st[i] = strides[i];
  a->bytes = 0;
  if (batch == 0 || dim == 0 || seqlen == 0) return SSM_OK;
  int64_t last = 0;
  for (int i = 0; i < 3; ++i) {
    int64_t reach;
    if (size[i] == 1) {
      // the only index of its axis: the stride is never used, and taken as the contiguous one
      st[i] = i == 2 ? 1 : i == 1 ? seqlen : dim * seqlen;
      continue;
    }
    if (st[i] < 0) return SSM_ERR_INVALID_ARG;
    if (!mul_ok(size[i] - 1, st[i], &reach) || reach > INT64_MAX - last) return SSM_ERR_UNSUPPORTED;
    last += reach;
  }
  if (last == INT64_MAX || !mul_ok(last + 1, esz, &a->bytes)) return SSM_ERR_UNSUPPORTED;
  if (output) {
    // Axes by stride: each must step past everything the smaller ones reach.
    int64_t reach = 0, floor = 0;
    bool used[3] = {false, false, false};
    for (int k = 0; k < 3; ++k) {
      int best = -1;
      for (int i = 0; i < 3; ++i)
        if (!used[i] && size[i] > 1 && (best < 0 || st[i] < st[best])) best = i;
      if (best < 0) break;
      used[best] = true;
      if (st[best] <= floor) return SSM_ERR_INVALID_ARG;
      reach += (size[best] - 1) * st[best];
      floor = reach;
    }
  }
  a->s = ssm::Strides{st[0], st[1], st[2]};
  const bool time = seqlen == 1 || st[2] == 1, chan = dim == 1 || st[1] == 1;
  if (!time && !chan) return SSM_ERR_UNSUPPORTED;
  // One step: channels contiguous is the order to use where it holds.
  a->order = chan && (!time || seqlen == 1) ? ssm::Order::Channel : ssm::Order::Time;
  return SSM_OK;
}

}  // namespace ssm_api
