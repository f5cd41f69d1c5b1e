// The grids that the C-ABI layer of the operators around the scan lets through (conv_api.cpp,
// step_api.cpp, norm_api.cpp), with the launches stubbed: every one has fewer than 2^32 work-items
// along each axis, counted here on its own from the sizes, and the calls just inside that are not
// refused. Host only; built and run by tests/test_block_launch_limits.py. Exit status 0 and
// "launch limits ok" on success.
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "block_launch.h"
#include "ssm_conv.h"
#include "ssm_norm.h"
#include "ssm_step.h"

namespace {

int g_launches = 0, g_fail = 0;
#define EXPECT(c)                                   \
  if (!(c)) {                                       \
    printf("FAILED line %d: %s\n", __LINE__, #c);   \
    ++g_fail;                                       \
  }

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
void items(int64_t workgroups, int64_t threads) {
  EXPECT(workgroups > 0 && __int128(workgroups) * threads < (__int128(1) << 32));
}

// Lanes of 8 steps along a row: a power of two, at most 64.
int64_t row_lanes(int64_t seqlen) {
  int64_t n = 1;
  while (n < 64 && n * 8 < seqlen) n *= 2;
  return n;
}

void conv(const ssm::ConvArgs& a, bool backward) {
  ++g_launches;
  if (a.order == ssm::Order::Channel && a.seqlen > 0) {
    items(up(a.seqlen, 128) * up(a.dim, 64), 256);
  } else {
    const int64_t lanes = row_lanes(a.seqlen);
    const int64_t tiles = backward ? 4 : ssm::conv_fwd_wave_tiles(a.batch, a.dim, a.seqlen, a.io);
    const int64_t runs = a.seqlen ? up(a.seqlen, 8 * lanes * tiles) : 1;
    items(up(up(a.dim, 64 / lanes) * runs, 4), 256);
  }
  if (backward) items(up(a.dim * (a.width + 1), 32), 512);
}

void norm(const ssm::NormArgs& a, const ssm::NormShape& s) {
  const int64_t cv = a.io == ssm::Io::BF16 ? 8 : 4, g = a.dim / a.groups;
  const int64_t blocks = up(up(g, cv << s.lanes_log2), s.waves);
  items(up(a.seqlen, int64_t(s.steps) * (64 >> s.lanes_log2)) * blocks * a.groups * a.batch, 64 * s.waves);
}

}  // namespace

namespace ssm {
int launch_conv_fwd(const ConvArgs& a, void*) { return conv(a, false), 0; }
int launch_conv_bwd(const ConvArgs& a, void*) { return conv(a, true), 0; }
int launch_conv_step(const ConvStepArgs& a, void*) {
  ++g_launches;
  items(up(a.dim, a.io == Io::BF16 ? 512 : 256), 256);
  return 0;
}
int launch_state_step(const StepArgs& a, void*) {
  ++g_launches;
  int64_t lanes = 1;
  while (lanes * 4 < a.dstate) lanes *= 2;
  items(up(a.dim, 4 * step_form(a.batch, a.dim, a.dstate).channels * (64 / lanes)), 256);
  return 0;
}
int launch_norm_fwd(const NormArgs& a, void*) {
  ++g_launches;
  norm(a, norm_fwd_shape(a));
  return 0;
}
int launch_norm_bwd(const NormArgs& a, void*) {
  ++g_launches;
  if (a.batch > 0 && a.seqlen > 0) norm(a, norm_bwd_shape(a));
  items(up(a.dim, 32), 1024);
  return 0;
}
}  // namespace ssm

namespace {

// Addresses 2^43 bytes apart: no tensor here is as large.
template <typename T = void>
T* at(int i) {
  return reinterpret_cast<T*>(uintptr_t(0x80000000000) * uintptr_t(i + 1));
}
using F = const float;

int conv_fwd(uint32_t io, const int64_t* st, int64_t b, int64_t d, int64_t L) {
  return ssm_conv_fwd(at(0), st, at<F>(1), nullptr, nullptr, nullptr, io, at(2), nullptr, b, d, 4, L, nullptr);
}
int conv_bwd(uint32_t io, const int64_t* st, int64_t b, int64_t d, int64_t L) {
  return ssm_conv_bwd(at(0), st, at<F>(1), nullptr, nullptr, nullptr, io, at(2), nullptr, at(3), st, at<float>(4),
                      nullptr, nullptr, at(5), INT64_MAX, b, d, 4, L, nullptr);
}
int scan_step(int64_t b, int64_t d, int64_t n) {
  return ssm_scan_step(at(0), d, at(1), d, at<F>(2), at(3), n, at(4), n, nullptr, nullptr, 0, nullptr, nullptr,
                       SSM_IO_F32, at<float>(5), at(6), b, b, d, n, nullptr);
}
int norm_fwd(uint32_t io, const int64_t* st, int64_t b, int64_t d, int64_t g, int64_t L) {
  return ssm_norm_fwd(at(0), st, nullptr, nullptr, at<F>(1), 1e-5f, io, at(2), st, nullptr, at(3), INT64_MAX, b, d, g,
                      L, nullptr);
}
int norm_bwd(uint32_t io, const int64_t* st, int64_t b, int64_t d, int64_t g, int64_t L) {
  return ssm_norm_bwd(at(0), st, nullptr, nullptr, at<F>(1), at<F>(2), at(3), st, io, at(4), st, nullptr, nullptr,
                      at<float>(5), at(6), INT64_MAX, b, d, g, L, nullptr);
}

// `st` is SSM_OK and launches, or SSM_ERR_UNSUPPORTED and does not.
void either(int st, int before) {
  EXPECT(st == SSM_OK || st == SSM_ERR_UNSUPPORTED);
  EXPECT((st == SSM_OK) == (g_launches > before));
}

}  // namespace

int main() {
  const int64_t one = 1;
  const uint32_t types[2] = {SSM_IO_F32, SSM_IO_BF16};
  // Every combination of sizes up to the ABI's, in both orders.
  int64_t sizes[80], n = 0;
  for (int k = 0; k < 31; k += 2) {
    sizes[n++] = one << k;
    sizes[n++] = (one << (k + 1)) - 1;
  }
  for (uint32_t io : types)
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < n; ++j)
        for (int64_t b : {one, int64_t(7), int64_t(65535), one << 20, one << 26}) {
          const int64_t d = sizes[i], L = sizes[j], token[3] = {d * L, 1, d};
          if (__int128(b) * d * L > (__int128(1) << 40)) continue;  // (of 2^43 bytes between tensors)
          for (const int64_t* st : {static_cast<const int64_t*>(nullptr), &token[0]}) {
            either(conv_fwd(io, st, b, d, L), g_launches);
            either(conv_bwd(io, st, b, d, L), g_launches);
            for (int64_t g : {one, d, d % 8 ? one : d / 8}) {
              either(norm_fwd(io, st, b, d, g, L), g_launches);
              either(norm_bwd(io, st, b, d, g, L), g_launches);
            }
          }
          if (L <= 256 && b <= 65535) either(scan_step(b, d, L), g_launches);
        }
  // Either side of the edges.
  EXPECT(conv_fwd(SSM_IO_F32, nullptr, 1, (one << 26) - 4, 512) == SSM_OK);
  EXPECT(conv_fwd(SSM_IO_F32, nullptr, 1, one << 26, 512) == SSM_ERR_UNSUPPORTED);
  EXPECT(conv_bwd(SSM_IO_F32, nullptr, 1, ((one << 28) - 32) / 5, 8) == SSM_OK);
  EXPECT(conv_bwd(SSM_IO_F32, nullptr, 1, (one << 28) / 5 + 1, 8) == SSM_ERR_UNSUPPORTED);
  EXPECT(scan_step(1, (one << 29) - 32, 256) == SSM_OK);
  EXPECT(scan_step(1, one << 29, 256) == SSM_ERR_UNSUPPORTED);
  EXPECT(norm_fwd(SSM_IO_BF16, nullptr, 130000, 4096, 512, 2) == SSM_OK);
  EXPECT(norm_fwd(SSM_IO_BF16, nullptr, 131072, 4096, 512, 2) == SSM_ERR_UNSUPPORTED);
  EXPECT(norm_bwd(SSM_IO_BF16, nullptr, 131072, 4096, 512, 2) == SSM_ERR_UNSUPPORTED);
  EXPECT(norm_bwd(SSM_IO_F32, nullptr, 1, one << 27, 1 << 20, 1) == SSM_ERR_UNSUPPORTED);
  if (g_fail) return 1;
  printf("launch limits ok (%d launches)\n", g_launches);
  return 0;
}
