// Host-only harness for the argument checks of the operators around the scan (conv_api.cpp,
// step_api.cpp, norm_api.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer, built with
// g++ and run by tests/test_block_sanitizers.py. The launches are stubbed: they check that what
// they are given fits what the kernels assume and touch no device. Every entry point is called
// with valid problems and with every combination of sizes and strides at the edges of int64.
// Exit status 0 and "block harness ok" on success.
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "block_launch.h"
#include "ssm_conv.h"
#include "ssm_norm.h"
#include "ssm_step.h"

namespace {
int g_launches = 0, g_fail = 0;
void expect(bool ok, const char* what, int line) {
  if (!ok) {
    printf("FAILED line %d: %s\n", line, what);
    ++g_fail;
  }
}
#define EXPECT(c) expect((c), #c, __LINE__)

const int64_t kMax = 2147483647;

// Workgroups and waves of a shape, as the launches form them, within a grid's limits.
void fits_norm(const ssm::NormArgs& a, const ssm::NormShape& s) {
  EXPECT(s.waves >= 1 && s.waves <= 16 && s.cblocks >= 1 && s.tiles >= 1 && s.lanes_log2 >= 0 && s.lanes_log2 <= 6);
  EXPECT(s.tiles * s.cblocks <= kMax / a.groups / a.batch);
  const int64_t cv = a.io == ssm::Io::BF16 ? 8 : 4, g = a.dim / a.groups;
  EXPECT(s.cblocks * s.waves * (cv << s.lanes_log2) >= g);
  EXPECT(s.tiles * s.steps * (64 >> s.lanes_log2) >= a.seqlen);
  EXPECT(s.split || s.cblocks == 1);
  EXPECT(!s.split || a.workspace);
}

void fits_norm(const ssm::NormArgs& a, bool backward) {
  for (const ssm::NormOrders o : {ssm::NormOrders{true, true}, ssm::NormOrders{false, true},
                                  ssm::NormOrders{false, false}})
    fits_norm(a, backward ? ssm::norm_bwd_shape(a.batch, a.dim, a.groups, a.seqlen, a.io, o)
                          : ssm::norm_fwd_shape(a.batch, a.dim, a.groups, a.seqlen, a.io, o));
}
}  // namespace

namespace ssm {
int launch_conv_fwd(const ConvArgs& a, void*) {
  ++g_launches;
  EXPECT(a.batch > 0 && a.batch <= 65535 && a.dim > 0 && a.dim <= kMax && a.seqlen <= kMax);
  EXPECT(a.seqlen == 0 || (a.order == Order::Time ? (a.xs.step == 1 || a.seqlen == 1)
                                                   : (a.xs.channel == 1 || a.dim == 1)));
  return 0;
}
int launch_conv_bwd(const ConvArgs& a, void*) {
  ++g_launches;
  EXPECT(a.dim > 0 && a.workspace || a.batch == 0);
  return 0;
}
int launch_conv_step(const ConvStepArgs& a, void*) {
  ++g_launches;
  EXPECT(a.batch > 0 && a.batch <= 65535 && a.nslots <= kMax && (a.slots || a.nslots >= a.batch));
  return 0;
}
int launch_state_step(const StepArgs& a, void*) {
  ++g_launches;
  EXPECT(a.batch > 0 && a.batch <= 65535 && a.dstate >= 1 && a.dstate <= 256 && a.dim <= kMax);
  EXPECT(a.headdim == 0 || a.dim % a.headdim == 0);
  return 0;
}
int launch_norm_fwd(const NormArgs& a, void*) {
  ++g_launches;
  fits_norm(a, false);
  return 0;
}
int launch_norm_bwd(const NormArgs& a, void*) {
  ++g_launches;
  if (a.batch > 0 && a.seqlen > 0) fits_norm(a, true);
  return 0;
}
}  // namespace ssm

namespace {

// Fake addresses so far apart that only sizes of the whole address space overlap.
template <typename T = void>
T* at(int i) {
  return reinterpret_cast<T*>(uintptr_t(0x100000000000) * uintptr_t(i + 1));
}

const int64_t kBig[] = {0, 1, 2, 3, 63, 65, 1023, 65535, 65536, 1 << 20, int64_t(1) << 31, (int64_t(1) << 31) - 1,
                        int64_t(1) << 40, int64_t(1) << 62, INT64_MAX / 2, INT64_MAX, -1, INT64_MIN};
const int64_t kFew[] = {0, 1, 5, 65536, (int64_t(1) << 31) - 1, int64_t(1) << 62, INT64_MAX, -1};

bool status(int st) {
  return st == SSM_OK || st == SSM_ERR_INVALID_ARG || st == SSM_ERR_UNSUPPORTED || st == SSM_ERR_MISALIGNED;
}

void conv() {
  const uint32_t bf = SSM_IO_BF16 | SSM_CONV_SILU;
  int before = g_launches;
  EXPECT(ssm_conv_fwd(at(0), nullptr, at<const float>(1), nullptr, nullptr, nullptr, bf, at(2), at(3), 4, 2304, 4,
                      2048, nullptr) == SSM_OK);
  EXPECT(g_launches == ++before);
  const int64_t need = ssm_conv_bwd_workspace_bytes(4, 2304, 4, 2048, bf);
  const int64_t token[3] = {2432 * 2048, 1, 2432};
  EXPECT(ssm_conv_bwd(at(0), token, at<const float>(1), at<const float>(2), at(3), at<const int32_t>(4), bf, at(5),
                      at(6), at(7), token, at<float>(8), at<float>(9), at(10), at(11), need, 4, 2304, 4, 2048,
                      nullptr) == SSM_OK);
  EXPECT(g_launches == ++before);
  for (int64_t b : kBig)
    for (int64_t d : kBig)
      for (int64_t L : kBig) {
        EXPECT(status(ssm_conv_fwd(at(0), nullptr, at<const float>(1), nullptr, at(4), nullptr, bf, at(2), at(3), b, d,
                                   3, L, nullptr)));
        const int64_t ws = ssm_conv_bwd_workspace_bytes(b, d, 4, L, bf);
        EXPECT(ws >= -1);
        EXPECT(status(ssm_conv_bwd(at(0), nullptr, at<const float>(1), nullptr, nullptr, nullptr, bf, at(2), nullptr,
                                   at(3), nullptr, at<float>(4), nullptr, nullptr, at(5), ws, b, d, 4, L, nullptr)));
        EXPECT(status(ssm_conv_step(at(0), d, at(1), at<const float>(2), nullptr, at<const int32_t>(3), bf, at(4), b,
                                    L, d, 4, nullptr)));
      }
  for (int64_t sb : kFew)
    for (int64_t sc : kFew)
      for (int64_t stp : kFew)
        for (int64_t b : {int64_t(1), int64_t(7)}) {
          const int64_t s[3] = {sb, sc, stp};
          EXPECT(status(ssm_conv_fwd(at(0), s, at<const float>(1), nullptr, nullptr, nullptr, SSM_IO_F32, at(2),
                                     nullptr, b, 6, 2, 9, nullptr)));
          EXPECT(status(ssm_conv_bwd(at(0), s, at<const float>(1), nullptr, nullptr, nullptr, SSM_IO_F32, at(2),
                                     nullptr, at(3), s, at<float>(4), nullptr, nullptr, at(5), 1 << 20, b, 6, 2, 9,
                                     nullptr)));
        }
  for (int64_t x : kBig)
    EXPECT(status(ssm_conv_step(at(0), x, at(1), at<const float>(2), nullptr, nullptr, bf, at(4), 3, 5, 8, 4, nullptr)));
}

void steps() {
  const uint32_t bf = SSM_IO_BF16 | SSM_DELTA_SOFTPLUS;
  int before = g_launches;
  EXPECT(ssm_ssd_step(at(0), 8448, at(1), 64, at<const float>(2), at(3), 8448, at(4), 8448, at<const float>(5),
                      at(6), 4096, at<const float>(7), at<const int32_t>(8), bf, at<float>(9), at(10), 256, 320, 64,
                      64, 128, nullptr) == SSM_OK);
  EXPECT(g_launches == ++before);
  for (int64_t b : kBig)
    for (int64_t d : kBig)
      for (int64_t n : kBig)
        for (int64_t e : kFew) {
          EXPECT(status(ssm_scan_step(at(0), e, at(1), d, at<const float>(2), at(3), n, at(4), e, nullptr, at(5), b,
                                      nullptr, at<const int32_t>(6), bf, at<float>(7), at(8), b, e, d, n, nullptr)));
          EXPECT(status(ssm_ssd_step(at(0), d, at(1), n, at<const float>(2), at(3), n, at(4), e, nullptr, nullptr, b,
                                     nullptr, nullptr, bf, at<float>(7), at(8), b, e, d, e, n, nullptr)));
        }
}

void norms() {
  const int64_t token[3] = {2048 * 2048, 1, 2048};
  int before = g_launches;
  EXPECT(ssm_norm_fwd(at(0), nullptr, at(1), token, at<const float>(2), 1e-5f, SSM_IO_BF16, at(3), token,
                      at<float>(4), at(5), 1 << 20, 4, 2048, 1, 2048, nullptr) == SSM_OK);
  EXPECT(g_launches == ++before);
  for (int64_t b : kBig)
    for (int64_t d : kBig)
      for (int64_t L : kBig)
        for (int64_t g : {int64_t(1), int64_t(5), int64_t(65535), int64_t(0), INT64_MAX, int64_t(-1)})
          for (uint32_t io : {SSM_IO_F32, SSM_IO_BF16}) {
            EXPECT(status(ssm_norm_fwd(at(0), nullptr, at(1), nullptr, at<const float>(2), 0.0f, io, at(3), nullptr,
                                       at<float>(4), at(5), ssm_norm_fwd_workspace_bytes(b, d, g, L, io), b, d, g, L,
                                       nullptr)));
            const int64_t ws = ssm_norm_bwd_workspace_bytes(b, d, g, L, io);
            EXPECT(ws >= -1);
            EXPECT(status(ssm_norm_bwd(at(0), nullptr, nullptr, nullptr, at<const float>(2), at<const float>(3), at(4),
                                       nullptr, io, at(5), nullptr, nullptr, nullptr, at<float>(6), at(7), ws, b, d, g,
                                       L, nullptr)));
          }
  for (int64_t sb : kFew)
    for (int64_t sc : kFew)
      for (int64_t stp : kFew)
        for (int64_t L : {int64_t(1), int64_t(9)}) {
          const int64_t s[3] = {sb, sc, stp};
          EXPECT(status(ssm_norm_fwd(at(0), s, at(1), s, at<const float>(2), 1e-5f, SSM_IO_F32, at(3), s, nullptr, at(4),
                                     1 << 20, 4, 6, 2, L, nullptr)));
        }
}

}  // namespace

int main() {
  conv();
  steps();
  norms();
  if (g_fail) return 1;
  printf("block harness ok (%d launches)\n", g_launches);
  return 0;
}
