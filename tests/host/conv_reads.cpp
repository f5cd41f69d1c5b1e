// The convolution's kernels (csrc/conv_kernels.hip) in a CPU build, over the C ABI: values against a
// plain loop, and x behind each row's length in pages that no access may touch, so that a read
// there ends the process. Built and run by tests/test_block_conv_reads.py. Exit status 0 and
// "conv reads ok" on success.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>
#include <sys/mman.h>

#include <vector>

#include "device_math.h"
#include "ssm_conv.h"

namespace {

int g_fail = 0;
constexpr int64_t kPage = 4096;

struct Shape {
  int64_t b, d, L, W;
  std::vector<int32_t> n;  // the rows' lengths
  bool channel;            // channels contiguous: a step a page; else a channel's rows 2048 steps a page
};

float draw(uint32_t& s) { return float(int32_t(s = s * 1664525u + 1013904223u)) / 2147483648.0f; }
uint16_t bf(float v) { return uint16_t(ssm::bf16_bits(v)); }
float fl(uint16_t v) { return ssm::bf16_lo(v); }
double silu(double p) { return p / (1 + exp(-p)); }
double silu_grad(double p) {
  const double s = 1 / (1 + exp(-p));
  return s * (1 + p * (1 - s));
}

// One rounding to bf16 and the float32 arithmetic before it.
void near(double got, double want, double scale, const char* what) {
  if (!(fabs(got - want) <= fabs(want) / 256 + scale * 1e-4)) {
    if (++g_fail < 10) printf("%s: %g, expected %g\n", what, got, want);
  }
}

void run(const Shape& s, bool protect) {
  const int64_t b = s.b, d = s.d, L = s.L, W = s.W;
  uint32_t seed = uint32_t(b * 7 + d * 3 + L + W);
  // x: [b][L] pages of channels, or [b][d][L] with L a multiple of a page's 2048 steps
  const int64_t row_bytes = s.channel ? L * kPage : d * L * 2, bytes = b * row_bytes;
  auto* mem = static_cast<char*>(mmap(nullptr, size_t(bytes), PROT_READ | PROT_WRITE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0));
  if (mem == MAP_FAILED) {
    ++g_fail;
    return;
  }
  auto* x = reinterpret_cast<uint16_t*>(mem);
  const int64_t xs[3] = {row_bytes / 2, s.channel ? 1 : L, s.channel ? kPage / 2 : 1};
  auto end = [&](int64_t i) { return int64_t(s.n[i] < 0 ? 0 : s.n[i] > L ? L : s.n[i]); };
  auto X = [&](int64_t i, int64_t c, int64_t t) -> uint16_t& { return x[i * xs[0] + c * xs[1] + t * xs[2]]; };
  for (int64_t i = 0; i < b; ++i)
    for (int64_t c = 0; c < d; ++c)
      for (int64_t t = 0; t < L; ++t) X(i, c, t) = t < end(i) ? bf(draw(seed)) : 0x7fc0;
  std::vector<float> w(d * W), bias(d), dw(d * W), db(d);
  for (float& v : w) v = draw(seed);
  for (float& v : bias) v = draw(seed);
  std::vector<uint16_t> init(b * d * (W - 1)), fin(init.size()), dfin(init.size()), dinit(init.size());
  std::vector<uint16_t> out(b * d * L), dout(out.size()), dx(out.size());
  for (auto* v : {&init, &dfin, &dout})
    for (uint16_t& e : *v) e = bf(draw(seed));
  if (protect)  // whole pages at and behind each row's end
    for (int64_t i = 0; i < b; ++i)
      for (int64_t k = 0; k < (s.channel ? 1 : d); ++k) {
        char* row = mem + i * row_bytes + k * L * 2;
        const int64_t from = s.channel ? end(i) * kPage : (end(i) * 2 + kPage - 1) / kPage * kPage;
        const int64_t all = s.channel ? L * kPage : L * 2;
        if (from < all) mprotect(row + from, size_t(all - from), PROT_NONE);
      }
  const uint32_t flags = SSM_IO_BF16 | SSM_CONV_SILU;
  // dx in x's order, dense
  const int64_t ds[3] = {d * L, s.channel ? 1 : L, s.channel ? d : 1};
  std::vector<char> raw(size_t(ssm_conv_bwd_workspace_bytes(b, d, W, L, flags)) + 256);
  void* ws = raw.data() + (256 - reinterpret_cast<uintptr_t>(raw.data()) % 256) % 256;
  int st = ssm_conv_fwd(x, xs, w.data(), bias.data(), init.data(), s.n.data(), flags, out.data(), fin.data(), b, d, W,
                        L, nullptr);
  if (st == SSM_OK)
    st = ssm_conv_bwd(x, xs, w.data(), bias.data(), init.data(), s.n.data(), flags, dout.data(), dfin.data(),
                      dx.data(), ds, dw.data(), db.data(), dinit.data(), ws, int64_t(raw.size()) - 256, b, d, W, L,
                      nullptr);
  if (st != SSM_OK) {
    printf("status %d\n", st);
    ++g_fail;
  }
  for (int64_t c = 0; c < d; ++c) {
    std::vector<double> sw(W, 0.0);
    double sb = 0;
    for (int64_t i = 0; i < b; ++i) {
      const int64_t n = end(i), row = i * d + c;
      std::vector<double> e(n + W - 1), de(n + W - 1, 0.0);
      for (int64_t k = 0; k < W - 1; ++k) e[k] = fl(init[row * (W - 1) + k]);
      for (int64_t t = 0; t < n; ++t) e[W - 1 + t] = fl(X(i, c, t));
      for (int64_t k = 0; k < W - 1; ++k) {
        near(fl(fin[row * (W - 1) + k]), e[n + k], 0, "final state");
        de[n + k] += fl(dfin[row * (W - 1) + k]);
      }
      for (int64_t t = 0; t < L; ++t) {
        double p = bias[c];
        if (t < n)
          for (int64_t k = 0; k < W; ++k) p += double(w[c * W + k]) * e[t + k];
        near(fl(out[row * L + t]), t < n ? silu(p) : 0.0, 1, "out");
        if (t >= n) continue;
        const double dp = fl(dout[row * L + t]) * silu_grad(p);
        for (int64_t k = 0; k < W; ++k) {
          de[t + k] += dp * double(w[c * W + k]);
          sw[k] += dp * e[t + k];
        }
        sb += dp;
      }
      for (int64_t t = 0; t < L; ++t)
        near(fl(dx[i * ds[0] + c * ds[1] + t * ds[2]]), t < n ? de[W - 1 + t] : 0.0, 1, "dx");
      for (int64_t k = 0; k < W - 1; ++k) near(fl(dinit[row * (W - 1) + k]), de[k], 1, "dinitial");
    }
    for (int64_t k = 0; k < W; ++k) near(dw[c * W + k], sw[k], double(b * L), "dweight");
    near(db[c], sb, double(b * L), "dbias");
  }
  munmap(mem, size_t(bytes));
  printf("b%ld d%ld L%ld W%ld %s %s: %d\n", long(b), long(d), long(L), long(W), s.channel ? "channel" : "time",
         protect ? "protected" : "open", g_fail);
  fflush(stdout);
}

}  // namespace

int main() {
  const Shape shapes[] = {
      {5, 70, 150, 4, {150, 37, 2, 0, 129}, true}, {3, 64, 40, 3, {33, 32, 31}, true},
      {2, 3, 9, 2, {1, 8}, true},                  {3, 65, 1, 4, {1, 0, -2}, true},
      {2, 2, 4096, 4, {2048, 0}, false},           {3, 3, 2048, 2, {0, 2048, 3000}, false}};
  for (bool protect : {false, true})
    for (const Shape& s : shapes) run(s, protect);
  if (g_fail) return 1;
  printf("conv reads ok\n");
  return 0;
}
