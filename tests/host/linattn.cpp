// The linear-attention kernels (csrc/linattn_*.hip) and those of the queries' and keys' norm
// (csrc/qk_kernels.hip) in a CPU build, over the C ABI: values against plain loops in 64 bits, every
// array in pages of its own with no access allowed behind its end (or before its start), and the steps
// behind each row's length NaN. Built and run by tests/test_linattn_cpu.py. Exit status 0 and "linattn
// ok" on success.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>
#include <sys/mman.h>
#include <unistd.h>

#include <vector>

#include "device_math.h"
#include "ssm_linattn.h"
#include "ssm_qk.h"

namespace {

int g_fail = 0;
uint32_t g_seed = 1;
double draw() {
  g_seed = g_seed * 1664525u + 1013904223u;
  return double(int32_t(g_seed)) / 2147483648.0;
}

bool g_front = false;

// n bytes that end where a closed page begins, or (g_front) start behind one.
struct Mem {
  char *base = nullptr, *p = nullptr;
  size_t whole = 0, bytes = 0;
  explicit Mem(size_t n) : bytes(n) {
    const bool front = g_front;
    const size_t page = 4096, pages = (n + page - 1) / page + 2;
    whole = pages * page;
    base = static_cast<char*>(mmap(nullptr, whole, PROT_READ | PROT_WRITE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0));
    if (base == MAP_FAILED) _exit(3);
    mprotect(base, page, PROT_NONE);
    mprotect(base + whole - page, page, PROT_NONE);
    p = front ? base + page : base + whole - page - n;
  }
  Mem(const Mem&) = delete;
  ~Mem() { munmap(base, whole); }
};

// Values of a storage type.
struct Array {
  bool bf;
  size_t n;
  Mem m;
  Array(size_t count, bool bf16) : bf(bf16), n(count), m(count * (bf16 ? 2 : 4)) {}
  double get(size_t i) const {
    return bf ? ssm::bf16_lo(reinterpret_cast<const uint16_t*>(m.p)[i]) : reinterpret_cast<const float*>(m.p)[i];
  }
  void set(size_t i, double v) {
    if (bf)
      reinterpret_cast<uint16_t*>(m.p)[i] = uint16_t(ssm::bf16_bits(float(v)));
    else
      reinterpret_cast<float*>(m.p)[i] = float(v);
  }
  Array& random(double scale = 1.0) {
    for (size_t i = 0; i < n; ++i) set(i, scale * draw());
    return *this;
  }
  Array& fill(double v) {
    for (size_t i = 0; i < n; ++i) set(i, v);
    return *this;
  }
  float* f() { return reinterpret_cast<float*>(m.p); }
  void* p() { return m.p; }
};

// The 2-norm of the difference over that of the result.
void near(const Array& got, const std::vector<double>& want, double tol, const char* what) {
  double d = 0, n = 0;
  bool finite = true;
  for (size_t i = 0; i < want.size(); ++i) {
    const double g = got.get(i);
    finite &= bool(isfinite(g));
    d += (g - want[i]) * (g - want[i]);
    n += want[i] * want[i];
  }
  const double rel = n > 0 ? sqrt(d / n) : sqrt(d);
  const bool ok = finite && rel <= tol;
  printf("  %s %.3g%s\n", what, rel, ok ? "" : finite ? " TOO FAR" : " NOT FINITE");
  if (!ok) ++g_fail;
}

struct Case {
  int64_t b, L, hk, h, dk, dv;
  bool bf, state;
  int decay;  // 0 none, 1 a head, 2 a step
  std::vector<int32_t> n;
};

double scale_of(const Case& c) { return 1 / sqrt(double(c.dk)); }

void attention(const Case& c) {
  printf("b%ld L%ld hk%ld h%ld dk%ld dv%ld %s decay%d%s\n", long(c.b), long(c.L), long(c.hk), long(c.h), long(c.dk),
         long(c.dv), c.bf ? "bf16" : "f32", c.decay, c.state ? " state" : "");
  fflush(stdout);
  g_seed = uint32_t(c.L * 7 + c.dk * 3 + c.dv);
  const int64_t b = c.b, L = c.L, hk = c.hk, h = c.h, dk = c.dk, dv = c.dv, group = h / hk;
  Array q(b * L * hk * dk, c.bf), k(b * L * hk * dk, c.bf), v(b * L * h * dv, c.bf), dout(b * L * h * dv, c.bf);
  Array g(c.decay == 1 ? h : b * L * h, false), s0(b * h * dv * dk, false), ds(b * h * dv * dk, false);
  q.random(), k.random(), v.random(), dout.random(), s0.random(), ds.random();
  for (size_t i = 0; i < g.n; ++i) g.set(i, -0.2 * (1 + draw()));
  if (c.decay == 2 && g.n > 5) g.set(g.n / 2, -INFINITY);  // a reset
  auto end = [&](int64_t i) { return c.n.empty() ? L : int64_t(c.n[i] < 0 ? 0 : c.n[i] > L ? L : c.n[i]); };
  for (int64_t i = 0; i < b; ++i)
    for (int64_t t = end(i); t < L; ++t) {
      for (int64_t x = 0; x < hk * dk; ++x) q.set((i * L + t) * hk * dk + x, NAN), k.set((i * L + t) * hk * dk + x, NAN);
      for (int64_t x = 0; x < h * dv; ++x) v.set((i * L + t) * h * dv + x, NAN), dout.set((i * L + t) * h * dv + x, NAN);
      if (c.decay == 2)
        for (int64_t x = 0; x < h; ++x) g.set((i * L + t) * h + x, NAN);
    }
  const uint32_t flags = c.bf ? SSM_IO_BF16 : SSM_IO_F32;
  const int64_t per_head[3] = {0, 0, 1};
  const float scale = float(scale_of(c));
  auto fine = [&](int st) {
    if (st != SSM_OK) printf("  status %d\n", st), ++g_fail;
  };
  // plain loops
  std::vector<double> o(b * L * h * dv, 0.0), fin(b * h * dv * dk), dq(b * L * hk * dk, 0.0), dkk(dq), dvv(o),
      dg(c.decay == 1 ? h : b * L * h, 0.0), di(fin);
  for (int64_t i = 0; i < b; ++i)
    for (int64_t x = 0; x < h; ++x) {
      const int64_t n = end(i), y = x / group;
      auto K = [&](const Array& a, int64_t t, int64_t e) { return a.get(((i * L + t) * hk + y) * dk + e); };
      auto V = [&](const Array& a, int64_t t, int64_t e) { return a.get(((i * L + t) * h + x) * dv + e); };
      auto keep = [&](int64_t t) {
        return c.decay == 0 ? 1.0 : exp(c.decay == 1 ? g.get(x) : g.get((i * L + t) * h + x));
      };
      std::vector<std::vector<double>> S(n + 1, std::vector<double>(dv * dk));
      for (int64_t e = 0; e < dv * dk; ++e) S[0][e] = c.state ? s0.get((i * h + x) * dv * dk + e) : 0.0;
      for (int64_t t = 0; t < n; ++t)
        for (int64_t e = 0; e < dv; ++e) {
          double sum = 0;
          for (int64_t f = 0; f < dk; ++f) {
            S[t + 1][e * dk + f] = keep(t) * S[t][e * dk + f] + V(v, t, e) * K(k, t, f);
            sum += S[t + 1][e * dk + f] * K(q, t, f);
          }
          o[((i * L + t) * h + x) * dv + e] = scale * sum;
        }
      for (int64_t e = 0; e < dv * dk; ++e) fin[(i * h + x) * dv * dk + e] = S[n][e];
      std::vector<double> R(dv * dk);
      for (int64_t e = 0; e < dv * dk; ++e) R[e] = c.state ? ds.get((i * h + x) * dv * dk + e) : 0.0;
      for (int64_t t = n - 1; t >= 0; --t) {
        double dot = 0;
        for (int64_t e = 0; e < dv; ++e)
          for (int64_t f = 0; f < dk; ++f) {
            double& r = R[e * dk + f];
            r += scale * V(dout, t, e) * K(q, t, f);
            dq[((i * L + t) * hk + y) * dk + f] += scale * V(dout, t, e) * S[t + 1][e * dk + f];
            dkk[((i * L + t) * hk + y) * dk + f] += r * V(v, t, e);
            dvv[((i * L + t) * h + x) * dv + e] += r * K(k, t, f);
            dot += r * S[t][e * dk + f] * keep(t);
            r *= keep(t);
          }
        if (c.decay) dg[c.decay == 1 ? x : (i * L + t) * h + x] += dot;
      }
      for (int64_t e = 0; e < dv * dk; ++e) di[(i * h + x) * dv * dk + e] = R[e];
    }
  // One more rounding of the pairs' weights next to that of the result in bf16; fp32 sums else.
  const double tol = c.bf ? 4e-3 : 2e-6, tol32 = 2e-6;
  {
    const int64_t need = ssm_linattn_fwd_workspace_bytes(b, L, h, dk, dv, flags);
    Mem ws(size_t((need + 255) / 256 * 256));
    Array out(b * L * h * dv, c.bf), final_state(b * h * dv * dk, false);
    out.fill(7), final_state.fill(7);
    fine(ssm_linattn_fwd(q.p(), nullptr, k.p(), nullptr, v.p(), nullptr, c.decay ? g.f() : nullptr,
                         c.decay == 1 ? per_head : nullptr, c.state ? s0.f() : nullptr,
                         c.n.empty() ? nullptr : c.n.data(), scale, flags, out.p(), final_state.f(), ws.p, need, b, L,
                         hk, h, dk, dv, nullptr));
    printf(" workspace %ld\n", long(need));
    near(out, o, tol, "out");
    near(final_state, fin, tol32, "final_state");
  }
  {
    const uint32_t f = flags | (c.decay == 1 ? SSM_LINATTN_HEAD_DG : 0);
    const int64_t need = ssm_linattn_bwd_workspace_bytes(b, L, h, dk, dv, f);
    Mem ws(size_t((need + 255) / 256 * 256));
    Array aq(dq.size(), c.bf), ak(dq.size(), c.bf), av(o.size(), c.bf), ag(dg.size(), false), ai(di.size(), false);
    aq.fill(7), ak.fill(7), av.fill(7), ag.fill(7), ai.fill(7);
    fine(ssm_linattn_bwd(q.p(), nullptr, k.p(), nullptr, v.p(), nullptr, dout.p(), nullptr,
                         c.decay ? g.f() : nullptr, c.decay == 1 ? per_head : nullptr, c.state ? s0.f() : nullptr,
                         c.n.empty() ? nullptr : c.n.data(), c.state ? ds.f() : nullptr, scale, f, aq.p(), ak.p(),
                         av.p(), c.decay ? ag.f() : nullptr, ai.f(), ws.p, need, b, L, hk, h, dk, dv, nullptr));
    near(aq, dq, tol, "dq");
    near(ak, dkk, tol, "dk");
    near(av, dvv, tol, "dv");
    near(ai, di, tol32, "dinitial");
    if (c.decay) near(ag, dg, 5e-6, "dg");
  }
  fflush(stdout);
}

void token(int64_t b, int64_t ns, int64_t hk, int64_t h, int64_t dk, int64_t dv, bool bf,
           const std::vector<int32_t>& slots) {
  printf("step b%ld of %ld hk%ld h%ld dk%ld dv%ld %s\n", long(b), long(ns), long(hk), long(h), long(dk), long(dv),
         bf ? "bf16" : "f32");
  Array q(b * hk * dk, bf), k(b * hk * dk, bf), v(b * h * dv, bf), g(b * h, false), s(ns * h * dv * dk, false),
      out(b * h * dv, bf);
  q.random(), k.random(), v.random(), s.random(), out.fill(7);
  for (size_t i = 0; i < g.n; ++i) g.set(i, -0.3 * (1 + draw()));
  std::vector<double> S(s.n), o(out.n, 0.0);
  for (size_t i = 0; i < s.n; ++i) S[i] = s.get(i);
  for (int64_t i = 0; i < b; ++i) {
    const int64_t at = slots.empty() ? i : slots[i];
    if (at < 0 || at >= ns) continue;
    for (int64_t x = 0; x < h; ++x)
      for (int64_t e = 0; e < dv; ++e)
        for (int64_t f = 0; f < dk; ++f) {
          const int64_t y = x / (h / hk);
          double& r = S[((at * h + x) * dv + e) * dk + f];
          r = exp(g.get(i * h + x)) * r + v.get((i * h + x) * dv + e) * k.get((i * hk + y) * dk + f);
          o[(i * h + x) * dv + e] += r * q.get((i * hk + y) * dk + f) / sqrt(double(dk));
        }
  }
  const int st = ssm_linattn_step(q.p(), nullptr, k.p(), nullptr, v.p(), nullptr, g.f(), nullptr,
                                  slots.empty() ? nullptr : slots.data(), float(1 / sqrt(double(dk))),
                                  bf ? SSM_IO_BF16 : SSM_IO_F32, s.f(), out.p(), b, ns, hk, h, dk, dv, nullptr);
  if (st != SSM_OK) printf("  status %d\n", st), ++g_fail;
  near(out, o, bf ? 3e-3 : 2e-6, "out");
  near(s, S, 2e-6, "state");
  fflush(stdout);
}

void norms(int64_t b, int64_t L, int64_t hq, int64_t hk, int64_t d, int64_t rot, bool bf, bool inter, bool places) {
  printf("qk b%ld L%ld %ld+%ld heads of %ld rot %ld %s%s\n", long(b), long(L), long(hq), long(hk), long(d), long(rot),
         bf ? "bf16" : "f32", inter ? " interleaved" : "");
  const int64_t rows = places ? 3 * L : L, half = rot / 2;
  Array q(b * L * hq * d, bf), k(b * L * hk * d, bf), qw(d, false), kw(d, false), cs(rows * half, false),
      sn(rows * half, false), gq(q.n, bf), gk(k.n, bf);
  q.random(), k.random(), gq.random(), gk.random();
  for (int64_t i = 0; i < d; ++i) qw.set(i, 1 + 0.2 * draw()), kw.set(i, 1 + 0.2 * draw());
  for (int64_t i = 0; i < rows * half; ++i) {
    const double a = 3 * draw();
    cs.set(i, cos(a)), sn.set(i, sin(a));
  }
  std::vector<int32_t> pos;
  if (places)
    for (int64_t i = 0; i < b * L; ++i) pos.push_back(i % 5 == 3 ? -1 : int32_t((i * 7) % (rows + 2)));
  const double eps = 1e-6;
  std::vector<double> yq(q.n, 0.0), yk(k.n, 0.0), dq(q.n, 0.0), dk(k.n, 0.0), dqw(d, 0.0), dkw(d, 0.0);
  for (int side = 0; side < 2; ++side) {
    const int64_t H = side ? hk : hq;
    const Array &x = side ? k : q, &w = side ? kw : qw, &g = side ? gk : gq;
    std::vector<double>&y = side ? yk : yq, &dx = side ? dk : dq, &dw = side ? dkw : dqw;
    for (int64_t row = 0; row < b * L * H; ++row) {
      const int64_t step = row / H, at = places ? pos[step] : step % L;
      if (rot && (at < 0 || at >= rows)) continue;
      double sum = 0;
      for (int64_t e = 0; e < d; ++e) sum += x.get(row * d + e) * x.get(row * d + e);
      const double r = 1 / sqrt(sum / d + eps);
      std::vector<double> u(d), back(d);
      for (int64_t e = 0; e < d; ++e) u[e] = w.get(e) * r * x.get(row * d + e), back[e] = g.get(row * d + e);
      std::vector<double> o = u;
      for (int64_t e = 0; e < half; ++e) {
        const int64_t i = inter ? 2 * e : e, j = inter ? 2 * e + 1 : e + half;
        const double c = cs.get(at * half + e), s = sn.get(at * half + e);
        o[i] = u[i] * c - u[j] * s, o[j] = u[j] * c + u[i] * s;
        const double gi = back[i], gj = back[j];
        back[i] = gi * c + gj * s, back[j] = gj * c - gi * s;
      }
      double mean = 0;
      for (int64_t e = 0; e < d; ++e) {
        y[row * d + e] = o[e];
        const double n = r * x.get(row * d + e);
        dw[e] += back[e] * n;
        mean += back[e] * w.get(e) * n / d;
      }
      for (int64_t e = 0; e < d; ++e) dx[row * d + e] = r * (back[e] * w.get(e) - r * x.get(row * d + e) * mean);
    }
  }
  const uint32_t flags = (bf ? SSM_IO_BF16 : SSM_IO_F32) | (inter ? SSM_QK_INTERLEAVED : 0);
  const int32_t* at = places ? pos.data() : nullptr;
  Array oq(q.n, bf), ok(k.n, bf), aq(q.n, bf), ak(k.n, bf), aqw(d, false), akw(d, false);
  oq.fill(7), ok.fill(7), aq.fill(7), ak.fill(7), aqw.fill(7), akw.fill(7);
  const float* c = rot ? cs.f() : nullptr;
  const float* s = rot ? sn.f() : nullptr;
  int st = ssm_qk_norm_fwd(q.p(), nullptr, k.p(), nullptr, qw.f(), kw.f(), c, s, at, 1e-6f, flags, oq.p(), ok.p(), b, L,
                           hq, hk, d, rot, rot ? rows : 0, nullptr);
  const int64_t need = ssm_qk_norm_bwd_workspace_bytes(b, L, hq, hk, d, rot, flags);
  Mem ws(size_t((need + 255) / 256 * 256));
  if (st == SSM_OK)
    st = ssm_qk_norm_bwd(q.p(), nullptr, k.p(), nullptr, gq.p(), nullptr, gk.p(), nullptr, qw.f(), kw.f(), c, s, at,
                         1e-6f, flags, aq.p(), ak.p(), aqw.f(), akw.f(), ws.p, need, b, L, hq, hk, d, rot,
                         rot ? rows : 0, nullptr);
  if (st != SSM_OK) printf("  status %d\n", st), ++g_fail;
  const double tol = bf ? 3e-3 : 2e-6;
  near(oq, yq, tol, "q"), near(ok, yk, tol, "k"), near(aq, dq, tol, "dq"), near(ak, dk, tol, "dk");
  near(aqw, dqw, 5e-6, "dq_weight"), near(akw, dkw, 5e-6, "dk_weight");
  fflush(stdout);
}

}  // namespace

// Argument: the side of every array that a closed page follows (back) or comes before (front).
int main(int argc, char** argv) {
  const std::vector<Case> cases = {
      {1, 1, 1, 1, 16, 16, true, true, 2, {}},       {2, 70, 1, 2, 32, 40, true, true, 2, {70, 3}},
      {1, 130, 1, 2, 128, 64, true, false, 2, {}},   {1, 65, 2, 2, 64, 100, true, true, 1, {}},
      {1, 600, 1, 1, 20, 72, true, true, 1, {}},     {1, 67, 1, 1, 192, 256, true, true, 0, {}},
      {3, 70, 1, 3, 33, 17, false, true, 2, {0, 70, 33}}, {1, 300, 1, 1, 100, 80, false, false, 1, {}},
      {1, 40, 1, 1, 256, 130, false, true, 2, {}},   {2, 129, 1, 1, 96, 128, true, true, 2, {129, 64}},
      {1, 0, 1, 1, 16, 16, true, true, 2, {}},
  };
  g_front = argc > 1 && argv[1][0] == 'f';
  for (const Case& c : cases) attention(c);
  token(3, 5, 2, 4, 128, 64, true, {4, 0, 2});
  token(4, 4, 1, 2, 100, 50, false, {1, 1, -1, 1});
  token(2, 2, 1, 1, 256, 256, true, {});
  token(2, 3, 1, 1, 3, 5, false, {2, 7});
  norms(2, 3, 4, 2, 128, 128, true, false, true);
  norms(1, 5, 3, 3, 96, 48, false, true, false);
  norms(1, 4, 1, 1, 33, 10, true, false, true);
  norms(1, 4, 2, 1, 256, 2, false, true, false);
  norms(2, 2, 5, 1, 64, 0, true, false, false);
  if (g_fail) return 1;
  printf("linattn ok\n");
  return 0;
}
