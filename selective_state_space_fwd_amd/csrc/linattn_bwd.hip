// Gradient of linear attention with a decay for each head (include/ssm_linattn.h) on the gfx950
// matrix cores.
//
// With S the state at a chunk's start, R the adjoint of the state at its end, D_ts = exp(cs_t -
// cs_s) for s <= t (0 else), e_t = exp(cs_t) and f_s = exp(cs_end - cs_s):
//
//   dq_t = scale (sum_s D_ts (do_t . v_s) k_s + e_t S^T do_t)
//   dk_s = scale sum_t D_ts (do_t . v_s) q_t + f_s R^T v_s
//   dv_s = scale sum_t D_ts (q_t . k_s) do_t + f_s R k_s
//   dg_t = sum_{i>=t>j} W_ij + sum_{i>=t} q_i . dq_i^S + sum_{j<t} k_j . dk_j^R + exp(cs_end) <R, S>
//
// where W_ij = scale D_ij (q_i . k_j)(do_i . v_j), and dq^S, dk^R are the parts through S and R:
// the pairs of steps, of the chunk and around it, between which the decay g_t lies. dg so needs
// no difference of sums over the sequence, whose rounding errors would stay where the decays
// have made dg small; W's rectangles are suffix sums of its row sums less its column sums, over
// one chunk, in 64 bits.
//
// linattn_state_kernel and linattn_join_kernel (linattn_kernels.hip) leave S and R of every chunk
// in the workspace, [dk][dv] in fp32; linattn_bwd_kernel then takes a (batch row, query head,
// chunk) per workgroup, the heads that share the query one after another (their dq and dk add
// up in its accumulators, in a fixed order). A wave owns a quarter of dk for dq and dk, a quarter
// of dv for dv, so that each value of S and R is split into operand pieces once.
//
// Roundings: the pairs' weights (scale D qk and scale D dov) are rounded to bf16 once, as operands,
// next to results in bf16. S and R enter in three bf16 pieces where dg, a result in fp32, comes
// of the product, and in two in dv.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_linattn.h"
#include "linattn_launch.h"

namespace ssm {
namespace {

struct BwdParams {
  HeadRows q, k, v, dout;
  const float* g;
  int64_t g_batch, g_step, g_head;
  const int32_t* lengths;
  const float* states;
  const float* adjoints;
  void *dq, *dk_out, *dv_out;
  float* dg;              // nullable: [batch, seqlen, heads]
  float* dg_sums;         // nullable: [batch, chunks, heads], of a chunk's steps each
  int64_t seqlen, chunks, state_floats;
  int qk_heads, heads, group, dk, dv, kpad, vpad;
  float scale;
};

template <typename Elem, int KP, int VP, bool kWhole>
__global__ __launch_bounds__(kLaThreads, KP <= 128 && VP <= 128 ? 2 : 1) void linattn_bwd_kernel(BwdParams p) {
  constexpr int C = chunk_of<Elem>(), T = C / 16, SB = C / 32;
  constexpr uint32_t E = sizeof(Elem);
  constexpr int NK = KP / 64, NV = VP / 64;  // 16-wide tiles of dk and dv a wave owns
  constexpr int QP = la_pitch<Elem>(KP), OP = la_pitch<Elem>(VP), PP = la_pitch<Elem>(C);
  __shared__ __attribute__((aligned(16))) Elem sQ[C * QP], sK[C * QP], sV[C * OP], sO[C * OP];
  __shared__ __attribute__((aligned(16))) Elem sP[C * PP], sD[C * PP];  // weights by rows s: scale D qk, scale D dov
  __shared__ Decays<C> dec;
  __shared__ float sRow[T][C], sCol[T][C], sQs[4][C], sKs[4][C], sX[4];

  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = threadIdx.x & 63, r = l & 15, g = l >> 4;
  uint32_t at = xcd_order(blockIdx.x, gridDim.x);
  const int hk = int(at % uint32_t(p.qk_heads));
  at /= uint32_t(p.qk_heads);
  const int64_t c = at % uint32_t(p.chunks), b = at / uint32_t(p.chunks), t0 = c * C;
  const int64_t end = row_end(p.lengths, b, p.seqlen);
  const int rows = p.seqlen - t0 < C ? int(p.seqlen - t0) : C;
  const int live = end <= t0 ? 0 : end - t0 < C ? int(end - t0) : C;
  const int64_t q_step = int64_t(p.qk_heads) * p.dk, v_step = int64_t(p.heads) * p.dv;
  Elem* dq = static_cast<Elem*>(p.dq) + (b * p.seqlen + t0) * q_step + hk * p.dk;
  Elem* dk = static_cast<Elem*>(p.dk_out) + (b * p.seqlen + t0) * q_step + hk * p.dk;

  la_f32x4 aq[NK][T], ak[NK][T];
#pragma unroll
  for (int n = 0; n < NK; ++n)
#pragma unroll
    for (int i = 0; i < T; ++i) aq[n][i] = ak[n][i] = la_f32x4{0, 0, 0, 0};

  // rows a..a+3 of dim columns, steps 16 i + r; zero behind the end.
  auto put = [&](Elem* base, int64_t step, int i, int col, int dim, la_f32x4 v) {
    const int t = 16 * i + r;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = t < live ? v[e] : 0.0f;
    store4_at<Elem, kWhole>(Buf(base, kLaBytes), uint32_t(t) * uint32_t(step) * E + uint32_t(col) * E, dim - col,
                            t < rows, v);
  };

  if (live > 0) {
    {
      TileLoad<Elem, C, KP, kWhole> lq, lk;
      lq.load(static_cast<const Elem*>(p.q.p) + b * p.q.batch + hk * p.q.head + t0 * p.q.step,
              uint32_t(p.q.step) * E, live, p.dk);
      lk.load(static_cast<const Elem*>(p.k.p) + b * p.k.batch + hk * p.k.head + t0 * p.k.step,
              uint32_t(p.k.step) * E, live, p.dk);
      lq.store(sQ);
      lk.store(sK);
    }
    // Tiles of pairs above the diagonal that share an operand with one below it.
    if (threadIdx.x < 64) {
#pragma unroll
      for (int i = 0; i < T; i += 2) {
        put4(&sP[(16 * (i + 1) + r) * PP + 16 * i + 4 * g], la_f32x4{0, 0, 0, 0});
        put4(&sD[(16 * (i + 1) + r) * PP + 16 * i + 4 * g], la_f32x4{0, 0, 0, 0});
      }
    }
  }

  for (int hh = 0; hh < p.group; ++hh) {
    const int h = hk * p.group + hh;
    Elem* dv = static_cast<Elem*>(p.dv_out) + (b * p.seqlen + t0) * v_step + h * p.dv;
    if (live == 0) {
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < T; ++i) put(dv, v_step, i, 16 * (NV * w + n) + 4 * g, p.dv, la_f32x4{0, 0, 0, 0});
      if (p.dg && int(threadIdx.x) < rows) p.dg[(b * p.seqlen + t0 + threadIdx.x) * p.heads + h] = 0.0f;
      if (p.dg_sums && threadIdx.x == 0) p.dg_sums[(b * p.chunks + c) * p.heads + h] = 0.0f;
      continue;
    }
    const float* S = p.states + ((b * p.heads + h) * p.chunks + c) * p.state_floats;
    const float* R = p.adjoints + ((b * p.heads + h) * p.chunks + c) * p.state_floats;
    {
      TileLoad<Elem, C, VP, kWhole> lv, lo;
      double gate = 0.0;
      lv.load(static_cast<const Elem*>(p.v.p) + b * p.v.batch + h * p.v.head + t0 * p.v.step,
              uint32_t(p.v.step) * E, live, p.dv);
      lo.load(static_cast<const Elem*>(p.dout.p) + b * p.dout.batch + h * p.dout.head + t0 * p.dout.step,
              uint32_t(p.dout.step) * E, live, p.dv);
      if (w == 0) gate = load_decay(p.g ? p.g + b * p.g_batch + h * p.g_head : nullptr, p.g_step, t0, live);
      lds_barrier();  // every wave has read the head before
      lv.store(sV);
      lo.store(sO);
      if (w == 0) dec.set(gate);
    }
    lds_barrier();

    // The pairs: tile (i, j) as rows t of columns s, stored by rows s.
    const WaveTiles mine = wave_tiles<C>(w);
    auto pairs = [&](int i, int j, const Frag<Elem>(&qf)[KP / 32], const Frag<Elem>(&of)[VP / 32]) {
      la_f32x4 a = {0, 0, 0, 0}, d = {0, 0, 0, 0};
#pragma unroll
      for (int kb = 0; kb < KP / 32; ++kb) a = mma(qf[kb], row_frag(sK, QP, 16 * j + r, 32 * kb), a);
#pragma unroll
      for (int vb = 0; vb < VP / 32; ++vb) d = mma(of[vb], row_frag(sV, OP, 16 * j + r, 32 * vb), d);
      const int s = 16 * j + r;
      const typename Decays<C>::Sum from = dec.sum[s];
      float wrow[4], wcol = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * i + 4 * g + e;
        const float m = s <= t ? p.scale * Decays<C>::between(dec.sum[t], from) : 0.0f;
        d[e] = s <= t ? d[e] * m : 0.0f;
        wrow[e] = s < t ? a[e] * d[e] : 0.0f;
        a[e] = s <= t ? a[e] * m : 0.0f;
        wcol += wrow[e];
      }
      put4(&sP[s * PP + 16 * i + 4 * g], a);
      put4(&sD[s * PP + 16 * i + 4 * g], d);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float sum = sum_lanes<4>(wrow[e]);
        if (r == 0) sRow[j][16 * i + 4 * g + e] = sum;
      }
      wcol += __shfl_xor(wcol, 16, 64);
      wcol += __shfl_xor(wcol, 32, 64);
      if (g == 0) sCol[i][s] = wcol;
    };
    {
      Frag<Elem> qf[KP / 32], of[VP / 32];
      auto rows_at = [&](int i) {
#pragma unroll
        for (int kb = 0; kb < KP / 32; ++kb) qf[kb] = row_frag(sQ, QP, 16 * i + r, 32 * kb);
#pragma unroll
        for (int vb = 0; vb < VP / 32; ++vb) of[vb] = row_frag(sO, OP, 16 * i + r, 32 * vb);
      };
      rows_at(mine.i);
      for (int j = mine.j0; j < mine.j1; ++j) pairs(mine.i, j, qf, of);
      if (mine.more) {
        rows_at(0);
        pairs(0, 0, qf, of);
      }
    }
    lds_barrier();

    // dq and dk of this wave's columns of dk.
    float dots = 0.0f;  // <R, S> over them
    float qs[T], ks[T];
#pragma unroll
    for (int i = 0; i < T; ++i) qs[i] = ks[i] = 0.0f;
#pragma unroll
    for (int n = 0; n < NK; ++n) {
      const int k0 = 16 * (NK * w + n);
      if (k0 >= p.dk) break;
      la_f32x4 xq[T], xk[T];
#pragma unroll
      for (int i = 0; i < T; ++i) xq[i] = xk[i] = la_f32x4{0, 0, 0, 0};
#pragma unroll
      for (int vb = 0; vb < VP / 32; ++vb) {
        if (32 * vb >= p.vpad) break;
        const int64_t off = int64_t(k0 + r) * p.vpad + 32 * vb + 8 * g;
        const la_f32x4 s0 = *reinterpret_cast<const la_f32x4*>(S + off),
                       s1 = *reinterpret_cast<const la_f32x4*>(S + off + 4),
                       r0 = *reinterpret_cast<const la_f32x4*>(R + off),
                       r1 = *reinterpret_cast<const la_f32x4*>(R + off + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dots = __builtin_fmaf(s0[e], r0[e], dots);
          dots = __builtin_fmaf(s1[e], r1[e], dots);
        }
        Pieces<Elem, 3> ps, pr;
        ps.split({s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]});
        pr.split({r0[0], r0[1], r0[2], r0[3], r1[0], r1[1], r1[2], r1[3]});
#pragma unroll
        for (int i = 0; i < T; ++i) {
          xq[i] = mma(ps, row_frag(sO, OP, 16 * i + r, 32 * vb), xq[i]);
          xk[i] = mma(pr, row_frag(sV, OP, 16 * i + r, 32 * vb), xk[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const int t = 16 * i + r;
        const float into = dec.into[t] * p.scale, onto = dec.onto[t];
        const la_f32x4 qv = get4(&sQ[t * QP + k0 + 4 * g]), kv = get4(&sK[t * QP + k0 + 4 * g]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          xq[i][e] *= into;
          xk[i][e] *= onto;
          qs[i] = __builtin_fmaf(qv[e], xq[i][e], qs[i]);
          ks[i] = __builtin_fmaf(kv[e], xk[i][e], ks[i]);
          aq[n][i][e] += xq[i][e];
          ak[n][i][e] += xk[i][e];
        }
      }
#pragma unroll
      for (int sb = 0; sb < SB; ++sb) {
        const Frag<Elem> kf = col_frag(sK, QP, 32 * sb, k0), qf = col_frag(sQ, QP, 32 * sb, k0);
#pragma unroll
        for (int i = 0; i < T; ++i) {
          if (i / 2 >= sb) aq[n][i] = mma(kf, col_frag(sD, PP, 32 * sb, 16 * i), aq[n][i]);
          if (i / 2 <= sb) ak[n][i] = mma(qf, row_frag(sD, PP, 16 * i + r, 32 * sb), ak[n][i]);
        }
      }
    }
    // dv of this wave's columns of dv.
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int v0 = 16 * (NV * w + n);
      if (v0 >= p.dv) break;
      la_f32x4 av[T];
#pragma unroll
      for (int i = 0; i < T; ++i) av[i] = la_f32x4{0, 0, 0, 0};
#pragma unroll
      for (int kb = 0; kb < KP / 32; ++kb) {
        if (32 * kb >= p.kpad) break;
        const float* from = R + int64_t(32 * kb + 8 * g) * p.vpad + v0 + r;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = from[e * p.vpad];
        Pieces<Elem, 2> pr;
        pr.split(x);
#pragma unroll
        for (int i = 0; i < T; ++i) av[i] = mma(pr, row_frag(sK, QP, 16 * i + r, 32 * kb), av[i]);
      }
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const float onto = dec.onto[16 * i + r];
#pragma unroll
        for (int e = 0; e < 4; ++e) av[i][e] *= onto;
      }
#pragma unroll
      for (int sb = 0; sb < SB; ++sb) {
        const Frag<Elem> of = col_frag(sO, OP, 32 * sb, v0);
#pragma unroll
        for (int i = 0; i < T; ++i)
          if (i / 2 <= sb) av[i] = mma(of, row_frag(sP, PP, 16 * i + r, 32 * sb), av[i]);
      }
#pragma unroll
      for (int i = 0; i < T; ++i) put(dv, v_step, i, v0 + 4 * g, p.dv, av[i]);
    }
    if (p.dg || p.dg_sums) {
#pragma unroll
      for (int i = 0; i < T; ++i) {
        float a = qs[i], d = ks[i];
        a += __shfl_xor(a, 16, 64);
        a += __shfl_xor(a, 32, 64);
        d += __shfl_xor(d, 16, 64);
        d += __shfl_xor(d, 32, 64);
        if (g == 0) {
          sQs[w][16 * i + r] = a;
          sKs[w][16 * i + r] = d;
        }
      }
      dots = sum_lanes<6>(dots);
      if (l == 0) sX[w] = dots;
      lds_barrier();
      if (w == 0) {
        const int t = l < C ? l : C - 1, i = t / 16;
        double down = 0.0, up = 0.0;
#pragma unroll
        for (int j = 0; j < T; ++j) {
          if (j <= i) down += sRow[j][t];
          if (j >= i) down -= sCol[j][t];
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          down += sQs[x][t];
          up += sKs[x][t];
        }
        if (l >= C) down = up = 0.0;
        const double before = wave_prefix_f64(down), all = dpp_f64(before, 63);
        const double behind = wave_prefix_f64(up) - up;
        const double around = double(dec.total) * (double(sX[0]) + sX[1] + sX[2] + sX[3]);
        double dg = all - before + down + behind + around;
        if (l >= live) dg = 0.0;
        if (p.dg && l < rows) p.dg[(b * p.seqlen + t0 + l) * p.heads + h] = float(dg);
        if (p.dg_sums) {
          const double sum = dpp_f64(wave_prefix_f64(dg), 63);
          if (l == 0) p.dg_sums[(b * p.chunks + c) * p.heads + h] = float(sum);
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NK; ++n)
#pragma unroll
    for (int i = 0; i < T; ++i) {
      put(dq, q_step, i, 16 * (NK * w + n) + 4 * g, p.dk, aq[n][i]);
      put(dk, q_step, i, 16 * (NK * w + n) + 4 * g, p.dk, ak[n][i]);
    }
}

// The sum over rows of sums[row][head], a workgroup a head, in a fixed order.
__global__ __launch_bounds__(256) void linattn_dg_kernel(const float* sums, int64_t rows, int heads, float* dg) {
  __shared__ double part[256];
  const int h = blockIdx.x;
  double a = 0.0;
  for (int64_t i = threadIdx.x; i < rows; i += 256) a += sums[i * heads + h];
  part[threadIdx.x] = a;
  __syncthreads();
  for (int m = 128; m > 0; m >>= 1) {
    if (int(threadIdx.x) < m) part[threadIdx.x] += part[threadIdx.x + m];
    __syncthreads();
  }
  if (threadIdx.x == 0) dg[h] = float(part[0]);
}

template <typename Elem, int KP, int VP>
void run_bwd_kernel(const BwdParams& p, int64_t groups, bool whole, hipStream_t s) {
  const dim3 grid{uint32_t(groups)}, block{kLaThreads};
  if (whole) hipLaunchKernelGGL((linattn_bwd_kernel<Elem, KP, VP, true>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((linattn_bwd_kernel<Elem, KP, VP, false>), grid, block, 0, s, p);
}

template <typename Elem>
void run_bwd(const BwdParams& p, int64_t groups, bool whole, hipStream_t s) {
  if (p.dk > 128 || p.dv > 128) return run_bwd_kernel<Elem, 256, 256>(p, groups, whole, s);
  if (p.dk > 64 && p.dv > 64) return run_bwd_kernel<Elem, 128, 128>(p, groups, whole, s);
  if (p.dk > 64) return run_bwd_kernel<Elem, 128, 64>(p, groups, whole, s);
  if (p.dv > 64) return run_bwd_kernel<Elem, 64, 128>(p, groups, whole, s);
  run_bwd_kernel<Elem, 64, 64>(p, groups, whole, s);
}

}  // namespace

int launch_linattn_bwd(const LinattnArgs& a, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (launch_linattn_chunk_states(a, stream) != 0) return -1;
  const int64_t c = linattn_chunk(a.io), chunks = (a.seqlen + c - 1) / c;
  const int64_t floats = linattn_state_floats(a.dk, a.dv), rows = a.batch * a.heads * chunks;
  BwdParams p{};
  p.q = a.q, p.k = a.k, p.v = a.v, p.dout = a.dout;
  p.g = a.g;
  p.g_batch = a.g_batch, p.g_step = a.g_step, p.g_head = a.g_head;
  p.lengths = a.lengths;
  p.states = a.workspace;
  p.adjoints = a.workspace + rows * floats;
  p.dq = a.dq, p.dk_out = a.dk_, p.dv_out = a.dv_;
  float* sums = a.workspace + 2 * rows * floats + rows;
  p.dg = a.dg_per_head ? nullptr : a.dg;
  p.dg_sums = a.dg && a.dg_per_head ? sums : nullptr;
  p.seqlen = a.seqlen, p.chunks = chunks, p.state_floats = floats;
  p.qk_heads = int(a.qk_heads), p.heads = int(a.heads), p.group = int(a.heads / a.qk_heads);
  p.dk = int(a.dk), p.dv = int(a.dv);
  p.kpad = int(linattn_pad(a.dk, 32)), p.vpad = int(linattn_pad(a.dv, 32));
  p.scale = a.scale;
  const int64_t groups = a.batch * a.qk_heads * chunks;
  const bool whole = linattn_whole(a, true);
  if (groups > 0) {
    if (a.io == Io::BF16) run_bwd<uint16_t>(p, groups, whole, s);
    else run_bwd<float>(p, groups, whole, s);
    if (hipGetLastError() != hipSuccess) return -1;
  }
  if (p.dg_sums) {
    hipLaunchKernelGGL(linattn_dg_kernel, dim3(uint32_t(a.heads)), dim3(256), 0, s, sums, a.batch * chunks,
                       int(a.heads), a.dg);
    if (hipGetLastError() != hipSuccess) return -1;
  }
  return 0;
}

}  // namespace ssm
