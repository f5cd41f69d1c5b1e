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
// the pairs of steps, of the chunk and around it, between which the decay g_t lies. dg so only adds
// terms that the decay scales: no difference of sums, over the sequence or the chunk, whose rounding
// errors would stay where a decay has made dg small. W's rectangle (rows from t on, columns before t) is made of the
// tiles that lie in it, of row sums of the tiles beside t's block, column sums of those below it, and
// of a rectangle of the block's own tile.
//
// linattn_state_kernel and linattn_join_kernel (linattn_kernels.hip) leave S and R of every chunk
// in the workspace, [dk][dv] in fp32; linattn_bwd_kernel then takes a (batch row, query head,
// chunk) per workgroup, the heads that share the query one after another (their dq and dk add
// up in its accumulators, in a fixed order). A wave owns an eighth of dk for dq and dk, an eighth of dv
// for dv, so that each value of S and R is split into operand pieces once.
//
// Roundings: the pairs' weights (scale D qk and scale D dov) are rounded to bf16 once, as operands,
// next to results in bf16. S and R enter in three bf16 pieces where dg, a result in fp32, comes
// of the product, and in two in dv.
//
// Measured, bf16, this kernel | the walk that leaves S and R: b4, 8 heads of 128 for 32 of 64, 2048 steps
// 157 | 127 us, reading 370 MB and writing 70 | 106 and 268; b1, 16 heads of 128 x 128, 16384 steps 306 | 195 (and 104
// for a first walk that finds its segments' starts). The two pass S and R through memory, 8 bytes a value
// each way; recomputing them in this kernel (several chunks a workgroup) was slower by a seventh, for want of
// registers. What bounds it: no unit is full (matrix cores 14%, LDS 28%, VALU 38% of its cycles, memory at half of
// a copy's rate); registers hold a CU to one workgroup, whose loads, pairs, states and stores follow one another.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

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

constexpr int kBwdThreads = 512;

// The pair tiles (i, j), j0 <= j < j1, of each of the eight waves: two at most. The last two have none:
// they do the next head's decays and the last one's dg meanwhile.
struct BwdTiles {
  int i, j0, j1;
};
template <int C>
__device__ __forceinline__ BwdTiles bwd_tiles(int w) {
  if constexpr (C == 64) {
    if (w == 0) return {3, 0, 2};
    if (w == 1) return {3, 2, 4};
    if (w == 2) return {2, 0, 2};
    if (w == 3) return {2, 2, 3};
    if (w == 4) return {1, 0, 2};
    return {0, 0, w == 5 ? 1 : 0};
  } else {
    if (w == 0) return {1, 0, 1};
    if (w == 1) return {1, 1, 2};
    return {0, 0, w == 2 ? 1 : 0};
  }
}

// What dg of one head comes from, by step of the chunk.
template <int C>
struct DgParts {
  float row[C / 16][C];      // of W: row sums of the tiles (i, j), j < i, by j; the tile (i, i)'s rectangles
  float col[C / 16][C];      // column sums of the tiles (i, j), j < i, by i
  float qs[8][C], ks[8][C];  // q . dq^S and k . dk^R, by wave
  float x[8], total;
};

template <typename Elem, int KP, int VP, bool kWhole>
__global__ __launch_bounds__(kBwdThreads, 2) void linattn_bwd_kernel(BwdParams p) {
  constexpr int C = linattn_bwd_chunk(sizeof(Elem) == 2 ? Io::BF16 : Io::F32, KP, VP);
  constexpr int T = C / 16, SB = C / 32, KB = KP / 32, VB = VP / 32;
  constexpr uint32_t E = sizeof(Elem);
  // The largest sizes keep fewer operands at a time, for want of registers.
  constexpr int kUnroll = KB + VB > 8 ? 1 : 8;
  // The 16-wide column tiles of dk and dv that a wave owns, for all steps; where there are only four,
  // one for half of the steps.
  constexpr bool kHalfK = KP < 128, kHalfV = VP < 128;
  constexpr int NK = kHalfK ? 1 : KP / 128, NV = kHalfV ? 1 : VP / 128;
  constexpr int TK = kHalfK ? T / 2 : T, TV = kHalfV ? T / 2 : T;
  // The states' operands are loaded ahead of the pairs where registers are left for them (b4, 8 heads of 128 for 32
  // of 64, 2048 steps, the whole gradient: 263 us, 273 with each where it is used); 128 x 128 has none to spare.
  constexpr bool kAhead = NK * VB <= 2;
  // Where they are not, two blocks of them at a time in bf16: b1, 16 heads of 128 x 128, 16384 steps, the whole
  // gradient: 588 us; all four, which spill, 672. (fp32, 8192 steps: two 632, all 634.)
  constexpr int kStateUnroll = !kAhead && E == 2 && kUnroll > 2 ? 2 : kUnroll;
  constexpr int QP = la_pitch<Elem>(KP), OP = la_pitch<Elem>(VP), PP = la_pitch<Elem>(C);
  __shared__ __attribute__((aligned(16))) Elem sQ[C * QP], sK[C * QP], sV[C * OP], sO[C * OP];
  __shared__ __attribute__((aligned(16))) Elem sP[C * PP], sD[C * PP];  // weights by rows s: scale D qk, scale D dov
  __shared__ __attribute__((aligned(16))) Decays<C> decays[2];          // of even and odd heads
  __shared__ DgParts<C> parts[2];
  __shared__ int again;

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
  const int kt = kHalfK ? w & 3 : NK * w, ik = kHalfK ? (w >> 2) * TK : 0;
  const int vt = kHalfV ? w & 3 : NV * w, iv = kHalfV ? (w >> 2) * TV : 0;

  la_f32x4 aq[NK][TK], ak[NK][TK];
#pragma unroll
  for (int n = 0; n < NK; ++n)
#pragma unroll
    for (int i = 0; i < TK; ++i) aq[n][i] = ak[n][i] = la_f32x4{0, 0, 0, 0};

  // Columns col .. + 3 of step 16 i + r; zero behind the end.
  auto put = [&](Elem* base, int64_t step, int i, int col, int dim, la_f32x4 v) {
    const int t = 16 * i + r;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = t < live ? v[e] : 0.0f;
    store4_at<Elem, kWhole>(Buf(base, kLaBytes), uint32_t(t) * uint32_t(step) * E + uint32_t(col) * E, dim - col,
                            t < rows, v);
  };
  auto dv_of = [&](int h) { return static_cast<Elem*>(p.dv_out) + (b * p.seqlen + t0) * v_step + int64_t(h) * p.dv; };

  if (live == 0) {
    for (int h = hk * p.group; h < (hk + 1) * p.group; ++h) {
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < TV; ++i) put(dv_of(h), v_step, iv + i, 16 * (vt + n) + 4 * g, p.dv, la_f32x4{0, 0, 0, 0});
      if (p.dg && int(threadIdx.x) < rows) p.dg[(b * p.seqlen + t0 + threadIdx.x) * p.heads + h] = 0.0f;
      if (p.dg_sums && threadIdx.x == 0) p.dg_sums[(b * p.chunks + c) * p.heads + h] = 0.0f;
    }
  } else {
    TileLoad<Elem, C, VP, kWhole, kBwdThreads> lv, lo;
    auto fetch = [&](int hh) {
      const int64_t h = hk * p.group + hh;
      const int n = hh < p.group ? live : 0;
      lv.load(static_cast<const Elem*>(p.v.p) + b * p.v.batch + (n ? h : 0) * p.v.head + t0 * p.v.step,
              uint32_t(p.v.step) * E, n, p.dv);
      lo.load(static_cast<const Elem*>(p.dout.p) + b * p.dout.batch + (n ? h : 0) * p.dout.head + t0 * p.dout.step,
              uint32_t(p.dout.step) * E, n, p.dv);
    };
    auto gate_of = [&](int hh) {
      return load_decay(p.g ? p.g + b * p.g_batch + int64_t(hk) * p.group * p.g_head : nullptr, p.g_step, t0,
                        hh < p.group ? live : 0, int64_t(hh < p.group ? hh : 0) * p.g_head);
    };
    // dg of the head whose parts lie in parts[hh & 1], by one wave.
    auto finish = [&](int hh) {
      const DgParts<C>& d = parts[hh & 1];
      const int h = hk * p.group + hh, t = l < C ? l : C - 1, i = t / 16;
      const bool on = l < C;
      // W's rectangle: in the block's own tile; of the tiles (i, j) the rows from t on, and those (y, j), j < i < y,
      // which lie in it whole; of the tiles (y, i) the columns before t. (Everything is loaded first, whatever comes of
      // it, so that the loads are one wait.)
      float row[T], col[T], qs[8], ks[8], x[8];
#pragma unroll
      for (int j = 0; j < T; ++j) {
        row[j] = d.row[j][t];
        col[j] = d.col[j][t];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        qs[j] = d.qs[j][t];
        ks[j] = d.ks[j][t];
        x[j] = d.x[j];
      }
      float rect = 0.0f, cols = 0.0f;
#pragma unroll
      for (int j = 0; j < T; ++j) rect = on && j == i ? row[j] : rect;
#pragma unroll
      for (int j = 0; j + 1 < T; ++j) {
        const float rows_on = row_suffix(on && i > j ? row[j] : 0.0f);
        rect += rows_on;
#pragma unroll
        for (int y = j + 2; y < T; ++y) {
          const float tile = lane_value(rows_on, 16 * y);
          rect += on && i > j && i < y ? tile : 0.0f;
        }
      }
#pragma unroll
      for (int j = 1; j < T; ++j) cols += on && j > i ? col[j] : 0.0f;
      rect += dpp_move<0x111>(row_prefix(cols));
      float down = 0.0f, up = 0.0f;
      double around = 0.0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool mine = on && (!kHalfK || (j >> 2) == i / TK);
        down += mine ? qs[j] : 0.0f;
        up += mine ? ks[j] : 0.0f;
        if (!kHalfK || j < 4) around += x[j];
      }
      float dg = float(double(rect) + wave_from(down) + wave_before(up) + double(d.total) * around);
      if (l >= live) dg = 0.0f;
      if (p.dg && l < rows) p.dg[(b * p.seqlen + t0 + l) * p.heads + h] = dg;
      if (p.dg_sums) {
        const double sum = dpp_f64(wave_prefix_f64(dg), 63);
        if (l == 0) p.dg_sums[(b * p.chunks + c) * p.heads + h] = float(sum);
      }
    };
    const bool any_dg = p.dg || p.dg_sums;
    unsigned long long met = 0;  // lanes with results that are not finite
    auto look = [&](float x) { met |= __ballot(!(__builtin_fabsf(x) < __builtin_inff())); };
    float gate = 0.0f;
    auto begin = [&] {
      gate = gate_of(1);
      const float first = gate_of(0);
      if (w == 6) decays[0].set_apart(first);
    };
    begin();
    {
      TileLoad<Elem, C, KP, kWhole, kBwdThreads> lq, lk;
      lq.load(static_cast<const Elem*>(p.q.p) + b * p.q.batch + hk * p.q.head + t0 * p.q.step,
              uint32_t(p.q.step) * E, live, p.dk);
      lk.load(static_cast<const Elem*>(p.k.p) + b * p.k.batch + hk * p.k.head + t0 * p.k.step,
              uint32_t(p.k.step) * E, live, p.dk);
      fetch(0);
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
    if (threadIdx.x == 0) again = 0;

    // All heads. alone: dq, dk and dv only, the pairs of steps one by one.
    auto heads = [&](auto one_by_one, int r, int g) {
      constexpr bool alone = decltype(one_by_one)::value;
      const bool want_dg = !alone && any_dg;
      // (The second form is to be small: it is hardly ever run.)
      constexpr bool ahead = kAhead && !alone, column_ahead = NV * KB <= 4 && !alone;
      constexpr int unroll = alone ? 1 : kUnroll, state_unroll = alone ? 1 : kStateUnroll;
      for (int hh = 0; hh < p.group; ++hh) {
        const int h = hk * p.group + hh;
        const int64_t state = ((b * p.heads + h) * p.chunks + c) * p.state_floats;
        const Buf S(p.states + state, uint32_t(p.state_floats) * 4), R(p.adjoints + state, uint32_t(p.state_floats) * 4);
        const Decays<C>& dec = decays[hh & 1];
        DgParts<C>& part = parts[hh & 1];
        // Row k of a state, values v of a block of 32: operands of dq and dk.
        auto state_at = [&](int n, int vb) {
          const int k = 16 * (kt + n) + r, v = 32 * vb + 8 * g;
          return k < p.kpad && v < p.vpad ? uint32_t(k * p.vpad + v) * 4u : kLaOob;
        };
        uint4 fs[ahead ? NK : 1][VB][2], fr[ahead ? NK : 1][VB][2];

        lds_barrier();  // every wave has read the head before
        lv.store(sV);
        lo.store(sO);
        lds_barrier();
        // (ahead of the loads, which it would wait for)
        if (w == 6 && hh + 1 < p.group) decays[(hh + 1) & 1].set_apart(gate);
        if constexpr (ahead) {
#pragma unroll
          for (int n = 0; n < NK; ++n)
#pragma unroll
            for (int vb = 0; vb < VB; ++vb) {
              const uint32_t off = state_at(n, vb);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                fs[n][vb][e] = S.load16(off + 16u * e);
                fr[n][vb][e] = R.load16(off + 16u * e);
              }
            }
        }
        gate = gate_of(hh + 2);
        fetch(hh + 1);

        // The pairs: tile (i, j) as rows t of columns s, stored by rows s.
        const BwdTiles mine = bwd_tiles<C>(w);
        if (mine.j1 > mine.j0) {
          const int i = mine.i;
          for (int j = mine.j0; j < mine.j1; ++j) {
            la_f32x4 a = {0, 0, 0, 0}, d = {0, 0, 0, 0};
#pragma unroll unroll
            for (int kb = 0; kb < KB; ++kb)
              a = mma(row_frag(sQ, QP, 16 * i + r, 32 * kb), row_frag(sK, QP, 16 * j + r, 32 * kb), a);
#pragma unroll unroll
            for (int vb = 0; vb < VB; ++vb)
              d = mma(row_frag(sO, OP, 16 * i + r, 32 * vb), row_frag(sV, OP, 16 * j + r, 32 * vb), d);
            const int s = 16 * j + r;
            float keep[4], wrow[4], wcol = 0.0f;
            dec.onwards(s, 16 * i + 4 * g, keep);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int t = 16 * i + 4 * g + e;
              const float m = p.scale * keep[e], da = d[e] * m, aa = a[e] * m, ww = a[e] * da;
              d[e] = s <= t ? da : 0.0f;
              a[e] = s <= t ? aa : 0.0f;
              wrow[e] = s < t ? ww : 0.0f;
              wcol += wrow[e];
            }
            put4(&sP[s * PP + 16 * i + 4 * g], a);
            put4(&sD[s * PP + 16 * i + 4 * g], d);
            if (want_dg && i == j) {
              // Rows from column s's own step on, columns before it.
              float rect = 0.0f;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float before = row_prefix(dpp_move<0x111>(wrow[e]));  // (row_shr 1)
                rect += 4 * g + e >= r ? before : 0.0f;
              }
              rect += __shfl_xor(rect, 16, 64);
              rect += __shfl_xor(rect, 32, 64);
              if (g == 0) part.row[i][s] = rect;
            } else if (want_dg) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float sum = sum_lanes<4>(wrow[e]);
                if (r == 0) part.row[j][16 * i + 4 * g + e] = sum;
              }
              wcol += __shfl_xor(wcol, 16, 64);
              wcol += __shfl_xor(wcol, 32, 64);
              if (g == 0) part.col[i][s] = wcol;
            }
          }
        }
        if (w == 7 && hh > 0 && want_dg) finish(hh - 1);
        lds_barrier();

        // Column v of R, values k of a block of 32: operands of dv.
        float rk[column_ahead ? NV : 1][KB][8];
        auto load_column = [&](int n, int kb, float (&x)[8]) {
          const int v = 16 * (vt + n) + r, k = 32 * kb + 8 * g;
          const uint32_t off = v < p.vpad && k < p.kpad ? uint32_t(k * p.vpad + v) * 4u : kLaOob;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(R.load4(off + uint32_t(e * p.vpad) * 4u));
        };

        // dq and dk of this wave's columns of dk.
        float dots = 0.0f;  // <R, S> over them
        float qs[TK], ks[TK];
#pragma unroll
        for (int i = 0; i < TK; ++i) qs[i] = ks[i] = 0.0f;
#pragma unroll
        for (int n = 0; n < NK; ++n) {
          const int k0 = 16 * (kt + n);
          la_f32x4 xq[TK], xk[TK];
#pragma unroll
          for (int i = 0; i < TK; ++i) xq[i] = xk[i] = la_f32x4{0, 0, 0, 0};
#pragma unroll state_unroll
          for (int vb = 0; vb < VB; ++vb) {
            uint4 words[2][2];
            if constexpr (ahead) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                words[0][e] = fs[n][vb][e];
                words[1][e] = fr[n][vb][e];
              }
            } else {
              const uint32_t off = state_at(n, vb);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                words[0][e] = S.load16(off + 16u * e);
                words[1][e] = R.load16(off + 16u * e);
              }
            }
            float sv[8], rv[8];
            widen_raw16<float>(words[0][0], sv);
            widen_raw16<float>(words[0][1], sv + 4);
            widen_raw16<float>(words[1][0], rv);
            widen_raw16<float>(words[1][1], rv + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) dots = __builtin_fmaf(sv[e], rv[e], dots);
            Pieces<Elem, 3> ps, pr;
            ps.split(sv);
            pr.split(rv);
#pragma unroll
            for (int i = 0; i < TK; ++i) {
              const Frag<Elem> fo = row_frag(sO, OP, 16 * (ik + i) + r, 32 * vb),
                               fv = row_frag(sV, OP, 16 * (ik + i) + r, 32 * vb);
#pragma unroll
              for (int e = ps.kCount - 1; e >= 0; --e) {  // the small ones first, the two sums in turn
                xq[i] = mma(piece(ps, e), fo, xq[i]);
                xk[i] = mma(piece(pr, e), fv, xk[i]);
              }
            }
          }
          // (by now the states' registers are free again)
          if (column_ahead && n == NK - 1) {
#pragma unroll
            for (int m = 0; m < NV; ++m)
#pragma unroll
              for (int kb = 0; kb < KB; ++kb) load_column(m, kb, rk[column_ahead ? m : 0][kb]);
          }
#pragma unroll
          for (int i = 0; i < TK; ++i) {
            const int t = 16 * (ik + i) + r;
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
            if constexpr (!alone) {
#pragma unroll
              for (int i = 0; i < TK; ++i) {
                if ((ik + i) / 2 >= sb) aq[n][i] = mma(kf, col_frag(sD, PP, 32 * sb, 16 * (ik + i)), aq[n][i]);
                if ((ik + i) / 2 <= sb) ak[n][i] = mma(qf, row_frag(sD, PP, 16 * (ik + i) + r, 32 * sb), ak[n][i]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < TK; ++i) {
                const int s = 16 * (ik + i) + r, b0 = 32 * sb, b1 = b0 + 32, col = k0 + 4 * g;
                aq[n][i] = steps_alone(sD + s, PP, sK + col, QP, b0, s < b1 ? s + 1 : b1, aq[n][i]);
                ak[n][i] = steps_alone(sD + s * PP, 1, sQ + col, QP, s > b0 ? s : b0, b1, ak[n][i]);
              }
            }
          }
        }
        // dv of this wave's columns of dv.
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          const int v0 = 16 * (vt + n);
          la_f32x4 av[TV];
#pragma unroll
          for (int i = 0; i < TV; ++i) av[i] = la_f32x4{0, 0, 0, 0};
#pragma unroll unroll
          for (int kb = 0; kb < KB; ++kb) {
            Pieces<Elem, 2> pr;
            if constexpr (column_ahead) {
              pr.split(rk[n][kb]);
            } else {
              float x[8];
              load_column(n, kb, x);
              pr.split(x);
            }
#pragma unroll
            for (int i = 0; i < TV; ++i) {
              const Frag<Elem> fk = row_frag(sK, QP, 16 * (iv + i) + r, 32 * kb);
#pragma unroll
              for (int e = pr.kCount - 1; e >= 0; --e) av[i] = mma(piece(pr, e), fk, av[i]);
            }
          }
#pragma unroll
          for (int i = 0; i < TV; ++i) {
            const float onto = dec.onto[16 * (iv + i) + r];
#pragma unroll
            for (int e = 0; e < 4; ++e) av[i][e] *= onto;
          }
#pragma unroll
          for (int sb = 0; sb < SB; ++sb) {
            const Frag<Elem> of = col_frag(sO, OP, 32 * sb, v0);
            if constexpr (!alone) {
#pragma unroll
              for (int i = 0; i < TV; ++i)
                if ((iv + i) / 2 <= sb) av[i] = mma(of, row_frag(sP, PP, 16 * (iv + i) + r, 32 * sb), av[i]);
            } else {
#pragma unroll
              for (int i = 0; i < TV; ++i) {
                const int s = 16 * (iv + i) + r, b0 = 32 * sb, b1 = b0 + 32;
                av[i] = steps_alone(sP + s * PP, 1, sO + v0 + 4 * g, OP, s > b0 ? s : b0, b1, av[i]);
              }
            }
          }
          if constexpr (!alone) look((av[0][0] + av[0][1]) + (av[0][2] + av[0][3]));
#pragma unroll
          for (int i = 0; i < TV; ++i) put(dv_of(h), v_step, iv + i, v0 + 4 * g, p.dv, av[i]);
        }
        if (want_dg) {
#pragma unroll
          for (int i = 0; i < TK; ++i) {
            float a = qs[i], d = ks[i];
            a += __shfl_xor(a, 16, 64);
            a += __shfl_xor(a, 32, 64);
            d += __shfl_xor(d, 16, 64);
            d += __shfl_xor(d, 32, 64);
            if (g == 0) {
              part.qs[w][16 * (ik + i) + r] = a;
              part.ks[w][16 * (ik + i) + r] = d;
            }
          }
          dots = sum_lanes<6>(dots);
          if (l == 0) {
            part.x[w] = dots;
            if (w == 0) part.total = dec.total;
          }
        }
      }
    };
    heads(std::false_type{}, r, g);
    // The weights of the pairs above the diagonal are zeros, which a value of q, k or dout that is not finite turns to
    // NaN in steps that it has no part in: a workgroup that met one forms dq, dk and dv again. It shows in the results
    // of the last steps (dq) or the first (dk, dv), whose sums are over all pairs. (Afterwards, since a branch around the
    // products took the registers of the loads on their way, and by the results, which are fewer than the values. b4, 8
    // heads of 128 for 32 of 64, 2048 steps, the whole gradient: 262.2 us, 260.4 without this, 495 with the branch.)
    float sum = 0.0f;
#pragma unroll
    for (int n = 0; n < NK; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += aq[n][TK - 1][e] + ak[n][0][e];
    look(sum);
    if (met != 0 && l == 0) again = 1;
    lds_barrier();
    if (any_dg && w == 7) finish(p.group - 1);
    if (__builtin_expect(__builtin_amdgcn_readfirstlane(again), 0)) {
#pragma unroll
      for (int n = 0; n < NK; ++n)
#pragma unroll
        for (int i = 0; i < TK; ++i) aq[n][i] = ak[n][i] = la_f32x4{0, 0, 0, 0};
      begin();
      fetch(0);
      heads(std::true_type{}, not_ahead(r), not_ahead(g));
    }
  }
#pragma unroll
  for (int n = 0; n < NK; ++n)
#pragma unroll
    for (int i = 0; i < TK; ++i) {
      put(dq, q_step, ik + i, 16 * (kt + n) + 4 * g, p.dk, aq[n][i]);
      put(dk, q_step, ik + i, 16 * (kt + n) + 4 * g, p.dk, ak[n][i]);
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
  const dim3 grid{uint32_t(groups)}, block{kBwdThreads};
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
  const int64_t c = linattn_bwd_chunk(a.io, a.dk, a.dv), chunks = (a.seqlen + c - 1) / c;
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
