// Linear attention with a decay for each head on the gfx950 matrix cores (include/ssm_linattn.h).
//
//   S_t = exp(g_t) S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t
//
// In chunks of C steps, with cs_t the running sum of g over the chunk:
//
//   o_t   = scale sum_{s<=t} exp(cs_t - cs_s) (q_t . k_s) v_s + scale exp(cs_t) S_in q_t
//   S_out = exp(cs_end) S_in + sum_s exp(cs_end - cs_s) v_s k_s^T
//
// linattn_fwd_kernel: one workgroup walks the chunks of a (batch row, head, tile of 64 or 128 value
// channels, segment of the sequence), the state dk x its channels in the accumulators of its
// four waves (16 or 32 channels each), which are the state's product's operand as they stand.
// A sequence is one segment where batch rows and heads fill the device; else
// linattn_state_kernel finds what each segment adds to the state, linattn_join_kernel the state
// at each segment's start, and the segments run side by side.
//
// Roundings: the pairs' weights are rounded to bf16 once, as an operand, like the result (its error
// is as large as the result's own rounding). The state enters its product in two bf16 pieces
// (16 bits): in one its error would add to that of the weights. What is added to the state enters
// in three pieces, all 24 bits, since the state is a result in fp32.
//
// Values that are not finite: a NaN or infinity is in the results of its own and later steps and in none before, as in
// the recurrence, although a chunk's product passes over all pairs of its steps. (The check of a chunk's values
// costs the whole-row forms between -3% and +1%: b8, 32 heads of 128 x 64 113.4 -> 109.8 us, fp32 b4 178.8 -> 180.1.)
//
// Measured, bf16: b4, 8 heads of 128 for 32 of 64, 2048 steps 80.1 us in all, 52 the forward, 30 the segments'
// states, 7 the join (must move 106 MB, 21 us at a copy's rate; the three launches move 226); b1, 16 heads of
// 128 x 128, 65536 steps 428, of which 337, 167 and 14 where each runs alone (must move 1076 MB, 210 us; they move 1748,
// 4.1 TB/s). The long one is near memory's rate on what a second pass over k and v costs; the short one waits: a
// chunk's products, decays and stores follow one another, and 214 registers and 55 KB of LDS hold it to two workgroups
// a CU. Near half of the LDS cycles are bank conflicts, from the operands' 16 rows, four banks apart: at eight (32 bytes
// between rows) a third of them go, and no time with them.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_linattn.h"
#include "linattn_launch.h"

namespace ssm {
namespace {

// ---------------------------------------------------------------- forward

struct FwdParams {
  HeadRows q, k, v;
  const float* g;
  int64_t g_batch, g_step, g_head;
  const float* initial;
  const int32_t* lengths;
  void* out;
  float* final_state;
  const float* states;   // nullable: [batch, heads, segments, pad(dv), pad(dk)], segment starts
  int64_t seqlen, chunks, per, segments;
  int64_t kpad, state_floats;
  int heads, group, dk, dv, value_tiles;
  float scale;
};

template <typename Elem, int KP, int NV, bool kWhole>
__global__ __launch_bounds__(kLaThreads, KP <= 128 ? 2 : 1) void linattn_fwd_kernel(FwdParams p) {
  constexpr int C = chunk_of<Elem>(), T = C / 16, SB = C / 32, VT = 64 * NV, KB = KP / 32;
  constexpr int QP = la_pitch<Elem>(KP), VP = la_pitch<Elem>(VT), PP = la_pitch<Elem>(C);
  __shared__ __attribute__((aligned(16))) Elem sQ[C * QP], sK[C * QP], sV[C * VP], sP[C * PP];
  __shared__ __attribute__((aligned(16))) Decays<C> decays[2];  // of even and odd chunks

  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = threadIdx.x & 63, r = l & 15, g = l >> 4;
  uint32_t at = xcd_order(blockIdx.x, gridDim.x);
  const int vt = int(at % uint32_t(p.value_tiles));
  at /= uint32_t(p.value_tiles);
  const int h = int(at % uint32_t(p.heads));
  at /= uint32_t(p.heads);
  const int64_t seg = at % uint32_t(p.segments), b = at / uint32_t(p.segments);
  const int hk = h / p.group, v0 = vt * VT;
  const Elem* q = static_cast<const Elem*>(p.q.p) + b * p.q.batch + hk * p.q.head;
  const Elem* k = static_cast<const Elem*>(p.k.p) + b * p.k.batch + hk * p.k.head;
  const Elem* v = static_cast<const Elem*>(p.v.p) + b * p.v.batch + h * p.v.head + v0;
  const float* gates = p.g ? p.g + b * p.g_batch + h * p.g_head : nullptr;
  Elem* out = static_cast<Elem*>(p.out) + (b * p.seqlen * p.heads + h) * p.dv;
  const int64_t out_step = int64_t(p.heads) * p.dv;
  const int64_t end = row_end(p.lengths, b, p.seqlen);
  const int64_t c0 = seg * p.per, c1 = c0 + p.per < p.chunks ? c0 + p.per : p.chunks;

  // The state: tiles (2 j, n) and (2 j + 1, n) are rows k = 32 j + 8 g + i and + 4 + i of column v =
  // vcol + 16 n + r, so that a lane has eight neighbouring k of one v.
  const int vcol = v0 + 16 * NV * w;
  la_f32x4 S[KP / 16][NV];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int vc = vcol + 16 * n + r;
    const float* from = nullptr;
    if (vc < p.dv) {
      if (p.states)
        from = p.states + ((b * p.heads + h) * p.segments + seg) * p.state_floats + vc * p.kpad;
      else if (p.initial)
        from = p.initial + ((b * p.heads + h) * p.dv + vc) * p.dk;
    }
#pragma unroll
    for (int j = 0; j < KP / 16; ++j) {
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      const int kr = 32 * (j / 2) + 8 * g + 4 * (j % 2);
      if (from && kr < p.dk) load_few<float, 4>(from + kr, p.dk - kr, s);
      S[j][n] = la_f32x4{s[0], s[1], s[2], s[3]};
    }
  }
  // Tiles of pairs above the diagonal that share an operand with one below it.
  if (threadIdx.x < 64) {
#pragma unroll
    for (int i = 0; i < T; i += 2) put4(&sP[(16 * i + r) * PP + 16 * (i + 1) + 4 * g], la_f32x4{0, 0, 0, 0});
  }

  TileLoad<Elem, C, KP, kWhole> lq, lk;
  TileLoad<Elem, C, VT, kWhole> lv;
  constexpr uint32_t E = sizeof(Elem);
  auto rows_of = [&](int64_t c) {
    const int64_t left = c < c1 ? end - c * C : 0;
    return left < 0 ? 0 : left < C ? int(left) : C;
  };
  const int v_left = p.dv - v0 < VT ? p.dv - v0 : VT;
  auto fetch = [&](int64_t c) {
    const int64_t t0 = c * C;
    const int rows = rows_of(c);
    lq.load(q + t0 * p.q.step, uint32_t(p.q.step) * E, rows, p.dk);
    lk.load(k + t0 * p.k.step, uint32_t(p.k.step) * E, rows, p.dk);
    lv.load(v + t0 * p.v.step, uint32_t(p.v.step) * E, rows, v_left);
  };
  // The last wave, with the fewest tiles of pairs, forms each chunk's decays a chunk ahead.
  float gate = load_decay(gates, p.g_step, (c0 + 1) * C, rows_of(c0 + 1));
  {
    const float first = load_decay(gates, p.g_step, c0 * C, rows_of(c0));
    if (w == 3) decays[c0 & 1].set(first);
  }
  if constexpr (kWhole) fetch(c0);
  for (int64_t c = c0; c < c1; ++c) {
    const int64_t t0 = c * C;
    const Buf to(out + t0 * out_step, kLaBytes);
    const int rows = p.seqlen - t0 < C ? int(p.seqlen - t0) : C;       // of out
    const int live = end <= t0 ? 0 : end - t0 < C ? int(end - t0) : C;  // that hold steps
    if (live > 0) {
      const Decays<C>& dec = decays[c & 1];
      // (Rows by elements take twice the registers on their way, and are loaded when their chunk begins: ahead of it they
      // made the kernel spill. b2, 16 heads of 100 x 100, 2048 steps in bf16 97.7 us, ahead 116.)
      if constexpr (!kWhole) fetch(c);
      lds_barrier();  // every wave has read the chunk before
      lq.store(sQ);
      lk.store(sK);
      lv.store(sV);
      lds_barrier();
      // (ahead of the loads for the next chunk, which it would wait for)
      if (w == 3) decays[(c + 1) & 1].set(gate);
      gate = load_decay(gates, p.g_step, (c + 2) * C, rows_of(c + 2));
      if constexpr (kWhole) fetch(c + 1);
      // The weights of the pairs s <= t, with the decay between them: tile (i, j) as rows s of
      // columns t, stored by rows t.
      const WaveTiles mine = wave_tiles<C>(w);
      auto weights = [&](int i, int j, const Frag<Elem>(&qf)[KB]) {
        la_f32x4 a = {0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) a = mma(row_frag(sK, QP, 16 * j + r, 32 * kb), qf[kb], a);
        const int t = 16 * i + r, s0 = 16 * j + 4 * g;
        float keep[4];
        dec.between(t, s0, keep);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float weight = a[e] * (p.scale * keep[e]);
          a[e] = s0 + e <= t ? weight : 0.0f;
        }
        put4(&sP[t * PP + s0], a);
      };
      {
        Frag<Elem> qf[KB];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) qf[kb] = row_frag(sQ, QP, 16 * mine.i + r, 32 * kb);
        for (int j = mine.j0; j < mine.j1; ++j) weights(mine.i, j, qf);
        if (mine.more) {
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) qf[kb] = row_frag(sQ, QP, r, 32 * kb);
          weights(0, 0, qf);
        }
      }
      Frag<Elem> vf[SB][NV];
#pragma unroll
      for (int sb = 0; sb < SB; ++sb)
#pragma unroll
        for (int n = 0; n < NV; ++n) vf[sb][n] = col_frag(sV, VP, 32 * sb, 16 * (NV * w + n));
      // Results as rows v of columns t: through the state first. Products of different sums follow each
      // other, so that none waits for the one before.
      la_f32x4 o[T][NV];
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int n = 0; n < NV; ++n) o[i][n] = la_f32x4{0, 0, 0, 0};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        Frag<Elem> f[T];
#pragma unroll
        for (int i = 0; i < T; ++i) f[i] = row_frag(sQ, QP, 16 * i + r, 32 * kb);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          const la_f32x4 x = S[2 * kb][n], y = S[2 * kb + 1][n];
          Pieces<Elem, 2> sp;
          sp.split({x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
#pragma unroll
          for (int e = sp.kCount - 1; e >= 0; --e)
#pragma unroll
            for (int i = 0; i < T; ++i) o[i][n] = mma(piece(sp, e), f[i], o[i][n]);
        }
      }
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const float into = dec.into[16 * i + r] * p.scale;
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][n][e] *= into;
      }
      lds_barrier();
      // Then the pairs. The weights of those above the diagonal are zeros, which a value that is not finite would turn to
      // NaN: a wave that has one in its columns sums the pairs below one by one.
      NotFinite odd;
#pragma unroll
      for (int sb = 0; sb < SB; ++sb)
#pragma unroll
        for (int n = 0; n < NV; ++n) odd.add(vf[sb][n]);
      if (__builtin_expect(!odd.any(), 1)) {
#pragma unroll
        for (int sb = 0; sb < SB; ++sb) {
          Frag<Elem> f[T];
#pragma unroll
          for (int i = 2 * sb; i < T; ++i) f[i] = row_frag(sP, PP, 16 * i + r, 32 * sb);
#pragma unroll
          for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int i = 2 * sb; i < T; ++i) o[i][n] = mma(vf[sb][n], f[i], o[i][n]);
        }
      } else {
        const int r1 = not_ahead(r), g1 = not_ahead(g);
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
          for (int n = 0; n < NV; ++n) {
            const int t = 16 * i + r1;
            o[i][n] = steps_alone(sP + t * PP, 1, sV + 16 * (NV * w + n) + 4 * g1, VP, 0, t + 1, o[i][n]);
          }
      }
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const int t = 16 * i + r;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          const int vr = vcol + 16 * n + 4 * g;
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][n][e] = t < live ? o[i][n][e] : 0.0f;
          store4_at<Elem, kWhole>(to, uint32_t(t) * uint32_t(out_step) * E + uint32_t(vr) * E, p.dv - vr, t < rows,
                                  o[i][n]);
        }
      }
      // The state at the chunk's end.
      const float total = dec.total;
      Pieces<Elem, 3> add[SB][NV];
#pragma unroll
      for (int sb = 0; sb < SB; ++sb) {
        float on[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) on[e] = dec.onto[32 * sb + 8 * g + e];
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          float x[8];
          widen_frag(vf[sb][n], x);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= on[e];
          add[sb][n].split(x);
        }
      }
#pragma unroll
      for (int j = 0; j < KP / 16; ++j)
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[j][n][e] *= total;
#pragma unroll
      for (int sb = 0; sb < SB; ++sb)
#pragma unroll
        for (int j4 = 0; j4 < KP / 16; j4 += 4) {
          Frag<Elem> f[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] = col_frag_paired(sK, QP, 32 * sb, 32 * ((j4 + j) / 2), j % 2);
#pragma unroll
          for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int e = add[sb][n].kCount - 1; e >= 0; --e)
#pragma unroll
              for (int j = 0; j < 4; ++j) S[j4 + j][n] = mma(f[j], piece(add[sb][n], e), S[j4 + j][n]);
        }
    } else {
      // Behind the row's end: zeros, and the state stays.
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const int t = 16 * i + r;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          const int vr = vcol + 16 * n + 4 * g;
          store4_at<Elem, kWhole>(to, uint32_t(t) * uint32_t(out_step) * E + uint32_t(vr) * E, p.dv - vr, t < rows,
                                  la_f32x4{0, 0, 0, 0});
        }
      }
    }
  }
  if (p.final_state && seg == p.segments - 1) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int vc = vcol + 16 * n + r;
      if (vc >= p.dv) continue;
      float* to = p.final_state + ((b * p.heads + h) * p.dv + vc) * p.dk;
#pragma unroll
      for (int j = 0; j < KP / 16; ++j) {
        const int kr = 32 * (j / 2) + 8 * g + 4 * (j % 2);
        const float s[4] = {S[j][n][0], S[j][n][1], S[j][n][2], S[j][n][3]};
        if (kr < p.dk) store_few<float, 4>(to + kr, p.dk - kr, s);
      }
    }
  }
}

// ---------------------------------------------------------------- states of segments

// What the steps of a segment add to a state: sum_s weight_s y_s x_s^T, rows y, x contiguous. Forward
// (x = k, y = v, or exchanged): weight_s = exp(sum of g behind s in the segment). Reverse (the
// adjoint: x and y of dout and q): weight_t = scale exp(sum of g from the segment's start to t).
struct StateParams {
  HeadRows x, y;
  int x_group, y_group;   // heads of the sequence to one of the array's
  int xd, yd;
  bool reverse;
  float scale;
  float* states;          // [batch, heads, segments, pad(yd), pad(xd)], what a segment adds
  // Walked instead: from the state at the segment's start, the state before every chunk.
  float* every;           // [batch, heads, chunks, pad(yd), pad(xd)]
  const float* starts;    // nullable (one segment): as states, joined
  const float* first;     // nullable: [batch, heads, xd, yd], the sequence's start, where starts is null
  float* last;            // nullable: the same, behind the last chunk of the walk
};

struct StatesParams {
  StateParams dir[2];
  const float* g;
  int64_t g_batch, g_step, g_head;
  const int32_t* lengths;
  float* totals;          // [batch, heads, segments]: log2 decay over the segment (not walked)
  int64_t seqlen, chunks, per, segments, rows;  // rows = batch * heads * segments
  int heads, y_tiles;
};

// kWalk: leave the state before every chunk.
template <typename Elem, int C, int XP, int NY, bool kWhole, bool kWalk>
__global__ __launch_bounds__(kLaThreads, XP <= 128 ? 2 : 1) void linattn_state_kernel(StatesParams p) {
  constexpr int SB = C / 32, YT = 64 * NY;
  constexpr int XPITCH = la_pitch<Elem>(XP), YPITCH = la_pitch<Elem>(YT);
  __shared__ __attribute__((aligned(16))) Elem sX[C * XPITCH], sY[C * YPITCH];
  __shared__ __attribute__((aligned(16))) Decays<C> decays[2];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = threadIdx.x & 63, r = l & 15, g = l >> 4;
  uint32_t at = xcd_order(blockIdx.x, gridDim.x);
  const int yt = int(at % uint32_t(p.y_tiles));
  at /= uint32_t(p.y_tiles);
  const int which = at >= uint32_t(p.rows) ? 1 : 0;
  const StateParams& d = p.dir[which];
  at -= which ? uint32_t(p.rows) : 0;
  const int64_t state = at;
  const int64_t seg = at % uint32_t(p.segments);
  at /= uint32_t(p.segments);
  const int h = int(at % uint32_t(p.heads));
  const int64_t b = at / uint32_t(p.heads);
  const int y0 = yt * YT;
  const Elem* x = static_cast<const Elem*>(d.x.p) + b * d.x.batch + (h / d.x_group) * d.x.head;
  const Elem* y = static_cast<const Elem*>(d.y.p) + b * d.y.batch + (h / d.y_group) * d.y.head + y0;
  const float* gates = p.g ? p.g + b * p.g_batch + h * p.g_head : nullptr;
  const int64_t end = row_end(p.lengths, b, p.seqlen);
  const int64_t c0 = seg * p.per, c1 = c0 + p.per < p.chunks ? c0 + p.per : p.chunks, n = c1 - c0;

  const int xpad = int(linattn_pad(d.xd, 32)), ypad = int(linattn_pad(d.yd, 32));
  const int64_t floats = int64_t(xpad) * ypad, ext = (b * p.heads + h) * int64_t(d.xd) * d.yd;
  // Tile (j, m): rows x = 16 j + 4 g + i of column y = y0 + 16 (NY w + m) + r.
  la_f32x4 S[XP / 16][NY];
#pragma unroll
  for (int j = 0; j < XP / 16; ++j)
#pragma unroll
    for (int m = 0; m < NY; ++m) {
      const int yc = y0 + 16 * (NY * w + m) + r, xr = 16 * j + 4 * g;
      S[j][m] = la_f32x4{0, 0, 0, 0};
      if constexpr (kWalk) {
        if (d.starts && yc < ypad && xr < xpad)
          S[j][m] = *reinterpret_cast<const la_f32x4*>(d.starts + state * floats + int64_t(yc) * xpad + xr);
        if (d.first && yc < d.yd) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (xr + e < d.xd) S[j][m][e] = d.first[ext + int64_t(xr + e) * d.yd + yc];
        }
      }
    }
  // (without branches, so that the loads of the next chunk can be waited for without these)
  auto store = [&](float* base) {
    const Buf to(base, uint32_t(floats) * 4);
#pragma unroll
    for (int m = 0; m < NY; ++m) {
      const int yc = y0 + 16 * (NY * w + m) + r;
#pragma unroll
      for (int j = 0; j < XP / 16; ++j) {
        const int xr = 16 * j + 4 * g;
        to.store16(__builtin_bit_cast(uint4, S[j][m]), yc < ypad && xr < xpad ? uint32_t(yc * xpad + xr) * 4u : kLaOob);
      }
    }
  };
  double all = 0.0;
  // Two chunks on their way at a time: a chunk takes less time than memory to answer.
  TileLoad<Elem, C, XP, kWhole> lx[2];
  TileLoad<Elem, C, YT, kWhole> ly[2];
  constexpr uint32_t E = sizeof(Elem);
  const int y_left = d.yd - y0 < YT ? d.yd - y0 : YT;
  auto chunk = [&](int64_t i) { return d.reverse ? c1 - 1 - i : c0 + i; };
  auto rows_of = [&](int64_t i) {
    const int64_t left = i < n ? end - chunk(i) * C : 0;
    return left < 0 ? 0 : left < C ? int(left) : C;
  };
  auto fetch = [&](int64_t i, int set) {
    const int64_t t0 = chunk(i) * C;
    const int rows = rows_of(i);
    lx[set].load(x + (rows ? t0 : 0) * d.x.step, uint32_t(d.x.step) * E, rows, d.xd);
    ly[set].load(y + (rows ? t0 : 0) * d.y.step, uint32_t(d.y.step) * E, rows, y_left);
  };
  auto gate_of = [&](int64_t i) {
    const int rows = rows_of(i);
    return load_decay(gates, p.g_step, rows ? chunk(i) * C : 0, rows);
  };
  // Chunks behind the row's end leave the state as it is: the first of a reverse walk.
  int64_t i0 = 0, i1 = n;
  if (d.reverse)
    while (i0 < n && rows_of(i0) == 0) ++i0;
  else
    while (i1 > 0 && rows_of(i1 - 1) == 0) --i1;
  float gate = gate_of(i0 + 1);
  {
    const float first = gate_of(i0);
    if (w == 0 && i0 < i1) all = decays[i0 & 1].set(first);
  }
  fetch(i0, 0);
  fetch(i0 + 1, 1);
  auto step = [&](int64_t i, int set) {
    const Decays<C>& dec = decays[i & 1];
    lds_barrier();
    lx[set].store(sX);
    ly[set].store(sY);
    lds_barrier();
    // (ahead of the loads for the chunk after the next, which it would wait for)
    if (w == 0 && i + 1 < i1) all += decays[(i + 1) & 1].set(gate);
    gate = gate_of(i + 2);
    fetch(i + 2, set);
    if constexpr (kWalk) store(d.every + ((b * p.heads + h) * p.chunks + chunk(i)) * floats);
    const float total = dec.total;
    Pieces<Elem, 3> add[SB][NY];
#pragma unroll
    for (int sb = 0; sb < SB; ++sb) {
      float weight[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int s = 32 * sb + 8 * g + e;
        weight[e] = d.reverse ? dec.into[s] * d.scale : dec.onto[s];
      }
#pragma unroll
      for (int m = 0; m < NY; ++m) {
        float v[8];
        widen_frag(col_frag(sY, YPITCH, 32 * sb, 16 * (NY * w + m)), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= weight[e];
        add[sb][m].split(v);
      }
    }
#pragma unroll
    for (int j = 0; j < XP / 16; ++j)
#pragma unroll
      for (int m = 0; m < NY; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[j][m][e] *= total;
#pragma unroll
    for (int sb = 0; sb < SB; ++sb)
#pragma unroll
      for (int j4 = 0; j4 < XP / 16; j4 += 4) {
        Frag<Elem> f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = col_frag(sX, XPITCH, 32 * sb, 16 * (j4 + j));
#pragma unroll
        for (int m = 0; m < NY; ++m)
#pragma unroll
          for (int e = add[sb][m].kCount - 1; e >= 0; --e)
#pragma unroll
            for (int j = 0; j < 4; ++j) S[j4 + j][m] = mma(f[j], piece(add[sb][m], e), S[j4 + j][m]);
      }
  };
  for (int64_t i = i0; i < i1; i += 2) {
    step(i, 0);
    if (i + 1 < i1) step(i + 1, 1);
  }
  if constexpr (!kWalk) store(d.states + state * floats);
  if (!kWalk && which == 0 && yt == 0 && threadIdx.x == 0) p.totals[state] = float(all);
  if (kWalk && d.last && seg == (d.reverse ? 0 : p.segments - 1)) {
#pragma unroll
    for (int m = 0; m < NY; ++m) {
      const int yc = y0 + 16 * (NY * w + m) + r;
#pragma unroll
      for (int j = 0; j < XP / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int xr = 16 * j + 4 * g + e;
          if (yc < d.yd && xr < d.xd) d.last[ext + int64_t(xr) * d.yd + yc] = S[j][m][e];
        }
    }
  }
}

// ---------------------------------------------------------------- the states at segments' starts

// In place, over the segments of a (batch row, head) in order: each state is exchanged for the one
// before it (forward: the state at the segment's start; reverse: the adjoint behind the
// segment). Four values a thread, loads eight segments ahead of the sums.
struct JoinDir {
  float* states;
  const float* first;   // nullable: [batch, heads, dv, dk]
  float* last;          // nullable: the same
  bool reverse;
};
struct JoinParams {
  JoinDir dir[2];
  const float* totals;
  int64_t segments, state_floats;
  int cols;                     // of a stored row, padded
  int row_count, col_count;     // without padding
  int64_t row_stride, col_stride;  // of `first` and `last`
  int64_t ext_floats;
  int64_t blocks;                  // workgroups of a head
};

__global__ __launch_bounds__(256) void linattn_join_kernel(JoinParams p) {
  const JoinDir& d = p.dir[blockIdx.y];
  const int64_t head = blockIdx.x / uint32_t(p.blocks);
  const int64_t at = (int64_t(blockIdx.x % uint32_t(p.blocks)) * 256 + threadIdx.x) * 4;
  if (at >= p.state_floats) return;
  const int row = int(at / p.cols), col = int(at % p.cols);
  float* base = d.states + head * p.segments * p.state_floats + at;
  const float* totals = p.totals + head * p.segments;
  const bool in = row < p.row_count;
  const int64_t ext = head * p.ext_floats + row * p.row_stride + col * p.col_stride;
  float s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = d.first && in && col + i < p.col_count ? d.first[ext + i * p.col_stride] : 0.0f;
  constexpr int kAhead = 8;
  for (int64_t n = 0; n < p.segments; n += kAhead) {
    la_f32x4 add[kAhead];
    float total[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t m = n + i < p.segments ? n + i : p.segments - 1, seg = d.reverse ? p.segments - 1 - m : m;
      add[i] = *reinterpret_cast<const la_f32x4*>(base + seg * p.state_floats);
      total[i] = totals[seg];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (n + i < p.segments) {
        const int64_t seg = d.reverse ? p.segments - 1 - (n + i) : n + i;
        *reinterpret_cast<la_f32x4*>(base + seg * p.state_floats) = la_f32x4{s[0], s[1], s[2], s[3]};
        const float keep = exp2_hw(total[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = __builtin_fmaf(keep, s[e], add[i][e]);
      }
    }
  }
  if (d.last && in) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < p.col_count) d.last[ext + i * p.col_stride] = s[i];
  }
}

// ---------------------------------------------------------------- launches

template <typename Elem, int C, int XP, int NY, bool kWalk>
void run_states(const StatesParams& p, int dirs, bool whole, hipStream_t s) {
  const dim3 grid{uint32_t(p.rows * p.y_tiles * dirs)}, block{kLaThreads};
  if (whole) hipLaunchKernelGGL((linattn_state_kernel<Elem, C, XP, NY, true, kWalk>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((linattn_state_kernel<Elem, C, XP, NY, false, kWalk>), grid, block, 0, s, p);
}

// 64 columns a workgroup where the state is walked (more workgroups) or has more than 128 rows (for want
// of registers), else up to 128.
template <typename Elem, int C, bool kWalk>
void run_states_of(StatesParams& p, int dirs, bool whole, hipStream_t s) {
  const int xd = p.dir[0].xd, yd = p.dir[0].yd, ny = kWalk || (p.per > 1 && dirs > 1) || yd <= 64 || xd > 128 ? 1 : 2;
  p.y_tiles = (yd + 64 * ny - 1) / (64 * ny);
  if (ny == 1) {
    if (xd <= 64) return run_states<Elem, C, 64, 1, kWalk>(p, dirs, whole, s);
    if (xd <= 128) return run_states<Elem, C, 128, 1, kWalk>(p, dirs, whole, s);
    return run_states<Elem, C, 256, 1, kWalk>(p, dirs, whole, s);
  }
  if constexpr (!kWalk) {
    if (xd <= 64) return run_states<Elem, C, 64, 2, false>(p, dirs, whole, s);
    run_states<Elem, C, 128, 2, false>(p, dirs, whole, s);
  }
}

// Chunks of c steps.
template <bool kWalk>
int run_all_states(StatesParams& p, int dirs, Io io, int c, bool whole, hipStream_t s) {
  if (io == Io::F32) run_states_of<float, 32, kWalk>(p, dirs, whole, s);
  else if (c == 64) run_states_of<uint16_t, 64, kWalk>(p, dirs, whole, s);
  else run_states_of<uint16_t, 32, kWalk>(p, dirs, whole, s);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

template <typename Elem, int KP, int NV>
void run_fwd_kernel(const FwdParams& p, int64_t groups, bool whole, hipStream_t s) {
  const dim3 grid{uint32_t(groups)}, block{kLaThreads};
  if (whole) hipLaunchKernelGGL((linattn_fwd_kernel<Elem, KP, NV, true>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((linattn_fwd_kernel<Elem, KP, NV, false>), grid, block, 0, s, p);
}

template <typename Elem>
void run_fwd(const FwdParams& p, int64_t groups, bool whole, hipStream_t s) {
  if (linattn_value_tile(p.dk, p.dv) == 64) {
    if (p.dk <= 64) return run_fwd_kernel<Elem, 64, 1>(p, groups, whole, s);
    if (p.dk <= 128) return run_fwd_kernel<Elem, 128, 1>(p, groups, whole, s);
    return run_fwd_kernel<Elem, 256, 1>(p, groups, whole, s);
  }
  if (p.dk <= 64) return run_fwd_kernel<Elem, 64, 2>(p, groups, whole, s);
  run_fwd_kernel<Elem, 128, 2>(p, groups, whole, s);
}

}  // namespace

// Both directions' states of every chunk, for the backward, as [dk][dv]: the states at the chunks'
// starts and the adjoints behind them (linattn_bwd_states says how and where).
int launch_linattn_chunk_states(const LinattnArgs& a, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const LinattnBwdStates st = linattn_bwd_states(a.batch, a.heads, a.dk, a.dv, a.seqlen, a.io);
  const int c = linattn_bwd_chunk(a.io, a.dk, a.dv), group = int(a.heads / a.qk_heads);
  const bool whole = linattn_whole(a, true);
  float *states = a.workspace, *adjoints = states + st.chunk_rows * st.floats;
  if (a.batch == 0) return 0;
  StatesParams p{};
  p.g = a.g;
  p.g_batch = a.g_batch, p.g_step = a.g_step, p.g_head = a.g_head;
  p.lengths = a.lengths;
  p.seqlen = a.seqlen, p.chunks = st.chunks, p.heads = int(a.heads);
  auto dir = [&](bool reverse) {
    StateParams d{};
    d.x = reverse ? a.dout : a.v;
    d.y = reverse ? a.q : a.k;
    d.x_group = 1, d.y_group = group;
    d.xd = int(a.dv), d.yd = int(a.dk);
    d.reverse = reverse;
    d.scale = reverse ? a.scale : 1.0f;
    return d;
  };
  JoinParams j{};
  j.state_floats = st.floats;
  j.cols = int(linattn_pad(a.dv, 32));
  j.row_count = int(a.dk), j.col_count = int(a.dv);
  j.row_stride = 1, j.col_stride = a.dk, j.ext_floats = a.dk * a.dv;
  j.blocks = linattn_join_blocks(st.floats);
  auto join = [&] {
    hipLaunchKernelGGL(linattn_join_kernel, dim3(uint32_t(j.blocks * a.batch * a.heads), 2), dim3(256), 0, s, j);
    return hipGetLastError() == hipSuccess ? 0 : -1;
  };
  // What each chunk, or segment, adds to the states: into `local`, the adjoints behind the states.
  auto add = [&](int64_t per, int64_t count, float* local, float* totals) {
    p.dir[0] = dir(false), p.dir[1] = dir(true);
    p.rows = a.batch * a.heads * count;
    p.per = per, p.segments = count;
    p.dir[0].states = local, p.dir[1].states = local + p.rows * st.floats;
    p.totals = totals;
    return run_all_states<false>(p, 2, a.io, c, whole, s);
  };
  if (!st.walked) {
    float* totals = adjoints + st.chunk_rows * st.floats;
    if (st.chunks > 0 && add(1, st.chunks, states, totals) != 0) return -1;
    j.totals = totals, j.segments = st.chunks;
    j.dir[0] = JoinDir{states, a.initial, nullptr, false};
    j.dir[1] = JoinDir{adjoints, a.dfinal, a.dinitial, true};
    return join();
  }
  const int64_t per = st.segments.per, count = st.segments.count;
  float* local = states + st.chunk_rows * (2 * st.floats + 4);
  if (count > 1) {
    float* totals = local + 2 * st.segment_rows * st.floats;
    if (add(per, count, local, totals) != 0) return -1;
    j.totals = totals, j.segments = count;
    j.dir[0] = JoinDir{local, a.initial, nullptr, false};
    j.dir[1] = JoinDir{local + st.segment_rows * st.floats, a.dfinal, nullptr, true};
    if (join() != 0) return -1;
  }
  p.dir[0] = dir(false), p.dir[1] = dir(true);
  p.rows = a.batch * a.heads * count;
  p.per = per, p.segments = count;
  p.totals = nullptr;
  p.dir[0].every = states, p.dir[1].every = adjoints;
  if (count > 1) {
    p.dir[0].starts = local;
    p.dir[1].starts = local + st.segment_rows * st.floats;
  } else {
    p.dir[0].first = a.initial;
    p.dir[1].first = a.dfinal;
  }
  p.dir[1].last = a.dinitial;
  return run_all_states<true>(p, 2, a.io, c, whole, s);
}

int launch_linattn_fwd(const LinattnArgs& a, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const LinattnSegments seg = linattn_segments(a.batch, a.heads, a.dk, a.dv, a.seqlen, a.io);
  const int64_t floats = linattn_state_floats(a.dv, a.dk), rows = a.batch * a.heads * seg.count;
  const int group = int(a.heads / a.qk_heads);
  const bool whole = linattn_whole(a, false);
  if (seg.count > 1) {
    StatesParams p{};
    p.dir[0] = StateParams{a.k, a.v, group, 1, int(a.dk), int(a.dv), false, 1.0f, a.workspace,
                           nullptr, nullptr, nullptr, nullptr};
    p.g = a.g;
    p.g_batch = a.g_batch, p.g_step = a.g_step, p.g_head = a.g_head;
    p.lengths = a.lengths;
    p.totals = a.workspace + rows * floats;
    p.seqlen = a.seqlen, p.chunks = seg.chunks, p.per = seg.per, p.segments = seg.count, p.rows = rows;
    p.heads = int(a.heads);
    if (run_all_states<false>(p, 1, a.io, linattn_chunk(a.io), whole, s) != 0) return -1;
    JoinParams j{};
    j.dir[0] = JoinDir{a.workspace, a.initial, nullptr, false};
    j.totals = p.totals;
    j.segments = seg.count, j.state_floats = floats;
    j.cols = int(linattn_pad(a.dk, 32));
    j.row_count = int(a.dv), j.col_count = int(a.dk);
    j.row_stride = a.dk, j.col_stride = 1, j.ext_floats = a.dk * a.dv;
    j.blocks = linattn_join_blocks(floats);
    hipLaunchKernelGGL(linattn_join_kernel, dim3(uint32_t(j.blocks * a.batch * a.heads)), dim3(256), 0, s, j);
    if (hipGetLastError() != hipSuccess) return -1;
  }
  FwdParams p{};
  p.q = a.q, p.k = a.k, p.v = a.v;
  p.g = a.g;
  p.g_batch = a.g_batch, p.g_step = a.g_step, p.g_head = a.g_head;
  p.initial = a.initial;
  p.lengths = a.lengths;
  p.out = a.out;
  p.final_state = a.final_state;
  p.states = seg.count > 1 ? a.workspace : nullptr;
  p.seqlen = a.seqlen, p.chunks = seg.chunks, p.per = seg.per, p.segments = seg.count;
  p.kpad = linattn_pad(a.dk, 32), p.state_floats = floats;
  p.heads = int(a.heads), p.group = group, p.dk = int(a.dk), p.dv = int(a.dv);
  p.value_tiles = int(linattn_value_tiles(a.dk, a.dv));
  p.scale = a.scale;
  if (a.io == Io::BF16) run_fwd<uint16_t>(p, rows * p.value_tiles, whole, s);
  else run_fwd<float>(p, rows * p.value_tiles, whole, s);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace ssm
