// Internal interface between the C-ABI layer of linear attention (linattn_api.cpp) and its
// kernels. Not installed; the public ABI is include/ssm_linattn.h.
#pragma once
#include <stdint.h>

#include "block_launch.h"

namespace ssm {

constexpr int kLinattnMaxDim = 256;  // dk and dv

// Steps of a chunk: 64, or 32 in fp32, whose tiles would not fit LDS at 256 columns otherwise.
constexpr int linattn_chunk(Io io) { return io == Io::BF16 ? 64 : 32; }
// The backward, whose four tiles and two of weights share LDS, takes 32 above 128 columns.
constexpr int linattn_bwd_chunk(Io io, int64_t dk, int64_t dv) {
  return io == Io::BF16 && dk <= 128 && dv <= 128 ? 64 : 32;
}

// A [batch, seqlen, heads, dim] array whose last axis is contiguous; element strides.
struct HeadRows {
  const void* p;
  int64_t batch, step, head;
};

struct LinattnArgs {
  HeadRows q, k, v;
  const float* g;            // nullable: log decays, strides below (0 along broadcast axes)
  int64_t g_batch, g_step, g_head;
  const float* initial;      // nullable: [batch, heads, dv, dk]
  const int32_t* lengths;    // nullable: [batch]
  void* out;                 // [batch, seqlen, heads, dv]
  float* final_state;        // nullable: [batch, heads, dv, dk]
  // backward
  HeadRows dout;
  const float* dfinal;       // nullable
  void *dq, *dk_, *dv_;      // contiguous
  float* dg;                 // nullable: [batch, seqlen, heads], or [heads] where dg_per_head
  bool dg_per_head;
  float* dinitial;           // nullable
  float* workspace;
  int64_t batch, seqlen, qk_heads, heads, dk, dv;
  float scale;
  Io io;
};

// Columns of dv that a workgroup of the forward takes: its waves keep the state of dk x that many
// in registers, with room for the operands next to it. (dk = dv = 128: 128 at a time 435 us for b1, 16 heads,
// 65536 steps and 216 for b4, 32 heads, 4096 steps; 64 at a time 504 and 245.)
constexpr int linattn_value_tile(int64_t dk, int64_t dv) { return dv <= 64 || dk > 128 ? 64 : 128; }
constexpr int64_t linattn_value_tiles(int64_t dk, int64_t dv) {
  return (dv + linattn_value_tile(dk, dv) - 1) / linattn_value_tile(dk, dv);
}
constexpr int64_t linattn_pad(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Into how many segments the sequences are cut where batch rows and heads are `base` workgroups: at
// most as many as leave all workgroups resident, two for each CU; and three at least, since the
// segments' states are a second pass over half of what the forward reads. Forward, 2048 steps of heads of
// 128 x 64, us in one segment | cut: base 128 114 | 80 in four (92 in three, 98 in six); 160 114 | 96 in three,
// 110 in four (640 workgroups); 192 113 | 131 in two; 256 115 | 138. The backward's walks, gradient in all:
// base 128 (4096 steps) 200 | 160 in four; 192 241 | 265 in two; 256 (2048 steps) 139 | 163. And only sequences of
// more than five chunks, whose walk takes as long as the two launches more. bf16, 16 heads of 128 x 128 and
// 64 of 128 x 64: 256 steps 24.0 18.3 | 26.3 28.8; 384 steps 32.5 24.9 | 29.4 30.9; 512 steps 41.6 31.3 | 31.0 32.8;
// fp32: 128 steps 31.7 21.5 | 29.3 28.6; 192 steps 43.9 29.2 | 31.4 33.4. (One number for all, by the 128 columns, which
// lose most: 64 columns, whose chunks take less time, would be 6 us faster whole at six chunks and near even at eight.)
constexpr int64_t kLinattnGroups = 512;
constexpr int64_t kLinattnWhole = 5;
inline int64_t linattn_cuts(int64_t base, int64_t chunks) {
  const int64_t want = base > 0 ? kLinattnGroups / base : 1;
  return want < 3 || chunks <= kLinattnWhole ? 1 : want < chunks ? want : chunks;
}

// How the forward cuts a sequence into segments that run side by side, each from a state that
// two small launches before it find.
struct LinattnSegments {
  int64_t chunks;   // of a row
  int64_t per;      // chunks of a segment
  int64_t count;
};
inline LinattnSegments linattn_segments(int64_t batch, int64_t heads, int64_t dk, int64_t dv, int64_t seqlen,
                                        Io io) {
  LinattnSegments s;
  const int64_t c = linattn_chunk(io);
  s.chunks = (seqlen + c - 1) / c;
  const int64_t base = batch * heads * linattn_value_tiles(dk, dv);
  const int64_t want = linattn_cuts(base, s.chunks);
  s.per = s.chunks > 0 ? (s.chunks + want - 1) / want : 1;
  s.count = s.chunks > 0 ? (s.chunks + s.per - 1) / s.per : 1;
  return s;
}

// Floats of one state in the workspace of the backward, [dk][dv], both padded so that operand
// reads stay inside.
inline int64_t linattn_state_floats(int64_t rows, int64_t cols) {
  return linattn_pad(rows, 32) * linattn_pad(cols, 32);
}

// The backward's states of every chunk. Walked: a workgroup of 64 columns of dk walks the chunks of a
// segment and leaves the state of each, from the segment's start, which is the sequence's, or is
// found by a first walk that leaves segments' states alone and the join. Else every chunk by
// itself, and the join over the chunks (all of them read and written once more), where they are
// few enough to stay in the caches and a walk would be cut. b4, 32 heads of 128 x 64, 2048 steps
// (268 MB): 126 us walked, 196 joined; b1, 16 heads of 128 x 128, 16384 steps (537 MB): 316 and 396; b3, 4
// heads of 64 x 100, 517 steps in fp32 (17 MB): 36 and 24. The whole gradient, us, walked | joined: b2, 32 heads
// of 128 x 64 (256 workgroups, not cut), 128 steps 28.0 | 33.6, 512 steps 54.3 | 62.4, fp32 86.9 | 106.9; 16 heads
// of 128 x 128, 192 steps 33.9 | 35.1, 256 steps 38.4 | 37.1, 512 steps (cut) 51.0 | 42.9.
constexpr int64_t kLinattnCached = int64_t(64) << 20;
struct LinattnBwdStates {
  bool walked;
  LinattnSegments segments;  // of the walk
  int64_t chunks, floats;
  // Workspace: states, adjoints, decays and dg sums of the chunks, then the same of the segments, in
  // floats (two more a row than those, to keep the states 16-byte aligned).
  int64_t chunk_rows, segment_rows, total;
};
inline LinattnBwdStates linattn_bwd_states(int64_t batch, int64_t heads, int64_t dk, int64_t dv, int64_t seqlen, Io io) {
  LinattnBwdStates s{};
  const int64_t c = linattn_bwd_chunk(io, dk, dv);
  s.chunks = (seqlen + c - 1) / c;
  s.floats = linattn_state_floats(dk, dv);
  s.chunk_rows = batch * heads * s.chunks;
  const int64_t base = batch * heads * 2 * ((dk + 63) / 64);
  s.walked = s.chunk_rows > 0 && (double(s.chunk_rows) * double(s.floats) * 8.0 > double(kLinattnCached) ||
                                  linattn_cuts(base, s.chunks) == 1);
  s.segments = LinattnSegments{s.chunks, s.chunks, 1};
  if (s.walked) {
    const int64_t want = linattn_cuts(base, s.chunks);
    s.segments.per = (s.chunks + want - 1) / want;
    s.segments.count = (s.chunks + s.segments.per - 1) / s.segments.per;
  }
  s.segment_rows = s.segments.count > 1 ? batch * heads * s.segments.count : 0;
  s.total = (s.chunk_rows + s.segment_rows) * (2 * s.floats + 4);
  return s;
}

inline int64_t linattn_join_blocks(int64_t state_floats) { return (state_floats / 4 + 255) / 256; }

// Rows of whole 16-byte words at 4-byte aligned addresses, those of the results too: a load a word and a store for four
// values, which a buffer makes in dwords; else each value by itself. (Results are contiguous, so that their rows
// are where their first value is.)
inline bool linattn_whole(const LinattnArgs& a, bool bwd) {
  const int64_t esz = a.io == Io::BF16 ? 2 : 4, word = 16 / esz, even = 4 / esz;
  auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; };
  auto rows = [&](const HeadRows& r) {
    return at(r.p) && r.batch % even == 0 && r.step % even == 0 && r.head % even == 0;
  };
  const bool results = bwd ? at(a.dq) && at(a.dk_) && at(a.dv_) : at(a.out);
  return a.dk % word == 0 && a.dv % word == 0 && rows(a.q) && rows(a.k) && rows(a.v) && (!bwd || rows(a.dout)) && results;
}

// Whether a chunk's rows, `step` elements apart, lie within the 32-bit byte offsets of the kernels.
inline bool linattn_reach(int64_t step, int64_t esz) { return step < (int64_t(1) << 30) / (64 * esz); }

int launch_linattn_chunk_states(const LinattnArgs& a, void* stream);
int launch_linattn_fwd(const LinattnArgs& a, void* stream);
int launch_linattn_bwd(const LinattnArgs& a, void* stream);

// ---------------------------------------------------------------- single tokens

constexpr int kLinattnStepWaves = 4;

// Rows of the state per lane, of 2^lg lanes a row (no more than a lane for each row's v): eight, for as
// many loads in flight, or four where eight would give a workgroup more rows than the head has. 32 heads of
// 128 x 64 (eight): 67 MB moved 12.7 us, 14.2 with four; 24 heads of 64 x 64 (four): 50 MB 10.2 us, 13.3 with
// eight. Two or sixteen were slower at both.
constexpr int linattn_step_most_rows(int lg) { return lg >= 3 ? 8 : 1 << lg; }
constexpr int linattn_step_less_rows(int lg) { return lg >= 3 ? 4 : 1 << lg; }

struct LinattnStepForm {
  int rows;
  int64_t tiles, groups;    // workgroups of a head, and of a batch row
};
inline LinattnStepForm linattn_step_form(int64_t heads, int64_t dk, int64_t dv) {
  const int lg = step_lanes_log2(dk), most = linattn_step_most_rows(lg), per = kLinattnStepWaves * (64 >> lg);
  LinattnStepForm f{};
  f.rows = most * per <= dv ? most : linattn_step_less_rows(lg);
  const int64_t tile = int64_t(f.rows) * per;
  f.tiles = (dv + tile - 1) / tile;
  f.groups = f.tiles * heads;
  return f;
}

struct LinattnStepArgs {
  HeadRows q, k, v;          // (no step axis)
  const float* g;            // nullable
  int64_t g_batch, g_head;
  float* state;              // [nslots, heads, dv, dk]
  const int32_t* slots;      // nullable
  void* out;                 // [batch, heads, dv]
  int64_t batch, nslots, qk_heads, heads, dk, dv;
  float scale;
  Io io;
};
int launch_linattn_step(const LinattnStepArgs& a, void* stream);

}  // namespace ssm
