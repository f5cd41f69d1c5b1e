// Internal interface between the C-ABI layer of the operators around the scan (conv_api.cpp,
// step_api.cpp, norm_api.cpp) and their kernels. Not installed; the public ABI is
// include/ssm_conv.h, ssm_step.h and ssm_norm.h.
#pragma once
#include <stdint.h>

#include <initializer_list>

#include "scan_launch.h"

namespace ssm {

// Element strides of a [batch, dim, seqlen] array.
struct Strides {
  int64_t batch, channel, step;
};

// Which of a tensor's axes is contiguous in memory. Time: runs of steps of one channel (what
// the scan takes); Channel: runs of channels of one step (a projection's output).
enum class Order : int { Time = 0, Channel = 1 };

// A HIP launch takes fewer than 2^32 work-items along an axis of its grid; the C-ABI layer refuses
// what would need more.
inline bool grid_fits(int64_t workgroups, int64_t threads) {
  return workgroups <= ((int64_t(1) << 32) - 1) / threads;
}

// Columns and slices of rows that a workgroup of the gradients' second launches sums.
constexpr int kReduceCols = 32;
constexpr int kConvReduceSlices = 16;
constexpr int kNormReduceSlices = 32;
inline int64_t reduce_groups(int64_t cols) { return (cols + kReduceCols - 1) / kReduceCols; }

// ---------------------------------------------------------------- short causal convolution

constexpr int kConvMinWidth = 2;
constexpr int kConvMaxWidth = 4;
// Steps per lane.
constexpr int kConvSteps = 8;
// Waves per workgroup.
constexpr int kConvWaves = 4;

// Everything a convolution launch needs, already validated by the C-ABI layer.
struct ConvArgs {
  const void* x;
  Strides xs;
  Order order;              // of x and dx
  const float* weight;      // [dim, width]
  const float* bias;        // nullable
  const void* initial;      // nullable: [batch, dim, width - 1]
  const int32_t* lengths;   // nullable: [batch]
  void* out;                // [batch, dim, seqlen]
  void* final_state;        // nullable: [batch, dim, width - 1]
  // backward
  const void* dout;         // [batch, dim, seqlen]
  const void* dfinal;       // nullable
  void* dx;
  Strides dxs;
  float* dweight;
  float* dbias;             // nullable
  void* dinitial;           // nullable
  float* workspace;         // conv_partials(...) x dim x (width + 1) floats
  int64_t batch, dim, width, seqlen;
  Io io;
  bool silu;
};

// Lanes along one row in the time-ordered kernels: the power of two, at most a wave, that
// covers the row with kConvSteps steps per lane.
inline int conv_row_lanes_log2(int64_t seqlen) {
  int lg = 0;
  while (lg < 6 && (int64_t(kConvSteps) << lg) < seqlen) ++lg;
  return lg;
}

// Channels a wave of the channel-ordered kernels covers.
constexpr int kConvWaveChannels = 64;

// Channels per lane of the channel-ordered kernels.
constexpr int kConvLaneChannels = 4;

// Steps one workgroup of the channel-ordered kernels covers (its waves lie along time).
constexpr int64_t kConvChannelTileSteps =
    int64_t(kConvSteps) * (64 * kConvLaneChannels / kConvWaveChannels) * kConvWaves;

// Consecutive tiles of a row that a wave of the time-ordered forward takes: two in bf16, for half the
// index arithmetic, by which bf16 is bound, once a row has two and one a wave gives twice the
// waves the device holds at a time. b4, 2304 channels, 2048 steps: 15.4 us against 16.9 (four
// tiles 17.9); b4, 3328 channels, 1536 steps (three tiles) 19.6 and 20.1; but b4, 4096 channels,
// 512 steps (one) 11.3 and 9.3; b16, 6000 channels, 100 steps 17.5 and 13.6. Few waves (b5, 523
// channels, 777 steps): 5.8 and 5.2. fp32, which memory binds (1536 channels, 65536 steps): 152
// and 147.
inline int conv_fwd_wave_tiles(int64_t batch, int64_t dim, int64_t seqlen, Io io) {
  const int lg = conv_row_lanes_log2(seqlen);
  const int64_t tile = int64_t(kConvSteps) << lg;
  const int64_t waves = batch * dim * ((seqlen + tile - 1) / tile) >> (6 - lg);
  return io == Io::BF16 && seqlen > tile && waves >= 16384 ? 2 : 1;
}

// Tiles of one row that one wave of the time-ordered backward walks.
constexpr int kConvBwdTiles = 4;

// The grid of a convolution's launch along its first axis (the second is the batch row): the runs of
// `run` steps of a row, and workgroups of 64 * kConvWaves lanes.
struct ConvGrid {
  int64_t tiles, waves, groups;
};

// Time order, `wave_tiles` tiles of a row per wave.
inline ConvGrid conv_time_grid(int64_t dim, int64_t seqlen, int wave_tiles) {
  const int lg = conv_row_lanes_log2(seqlen);
  const int64_t run = (int64_t(kConvSteps) << lg) * wave_tiles, rows = int64_t(1) << (6 - lg);
  ConvGrid g;
  g.tiles = seqlen > 0 ? (seqlen + run - 1) / run : 1;
  g.waves = (dim + rows - 1) / rows * g.tiles;
  g.groups = (g.waves + kConvWaves - 1) / kConvWaves;
  return g;
}

inline ConvGrid conv_chan_grid(int64_t dim, int64_t seqlen) {
  ConvGrid g;
  g.tiles = (seqlen + kConvChannelTileSteps - 1) / kConvChannelTileSteps;
  g.groups = g.tiles * ((dim + kConvWaveChannels - 1) / kConvWaveChannels);
  g.waves = g.groups * kConvWaves;
  return g;
}

// Partial sums of dweight and dbias per channel: one per batch row and run of steps.
inline int64_t conv_partials(int64_t batch, int64_t seqlen, Order order) {
  const int64_t run = order == Order::Channel
                          ? kConvChannelTileSteps
                          : int64_t(kConvBwdTiles) * (int64_t(kConvSteps) << conv_row_lanes_log2(seqlen));
  return batch * (seqlen > 0 ? seqlen / run + (seqlen % run != 0) : 1);
}

int launch_conv_fwd(const ConvArgs& a, void* stream);
int launch_conv_bwd(const ConvArgs& a, void* stream);

struct ConvStepArgs {
  const void* x;            // [batch, dim], rows x_stride apart
  int64_t x_stride;
  void* state;              // [nslots, dim, width - 1]
  const float* weight;
  const float* bias;        // nullable
  const int32_t* slots;     // nullable: row i is slot i
  void* out;                // [batch, dim]
  int64_t batch, nslots, dim, width;
  Io io;
  bool silu;
};
// Rows a lane takes: two once the rows fill the device's 8192 wave slots, one before that. 384 rows
// of 4352 bf16 channels: 9.6 us with one row, 8.8 with two, 10.2 with four; 8 rows of 2304:
// 2.9 us with one.
inline int conv_step_rows(int64_t batch, int64_t dim, Io io) {
  return (dim * (io == Io::BF16 ? 2 : 4) / 256 + 1) * batch > 8192 ? 2 : 1;
}

int launch_conv_step(const ConvStepArgs& a, void* stream);

// ---------------------------------------------------------------- single-token state step

// One step of the recurrence for `batch` rows against a cache of states. headdim 0: Mamba-1
// (A [dim, dstate], dt and dt_bias per channel); else Mamba-2 (A, dt and dt_bias per head of
// headdim channels).
struct StepArgs {
  const void* x;            // [batch, dim], rows x_stride apart; likewise dt, B, C, z
  const void* dt;
  const void* B;
  const void* C;
  const void* z;            // nullable
  int64_t x_stride, dt_stride, b_stride, c_stride, z_stride;
  const float* A;
  const float* D;           // nullable
  const float* dt_bias;     // nullable
  float* state;             // [nslots, dim, dstate]
  const int32_t* slots;     // nullable
  void* out;                // [batch, dim]
  int64_t batch, nslots, dim, dstate, headdim;
  Io io;
  bool softplus;
};
constexpr int64_t kStepMaxState = 256;
constexpr int kStepWaves = 4;

// Lanes of a channel: four states each, a power of two.
inline int step_lanes_log2(int64_t dstate) {
  int lg = 0;
  while ((int64_t(4) << lg) < dstate) ++lg;
  return lg;
}

// Channels a lane may hold (its wave has a lane for each), and those of small calls.
constexpr int step_most_channels(int lg) { return (1 << lg) < 8 ? (1 << lg) : 8; }
constexpr int step_few_channels(int lg) { return step_most_channels(lg) < 2 ? 1 : 2; }

// Eight channels per lane (fewer where a wave has no lane per channel) while that leaves a wave
// for every slot of the device, 8192; two below, for more waves. Mamba-2, 64 heads x 64, 128
// states, 256 rows, all through the caches: 197 us with eight channels, 205 with four, 284 with
// two, 200 with sixteen; 32 heads, 8 rows take 5.0 us with two (as with four, 7.9 with one).
// States of 128 MiB or more, half of what holds the last call's, go past the caches, which they
// would fill for nothing: those 256 rows then take 179 us, 6.0 TB/s (a copy of as much: 5.2).
// With three caches in turn, us, past and through: Mamba-1 256 rows of 4096 channels, 64 states
// 107 and 164, 512 rows, 16 states 60 and 85, Mamba-2 256 rows, 64 heads x 64, 64 states 96 and
// 107; but of 64 MiB, 256 rows of 4096 channels, 16 states, 40 and 32.
struct StepForm {
  int channels;
  bool past_caches;
  int64_t groups;  // along the grid's first axis (the second is the row)
};
inline StepForm step_form(int64_t batch, int64_t dim, int64_t dstate) {
  const int lg = step_lanes_log2(dstate), most = step_most_channels(lg), per_wave = 64 >> lg;
  const bool many = dim * batch / (most * per_wave) >= 8192;
  StepForm f{many ? most : step_few_channels(lg), many && batch * dim * dstate * 4 >= (int64_t(1) << 27), 0};
  const int64_t per = int64_t(kStepWaves) * f.channels * per_wave;
  f.groups = (dim + per - 1) / per;
  return f;
}

int launch_state_step(const StepArgs& a, void* stream);

// ---------------------------------------------------------------- gated RMS norm

// A tensor of [batch, dim, seqlen] values in either memory order.
struct View {
  const void* p;  // written through for outputs
  Strides s;
  Order order;
};

struct NormArgs {
  View y, z, out;           // z.p nullable (no gate)
  const float* weight;      // [dim]
  float* rstd;              // of every token and group: forward nullable, written; backward read
  Strides rs;               // of rstd, with the group in the place of the channel
  float eps;
  // backward (out unused)
  View dout, dy, dz;        // dz.p required when z is given
  float* dweight;           // [dim]
  float* workspace;         // backward: norm_partials(...) x dim floats; then, split, the blocks'
                            // sums: batch x groups x cblocks x seqlen floats
  int64_t batch, dim, groups, seqlen;
  Io io;
  bool norm_first;
};

// How a launch covers the tensors: a lane holds 16 bytes of channels by `steps` steps;
// 2^lanes_log2 lanes of a wave lie along the channels of one group, the others along time;
// `waves` waves of a workgroup along the channels. A workgroup covers a whole group, or, split,
// one of the group's `cblocks` blocks of channels.
struct NormShape {
  int steps, lanes_log2, waves;
  int64_t cblocks, tiles;    // tiles: workgroups along time
  bool split;
};

// all_channel: every tensor has its channels contiguous. dword_rows: every row of steps of the
// others (forward: of the result, if it is one) starts at a multiple of four bytes.
struct NormOrders {
  bool all_channel, dword_rows;
};

// Steps of a lane by storage type (Io), where some tensor has its steps contiguous.
constexpr int kNormFwdSteps[2] = {4, 8};
constexpr int kNormBwdSteps[2] = {4, 4};
// Most waves of a workgroup; waves of a split one, and its lanes along channels (8, with 8 along
// time).
constexpr int kNormMostWaves = 16;
constexpr int kNormSplitWaves = 4;
constexpr int kNormSplitLanes = 3;

// A group of g channels whole. Lanes along channels: all that the group has work for, then fewer,
// down to eight, while `good` waves still cover the group and the sequence has steps for the
// lanes freed. More than the most waves: not to be launched.
inline NormShape norm_whole_shape(int64_t g, int64_t seqlen, Io io, int steps, int good) {
  const int64_t cv = io == Io::BF16 ? 8 : 4;
  NormShape s{steps, 0, 0, 1, 0, false};
  int lg = 0;
  while (lg < 6 && (cv << lg) < g) ++lg;
  while (steps > 1 && lg > 3 && (g + (cv << (lg - 1)) - 1) / (cv << (lg - 1)) <= good &&
         int64_t(steps) * (64 >> lg) < seqlen)
    --lg;
  s.lanes_log2 = lg;
  const int64_t w = (g + (cv << lg) - 1) / (cv << lg), run = int64_t(steps) * (64 >> lg);
  s.waves = int(w <= kNormMostWaves ? w : kNormMostWaves + 1);
  s.tiles = seqlen / run + (seqlen % run != 0);
  return s;
}

inline NormShape norm_split_shape(int64_t g, int64_t seqlen, Io io, int steps) {
  const int64_t cv = io == Io::BF16 ? 8 : 4, wave = cv << kNormSplitLanes;
  const int64_t run = int64_t(steps) * (64 >> kNormSplitLanes), w = (g + wave - 1) / wave;
  NormShape s{steps, kNormSplitLanes, int(w < kNormSplitWaves ? w : kNormSplitWaves), 0, 0, true};
  s.cblocks = (w + s.waves - 1) / s.waves;
  s.tiles = seqlen / run + (seqlen % run != 0);
  return s;
}

// Bytes that a workgroup reads on end of a channel whose steps are contiguous.
inline int64_t norm_run_bytes(const NormShape& s, Io io) {
  return int64_t(s.steps) * (64 >> s.lanes_log2) * (io == Io::BF16 ? 2 : 4);
}

// all_channel: a lane holds one step. Else eight steps (bf16): b4, 2048 channels, 2048 steps
// take 20 us with eight waves a workgroup (100 MB: 5.1 TB/s), 21.8 with four, 21 with sixteen,
// and 21.4 with four steps a lane. Sixteen waves where eight would read less than 32 bytes on
// end, if that leaves workgroups for most CUs: b4, 2048 channels, 2048 steps, fp32, all tensors
// so ordered, 57 and 41 us; b4, 4096 channels, 2048 steps, bf16, 57 and 43 (but b1, 4096
// channels, 1024 steps, 64 workgroups, 11 and 15). Split where a group does not fit, and where a
// workgroup would write 16 bytes on end of a result at odd addresses: b1, 4096 channels, 1023
// steps, 27 us whole and 19 split; with the result in channel order 13 and 18.
inline NormShape norm_fwd_shape(int64_t batch, int64_t dim, int64_t groups, int64_t seqlen, Io io,
                                NormOrders o) {
  const int steps = kNormFwdSteps[int(io)];
  NormShape s = norm_whole_shape(dim / groups, seqlen, io, o.all_channel ? 1 : steps, 8);
  if (!o.all_channel && norm_run_bytes(s, io) < 32) {
    const NormShape more = norm_whole_shape(dim / groups, seqlen, io, steps, kNormMostWaves);
    if (more.tiles * groups * batch >= 192 && norm_run_bytes(more, io) >= 32) s = more;
  }
  const bool split = s.waves > kNormMostWaves ||
                     (!o.all_channel && !o.dword_rows && norm_run_bytes(s, io) < 32 && seqlen > steps);
  return split ? norm_split_shape(dim / groups, seqlen, io, steps) : s;
}

// The backward takes squares of channels by steps whatever the orders (a lane of one step would
// leave a partial sum of dweight per token). With the channels contiguous throughout eight
// waves a workgroup are best (two workgroups a CU); a tensor with steps contiguous wants more
// steps in a workgroup: b4, 2048 channels, 2048 steps, bf16, y so ordered 51 us with eight
// waves, 44 with sixteen; none so ordered 33 and 39. Split where such a tensor's channels would
// be read by less than 32 bytes on end (b1, 2722 channels, 2920 steps: 46 us whole, 40 split;
// b8, 8192 channels, 512 steps: 141 and 105; b4, 2048 channels, 2048 steps: 41 and 53), or the
// workgroups are a quarter of the CUs (b1, 2048 channels, 512 steps: 16.5 and 14.2).
inline NormShape norm_bwd_shape(int64_t batch, int64_t dim, int64_t groups, int64_t seqlen, Io io,
                                NormOrders o) {
  const int steps = kNormBwdSteps[int(io)];
  const NormShape s = norm_whole_shape(dim / groups, seqlen, io, steps, o.all_channel ? 8 : 16);
  const bool split = s.waves > kNormMostWaves ||
                     (!o.all_channel && seqlen > steps &&
                      (norm_run_bytes(s, io) < 32 || (s.tiles * groups * batch < 64 && s.waves > kNormSplitWaves)));
  return split ? norm_split_shape(dim / groups, seqlen, io, steps) : s;
}

// The tensors of a launch, for the choice of its shape.
inline NormOrders norm_orders(const NormArgs& a, std::initializer_list<const View*> views) {
  NormOrders o{true, true};
  const int64_t esz = a.io == Io::BF16 ? 2 : 4;
  for (const View* v : views) {
    if (!v->p || v->order == Order::Channel) continue;
    o.all_channel = false;
    if (reinterpret_cast<uintptr_t>(v->p) % 4 || v->s.channel * esz % 4 || (a.batch > 1 && v->s.batch * esz % 4))
      o.dword_rows = false;
  }
  return o;
}

inline NormShape norm_fwd_shape(const NormArgs& a) {
  const NormOrders all = norm_orders(a, {&a.y, &a.z, &a.out}), result = norm_orders(a, {&a.out});
  return norm_fwd_shape(a.batch, a.dim, a.groups, a.seqlen, a.io, {all.all_channel, result.dword_rows});
}

inline NormShape norm_bwd_shape(const NormArgs& a) {
  return norm_bwd_shape(a.batch, a.dim, a.groups, a.seqlen, a.io,
                        norm_orders(a, {&a.y, &a.z, &a.dout, &a.dy, &a.dz}));
}

inline bool norm_fits(const NormArgs& a, const NormShape& s) {
  return grid_fits(s.tiles * s.cblocks * a.groups * a.batch, 64 * s.waves);
}

// Partial sums of dweight per channel: one per batch row and tile of steps.
inline int64_t norm_partials(int64_t batch, const NormShape& s) { return batch * s.tiles; }

int launch_norm_fwd(const NormArgs& a, void* stream);
int launch_norm_bwd(const NormArgs& a, void* stream);

}  // namespace ssm
