// C-ABI entry points of the short causal convolution (declared in include/ssm_conv.h).
// Argument checking happens here, before any HIP call; the launches are in conv_kernels.hip.
#include <stdint.h>

#include "api_util.h"
#include "block_launch.h"
#include "ssm_conv.h"
#include "strided.h"

using ssm_api::aligned;
using ssm_api::check_strided;
using ssm_api::kInt32Max;
using ssm_api::mul_ok;
using ssm_api::Ranges;
using ssm_api::StridedArray;

namespace {

struct ConvSizes {
  int64_t esz, elems, edge;  // elements of x and of a state
};

// Flags, sizes and the storage type; common to the prompt's forward and backward.
int check_sizes(uint32_t flags, int64_t batch, int64_t dim, int64_t width, int64_t seqlen, ConvSizes* z) {
  if (flags & ~uint32_t(SSM_IO_MASK | SSM_CONV_SILU)) return SSM_ERR_INVALID_ARG;
  if (batch < 0 || dim < 0 || width < 0 || seqlen < 0) return SSM_ERR_INVALID_ARG;
  const uint32_t io = flags & SSM_IO_MASK;
  if (io != SSM_IO_F32 && io != SSM_IO_BF16) return SSM_ERR_UNSUPPORTED;
  if (width < ssm::kConvMinWidth || width > ssm::kConvMaxWidth) return SSM_ERR_UNSUPPORTED;
  z->esz = io == SSM_IO_BF16 ? 2 : 4;
  int64_t rows, bytes;
  if (!mul_ok(batch, dim, &rows) || rows > kInt32Max || dim > kInt32Max || batch > 65535 ||
      seqlen > kInt32Max || !mul_ok(rows, seqlen, &z->elems) || !mul_ok(z->elems, z->esz, &bytes) ||
      dim > kInt32Max / (width + 1))
    return SSM_ERR_UNSUPPORTED;
  z->edge = rows * (width - 1);
  return SSM_OK;
}

// A single step has runs of no length either way: the time-ordered kernels' lanes then lie
// along the channels.
ssm::Order order_of(const StridedArray& a, int64_t seqlen) {
  return seqlen == 1 ? ssm::Order::Time : a.order;
}

// The launches of a call within what a grid takes; the channel-ordered kernels number all their
// workgroups in 32 bits.
bool launch_fits(int64_t batch, int64_t dim, int64_t width, int64_t seqlen, ssm::Order order, ssm::Io io,
                 bool backward) {
  if (backward && !ssm::grid_fits(ssm::reduce_groups(dim * (width + 1)), ssm::kReduceCols * ssm::kConvReduceSlices))
    return false;
  const bool time = order == ssm::Order::Time || seqlen == 0;
  const int wave_tiles = backward ? ssm::kConvBwdTiles : ssm::conv_fwd_wave_tiles(batch, dim, seqlen, io);
  const ssm::ConvGrid g =
      time ? ssm::conv_time_grid(dim, seqlen, wave_tiles) : ssm::conv_chan_grid(dim, seqlen);
  int64_t all;
  return ssm::grid_fits(g.groups, 64 * ssm::kConvWaves) &&
         (time || (mul_ok(g.groups, batch, &all) && all <= kInt32Max));
}

ssm::Io io_of(uint32_t flags) { return (flags & SSM_IO_MASK) == SSM_IO_BF16 ? ssm::Io::BF16 : ssm::Io::F32; }

ssm::ConvArgs common(const void* x, const StridedArray& xa, const float* weight, const float* bias,
                     const void* initial_state, const int32_t* lengths, uint32_t flags, int64_t batch,
                     int64_t dim, int64_t width, int64_t seqlen) {
  ssm::ConvArgs a{};
  a.x = x;
  a.xs = xa.s;
  a.order = order_of(xa, seqlen);
  a.weight = weight;
  a.bias = bias;
  a.initial = initial_state;
  a.lengths = lengths;
  a.batch = batch;
  a.dim = dim;
  a.width = width;
  a.seqlen = seqlen;
  a.io = io_of(flags);
  a.silu = (flags & SSM_CONV_SILU) != 0;
  return a;
}

}  // namespace

extern "C" {

int ssm_conv_fwd(const void* x, const int64_t* x_strides, const float* weight, const float* bias,
                 const void* initial_state, const int32_t* lengths, uint32_t flags, void* out,
                 void* final_state, int64_t batch, int64_t dim, int64_t width, int64_t seqlen,
                 void* stream) {
  ConvSizes z;
  if (int st = check_sizes(flags, batch, dim, width, seqlen, &z)) return st;
  StridedArray xa;
  if (int st = check_strided(x_strides, batch, dim, seqlen, z.esz, false, &xa)) return st;
  if (!launch_fits(batch, dim, width, seqlen, order_of(xa, seqlen), io_of(flags), false)) return SSM_ERR_UNSUPPORTED;
  if ((z.elems > 0 && (!x || !out)) || (dim > 0 && !weight)) return SSM_ERR_INVALID_ARG;
  const uintptr_t e = uintptr_t(z.esz);
  if (!aligned(x, e) || !aligned(out, e) || !aligned(initial_state, e) || !aligned(final_state, e) ||
      !aligned(weight, 4) || !aligned(bias, 4) || !aligned(lengths, 4))
    return SSM_ERR_MISALIGNED;
  Ranges r;
  r.add(x, xa.bytes, false);
  r.add(weight, dim * width * 4, false);
  r.add(bias, dim * 4, false);
  r.add(initial_state, z.edge * z.esz, false);
  r.add(lengths, batch * 4, false);
  r.add(out, z.elems * z.esz, true);
  r.add(final_state, z.edge * z.esz, true);
  if (r.clash()) return SSM_ERR_INVALID_ARG;
  if (batch == 0 || dim == 0 || (seqlen == 0 && !final_state)) return SSM_OK;
  ssm::ConvArgs a = common(x, xa, weight, bias, initial_state, lengths, flags, batch, dim, width, seqlen);
  a.out = out;
  a.final_state = final_state;
  return ssm::launch_conv_fwd(a, stream) == 0 ? SSM_OK : SSM_ERR_HIP;
}

int64_t ssm_conv_bwd_workspace_bytes(int64_t batch, int64_t dim, int64_t width, int64_t seqlen,
                                     uint32_t flags) {
  const uint32_t io = flags & SSM_IO_MASK;
  if (batch < 0 || dim < 0 || seqlen < 0 || width < ssm::kConvMinWidth || width > ssm::kConvMaxWidth ||
      (io != SSM_IO_F32 && io != SSM_IO_BF16))
    return -1;
  if (seqlen > kInt32Max || batch > 65535) return -1;
  const int64_t t = ssm::conv_partials(batch, seqlen, ssm::Order::Time);
  const int64_t c = ssm::conv_partials(batch, seqlen, ssm::Order::Channel);
  int64_t row, total;
  if (!mul_ok(dim, (width + 1) * 4, &row) || !mul_ok(t > c ? t : c, row, &total)) return -1;
  return total;
}

int ssm_conv_bwd(const void* x, const int64_t* x_strides, const float* weight, const float* bias,
                 const void* initial_state, const int32_t* lengths, uint32_t flags, const void* dout,
                 const void* dfinal, void* dx, const int64_t* dx_strides, float* dweight, float* dbias,
                 void* dinitial, void* workspace, int64_t workspace_bytes, int64_t batch, int64_t dim,
                 int64_t width, int64_t seqlen, void* stream) {
  ConvSizes z;
  if (int st = check_sizes(flags, batch, dim, width, seqlen, &z)) return st;
  StridedArray xa, dxa;
  if (int st = check_strided(x_strides, batch, dim, seqlen, z.esz, false, &xa)) return st;
  if (int st = check_strided(dx_strides, batch, dim, seqlen, z.esz, true, &dxa)) return st;
  if (z.elems > 0 && order_of(xa, seqlen) != order_of(dxa, seqlen)) return SSM_ERR_UNSUPPORTED;
  if (!launch_fits(batch, dim, width, seqlen, order_of(xa, seqlen), io_of(flags), true)) return SSM_ERR_UNSUPPORTED;
  const int64_t need = ssm_conv_bwd_workspace_bytes(batch, dim, width, seqlen, flags);
  if (need < 0) return SSM_ERR_UNSUPPORTED;
  if ((z.elems > 0 && (!x || !dout || !dx)) || (dim > 0 && (!weight || !dweight))) return SSM_ERR_INVALID_ARG;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SSM_ERR_INVALID_ARG;
  const uintptr_t e = uintptr_t(z.esz);
  if (!aligned(x, e) || !aligned(dout, e) || !aligned(dx, e) || !aligned(initial_state, e) ||
      !aligned(dfinal, e) || !aligned(dinitial, e) || !aligned(weight, 4) || !aligned(bias, 4) ||
      !aligned(lengths, 4) || !aligned(dweight, 4) || !aligned(dbias, 4) || !aligned(workspace, 256))
    return SSM_ERR_MISALIGNED;
  Ranges r;
  r.add(x, xa.bytes, false);
  r.add(weight, dim * width * 4, false);
  r.add(bias, dim * 4, false);
  r.add(initial_state, z.edge * z.esz, false);
  r.add(lengths, batch * 4, false);
  r.add(dout, z.elems * z.esz, false);
  r.add(dfinal, z.edge * z.esz, false);
  r.add(dx, dxa.bytes, true);
  r.add(dweight, dim * width * 4, true);
  r.add(dbias, dim * 4, true);
  r.add(dinitial, z.edge * z.esz, true);
  r.add(workspace, need, true);
  if (r.clash()) return SSM_ERR_INVALID_ARG;
  if (dim == 0) return SSM_OK;
  ssm::ConvArgs a = common(x, xa, weight, bias, initial_state, lengths, flags, batch, dim, width, seqlen);
  a.dout = dout;
  a.dfinal = dfinal;
  a.dx = dx;
  a.dxs = dxa.s;
  a.dweight = dweight;
  a.dbias = dbias;
  a.dinitial = dinitial;
  a.workspace = static_cast<float*>(workspace);
  return ssm::launch_conv_bwd(a, stream) == 0 ? SSM_OK : SSM_ERR_HIP;
}

int ssm_conv_step(const void* x, int64_t x_stride, void* state, const float* weight, const float* bias,
                  const int32_t* slots, uint32_t flags, void* out, int64_t batch, int64_t nslots, int64_t dim,
                  int64_t width, void* stream) {
  ConvSizes z;
  if (int st = check_sizes(flags, batch, dim, width, 1, &z)) return st;
  if (nslots < 0 || (!slots && nslots < batch)) return SSM_ERR_INVALID_ARG;
  int64_t cache, bytes, reach;
  if (nslots > kInt32Max || !mul_ok(nslots, dim, &cache) ||
      !mul_ok(cache, (width - 1) * z.esz, &bytes))
    return SSM_ERR_UNSUPPORTED;
  if (batch > 1 && x_stride < 0) return SSM_ERR_INVALID_ARG;
  if (!mul_ok(batch > 1 ? batch - 1 : 0, batch > 1 ? x_stride : 0, &reach) ||
      reach > INT64_MAX / z.esz - dim)
    return SSM_ERR_UNSUPPORTED;
  if ((z.elems > 0 && (!x || !out)) || (bytes > 0 && !state) || (dim > 0 && !weight)) return SSM_ERR_INVALID_ARG;
  const uintptr_t e = uintptr_t(z.esz);
  if (!aligned(x, e) || !aligned(out, e) || !aligned(state, e) || !aligned(weight, 4) || !aligned(bias, 4) ||
      !aligned(slots, 4))
    return SSM_ERR_MISALIGNED;
  Ranges r;
  if (z.elems > 0) r.add(x, (reach + dim) * z.esz, false);
  r.add(weight, dim * width * 4, false);
  r.add(bias, dim * 4, false);
  r.add(slots, batch * 4, false);
  r.add(out, z.elems * z.esz, true);
  r.add(state, bytes, true);
  if (r.clash()) return SSM_ERR_INVALID_ARG;
  if (batch == 0 || dim == 0) return SSM_OK;
  ssm::ConvStepArgs a{x, x_stride, state, weight, bias, slots, out, batch, nslots, dim, width,
                      io_of(flags), (flags & SSM_CONV_SILU) != 0};
  return ssm::launch_conv_step(a, stream) == 0 ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
