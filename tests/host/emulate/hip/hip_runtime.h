// Stands in for the HIP runtime where a kernel of csrc/ is compiled for the CPU by a host test: each
// lane of a workgroup is a thread, a workgroup runs after the other, LDS is static memory, and
// lanes exchange values at barriers of their wave or workgroup. For kernels whose lanes reach the
// same barriers and exchanges unless they have returned.
#pragma once
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <barrier>
#include <memory>
#include <thread>
#include <vector>

#define __global__
#define __device__
#define __forceinline__ inline
#define __launch_bounds__(...)
#define __shared__ static

struct uint4 {
  uint32_t x, y, z, w;
};
inline uint4 make_uint4(uint32_t x, uint32_t y, uint32_t z, uint32_t w) { return {x, y, z, w}; }
struct dim3 {
  unsigned x, y, z;
  dim3(unsigned a = 1, unsigned b = 1, unsigned c = 1) : x(a), y(b), z(c) {}
};
typedef void* hipStream_t;
inline int hipGetLastError() { return 0; }

inline float __uint_as_float(uint32_t v) { return __builtin_bit_cast(float, v); }
inline uint32_t __float_as_uint(float v) { return __builtin_bit_cast(uint32_t, v); }
inline float __int_as_float(int v) { return __builtin_bit_cast(float, v); }
inline int __float_as_int(float v) { return __builtin_bit_cast(int, v); }

namespace emulate {
struct Group {
  std::barrier<> all;
  std::vector<std::unique_ptr<std::barrier<>>> wave;
  uint32_t lanes[16][64];
  explicit Group(int threads) : all(threads) {
    for (int i = 0; i < threads / 64; ++i) wave.push_back(std::make_unique<std::barrier<>>(64));
  }
};
inline thread_local Group* group;
inline thread_local dim3 thread_idx, block_idx, grid_dim, block_dim;

// The value of lane `from` of this lane's wave (its own where there is none).
template <typename T>
T exchange(T v, int from) {
  static_assert(sizeof(T) == 4);
  const int w = int(thread_idx.x / 64), lane = int(thread_idx.x % 64);
  memcpy(&group->lanes[w][lane], &v, 4);
  group->wave[w]->arrive_and_wait();
  T r;
  memcpy(&r, &group->lanes[w][from < 0 || from > 63 ? lane : from], 4);
  group->wave[w]->arrive_and_wait();
  return r;
}

template <typename F>
void launch(dim3 grid, dim3 block, F kernel) {
  for (unsigned y = 0; y < grid.y; ++y)
    for (unsigned x = 0; x < grid.x; ++x) {
      Group g(int(block.x));
      std::vector<std::thread> lanes;
      for (unsigned t = 0; t < block.x; ++t)
        lanes.emplace_back([&, t] {
          group = &g;
          thread_idx = dim3(t);
          block_idx = dim3(x, y);
          grid_dim = grid;
          block_dim = block;
          kernel();
          g.wave[t / 64]->arrive_and_drop();
          g.all.arrive_and_drop();
        });
      for (std::thread& l : lanes) l.join();
    }
}
}  // namespace emulate

#define threadIdx emulate::thread_idx
#define blockIdx emulate::block_idx
#define gridDim emulate::grid_dim
#define blockDim emulate::block_dim
#define hipLaunchKernelGGL(kernel, grid, block, lds, stream, ...) \
  emulate::launch(grid, block, [=] { kernel(__VA_ARGS__); })

inline void __syncthreads() { emulate::group->all.arrive_and_wait(); }
template <typename T>
T __shfl(T v, int from, int) {
  return emulate::exchange(v, from);
}
template <typename T>
T __shfl_xor(T v, int m, int) {
  return emulate::exchange(v, int(threadIdx.x % 64) ^ m);
}
template <typename T>
T __shfl_down(T v, int by, int) {
  return emulate::exchange(v, int(threadIdx.x % 64) + by);
}
inline unsigned long long __ballot(int on) {
  unsigned long long m = 0;
  for (int i = 0; i < 64; ++i) m |= (unsigned long long)(emulate::exchange(on, i) != 0) << i;
  return m;
}
template <typename T>
T __builtin_amdgcn_readfirstlane(T v) {
  return v;  // (the same in every lane of a wave)
}
inline int __builtin_amdgcn_update_dpp(int, int v, int, int, int, bool) { return v; }  // (not reached)
