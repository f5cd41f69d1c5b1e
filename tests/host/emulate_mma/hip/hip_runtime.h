// Stands in for the HIP runtime where kernels of csrc/ that use the matrix instructions are compiled
// for the CPU by a host test: each lane of a workgroup is a fiber of one thread, workgroups run one
// after the other, LDS is static memory, and lanes exchange values where all of their wave (or of
// a row that is on together) meet. Lanes of a wave reach the same exchanges unless they have
// returned.
#pragma once
#include <math.h>
#include <setjmp.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <ucontext.h>

#include <functional>
#include <vector>

#define __global__
#define __device__
#define __host__
#define __forceinline__ inline
#define __launch_bounds__(...)
#define __shared__ static

struct uint2 {
  uint32_t x, y;
};
struct uint4 {
  uint32_t x, y, z, w;
};
struct int2 {
  int x, y;
};
struct float4 {
  float x, y, z, w;
};
inline uint2 make_uint2(uint32_t x, uint32_t y) { return {x, y}; }
inline uint4 make_uint4(uint32_t x, uint32_t y, uint32_t z, uint32_t w) { return {x, y, z, w}; }
struct dim3 {
  unsigned x, y, z;
  dim3(unsigned a = 1, unsigned b = 1, unsigned c = 1) : x(a), y(b), z(c) {}
};
typedef void* hipStream_t;
constexpr int hipSuccess = 0;
inline int hipGetLastError() { return 0; }

inline float __uint_as_float(uint32_t v) { return __builtin_bit_cast(float, v); }
inline uint32_t __float_as_uint(float v) { return __builtin_bit_cast(uint32_t, v); }
inline float __int_as_float(int v) { return __builtin_bit_cast(float, v); }
inline int __float_as_int(float v) { return __builtin_bit_cast(int, v); }

namespace emulate {

struct Meeting {  // of `alive` lanes
  int alive = 0, here = 0;
  long turn = 0;
};
// A fiber starts by its context and is switched to by jumps, which make no system call.
struct Jump {
  jmp_buf at;
  bool set;
};
inline Jump scheduler;
inline std::vector<Jump> jumps;
inline std::vector<ucontext_t> fibers;
inline std::vector<char> done;
inline std::vector<std::vector<char>> stacks;
inline int now;
inline Meeting wave_meets[16], all_meet;
inline char slot[1024][32];
inline dim3 thread_idx, block_idx, grid_dim, block_dim;
inline std::function<void()> body;

inline void yield() {
  jumps[now].set = true;
  if (!_setjmp(jumps[now].at)) _longjmp(scheduler.at, 1);
}
inline void resume(int t) {
  if (_setjmp(scheduler.at)) return;
  if (jumps[t].set) _longjmp(jumps[t].at, 1);
  setcontext(&fibers[t]);
}
inline void close(Meeting& m) {
  m.here = 0;
  ++m.turn;
}
inline void meet(Meeting& m) {
  const long turn = m.turn;
  if (++m.here == m.alive)
    close(m);
  else
    while (m.turn == turn) yield();
}
inline Meeting& my_wave() { return wave_meets[now / 64]; }
inline void leave(Meeting& m) {
  if (--m.alive == m.here && m.alive > 0) close(m);
}
inline void fiber() {
  body();
  done[now] = 1;
  leave(wave_meets[now / 64]);
  leave(all_meet);
  for (;;) yield();
}

// Every lane's value of T, by lane of this wave, handed to f between two meetings.
template <typename T, typename F>
auto with_wave(const T& mine, F f) {
  static_assert(sizeof(T) <= 32);
  const int base = now / 64 * 64;
  memcpy(slot[now], &mine, sizeof(T));
  meet(my_wave());
  auto r = f([&](int lane) {
    T v;
    memcpy(&v, slot[base + lane], sizeof(T));
    return v;
  });
  meet(my_wave());
  return r;
}

inline void launch(dim3 grid, dim3 block, std::function<void()> kernel) {
  body = std::move(kernel);
  const int n = int(block.x);
  fibers.resize(n);
  jumps.resize(n);
  done.resize(n);
  stacks.resize(n);
  grid_dim = grid;
  block_dim = block;
  for (unsigned y = 0; y < grid.y; ++y)
    for (unsigned x = 0; x < grid.x; ++x) {
      block_idx = dim3(x, y);
      all_meet = Meeting{n};
      for (int w = 0; w < n / 64; ++w) wave_meets[w] = Meeting{64};
      for (int t = 0; t < n; ++t) {
        done[t] = 0;
        jumps[t].set = false;
        stacks[t].resize(1 << 20);
        getcontext(&fibers[t]);
        fibers[t].uc_stack.ss_sp = stacks[t].data();
        fibers[t].uc_stack.ss_size = stacks[t].size();
        fibers[t].uc_link = nullptr;
        makecontext(&fibers[t], fiber, 0);
      }
      for (int left = n; left > 0;)
        for (int t = 0; t < n; ++t) {
          if (done[t]) continue;
          now = t;
          thread_idx = dim3(unsigned(t));
          resume(t);
          if (done[t]) --left;
        }
    }
}
}  // namespace emulate

#define threadIdx emulate::thread_idx
#define blockIdx emulate::block_idx
#define gridDim emulate::grid_dim
#define blockDim emulate::block_dim
#define hipLaunchKernelGGL(kernel, grid, block, lds, stream, ...) \
  emulate::launch(grid, block, [=] { kernel(__VA_ARGS__); })

inline void __syncthreads() { emulate::meet(emulate::all_meet); }
// Lanes that have returned keep the value they last gave.
template <typename T>
T __shfl(T v, int from, int) {
  const int lane = emulate::now % 64;
  return emulate::with_wave(v, [&](auto of) { return of(from < 0 || from > 63 ? lane : from); });
}
template <typename T>
T __shfl_xor(T v, int m, int) {
  return __shfl(v, (emulate::now % 64) ^ m, 64);
}
inline unsigned long long __ballot(int on) {
  return emulate::with_wave(on, [](auto of) {
    unsigned long long m = 0;
    for (int i = 0; i < 64; ++i) m |= (unsigned long long)(of(i) != 0) << i;
    return m;
  });
}
inline int __builtin_amdgcn_readlane(int v, int lane) {
  return emulate::with_wave(v, [&](auto of) { return of(lane); });
}
template <typename T>
T __builtin_amdgcn_readfirstlane(T v) {
  return v;  // (the same in every lane of a wave)
}
inline int __builtin_amdgcn_update_dpp(int old, int v, int ctrl, int, int, bool) {
  const int lane = emulate::now % 64, row = lane & ~15, i = lane & 15;
  int from = -1;
  if (ctrl < 0x100) from = (lane & ~3) + ((ctrl >> (2 * (lane & 3))) & 3);  // quad_perm
  else if (ctrl > 0x110 && ctrl < 0x120) from = i >= (ctrl & 15) ? lane - (ctrl & 15) : -1;  // row_shr
  else if (ctrl == 0x140) from = row + 15 - i;                                // row_mirror
  else if (ctrl == 0x141) from = (lane & ~7) + 7 - (lane & 7);                // row_half_mirror
  else abort();
  return emulate::with_wave(v, [&](auto of) { return from < 0 ? old : of(from); });
}

namespace emulate {
typedef float f4 __attribute__((ext_vector_type(4)));
typedef short h4 __attribute__((ext_vector_type(4)));
struct Bf8 {
  uint16_t v[8];
};
inline float wide(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }
}  // namespace emulate

template <typename V>
emulate::f4 __builtin_amdgcn_mfma_f32_16x16x32_bf16(V a, V b, emulate::f4 c, int, int, int) {
  struct Two {
    emulate::Bf8 a, b;
  } mine{__builtin_bit_cast(emulate::Bf8, a), __builtin_bit_cast(emulate::Bf8, b)};
  const int lane = emulate::now % 64, r = lane & 15, g = lane >> 4;
  return emulate::with_wave(mine, [&](auto of) {
    double s[4] = {c[0], c[1], c[2], c[3]};
    for (int k8 = 0; k8 < 4; ++k8) {
      const Two col = of(16 * k8 + r);
      for (int e = 0; e < 4; ++e) {
        const Two row = of(16 * k8 + 4 * g + e);
        for (int i = 0; i < 8; ++i) s[e] += double(emulate::wide(row.a.v[i])) * emulate::wide(col.b.v[i]);
      }
    }
    return emulate::f4{float(s[0]), float(s[1]), float(s[2]), float(s[3])};
  });
}
inline emulate::f4 __builtin_amdgcn_mfma_f32_16x16x4f32(float a, float b, emulate::f4 c, int, int, int) {
  struct Two {
    float a, b;
  } mine{a, b};
  const int lane = emulate::now % 64, r = lane & 15, g = lane >> 4;
  return emulate::with_wave(mine, [&](auto of) {
    double s[4] = {c[0], c[1], c[2], c[3]};
    for (int k = 0; k < 4; ++k)
      for (int e = 0; e < 4; ++e) s[e] += double(of(16 * k + 4 * g + e).a) * of(16 * k + r).b;
    return emulate::f4{float(s[0]), float(s[1]), float(s[2]), float(s[3])};
  });
}
// Of each 16 lanes, lane i receives column i of the four rows of 16 elements that they hold together.
inline emulate::h4 __builtin_amdgcn_ds_read_tr16_b64_v4i16(const emulate::h4* p) {
  emulate::h4 mine;
  memcpy(&mine, p, 8);
  const int lane = emulate::now % 64, base = lane & ~15, i = lane & 15;
  return emulate::with_wave(mine, [&](auto of) {
    emulate::h4 v;
    for (int j = 0; j < 4; ++j) v[j] = of(base + 4 * j + i / 4)[i % 4];
    return v;
  });
}
