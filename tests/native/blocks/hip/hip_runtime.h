// Blocks of a kernel run on the host, for tests of what does not show on a device: the
// same source, compiled by the host compiler with this header in the runtime's place.
//
// Every thread of a block is a context of its own.  A wave's threads meet where the wave
// exchanges values, a block's where it has a barrier; between two barriers the waves run
// one after another in an order that the program chooses (blocks::order), and between two
// exchanges a wave's threads do.  What a block gives out must not depend on that order;
// where it does, threads touch the same memory without anything that keeps one from the
// other.  Threads that do not meet at the same place are reported (blocks::fault).
#pragma once

#include <setjmp.h>
#include <stdint.h>
#include <string.h>
#include <ucontext.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <functional>
#include <string>
#include <vector>

#define __global__
#define __device__
#define __host__
#define __shared__ static
#define __forceinline__ inline
#define __launch_bounds__(...)

typedef int hipError_t;
typedef void* hipStream_t;
typedef void* hipEvent_t;
enum { hipSuccess = 0 };
inline hipError_t hipGetLastError() { return hipSuccess; }

struct dim3 {
  unsigned x, y, z;
  dim3(unsigned x = 1, unsigned y = 1, unsigned z = 1) : x(x), y(y), z(z) {}
};
struct alignas(8) int2 {
  int32_t x, y;
};
struct alignas(8) uint2 {
  uint32_t x, y;
};
struct alignas(16) uint4 {
  uint32_t x, y, z, w;
};

namespace blocks {

enum Order { kForward, kBackward };   // by their numbers
inline Order order = kForward;
inline std::string fault;   // the first one

struct Thread {
  ucontext_t at;    // where it begins,
  jmp_buf where;    // and where it goes on
  std::vector<char> stack;
  int tid;
  bool begun;
  int place;        // line of the exchange or barrier that it waits at; 0: it runs
  bool barrier, ended;
  uint64_t gives;   // what it brought there, and what it takes away
  uint64_t takes;
};
inline std::vector<Thread> threads;
inline Thread* now = nullptr;
inline jmp_buf home;
inline dim3 grid, block, index, number;   // number: the running thread's
inline const std::function<void()>* body = nullptr;
using Meet = void (*)(Thread* lanes, int n);
inline Meet meet = nullptr;

inline void fail(const std::string& what) {
  if (fault.empty()) fault = what;
}
inline uint64_t wait(int place, bool barrier, uint64_t gives, Meet how) {
  Thread* t = now;
  t->place = place;
  t->barrier = barrier;
  t->gives = gives;
  meet = how;
  if (!_setjmp(t->where)) _longjmp(home, 1);
  return t->takes;
}
inline void begin() {
  (*body)();
  now->ended = true;
  _longjmp(home, 1);
}
inline void go_on(Thread& t) {
  now = &t;
  number = dim3((unsigned)t.tid);
  t.place = 0;
  if (_setjmp(home)) return;
  if (t.begun) _longjmp(t.where, 1);
  t.begun = true;
  setcontext(&t.at);
}
// A wave up to its next barrier or its end; false: its threads do not meet.
inline bool run_wave(Thread* lanes, int n) {
  for (;;) {
    for (int i = 0; i < n; ++i) {
      Thread& t = lanes[order == kForward ? i : n - 1 - i];
      if (!t.ended) go_on(t);
    }
    const Thread* first = nullptr;
    bool apart = false;
    for (int i = 0; i < n; ++i) {
      if (lanes[i].ended) continue;
      if (!first) first = &lanes[i];
      apart |= lanes[i].place != first->place || lanes[i].barrier != first->barrier;
    }
    if (!first) return true;
    if (apart) {
      fail("threads of a wave wait at different places, one in line " + std::to_string(first->place));
      return false;
    }
    if (first->barrier) return true;
    meet(lanes, n);
  }
}
inline void run_block(int n) {
  const int waves = (n + 63) / 64;
  for (int t = 0; t < n; ++t) {
    Thread& th = threads[t];
    th.tid = t;
    th.ended = th.barrier = th.begun = false;
    th.place = 0;
    getcontext(&th.at);
    th.at.uc_stack.ss_sp = th.stack.data();
    th.at.uc_stack.ss_size = th.stack.size();
    th.at.uc_link = nullptr;
    makecontext(&th.at, begin, 0);
  }
  for (;;) {
    for (int i = 0; i < waves; ++i) {
      const int w = order == kForward ? i : waves - 1 - i;
      if (!run_wave(&threads[w * 64], std::min(64, n - w * 64))) return;
    }
    const Thread* first = nullptr;
    bool apart = false;
    for (int t = 0; t < n; ++t) {
      if (threads[t].ended) continue;
      if (!first) first = &threads[t];
      apart |= threads[t].place != first->place;
    }
    if (!first) return;
    if (apart) return fail("waves wait at different barriers, one in line " + std::to_string(first->place));
    uint64_t any = 0;   // (threads that ended take no part)
    for (int t = 0; t < n; ++t)
      if (!threads[t].ended) any |= threads[t].gives;
    for (int t = 0; t < n; ++t) threads[t].takes = any;
  }
}
inline void launch(const std::function<void()>& kernel, dim3 g, dim3 b) {
  const int n = (int)(b.x * b.y * b.z);
  if ((int)threads.size() < n) threads.resize(n);
  for (Thread& t : threads)
    if (t.stack.empty()) t.stack.resize(64 << 10);
  grid = g;
  block = b;
  body = &kernel;
  for (unsigned z = 0; z < g.z && fault.empty(); ++z)
    for (unsigned y = 0; y < g.y && fault.empty(); ++y)
      for (unsigned x = 0; x < g.x && fault.empty(); ++x) {
        index = dim3(x, y, z);
        run_block(n);
      }
}

// Lane `from(i)` of a wave's values, to lane i.
template <typename F>
inline uint64_t exchange(int place, uint64_t v, const F& from) {
  // (every lane has its own `from`: it sends along what it wants)
  struct Wish {
    uint64_t v;
    int src;
  };
  Wish w{v, from((int)(number.x & 63u))};
  return wait(place, false, (uint64_t)(uintptr_t)&w,
              [](Thread* lanes, int n) {
                for (int i = 0; i < n; ++i) {
                  if (lanes[i].ended) continue;
                  const int src = ((const Wish*)(uintptr_t)lanes[i].gives)->src;
                  const Thread& o = lanes[src >= 0 && src < n && !lanes[src].ended ? src : i];
                  lanes[i].takes = ((const Wish*)(uintptr_t)o.gives)->v;
                }
              });
}
inline uint64_t votes(int place, bool p) {
  return wait(place, false, p,
              [](Thread* lanes, int n) {
                uint64_t all = 0;
                for (int i = 0; i < n; ++i)
                  if (!lanes[i].ended) all |= (lanes[i].gives & 1u) << i;
                for (int i = 0; i < n; ++i) lanes[i].takes = all;
              });
}
template <typename T, typename F>
inline T moved(int place, T x, const F& from) {
  uint64_t v = 0;
  memcpy(&v, &x, sizeof(T));
  v = exchange(place, v, from);
  memcpy(&x, &v, sizeof(T));
  return x;
}

}  // namespace blocks

#define threadIdx (blocks::number)
#define blockIdx (blocks::index)
#define blockDim (blocks::block)
#define gridDim (blocks::grid)

#define __syncthreads() ((void)blocks::wait(__LINE__, true, 0, nullptr))
#define __syncthreads_or(p) ((int)blocks::wait(__LINE__, true, (p) ? 1 : 0, nullptr))
#define __ballot(p) ((unsigned long long)blocks::votes(__LINE__, (p)))
#define __any(p) (blocks::votes(__LINE__, (p)) != 0)
#define __shfl(x, src) (blocks::moved(__LINE__, (x), [&](int) { return (int)(src)&63; }))
#define __shfl_xor(x, d) (blocks::moved(__LINE__, (x), [&](int i) { return i ^ (int)(d); }))
#define __shfl_up(x, d) (blocks::moved(__LINE__, (x), [&](int i) { return i - (int)(d); }))
#define __builtin_amdgcn_wave_barrier() ((void)blocks::votes(__LINE__, false))
#define __builtin_amdgcn_readfirstlane(x) (x)   // (of values that all lanes have alike)

inline int __popcll(unsigned long long x) { return __builtin_popcountll(x); }
inline uint32_t __umulhi(uint32_t a, uint32_t b) { return (uint32_t)((uint64_t)a * b >> 32); }
template <typename To, typename From>
inline To blocks_bits(From x) {
  To y;
  memcpy(&y, &x, sizeof y);
  return y;
}
inline uint32_t __float_as_uint(float x) { return blocks_bits<uint32_t>(x); }
inline float __uint_as_float(uint32_t x) { return blocks_bits<float>(x); }
inline float __int_as_float(int x) { return blocks_bits<float>(x); }
inline uint32_t blocks_mbcnt(uint32_t m, uint32_t base, int from) {
  const int below = (int)(threadIdx.x & 63u) - from;
  return base + (uint32_t)__builtin_popcount(below <= 0 ? 0u : (below >= 32 ? m : m & ((1u << below) - 1u)));
}
#define __builtin_amdgcn_mbcnt_lo(m, base) blocks_mbcnt((m), (base), 0)
#define __builtin_amdgcn_mbcnt_hi(m, base) blocks_mbcnt((m), (base), 32)
// Instructions of helpers that the tested kernels do not call.
struct BlocksNone {
  uint32_t bits;
  template <typename T>
  operator T() const {
    abort();
  }
};
template <typename... A>
inline BlocksNone blocks_none(const A&...) {
  abort();
}
#define __builtin_amdgcn_cvt_pk_f32_fp8 blocks_none
#define __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8 blocks_none
#define __builtin_amdgcn_cvt_scalef32_pk_f16_fp8 blocks_none
#define __builtin_amdgcn_update_dpp blocks_none
#define __builtin_amdgcn_readlane blocks_none
#define __builtin_amdgcn_mfma_f32_16x16x32_bf16 blocks_none
#define __builtin_amdgcn_mfma_f32_16x16x32_f16 blocks_none
#define __builtin_amdgcn_mfma_f32_32x32x16_bf16 blocks_none
#define __builtin_amdgcn_mfma_f32_32x32x16_f16 blocks_none
#define __builtin_amdgcn_global_load_lds blocks_none
template <typename T>
inline T atomicAdd(T* p, T x) {
  const T old = *p;
  *p = old + x;
  return old;
}
using std::max;
using std::min;

#define hipLaunchKernelGGL(kernel, g, b, lds, stream, ...) blocks::launch([&] { (kernel)(__VA_ARGS__); }, (g), (b))
