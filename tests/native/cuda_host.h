// What a kernel needs of CUDA to run on the host (test-suite only): every thread is a fiber that
// runs until it has to wait for others, warps take their turns in a given order of priority.
#pragma once

#include <stdint.h>
#include <string.h>
#include <ucontext.h>

#include <algorithm>
#include <functional>
#include <map>
#include <memory>
#include <utility>
#include <vector>

#define __device__
#define __global__
#define __forceinline__ inline
#define __launch_bounds__(...)

namespace sim {

struct Index {
  unsigned x;
};
struct Barrier {
  int size = 0, arrived = 0, passed = 0;
};
struct Thread {
  ucontext_t context;
  std::unique_ptr<char[]> stack;
  Index block, thread;
  const Barrier* waits = nullptr;
  int until = 0;
  bool done = false;
};
struct Block {
  Barrier all, warps[32];
  uint64_t lanes[32][32];
  std::map<int, std::vector<char>> shared;
};

inline std::vector<Thread> threads;
inline std::vector<Block> blocks;
inline ucontext_t scheduler;
inline Thread* self;
inline std::function<void()> body;

inline void wait(Barrier& b) {
  const int turn = b.passed;
  if (++b.arrived == b.size) {
    b.arrived = 0;
    ++b.passed;
    return;
  }
  self->waits = &b;
  self->until = turn;
  swapcontext(&self->context, &scheduler);
}

inline void enter() {
  body();
  self->done = true;
  swapcontext(&self->context, &scheduler);
}

// order: warps (block * warps of a block + warp), first the one that runs whenever it can.
// False if all that is left waits for something that never comes.
inline bool run(int n_blocks, int n_threads, const int* order, std::function<void()> kernel) {
  const int warps = n_threads / 32;
  body = std::move(kernel);
  blocks = std::vector<Block>(n_blocks);
  threads = std::vector<Thread>(static_cast<size_t>(n_blocks) * n_threads);
  for (auto& b : blocks) {
    b.all.size = n_threads;
    for (auto& w : b.warps) w.size = 32;
  }
  for (size_t i = 0; i < threads.size(); ++i) {
    Thread& t = threads[i];
    t.block.x = static_cast<unsigned>(i / n_threads);
    t.thread.x = static_cast<unsigned>(i % n_threads);
    t.stack.reset(new char[1 << 16]);
    getcontext(&t.context);
    t.context.uc_stack.ss_sp = t.stack.get();
    t.context.uc_stack.ss_size = 1 << 16;
    t.context.uc_link = &scheduler;
    makecontext(&t.context, enter, 0);
  }
  for (;;) {
    Thread* next = nullptr;
    bool left = false;
    for (int w = 0; w < n_blocks * warps && !next; ++w)
      for (int lane = 0; lane < 32 && !next; ++lane) {
        Thread& t = threads[static_cast<size_t>(order[w]) * 32 + lane];
        if (t.done) continue;
        left = true;
        if (!t.waits || t.waits->passed != t.until) next = &t;
      }
    if (!next) return !left;
    next->waits = nullptr;
    self = next;
    swapcontext(&scheduler, &next->context);
  }
}

// Shared memory of the running block: one array a line of the source.
template <class T>
T& shared(int line, size_t bytes = sizeof(T)) {
  auto& a = blocks[self->block.x].shared[line];
  if (a.empty()) a.resize(bytes, 0x5A);
  return *reinterpret_cast<T*>(a.data());
}

inline Index grid;

}  // namespace sim

#define blockIdx (sim::self->block)
#define threadIdx (sim::self->thread)
#define gridDim (sim::grid)

inline void __syncthreads() { sim::wait(sim::blocks[sim::self->block.x].all); }
inline void __threadfence() {}
template <class T>
T __shfl_up_sync(unsigned, T x, int d) {
  sim::Block& b = sim::blocks[sim::self->block.x];
  const int warp = sim::self->thread.x / 32, lane = sim::self->thread.x % 32;
  memcpy(&b.lanes[warp][lane], &x, sizeof(T));
  sim::wait(b.warps[warp]);
  if (lane >= d) memcpy(&x, &b.lanes[warp][lane - d], sizeof(T));
  sim::wait(b.warps[warp]);
  return x;
}
template <class T>
T __ldg(const T* p) { return *p; }
template <class T>
T __ldcg(const T* p) { return *p; }
inline int atomicAdd(int* p, int x) { return std::exchange(*p, *p + x); }
inline int atomicOr(int* p, int x) { return std::exchange(*p, *p | x); }
