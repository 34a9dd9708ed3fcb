// device.h -- a CUDA kernel's source on the host, for tests: every thread of a cluster is a fiber that runs
// until it waits at a barrier, a warp's exchange or the cluster's barrier, and the fiber that goes on
// next is the first, of those that can, in an order that the test gives.  A kernel whose accesses are all
// ordered by its barriers has one result whatever the order; where a barrier is missing, an order that holds one
// thread, warp or block back shows it.  Nothing is said about the time between barriers: a
// thread may be arbitrarily late.
//
// A warp's exchange (shuffle, ballot, reduction) takes all 32 threads.  Blocks' shared memory starts as 0xa5.  Ends a
// run with an error: threads that wait for one another, a block's shared memory named from the cluster after
// that block has ended, a launch that the stand-in does not know.
#pragma once

#include <setjmp.h>
#include <ucontext.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <memory>
#include <numeric>
#include <set>
#include <utility>
#include <type_traits>
#include <vector>

#define __device__
#define __host__
#define __global__
#define __forceinline__ inline
#define __noinline__ __attribute__((noinline))
#define __launch_bounds__(...)
#define __grid_constant__
#define __align__(n) alignas(n)

struct uint2 { uint32_t x, y; };
struct uint4 { uint32_t x, y, z, w; };
inline uint2 make_uint2(uint32_t x, uint32_t y) { return {x, y}; }
inline uint4 make_uint4(uint32_t x, uint32_t y, uint32_t z, uint32_t w) { return {x, y, z, w}; }
struct dim3 {
  unsigned x, y, z;
  dim3(unsigned a = 1, unsigned b = 1, unsigned c = 1) : x(a), y(b), z(c) {}
};

namespace threads {

struct Fiber;
struct Barrier {  // of `expected` arrivals (less those that have ended)
  int expected = 0, arrived = 0;
  unsigned phase = 0;
  std::vector<Fiber *> waiting;
  void look();
  unsigned arrive() {
    const unsigned p = phase;
    ++arrived;
    look();
    return p;
  }
  void drop() { --expected, look(); }
};
struct Warp {
  Barrier all;
  uint64_t value[2][32];  // (a thread is at most one exchange ahead of another)
};
struct Block {
  Barrier all;
  uint64_t pred[2] = {};  // __syncthreads_count
  int left = 0;
  std::unique_ptr<uint64_t[]> fixed, dynamic;
  size_t fixed_bytes = 0, dynamic_bytes = 0;
};
struct Fiber {
  ucontext_t start;
  jmp_buf at;  // (a swap of contexts would call the system each time)
  bool begun = false;
  std::unique_ptr<char[]> stack;
  unsigned cluster_phase = 0, votes = 0, exchanges = 0;
  Block *block;
  Warp *warp;
  Barrier *cluster;
  int thread, rank, place;  // place: in the order
  dim3 block_index;
  bool done = false;
};

struct Machine {
  std::vector<Fiber> fibers;
  std::vector<Block> blocks;
  std::vector<Warp> warps;
  Barrier cluster;
  std::set<std::pair<int, Fiber *>> ready;
  Fiber *now = nullptr;
  jmp_buf home;
  void (*body)(void *);
  void *arg;
};
inline Machine *machine = nullptr;
inline Fiber &self() { return *machine->now; }
[[noreturn]] inline void fail(const char *what) {
  std::fprintf(stderr, "%s\n", what);
  std::exit(3);
}

inline void leave(Fiber &f) {
  if (_setjmp(f.at) == 0) _longjmp(machine->home, 1);
}
inline void Barrier::look() {
  if (arrived == 0 || arrived < expected) return;
  arrived = 0, ++phase;
  for (Fiber *f : waiting) machine->ready.insert({f->place, f});
  waiting.clear();
}
// (a thread that does not have to wait lets those before it in the order go on all the same)
inline void wait(Barrier &b, unsigned phase) {
  Fiber &f = self();
  if (b.phase == phase) b.waiting.push_back(&f);
  else machine->ready.insert({f.place, &f});
  leave(f);
}
inline void sync(Barrier &b) { wait(b, b.arrive()); }

// A warp's exchange: this thread's value for all of its threads.
inline const uint64_t *exchange(uint64_t v) {
  Fiber &f = self();
  uint64_t *const values = f.warp->value[f.exchanges++ & 1];
  values[f.thread % 32] = v;
  sync(f.warp->all);
  return values;
}
template <class T>
uint64_t bits(T v) {
  uint64_t b = 0;
  std::memcpy(&b, &v, sizeof v);
  return b;
}
template <class T>
T from_bits(uint64_t b) {
  T v;
  std::memcpy(&v, &b, sizeof v);
  return v;
}

inline void entry() {
  Machine *const m = machine;
  m->body(m->arg);
  Fiber &f = self();
  f.done = true;
  --f.block->left;
  f.warp->all.drop(), f.block->all.drop(), m->cluster.drop();
  leave(f);
}

constexpr size_t kGuard = 16;  // words behind (and, for alignment, before) a block's shared memory, which stay as they are
inline uint8_t *aligned(const std::unique_ptr<uint64_t[]> &p) { return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p.get()) + 15) / 16 * 16); }

// One cluster of `ranks` blocks: body(arg) in every thread.  order[i]: the i-th thread (rank * block + thread) that
// goes on where it can.
inline void run_cluster(int ranks, int block, dim3 first, size_t fixed, size_t dynamic, const std::vector<int> &order,
                        void (*body)(void *), void *arg) {
  Machine m;
  const int n = ranks * block;
  m.body = body, m.arg = arg;
  m.fibers = std::vector<Fiber>(n);
  m.blocks = std::vector<Block>(ranks);
  m.warps = std::vector<Warp>(n / 32);
  m.cluster.expected = n;
  for (Warp &w : m.warps) w.all.expected = 32;
  for (Block &b : m.blocks) {
    b.all.expected = b.left = block;
    b.fixed_bytes = fixed, b.dynamic_bytes = dynamic;
    for (auto [at, bytes] : {std::pair(&b.fixed, fixed), std::pair(&b.dynamic, dynamic)}) {
      *at = std::make_unique<uint64_t[]>(bytes / 8 + kGuard);
      std::memset(at->get(), 0xa5, (bytes / 8 + kGuard) * 8);
    }
  }
  machine = &m;
  constexpr size_t kStack = 64 << 10;
  for (int i = 0; i < n; ++i) {
    Fiber &f = m.fibers[i];
    f.block = &m.blocks[i / block], f.warp = &m.warps[i / 32], f.cluster = &m.cluster;
    f.thread = i % block, f.rank = i / block;
    f.block_index = dim3(first.x + f.rank, first.y, first.z);
    f.stack = std::unique_ptr<char[]>(new char[kStack]);
    getcontext(&f.start);
    f.start.uc_stack.ss_sp = f.stack.get(), f.start.uc_stack.ss_size = kStack;
    f.start.uc_link = nullptr;
    makecontext(&f.start, entry, 0);
  }
  for (int i = 0; i < n; ++i) {
    Fiber &f = m.fibers[order[i]];
    f.place = i;
    m.ready.insert({i, &f});
  }
  int left = n;
  while (!m.ready.empty()) {
    m.now = m.ready.begin()->second;
    m.ready.erase(m.ready.begin());
    if (_setjmp(m.home) == 0) {
      if (m.now->begun) _longjmp(m.now->at, 1);
      m.now->begun = true;
      setcontext(&m.now->start);
    }
    left -= m.now->done;
  }
  if (left) fail("threads wait for one another");
  for (Block &b : m.blocks)
    for (auto [at, bytes] : {std::pair(&b.fixed, fixed), std::pair(&b.dynamic, dynamic)})
      for (size_t i = bytes; i < bytes + 8 * (kGuard - 2); ++i)
        if (aligned(*at)[i] != 0xa5) fail("written behind shared memory");
  machine = nullptr;
}

// Orders: the threads as they are numbered; in reverse; one rank, warp or lane behind all others; mixed.
inline std::vector<int> order_of(int ranks, int block, int which, unsigned seed) {
  std::vector<int> o(ranks * block);
  std::iota(o.begin(), o.end(), 0);
  unsigned s = seed * 2654435761u + 12345u;
  auto next = [&] { return s = s * 1664525u + 1013904223u, s >> 8; };
  if (which == 1) std::reverse(o.begin(), o.end());
  auto behind = [&](auto late) { std::stable_partition(o.begin(), o.end(), [&](int i) { return !late(i); }); };
  if (which == 2) behind([&, r = int(next() % ranks)](int i) { return i / block == r; });
  if (which == 3) behind([&, w = int(next() % (ranks * block / 32))](int i) { return i / 32 == w; });
  if (which == 4) behind([&, w = int(next() % 32)](int i) { return i % 32 == w; });
  if (which == 5)
    for (size_t i = o.size() - 1; i; --i) std::swap(o[i], o[next() % (i + 1)]);
  return o;
}
inline int which_order = 0;
inline unsigned order_seed = 0;

template <class T>
T &shared() {
  Block &b = *self().block;
  if (sizeof(T) > b.fixed_bytes) fail("more shared memory than was laid out");
  return *reinterpret_cast<T *>(aligned(b.fixed));
}
inline void *dynamic() { return aligned(self().block->dynamic); }
template <class T>
T *in_rank(T *p, int rank) {
  Fiber &f = self();
  Block &own = *f.block, &other = (&own - f.rank)[rank];
  if (other.left == 0) fail("shared memory of a block that has ended");
  const auto move = [&](std::unique_ptr<uint64_t[]> Block::*m, size_t bytes) -> T * {
    uint8_t *const at = reinterpret_cast<uint8_t *>(p), *const base = aligned(own.*m);
    return at < base || at >= base + bytes ? nullptr : reinterpret_cast<T *>(aligned(other.*m) + (at - base));
  };
  if (T *q = move(&Block::fixed, own.fixed_bytes)) return q;
  if (T *q = move(&Block::dynamic, own.dynamic_bytes)) return q;
  fail("not shared memory");
}

}  // namespace threads

struct ThreadIndex {
  struct X { operator unsigned() const { return (unsigned)threads::self().thread; } } x;
};
inline ThreadIndex threadIdx;
#define blockIdx (threads::self().block_index)

// ---- a warp and a block ----
inline void full(unsigned mask) {
  if (mask != 0xffffffffu) threads::fail("an exchange of a part of a warp");
}
inline void __syncwarp() { threads::exchange(0); }
inline void __syncthreads() { threads::sync(threads::self().block->all); }
inline int __syncthreads_count(int pred) {
  threads::Fiber &f = threads::self();
  uint64_t &n = f.block->pred[f.votes++ & 1];
  n += pred != 0;
  __syncthreads();
  const int r = (int)n;
  __syncthreads();  // (all have read it)
  n = 0;
  __syncthreads();
  return r;
}
template <class T>
T __shfl_sync(unsigned mask, T v, int lane) {
  full(mask);
  return threads::from_bits<T>(threads::exchange(threads::bits(v))[lane & 31]);
}
template <class T>
T __shfl_xor_sync(unsigned mask, T v, int x) {
  full(mask);
  return threads::from_bits<T>(threads::exchange(threads::bits(v))[threads::self().thread % 32 ^ x]);
}
template <class T>
T __shfl_up_sync(unsigned mask, T v, int d) {
  full(mask);
  const int lane = threads::self().thread % 32;
  return threads::from_bits<T>(threads::exchange(threads::bits(v))[lane >= d ? lane - d : lane]);
}
inline unsigned __ballot_sync(unsigned mask, int pred) {
  full(mask);
  const uint64_t *const v = threads::exchange(pred != 0);
  unsigned r = 0;
  for (int i = 0; i < 32; ++i) r |= (unsigned)v[i] << i;
  return r;
}
inline unsigned __reduce_max_sync(unsigned mask, unsigned x) {
  full(mask);
  const uint64_t *const v = threads::exchange(x);
  return (unsigned)*std::max_element(v, v + 32);
}
inline unsigned __reduce_min_sync(unsigned mask, unsigned x) {
  full(mask);
  const uint64_t *const v = threads::exchange(x);
  return (unsigned)*std::min_element(v, v + 32);
}
inline uint32_t atomicAdd(uint32_t *p, uint32_t v) { return *p += v, *p - v; }

// ---- arithmetic (compiled without contraction) ----
using std::fabs;
inline uint32_t __float_as_uint(float x) { return (uint32_t)threads::bits(x); }
inline float __uint_as_float(uint32_t x) { return threads::from_bits<float>(x); }
inline float __fadd_rn(float a, float b) { return a + b; }
inline float __fsub_rn(float a, float b) { return a - b; }
inline float __fmul_rn(float a, float b) { return a * b; }
inline float __fdiv_rn(float a, float b) { return a / b; }
inline float __fmaf_rn(float a, float b, float c) { return std::fmaf(a, b, c); }
inline int __float2int_rn(float x) { return (int)std::nearbyintf(x); }
inline float __double2float_ru(double x) {
  const float f = (float)x;
  return (double)f < x ? std::nextafterf(f, INFINITY) : f;
}
inline uint32_t __funnelshift_rc(uint32_t lo, uint32_t hi, uint32_t by) {
  return (uint32_t)(((uint64_t)hi << 32 | lo) >> std::min(by, 32u));
}
inline uint64_t __umul64hi(uint64_t a, uint64_t b) { return (uint64_t)((unsigned __int128)a * b >> 64); }
inline int __popc(uint32_t x) { return __builtin_popcount(x); }
inline int __ffs(uint32_t x) { return __builtin_ffs((int)x); }
template <class A, class B>
std::common_type_t<A, B> min(A a, B b) { return (std::common_type_t<A, B>)a < (std::common_type_t<A, B>)b ? a : b; }
template <class A, class B>
std::common_type_t<A, B> max(A a, B b) { return (std::common_type_t<A, B>)a < (std::common_type_t<A, B>)b ? b : a; }
using __half = uint16_t;  // (its bits)
inline __half __ushort_as_half(uint16_t x) { return x; }
inline float __half2float(__half h) {
  const float v = std::ldexp(float(h >> 10 & 31 ? (h & 1023) | 1024 : h & 1023), std::max(h >> 10 & 31, 1) - 25);
  const float r = (h >> 10 & 31) == 31 ? (h & 1023 ? NAN : INFINITY) : v;
  return h & 0x8000 ? -r : r;
}

// ---- cooperative groups ----
namespace cooperative_groups {
struct cluster_group {
  unsigned block_rank() const { return (unsigned)threads::self().rank; }
  unsigned num_blocks() const { return (unsigned)threads::machine->blocks.size(); }
  void barrier_arrive() const { threads::self().cluster_phase = threads::machine->cluster.arrive(); }
  void barrier_wait() const { threads::wait(threads::machine->cluster, threads::self().cluster_phase); }
  void sync() const { barrier_arrive(), barrier_wait(); }
  template <class T>
  T *map_shared_rank(T *p, int rank) const { return threads::in_rank(p, rank); }
};
inline cluster_group this_cluster() { return {}; }
}  // namespace cooperative_groups
