// kv_evict.cu -- mq_kv_evict: the rows that stay are chosen per (sequence, kv head) by one CTA,
// then copied in order.
//
// Choice: a weight sum maps to an unsigned key in the order of the values (NaN above all, -0 as
// 0); the smallest key of the rows that stay is found bit by bit from the top, counting the
// candidates at or above each trial key; rows equal to it stay from the lowest position on.
#include "kv.cuh"

namespace mq {
namespace {

constexpr int kSelThreads = 256;

__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t b = __float_as_uint(w + 0.f);  // -0 becomes 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Sum over the CTA (every thread gets it); buf: one int per warp.
__device__ int block_sum(int v, int *buf) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
  for (int w = 0; w < kSelThreads / 32; ++w) s += buf[w];
  return s;
}
// Threads before this one whose flag is set, and the CTA's count of them.
__device__ int block_rank(bool f, int *buf, int *total) {
  const unsigned b = __ballot_sync(0xffffffffu, f);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) buf[warp] = __popc(b);
  __syncthreads();
  int before = __popc(b & ((1u << lane) - 1)), all = 0;
  for (int w = 0; w < kSelThreads / 32; ++w) {
    if (w < warp) before += buf[w];
    all += buf[w];
  }
  *total = all;
  return before;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a) {
  __shared__ int buf[kSelThreads / 32];
  grid_dependency();
  const int s = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  const int raw = a.len[s], n = clamped_len(raw, a.max_len);
  if (h == 0 && tid == 0) {
    if (raw != n) index_error(a.status, kIdxEvictLen, raw);
    a.new_len[s] = min(n, a.keep);
  }
  int32_t *kept = a.kept + (int64_t(s) * a.c.hkv + h) * a.keep;
  if (n <= a.keep) {
    for (int i = tid; i < a.keep; i += kSelThreads) kept[i] = i < n ? i : -1;
    return;
  }
  const int32_t *pages = a.pages + s * a.pages_ld;
  const int lo = a.sink, hi = n - a.recent, need = a.keep - a.sink - a.recent;
  auto key = [&](int i) -> uint32_t {
    const int64_t r = kv_row(a.c, pages, h, i);
    return r < 0 ? order_key(0.f) : order_key(a.c.sums[r]);
  };
  // the largest key T with at least `need` candidates at or above it
  uint32_t T = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t trial = T | (1u << bit);
    int c = 0;
    for (int i = lo + tid; i < hi; i += kSelThreads) c += key(i) >= trial;
    if (block_sum(c, buf) >= need) T = trial;
  }
  int above = 0;
  for (int i = lo + tid; i < hi; i += kSelThreads) above += key(i) > T;
  int ties = need - block_sum(above, buf);  // rows equal to T that stay
  int out = 0;
  for (int i0 = 0; i0 < n; i0 += kSelThreads) {
    const int i = i0 + tid;
    const bool middle = i >= lo && i < hi;
    const uint32_t k = middle ? key(i) : 0;
    int all;
    const int eq = block_rank(middle && k == T, buf, &all);
    const bool stay = i < n && (!middle || k > T || (k == T && eq < ties));
    ties -= min(ties, all);
    const int place = block_rank(stay, buf, &all);
    if (stay) kept[out + place] = i;
    out += all;
  }
}

__global__ void __launch_bounds__(256) evict_copy_kernel(EvictArgs a) {
  grid_dependency();
  const int s = blockIdx.y, h = blockIdx.z, lane = threadIdx.x & 31;
  const int j = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (j >= a.keep) return;
  const int src = a.kept[(int64_t(s) * a.c.hkv + h) * a.keep + j];
  if (src < 0) return;
  const int64_t r = kv_row(a.c, a.pages + s * a.pages_ld, h, src);
  const int64_t w = kv_row(a.c, a.new_pages + s * a.new_pages_ld, h, j);
  if (r < 0 || w < 0) {
    if (lane == 0)
      index_error(a.status, kIdxEvictPage,
                  r < 0 ? a.pages[s * a.pages_ld + src / a.c.page.d]
                        : a.new_pages[s * a.new_pages_ld + j / a.c.page.d]);
    return;
  }
  const int words = (a.c.type == MQ_Q8_0 ? a.c.dim : 2 * a.c.dim) / 16;
  for (int i = lane; i < words; i += 32) {
    reinterpret_cast<uint4 *>(a.c.k)[w * words + i] = reinterpret_cast<const uint4 *>(a.c.k)[r * words + i];
    reinterpret_cast<uint4 *>(a.c.v)[w * words + i] = reinterpret_cast<const uint4 *>(a.c.v)[r * words + i];
  }
  const int nb = a.c.dim / 32;
  if (a.c.type == MQ_Q8_0 && lane < nb) {
    a.c.ks[w * nb + lane] = a.c.ks[r * nb + lane];
    a.c.vs[w * nb + lane] = a.c.vs[r * nb + lane];
  }
  if (lane == 0) a.c.sums[w] = a.c.sums[r];
}

}  // namespace

mq_status launch_kv_evict(const EvictArgs &a, cudaStream_t s, const DeviceState *) {
  mq_status r = launch_dependent("evict_select_kernel", evict_select_kernel,
                                 dim3((unsigned)a.S, a.c.hkv, 1), dim3(kSelThreads, 1, 1), 0, s, a);
  if (r == MQ_OK)
    r = launch_dependent("evict_copy_kernel", evict_copy_kernel,
                         dim3((a.keep + 7) / 8, (unsigned)a.S, a.c.hkv), dim3(256, 1, 1), 0, s, a);
  return r;
}

}  // namespace mq
