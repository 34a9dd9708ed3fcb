// kv_evict.cu -- mq_kv_evict: the rows that stay are chosen per (sequence, kv head), then copied
// in order.
//
// Choice: a weight sum maps to an unsigned key in the order of the values (NaN above all, -0 as
// 0).  A thread block cluster of up to 16 blocks holds the candidates' keys of one kv head (a part
// of the positions each, 16 a thread in registers and further ones in shared memory) and finds the
// smallest key that stays by a radix selection from the top.  A histogram of the first 11 bits,
// whose bins that are not empty are added to rank 0's through distributed shared memory (every
// rank reading all of the others' took one more cluster barrier and eight times the reads), names
// the bin that holds it.  If that has at most 4096 keys, each block reads them all and counts
// their next 11 and 10 bits by itself; else these are counted over the cluster as well.  Rows
// equal to the key stay from the lowest position on; ballots and the cluster's counts give every
// row its place.  What bounds it: latency.  131072 rows of 4 heads take 19 us: a length, its pages
// and their sums read one after the other 5, four to six barriers and reads of the cluster about 1 us
// each; the rest (the histogram's additions in shared memory, the block's own barriers, its
// instructions' first fetch) has not been taken apart.  (It reads 4 bytes per row; counting bit by
// bit from global memory, one block per head, took 5.2 ms.)
//
// Copy: bounded by the bytes of the kept rows, read and written once.  A warp looks up 32 (or,
// when there are few, 16) rows, one per lane, then moves them 16 bytes a lane, eight loads in
// flight (32768 rows of 4 heads of 128, f16: 20.5 us, 6.5 TB/s).
#include <algorithm>
#include <cooperative_groups.h>

#include "kv.cuh"

namespace cg = cooperative_groups;

namespace mq {
namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kKeysHeld = 48 * 1024;  // per block, in shared memory, beside 16 K in registers
constexpr int kMaxCluster = 16;  // above 8 only where the device reports such clusters
constexpr uint32_t kList = 2 * kBins;  // keys of one bin that each block reads from the cluster's

// No weight's key is 0 (its float would be a NaN): it stands for no candidate.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t b = __float_as_uint(w + 0.f);  // -0 becomes 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct SelShared {
  uint32_t hist[kBins];
  uint32_t total[3][kBins];               // rank 0's: the cluster's histograms; the last two of
                                          // every rank: its keys of the first chosen bin
  uint32_t warp_sum[kSelWarps];
  uint32_t gt[kSelWarps], eq[kSelWarps];  // per warp: candidates above T, equal to it
  uint32_t rank_gt[kMaxCluster], rank_eq[kMaxCluster];
  uint32_t bin, above, in_bin;            // the bin chosen, candidates above it and in it
  uint32_t listed;                        // and their number
};

// Sum over the warps before this one of a value per warp in shared memory.
__device__ __forceinline__ uint32_t sum_before(const uint32_t *per_warp, int warp, int lane) {
  return __reduce_add_sync(0xffffffffu, lane < warp ? per_warp[lane] : 0u);
}

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const __grid_constant__ EvictArgs a,
                                                                      int held) {
  extern __shared__ __align__(16) uint32_t keys[];  // [held]
  __shared__ __align__(16) SelShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int s = blockIdx.y, h = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kBins; i += kSelThreads)
    sh.hist[i] = sh.total[0][i] = sh.total[1][i] = sh.total[2][i] = 0;
  if (tid == 0) sh.listed = 0;
  cluster.barrier_arrive();  // (the totals are clear; waited for before the first is added to)
  grid_dependency();
  const int raw = a.len[s], n = clamped_len(raw, a.max_len);
  if (h == 0 && rank == 0 && tid == 0 && raw != n) index_error(a.status, kIdxEvictLen, raw);
  int32_t *kept = a.kept + (int64_t(s) * a.c.hkv + h) * a.keep;
  const int share = rank * kSelThreads + tid, stride = ranks * kSelThreads;
  if (n <= a.keep) {  // (the whole cluster)
    for (int i = share; i < a.keep; i += stride) kept[i] = i < n ? i : -1;
    cluster.barrier_wait();
    return;
  }
  for (int i = share; i < a.sink; i += stride) kept[i] = i;
  for (int i = share; i < a.recent; i += stride) kept[a.keep - a.recent + i] = n - a.recent + i;

  // this block's candidates: positions [first, first + count), a run of whole 32s for each warp;
  // lane i of a warp has the run's i-th, 32 + i-th, ... candidate: the first NK in registers, then
  // `held` of the block in shared memory, others are read again
  const int all = n - a.recent - a.sink;
  const int per = (all + ranks - 1) / ranks;
  const int first = a.sink + rank * per, count = max(0, min(per, all - rank * per));
  const int run = (count + kSelThreads - 1) / kSelThreads * 32;
  const int r0 = min(warp * run, count), r1 = min(r0 + run, count);
  const int32_t *const pages = a.pages + s * a.pages_ld;
  constexpr int NK = 16;
  const int nk = (r1 - r0 + 31) / 32;  // (the same for the warp)
  auto valid = [&](int k) { return r0 + 32 * k + lane < r1; };
  auto read_key = [&](int k) -> uint32_t {
    if (!valid(k)) return 0;
    const uint32_t r = kv_row32(a.c, pages, h, first + r0 + 32 * k + lane);
    return order_key(r == kNoRow ? 0.f : a.c.sums[r]);
  };
  auto far_key = [&](int k) -> uint32_t {
    const int at = (k - NK) * kSelThreads + tid;
    return at < held ? keys[at] : read_key(k);
  };
  __syncthreads();
  uint32_t near[NK];
  {  // 16 page entries, then 16 sums on their way side by side: no branch but the way out (few
     // candidates: the rest of the unrolled code is not even fetched) and no use behind a load
    int page[NK];
    float w[NK];
    uint32_t pi[NK];
    auto pos = [&](int k) { return (uint32_t)(first + min(r0 + 32 * k + lane, r1 - 1)); };
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      if (k >= nk) break;
      pi[k] = quotient(pos(k), a.c.page);
      page[k] = pages[pi[k]];
    }
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      if (k >= nk) break;
      const bool known = (uint32_t)page[k] < (uint32_t)a.c.n_pages;
      const uint32_t row = (uint32_t)page[k] * (uint32_t)a.c.page_stride +
                           (uint32_t)h * (uint32_t)a.c.head_stride +
                           (pos(k) - pi[k] * a.c.page.d) * (uint32_t)a.c.slot_stride;
      near[k] = known;
      w[k] = a.c.sums[known ? row : 0];
    }
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      if (k >= nk) break;
      near[k] = valid(k) ? order_key(near[k] ? w[k] : 0.f) : 0;
    }
  }
  // counted by their top bits at once
#pragma unroll
  for (int k = 0; k < NK; ++k) {
    if (k >= nk) break;
    if (near[k]) atomicAdd(&sh.hist[near[k] >> 21], 1u);
  }
  for (int k = NK; k < nk; ++k) {
    const uint32_t v = read_key(k);
    const int at = (k - NK) * kSelThreads + tid;
    if (at < held) keys[at] = v;
    if (v) atomicAdd(&sh.hist[v >> 21], 1u);
  }
  cluster.barrier_wait();

  uint32_t need = a.keep - a.sink - a.recent;  // candidates that stay, of those not yet above
  uint32_t T = 0, ties = 0;                    // keys above T stay, and `ties` of those equal
  if (need == 0) {
    T = 0xffffffffu;
  } else {
    uint32_t prefix = 0;  // the chosen bits so far
    uint32_t *const list = sh.total[1];
    uint32_t listed = 0, part[kList / kSelThreads];  // this thread's of the cluster's listed keys
    bool own = ranks == 1;                           // the block's histogram is the whole one
    for (int pass = 0;; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      if (pass) {
        for (int i = tid; i < kBins; i += kSelThreads) sh.hist[i] = 0;
        __syncthreads();
        auto add = [&](uint32_t v) {
          if (v && v >> (shift + bits) == prefix)
            atomicAdd(&sh.hist[v >> shift & ((1u << bits) - 1)], 1u);
        };
        if (listed) {
#pragma unroll
          for (int i = 0; i < int(kList) / kSelThreads; ++i)
            if (i * kSelThreads + tid < listed) add(part[i]);
        } else {
#pragma unroll
          for (int k = 0; k < NK; ++k) {
            if (k >= nk) break;
            add(near[k]);
          }
          for (int k = NK; k < nk; ++k) add(far_key(k));
        }
      }
      __syncthreads();
      uint32_t *total = sh.hist;
      if (!own) {  // the bins that are not empty, to rank 0
        total = cluster.map_shared_rank(sh.total[pass], 0);
        for (int i = tid; i < kBins; i += kSelThreads)
          if (sh.hist[i]) atomicAdd(total + i, sh.hist[i]);
        cluster.sync();
      }
      // the cluster's counts of this thread's two bins, from the top bin down
      const int b1 = kBins - 1 - 2 * tid, b0 = b1 - 1;
      const uint2 c = *reinterpret_cast<const uint2 *>(total + b0);
      uint32_t inc = c.x + c.y;  // inclusive sum over the threads before
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, inc, k);
        if (lane >= k) inc += o;
      }
      if (lane == 31) sh.warp_sum[warp] = inc;
      __syncthreads();
      const uint32_t up1 = sum_before(sh.warp_sum, warp, lane) + inc - c.x - c.y;  // candidates above each bin
      const uint32_t up0 = up1 + c.y;
      if (up1 < need && need <= up1 + c.y) sh.bin = b1, sh.above = up1, sh.in_bin = c.y;
      if (up0 < need && need <= up0 + c.x) sh.bin = b0, sh.above = up0, sh.in_bin = c.x;
      __syncthreads();
      need -= sh.above;
      prefix = prefix << bits | sh.bin;
      if (pass == 2) {
        T = prefix, ties = need;
        break;
      }
      if (need == sh.in_bin && prefix != 0) {  // the whole bin stays
        T = (prefix << shift) - 1, ties = 0;
        break;
      }
      if (pass == 0 && !own && sh.in_bin <= kList) {
        // few keys share the first bits: each block lists its own, reads all of them, and what is
        // left to do needs no other block (a round over the cluster less, and no histogram's)
        auto give = [&](uint32_t v) {
          if (v && v >> shift == prefix) list[atomicAdd(&sh.listed, 1u)] = v;
        };
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          if (k >= nk) break;
          give(near[k]);
        }
        for (int k = NK; k < nk; ++k) give(far_key(k));
        cluster.sync();
        listed = sh.in_bin;
        const uint32_t n_of = lane < ranks ? *cluster.map_shared_rank(&sh.listed, lane) : 0;
        uint32_t upto = n_of;  // keys of the ranks up to this lane's
#pragma unroll
        for (int k = 1; k < kMaxCluster; k <<= 1) {
          const uint32_t o = __shfl_up_sync(0xffffffffu, upto, k);
          if (lane >= k) upto += o;
        }
#pragma unroll
        for (int i = 0; i < int(kList) / kSelThreads; ++i) {
          const uint32_t at = i * kSelThreads + tid;
          if (at - lane >= listed) break;
          uint32_t q = 0, before = 0;
#pragma unroll
          for (int k = 0; k < kMaxCluster - 1; ++k) {
            const uint32_t u = __shfl_sync(0xffffffffu, upto, k);
            if (k < ranks - 1 && at >= u) q = k + 1, before = u;
          }
          part[i] = at < listed ? *cluster.map_shared_rank(list + (at - before), q) : 0;
        }
        own = true;
      }
    }
  }

  // places, from the counts before a warp's run
  uint32_t gt = 0, eq = 0;
  auto tally = [&](uint32_t v) { gt += v > T, eq += v == T; };
#pragma unroll
  for (int k = 0; k < NK; ++k) {
    if (k >= nk) break;
    tally(near[k]);
  }
  for (int k = NK; k < nk; ++k) tally(far_key(k));
  gt = __reduce_add_sync(0xffffffffu, gt), eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) sh.gt[warp] = gt, sh.eq[warp] = eq;
  __syncthreads();
  if (warp == 0) {  // the block's counts, to every rank
    const uint32_t g = __reduce_add_sync(0xffffffffu, sh.gt[lane]);
    const uint32_t e = __reduce_add_sync(0xffffffffu, sh.eq[lane]);
    if (lane < ranks) {
      *cluster.map_shared_rank(&sh.rank_gt[rank], lane) = g;
      *cluster.map_shared_rank(&sh.rank_eq[rank], lane) = e;
    }
  }
  cluster.sync();  // (the last access to another block's shared memory lies before it)
  uint32_t gt_at = sum_before(sh.gt, warp, lane), eq_at = sum_before(sh.eq, warp, lane);
  for (int q = 0; q < rank; ++q) gt_at += sh.rank_gt[q], eq_at += sh.rank_eq[q];
  const uint32_t below = (1u << lane) - 1;
  if (eq == 0 || eq_at >= ties) {  // none of the warp's equal keys stays
    int32_t *at = kept + a.sink + gt_at + min(eq_at, ties);
    auto place = [&](int k, uint32_t v) {
      const unsigned stays = __ballot_sync(0xffffffffu, v > T);
      if (v > T) at[__popc(stays & below)] = first + r0 + 32 * k + lane;
      at += __popc(stays);
    };
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      if (k >= nk) break;
      place(k, near[k]);
    }
    for (int k = NK; k < nk; ++k) place(k, far_key(k));
    return;
  }
  auto place = [&](int k, uint32_t v) {  // (all lanes of the warp)
    const unsigned eqs = __ballot_sync(0xffffffffu, v == T);
    const bool stay = v > T || (v == T && eq_at + __popc(eqs & below) < ties);
    const unsigned stays = __ballot_sync(0xffffffffu, stay);
    if (stay) kept[a.sink + gt_at + min(eq_at, ties) + __popc(stays & below)] = first + r0 + 32 * k + lane;
    gt_at += __popc(stays) - (min(eq_at + __popc(eqs), ties) - min(eq_at, ties));
    eq_at += __popc(eqs);
  };
#pragma unroll
  for (int k = 0; k < NK; ++k) {
    if (k >= nk) break;
    place(k, near[k]);
  }
  for (int k = NK; k < nk; ++k) place(k, far_key(k));
}

// RB: bytes of a row; ROWS: rows of a warp (16 or 32).
template <int RB, int ROWS>
__global__ void __launch_bounds__(256) evict_copy_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int CH = RB / 16, STEPS = ROWS * CH / 32, NU = STEPS % 4 == 0 ? 4 : STEPS % 3 == 0 ? 3 : STEPS % 2 == 0 ? 2 : 1;
  const int s = blockIdx.y, h = blockIdx.z, lane = threadIdx.x & 31;
  const int j = (blockIdx.x * 8 + (threadIdx.x >> 5)) * ROWS + lane;
  grid_dependency();
  // (not by the choice, whose other blocks may still have to read the length: new_len may be len)
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0)
    a.new_len[s] = min(clamped_len(a.len[s], a.max_len), a.keep);
  if (j - lane >= a.keep) return;
  uint32_t from = 0, to = 0;
  bool on = false;
  if (lane < ROWS && j < a.keep) {
    const int src = a.kept[(int64_t(s) * a.c.hkv + h) * a.keep + j];
    if (src >= 0) {
      from = kv_row32(a.c, a.pages + s * a.pages_ld, h, src);
      to = kv_row32(a.c, a.new_pages + s * a.new_pages_ld, h, j);
      on = from != kNoRow && to != kNoRow;
      if (!on)
        index_error(a.status, kIdxEvictPage,
                    from == kNoRow ? a.pages[s * a.pages_ld + quotient(src, a.c.page)]
                          : a.new_pages[s * a.new_pages_ld + quotient(j, a.c.page)]);
    }
  }
  const unsigned live = __ballot_sync(0xffffffffu, on);
  if (live == 0) return;
  float sum = 0.f;
  if (on) sum = a.c.sums[from];
#pragma unroll 1
  for (int st = 0; st < STEPS; st += NU) {
    uint4 k[NU], v[NU];
    uint32_t dst[NU];
    bool ok[NU];
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int c = (st + i) * 32 + lane, row = c / CH, ch = c % CH;
      const uint32_t src = __shfl_sync(0xffffffffu, from, row);
      dst[i] = __shfl_sync(0xffffffffu, to, row);
      ok[i] = live >> row & 1;
      if (ok[i]) {
        k[i] = *reinterpret_cast<const uint4 *>(a.c.k + size_t(src) * RB + ch * 16);
        v[i] = *reinterpret_cast<const uint4 *>(a.c.v + size_t(src) * RB + ch * 16);
      }
    }
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int ch = ((st + i) * 32 + lane) % CH;
      if (ok[i]) {
        *reinterpret_cast<uint4 *>(a.c.k + size_t(dst[i]) * RB + ch * 16) = k[i];
        *reinterpret_cast<uint4 *>(a.c.v + size_t(dst[i]) * RB + ch * 16) = v[i];
      }
    }
  }
  if (!on) return;
  a.c.sums[to] = sum;
  if (a.c.type == MQ_Q8_0) {  // a lane its own row's scales
    constexpr int NB = RB / 32;
    const size_t f = size_t(from) * NB, t = size_t(to) * NB;
    __half ks[NB], vs[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) ks[i] = a.c.ks[f + i], vs[i] = a.c.vs[f + i];
#pragma unroll
    for (int i = 0; i < NB; ++i) a.c.ks[t + i] = ks[i], a.c.vs[t + i] = vs[i];
  }
}

template <int RB>
mq_status launch_copy(const EvictArgs &a, cudaStream_t s, const DeviceState *st) {
  const int64_t rows = a.S * a.c.hkv * a.keep;
  const bool few = rows < int64_t(st->sms) * 16 * 32;  // less than 16 warps of 32 rows per SM
  const int per_block = 8 * (few ? 16 : 32);
  const dim3 grid((a.keep + per_block - 1) / per_block, (unsigned)a.S, a.c.hkv);
  return launch_dependent("evict_copy_kernel", few ? evict_copy_kernel<RB, 16> : evict_copy_kernel<RB, 32>,
                          grid, dim3(256, 1, 1), 0, s, a);
}

}  // namespace

mq_status init_kv_evict(DeviceState *st) {
  const int bytes = kKeysHeld * 4;
  if (bytes + (int)sizeof(SelShared) > st->smem_optin)
    return fail(MQ_ERR_LAUNCH, "evict_select_kernel needs %d bytes of shared memory, the device allows %d",
                bytes + (int)sizeof(SelShared), st->smem_optin);
  cudaError_t e =
      cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  for (int i = 0; i < 5 && e == cudaSuccess; ++i) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1 << i);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = bytes;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1 << i, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&st->evict_clusters[i], evict_select_kernel, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      st->evict_clusters[i] = 0;
    }
  }
  return e == cudaSuccess ? MQ_OK : cuda_fail(e, "cudaFuncSetAttribute", "evict_select_kernel");
}

mq_status launch_kv_evict(const EvictArgs &a, cudaStream_t s, const DeviceState *st) {
  // blocks of a cluster: at least 4096 candidates each (4096 rows of 4 heads: 8.6 us by one block a
  // head, 9.5 by two; 16384: 14.7, 12.4 by two, 11.0 by four or eight; 32768: 13.4 by four, 12.5 by
  // eight; 131072: 20.0 by eight, 18.8 by sixteen), as long as all clusters are resident at once: 15
  // of eight blocks here, so that 16 heads of 32768 rows take 13.6 us by four blocks each and 21.4
  // by eight.
  int ranks = 1;
  for (int i = 1; i < 5 && (a.max_len >> i) >= 4096 && a.S * a.c.hkv <= st->evict_clusters[i]; ++i)
    ranks = 1 << i;
  const int per_rank = ((a.max_len + ranks - 1) / ranks + kSelThreads - 1) / kSelThreads * kSelThreads;
  const int held = std::max(0, std::min(per_rank - 16 * kSelThreads, kKeysHeld));
  mq_status r = launch_cluster("evict_select_kernel", evict_select_kernel,
                               dim3(ranks, (unsigned)a.S, a.c.hkv), dim3(kSelThreads, 1, 1),
                               size_t(held) * 4, s, ranks, a, held);
  if (r != MQ_OK) return r;
  switch (a.c.type == MQ_Q8_0 ? a.c.dim : 2 * a.c.dim) {
    case 64: return launch_copy<64>(a, s, st);
    case 96: return launch_copy<96>(a, s, st);
    case 128: return launch_copy<128>(a, s, st);
    case 192: return launch_copy<192>(a, s, st);
    case 256: return launch_copy<256>(a, s, st);
    case 384: return launch_copy<384>(a, s, st);
    default: return launch_copy<512>(a, s, st);
  }
}

}  // namespace mq
