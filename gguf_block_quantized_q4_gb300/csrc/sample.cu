// sample.cu -- mq_sample: the next token of each row of logits, by temperature, top-k, top-p and
// min-p, from one given uniform number per row.
//
// Mathematics.  With m the row's largest logit and T the temperature, token i weighs
// w_i = exp((l_i - m) / T) = 2^-y_i.  In the order of falling logits (equal ones by rising index)
// top-k keeps a prefix by its length and top-p one by its share of the sum, so both are a cut: the
// last (logit, index) that stays.  The token is the first, in the order of the indexes, at which the
// running sum of the weights that stay passes u times their sum.
//
// What bounds it: the logits are read once (64 rows of 151936: 5.8 us); then latency.  A thread block
// cluster holds a row in its shared memory, a slice of consecutive tokens per block, so everything
// behind the reading costs no memory traffic: the maximum (one exchange over the cluster), a cut
// (each two or three exchanges), the sums and the token (one).
//
// Weights are whole numbers in units of 2^-44 (44 bits for the largest; a token 2^-45 below it weighs
// nothing, and fewer than 2^19 tokens fit a 64-bit sum).  Sums of whole numbers do not depend on their
// order, so neither do results: not on the cluster's size, nor on the atomics.  The exponential
// (weight) is right to about 2^-27 of itself: binary32's own 2^-24 would move the running sum
// enough to name another token in one of a few hundred rows of flat logits.
//
// A cut: the row's tokens are counted, or their weights added, in 2048 bins of y (45 to each halving),
// which the cluster's blocks add to rank 0's; a scan names the bin that holds the cut.  The few
// tokens of that bin (or, for top-k, of all bins up to it) are listed and sorted by each block for
// itself.  Where they are more than a list holds (equal or nearly equal logits) three more rounds of
// bins, of the logit's bits, name the logit and a count of equals the index.
#include <cooperative_groups.h>

#include <algorithm>

#include "kv.cuh"
#include "sample.cuh"

namespace cg = cooperative_groups;

namespace mq {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048, kPer = kBins / kThreads;  // bins of a thread in a scan
constexpr int kList = 1024;                           // tokens listed and sorted
constexpr int kMaxRanks = 16;
constexpr int kUnit = 44;            // weights in units of 2^-kUnit
constexpr float kDeep = 45.f;        // y from which a token weighs nothing
constexpr float kBinsPerHalving = 45.f;
constexpr int kLastBin = kBins - 1;  // (2025 and up weigh nothing)

struct Shared {
  // the block's bins, low and high words; while a cut's tokens are sorted: its own list, all lists
  union {
    uint32_t bins[2][kBins];
    u64 list[2][kList];
  };
  uint32_t total[2][kBins];  // rank 0's: the cluster's bins
  u64 warp_sum[kWarps];
  uint32_t warp_key[kWarps], warp_index[kWarps];
  uint32_t rank_key[kMaxRanks], rank_index[kMaxRanks], rank_n[kMaxRanks];
  u64 rank_sum[kMaxRanks];
  u64 above, inside;  // of the bin that was chosen: what lies before it, and in it
  uint32_t bin, listed, cut_key, cut_index;
  float c_hi, c_lo, floor_less;
  u64 sum;
};

// Order of the logits as unsigned numbers (-0 as 0), and back.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

struct Scale {
  float top, hi, lo;  // m; log2(e) / T in two parts
};
// y of a logit, rounded: for the bins (it falls with the logit, never the other way round).
__device__ __forceinline__ float depth(const Scale &s, float x) { return __fmul_rn(__fsub_rn(s.top, x), s.hi); }
__device__ __forceinline__ int bin_of(const Scale &s, float x) {
  if (x == s.top) return 0;
  const float y = depth(s, x);
  return y < kDeep ? (int)(y * kBinsPerHalving) : kLastBin;  // (NaN: infinite logits, infinite temperatures)
}
// The weight 2^-y in units of 2^-kUnit.  The difference, its product with log2(e) / T and 1 + ln 2 f are
// carried in two parts; n is y rounded and f = n - y, so that 2^-y = 2^-n e^(f ln 2), whose
// series runs to the ninth power (|f ln 2| < 0.347: the tenth is 2^-37).
__device__ __forceinline__ u64 weight(const Scale &s, float x) {
  if (x == s.top) return u64(1) << kUnit;
  const float d = __fsub_rn(s.top, x), y = __fmul_rn(d, s.hi);
  if (!(y < kDeep)) return 0;
  const float b = __fsub_rn(d, s.top);
  const float e = __fsub_rn(__fsub_rn(s.top, __fsub_rn(d, b)), __fadd_rn(x, b));  // top - x - d
  const float less = __fmaf_rn(d, s.hi, -y) + __fmaf_rn(d, s.lo, e * s.hi);       // y's second part
  const float n = rintf(y), f = __fsub_rn(n, y);
  constexpr float ln2 = 0.693147182464599609375f, ln2_lo = -1.904654323148236e-9f;
  const float t = __fmul_rn(f, ln2);
  const float t_lo = __fmaf_rn(f, ln2, -t) + __fmaf_rn(f, ln2_lo, -less * ln2);
  float q = 1.f / 362880;
  q = fmaf(q, t, 1.f / 40320), q = fmaf(q, t, 1.f / 5040), q = fmaf(q, t, 1.f / 720);
  q = fmaf(q, t, 1.f / 120), q = fmaf(q, t, 1.f / 24), q = fmaf(q, t, 1.f / 6), q = fmaf(q, t, 0.5f);
  const float rest = fmaf(t * t, q, fmaf(t, t_lo, t_lo));
  const int mantissa = (1 << 30) + __float2int_rn(t * 0x1p30f) + __float2int_rn(rest * 0x1p30f);
  return (u64(uint32_t(mantissa)) << (kUnit - 30)) >> (int)n;
}

__device__ __forceinline__ u64 shfl_up(u64 v, int by) { return __shfl_up_sync(0xffffffffu, v, by); }

// Adds to a 64-bit sum kept as two words (a 64-bit atomic on shared memory is a loop of exchanges).
__device__ __forceinline__ void add_to(uint32_t *lo, uint32_t *hi, u64 v) {
  const uint32_t w = (uint32_t)v, before = atomicAdd(lo, w);
  const uint32_t up = (uint32_t)(v >> 32) + (before + w < before);
  if (up) atomicAdd(hi, up);
}

template <int IO>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a, int per_rank) {
  extern __shared__ __align__(16) float slice[];  // [per_rank]
  __shared__ __align__(16) Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.y;
  for (int i = tid; i < 2 * kBins; i += kThreads) (&sh.bins[0][0])[i] = (&sh.total[0][0])[i] = 0;
  if (tid == 0) sh.listed = 0;
  cluster.barrier_arrive();  // (every block's shared memory exists and is clear; waited for below)
  grid_dependency();

  const float T = a.temperature ? a.temperature[row] : 1.f;
  const int k = a.top_k ? a.top_k[row] : 0;
  const float p = a.top_p ? a.top_p[row] : 1.f, floor_p = a.min_p ? a.min_p[row] : 0.f;
  const float u = a.u[row];
  const bool greedy = !(T > 0.f), by_count = k > 0 && k < a.V, by_share = p < 1.f, by_floor = floor_p > 0.f;
  if (tid == 0 && !greedy) {
    const double c = 1.4426950408889634 / (double)T;
    sh.c_hi = (float)c, sh.c_lo = (float)(c - (double)sh.c_hi);
  }

  // ---- the slice: tokens first .. first + n - 1 ----
  // The row's 16-byte blocks in order, as it lies in memory; a token that is none is -inf.
  using E = typename std::conditional<IO == MQ_F32, float, uint16_t>::type;
  constexpr int EB = 16 / sizeof(E);  // elements of a block
  const E *const from = static_cast<const E *>(a.logits) + row * a.ld;
  const int off = (int)(reinterpret_cast<uintptr_t>(from) % 16 / sizeof(E));
  const int first = rank * per_rank - off;  // (below 0 in rank 0 where the row starts inside a block)
  const int n = max(0, min(per_rank, (int)a.V - first));
  auto read = [&](int i) { return load_io1(from, IO, i); };
  auto clean = [](float x) { return x == x ? x : -INFINITY; };
  float top = -INFINITY;
  {
    constexpr int U = 4;
    for (int c0 = tid; c0 * EB < n; c0 += U * kThreads) {
      uint4 v[U];
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const int i = first + (c0 + q * kThreads) * EB;
        if (i >= 0 && i + EB <= a.V && (c0 + q * kThreads) * EB < n) v[q] = *reinterpret_cast<const uint4 *>(from + i);
      }
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const int at = (c0 + q * kThreads) * EB, i = first + at;
        if (at >= n) break;
        float x[EB];
        if (i >= 0 && i + EB <= a.V) {
          const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
          for (int e = 0; e < EB; ++e) {
            if (IO == MQ_F32) {
              x[e] = __uint_as_float(w[e % 4]);
            } else {
              const uint16_t h = (uint16_t)(w[e / 2 % 4] >> 16 * (e & 1));
              x[e] = IO == MQ_BF16 ? __uint_as_float(uint32_t(h) << 16) : __half2float(__ushort_as_half(h));
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < EB; ++e) x[e] = i + e >= 0 && i + e < a.V ? read(i + e) : -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < EB; ++e) x[e] = clean(x[e]), top = fmaxf(top, x[e]);
#pragma unroll
        for (int e = 0; e < EB; e += 4)
          *reinterpret_cast<float4 *>(slice + at + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
      }
    }
  }
  // (what the last block of 16 bytes has past the slice's end is -inf and belongs to no token)
  const int run = ((n + kThreads - 1) / kThreads) | 1;  // a thread's tokens, for passes in order: an
  const int r0 = min(tid * run, n), r1 = min(r0 + run, n);  // odd number, so no two share a bank

  // ---- the maximum ----
  uint32_t top_key = __reduce_max_sync(0xffffffffu, key_of(top));
  if (lane == 0) sh.warp_key[warp] = top_key;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top_key = max(top_key, sh.warp_key[w]);
  uint32_t top_index = 0xffffffffu;
  if (greedy) {  // the block's first token with its maximum
    for (int i = r0; i < r1; ++i)
      if (key_of(slice[i]) == top_key) {
        top_index = first + i;
        break;
      }
    top_index = __reduce_min_sync(0xffffffffu, top_index);
    if (lane == 0) sh.warp_index[warp] = top_index;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) top_index = min(top_index, sh.warp_index[w]);
  }
  cluster.barrier_wait();
  if (tid < ranks) {
    *cluster.map_shared_rank(&sh.rank_key[rank], tid) = top_key;
    *cluster.map_shared_rank(&sh.rank_index[rank], tid) = top_index;
  }
  cluster.sync();
  for (int q = 0; q < ranks; ++q) {
    const uint32_t key = sh.rank_key[q];
    if (key > top_key) top_key = key, top_index = sh.rank_index[q];
    else if (key == top_key) top_index = min(top_index, sh.rank_index[q]);
  }
  const Scale s = {logit_of(top_key), sh.c_hi, sh.c_lo};
  auto finish = [&](int token, float logprob) {
    a.token[row] = token;
    if (a.logprob) a.logprob[row] = logprob;
  };
  if (greedy || s.top == -INFINITY) {
    if (rank == 0 && tid == 0) {
      if (s.top == -INFINITY)
        finish(-1, -INFINITY);
      else
        finish((int)top_index, 0.f);
    }
    return;
  }

  // ---- the cuts ----
  uint32_t cut_key = 0, cut_index = 0xffffffffu;  // the last that stays: no cut yet
  auto stays = [&](uint32_t key, int i) { return key > cut_key || (key == cut_key && (uint32_t)(first + i) <= cut_index); };

  // Sums over the threads up to this one, and over all (sh.sum).
  auto scan = [&](u64 v) {
    u64 upto = v;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const u64 o = shfl_up(upto, i);
      if (lane >= i) upto += o;
    }
    __syncthreads();  // (the sums before have been read)
    if (lane == 31) sh.warp_sum[warp] = upto;
    __syncthreads();
    u64 all = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) before = all;
      all += sh.warp_sum[w];
    }
    if (tid == 0) sh.sum = all;
    return before + upto;
  };
  bool fresh = true;  // the bins are clear
  auto clear = [&] {
    if (!fresh) {
      cluster.sync();  // (the totals, and what is listed in the bins' place, have been read)
      for (int i = tid; i < 2 * kBins; i += kThreads) (&sh.bins[0][0])[i] = (&sh.total[0][0])[i] = 0;
      cluster.sync();
    }
    fresh = false;
  };
  // The bins, filled by add(), over the cluster; then the bin at which their sum reaches need(sum of all):
  // sh.bin, sh.above, sh.inside.
  auto choose = [&](auto add, auto need) {
    clear();
    add();
    __syncthreads();
    uint32_t(*total)[kBins] = sh.bins;
    if (ranks > 1) {
      total = reinterpret_cast<uint32_t(*)[kBins]>(cluster.map_shared_rank(&sh.total[0][0], 0));
      for (int i = tid; i < kBins; i += kThreads) {
        const u64 v = (u64)sh.bins[1][i] << 32 | sh.bins[0][i];
        if (v) add_to(&total[0][i], &total[1][i], v);
      }
      cluster.sync();
    }
    const uint4 lo = *reinterpret_cast<const uint4 *>(&total[0][kPer * tid]);
    const uint4 hi = *reinterpret_cast<const uint4 *>(&total[1][kPer * tid]);
    const u64 v[kPer] = {(u64)hi.x << 32 | lo.x, (u64)hi.y << 32 | lo.y, (u64)hi.z << 32 | lo.z, (u64)hi.w << 32 | lo.w};
    const u64 mine = v[0] + v[1] + v[2] + v[3];
    u64 before = scan(mine) - mine;
    __syncthreads();
    const u64 wanted = need(sh.sum);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      if (before < wanted && wanted <= before + v[q]) sh.bin = kPer * tid + q, sh.above = before, sh.inside = v[q];
      before += v[q];
    }
    __syncthreads();
    return wanted;
  };
  static_assert(kPer == 4, "a thread reads four bins at once");

  // Lists the cluster's tokens that wanted() names, sorted: the largest key first, equal ones by their
  // index.  False where they are too many.
  u64 *const sorted = sh.list[1];
  auto list = [&](auto wanted) -> int {
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const float x = slice[i];
      if (!wanted(x, i)) continue;
      const uint32_t at = atomicAdd(&sh.listed, 1u);
      if (at < kList) sh.list[0][at] = (u64)key_of(x) << 32 | ~(uint32_t)(first + i);
    }
    __syncthreads();
    if (tid < ranks) *cluster.map_shared_rank(&sh.rank_n[rank], tid) = sh.listed;
    cluster.sync();
    int all = 0;
    for (int q = 0; q < ranks; ++q) all += (int)min(sh.rank_n[q], (uint32_t)kList + 1);
    if (tid == 0) sh.listed = 0;
    if (all > kList) return -1;
    int size = 32;  // a power of two
    while (size < all) size *= 2;
    for (int i = tid; i < size; i += kThreads) {
      u64 v = 0;
      int at = i;
      for (int q = 0; q < ranks && at >= 0; ++q) {
        const int there = (int)sh.rank_n[q];
        if (at < there) v = cluster.map_shared_rank(sh.list[0], q)[at], at = -1;
        else at -= there;
      }
      sorted[i] = v;
    }
    __syncthreads();
    for (int len = 2; len <= size; len *= 2)  // bitonic
      for (int gap = len / 2; gap; gap /= 2) {
        for (int t = tid; t < size / 2; t += kThreads) {
          const int i = 2 * t - (t & (gap - 1)), j = i + gap;
          const u64 x = sorted[i], y = sorted[j];
          if ((x < y) == ((i & len) == 0)) sorted[i] = y, sorted[j] = x;
        }
        __syncthreads();
      }
    return all;
  };
  auto cut_at = [&](int at) { cut_key = (uint32_t)(sorted[at] >> 32), cut_index = ~(uint32_t)sorted[at]; };
  // The cut in the sorted list's first `most` tokens at which the weights' sum, from `above` on,
  // reaches need(its sum over them).
  auto cut_by_weight = [&](int most, u64 above, auto need) {
    u64 w[kList / kThreads], mine = 0;
#pragma unroll
    for (int q = 0; q < kList / kThreads; ++q) {
      const int i = kList / kThreads * tid + q;
      w[q] = i < most ? weight(s, logit_of((uint32_t)(sorted[i] >> 32))) : 0;
      mine += w[q];
    }
    u64 before = scan(mine) - mine + above;
    __syncthreads();
    const u64 wanted = need(above + sh.sum);
#pragma unroll
    for (int q = 0; q < kList / kThreads; ++q) {
      if (before < wanted && wanted <= before + w[q]) sh.bin = kList / kThreads * tid + q;
      before += w[q];
    }
    __syncthreads();
    cut_at(sh.bin);
  };
  // The first token in order at which the sum of amount(), over the cluster's blocks in order, passes
  // `target`: true in the block that has it, whose thread calls found(index).
  auto find = [&](auto amount, auto target, auto found) {
    u64 mine = 0;
    for (int i = r0; i < r1; ++i) mine += amount(i);
    const u64 before = scan(mine) - mine;
    __syncthreads();
    if (tid < ranks) *cluster.map_shared_rank(&sh.rank_sum[rank], tid) = sh.sum;
    cluster.sync();
    u64 all = 0, lead = 0;
    for (int q = 0; q < ranks; ++q) {
      if (q == rank) lead = all;
      all += sh.rank_sum[q];
    }
    const u64 at = target(all);
    u64 sum = lead + before;
    if (at < sum || at >= sum + mine) return;
    for (int i = r0; i < r1; ++i) {
      sum += amount(i);
      if (at < sum) {
        found(i, all);
        break;
      }
    }
  };
  // The cut by the logits' bits where a list is too long: among the tokens of the chosen bin that stay
  // so far, the one at which their count or weight reaches `need`.
  auto cut_by_bits = [&](int bin, bool weights, u64 need) {
    uint32_t prefix = 0;
    for (int level = 0; level < 3; ++level) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
      choose(
          [&] {
            for (int i = tid; i < n; i += kThreads) {
              const float x = slice[i];
              const uint32_t key = key_of(x), rev = ~key;
              if (bin_of(s, x) != bin || !stays(key, i) || (level && rev >> (shift + bits) != prefix)) continue;
              const uint32_t digit = rev >> shift & ((1u << bits) - 1);
              if (weights) add_to(&sh.bins[0][digit], &sh.bins[1][digit], weight(s, x));
              else atomicAdd(&sh.bins[0][digit], 1u);
            }
          },
          [&](u64) { return need; });
      need -= sh.above;
      prefix = prefix << bits | sh.bin;
      __syncthreads();
    }
    const uint32_t key = ~prefix;
    if (weights) {
      const u64 w = weight(s, logit_of(key));
      need = (need + w - 1) / w;
    }
    find([&](int i) -> u64 { return key_of(slice[i]) == key && stays(key, i); }, [&](u64) { return need - 1; },
         [&](int i, u64) {
           for (int q = 0; q < ranks; ++q) *cluster.map_shared_rank(&sh.cut_index, q) = first + i;
         });
    cluster.sync();
    cut_key = key, cut_index = sh.cut_index;
  };
  auto share = [&](u64 all) {
    const double x = ceil((double)p * (double)all);
    return x >= 1.0 ? min((u64)x, all) : u64(1);
  };

  bool shared_out = !by_share;
  if (by_count) {
    choose(
        [&] {
          for (int i = tid; i < n; i += kThreads) atomicAdd(&sh.bins[0][bin_of(s, slice[i])], 1u);
        },
        [&](u64) { return (u64)k; });
    const int bin = (int)sh.bin, above = (int)sh.above;
    const u64 upto = sh.above + sh.inside;
    if (bin < kLastBin) {  // (else all that weighs something stays)
      if (upto <= kList) {
        list([&](float x, int) { return bin_of(s, x) <= bin; });
        if (by_share) cut_by_weight(k, 0, share);
        else cut_at(k - 1);
        shared_out = true;
      } else if (list([&](float x, int) { return bin_of(s, x) == bin; }) >= 0) {
        cut_at(k - above - 1);
      } else {
        cut_by_bits(bin, false, k - above);
      }
    }
  }
  if (!shared_out) {
    const u64 need = choose(
        [&] {
          for (int i = tid; i < n; i += kThreads) {
            const float x = slice[i];
            const int bin = bin_of(s, x);
            if (bin < kLastBin && stays(key_of(x), i)) add_to(&sh.bins[0][bin], &sh.bins[1][bin], weight(s, x));
          }
        },
        share);
    const int bin = (int)sh.bin;
    const u64 above = sh.above;
    const int listed = list([&](float x, int i) { return bin_of(s, x) == bin && stays(key_of(x), i); });
    if (listed >= 0) cut_by_weight(listed, above, [&](u64) { return need; });
    else cut_by_bits(bin, true, need - above);
  }

  // ---- the token ----
  float least = -INFINITY;  // min-p: w < min_p is l < m + T ln(min_p)
  if (by_floor && T < INFINITY) least = __double2float_ru((double)s.top + (double)T * log((double)fminf(floor_p, 1.f)));
  find(
      [&](int i) -> u64 {
        const float x = slice[i];
        return x >= least && stays(key_of(x), i) ? weight(s, x) : 0;
      },
      [&](u64 all) {
        const double x = (double)u * (double)all;
        return x > 0.0 ? min((u64)x, all - 1) : u64(0);
      },
      [&](int i, u64 all) {
        // ln w - ln(sum): of the sum the part past the largest weight where it is small
        const float x = slice[i], one = 0x1p-44f;
        const float l = x == s.top ? 0.f : -(float)(((double)s.top - (double)x) / (double)T);
        const u64 rest = all - min(all, u64(1) << kUnit);
        finish(first + i, l - log1pf((float)rest * one));
      });
}

}  // namespace

namespace {
// The slice of a block, in floats (whole 16-byte blocks of logits, one more for a row that starts
// inside one), and its shared memory.
int per_rank_of(int64_t V, int ranks) { return (int)((V + 8 + ranks - 1) / ranks + 7) / 8 * 8; }
size_t smem_of(int per_rank) { return size_t(per_rank) * 4; }
}  // namespace

mq_status init_sample(DeviceState *st) {
  cudaError_t e = cudaSuccess;
  auto set_up = [&](auto *kernel) {
    if (e != cudaSuccess) return;
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return;
    const int most = st->smem_optin - (int)fa.sharedSizeBytes;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return;
    st->sample_smem = most;
    for (int i = 0; i < 5; ++i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(1 << i);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = most;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = 1 << i, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&st->sample_clusters[i], kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        st->sample_clusters[i] = 0;
      }
    }
  };
  set_up(sample_kernel<MQ_F32>);
  set_up(sample_kernel<MQ_F16>);
  set_up(sample_kernel<MQ_BF16>);
  return e == cudaSuccess ? MQ_OK : cuda_fail(e, "cudaFuncSetAttribute", "sample_kernel");
}

mq_status launch_sample(const SampleArgs &a, cudaStream_t s, const DeviceState *st) {
  // Blocks of a cluster: so many that two blocks fit an SM (slices of 20 thousand logits), and where
  // the rows are few, twice as many as long as all blocks have an SM and 2048 logits of their own.
  int r = 0;
  while (r < 4 && per_rank_of(a.V, 1 << r) > 20 * 1024) ++r;
  while (r < 4 && a.B << (r + 1) <= st->sms && a.V >> (r + 1) >= 2048) ++r;
  while (r > 0 && st->sample_clusters[r] == 0) --r;
  const int ranks = 1 << r, per_rank = per_rank_of(a.V, ranks);
  if (st->sample_clusters[r] == 0 || smem_of(per_rank) > (size_t)st->sample_smem)
    return fail(MQ_ERR_SHAPE, "mq_sample: V=%lld does not fit the shared memory of a cluster of %d blocks",
                (long long)a.V, ranks);
  auto *kernel = a.io == MQ_F32 ? sample_kernel<MQ_F32> : a.io == MQ_F16 ? sample_kernel<MQ_F16> : sample_kernel<MQ_BF16>;
  return launch_cluster("sample_kernel", kernel, dim3(ranks, (unsigned)a.B, 1), dim3(kThreads, 1, 1), smem_of(per_rank),
                        s, ranks, a, per_rank);
}

}  // namespace mq
