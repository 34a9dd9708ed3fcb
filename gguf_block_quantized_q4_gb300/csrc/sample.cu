// sample.cu -- mq_sample: the next token of each row of logits, by temperature, top-k, top-p and
// min-p, from one given uniform number per row.
//
// Mathematics.  With m the row's largest logit and T the temperature, token i weighs
// w_i = exp((l_i - m) / T) = 2^-y_i.  In the order of falling logits (equal ones by rising index)
// top-k keeps a prefix by its length and top-p one by its share of the sum, so both are a cut: the
// last (logit, index) that stays.  The token is the first, in the order of the indexes, at which the
// running sum of the weights that stay passes u times their sum.
//
// What bounds it: the logits are read once (64 rows of 151936: 5.7 us); then latency.  A thread block
// cluster has a row, a run of consecutive tokens per block and of those one per warp, read 128 at a time:
// such a group's maximum stays in shared memory.  What follows the maximum (one exchange over the
// cluster) reads only the groups that can matter: a cut's tokens, or what a cut or min-p has left, are in
// the few groups whose maxima reach them.  Only rows without limits, the sum that top-p takes its share of,
// and flat rows read all logits again, then from the L2 cache.
//
// Weights are whole numbers in units of 2^-44 (44 bits for the largest; a token 2^-45 below it weighs
// nothing, and fewer than 2^19 tokens fit a 64-bit sum), of 2^-38 or 2^-34 in flat rows, whose deep
// weights then fit 32 bits, which a shared atomic adds in 10 cycles a warp (64 bits take 25).  Sums of whole
// numbers do not depend on their order, so neither do results: not on the cluster's size, nor on the
// atomics, nor on the row's place.  The exponential is right to 2^-27 of itself down to 2^-8 of the largest weight: binary32's own
// 2^-24 would move the running sum enough to name another token in one of a few hundred rows of
// flat logits.  Below that it is the hardware's (2^-21, the errors of either sign).
//
// A cut: the groups' maxima are counted in 2048 bins of y (45 to each halving), which the cluster's blocks
// add up; a scan names the bin down to which k of them lie.  There are at least k tokens down to that
// bin and hardly any more: these are listed, and sorted by each block for itself.  Where k is too large for
// that, or the listed tokens have too small a share, all tokens are counted, or their weights added, in
// the bins; the few tokens of the bin that holds the cut are listed then.  Where they are more than
// a list holds (nearly equal logits) the bin is divided in 2048 once more, and where that does not do
// (equal ones) three rounds of bins, of the logit's bits, name the logit and a count of equals the index.
//
// Measured (f32): one row of 151936 with top-k 40 and top-p 13.3 us, greedy 3.9, the temperature alone 10.3, top-p of
// a flat row 23 to 32; 64 such rows with limits of their own 44 to 58 us over twelve draws of these, 51 on average
// (nine times their bytes' time: rows of top-p pass over their logits three times, eight blocks each); 256
// with min-p 59.2 us (39% of a plain copy's rate); 16 rows of 32003 bf16 logits, most of them masked, top-p
// 20.2 us.  (First form 25.0, 76.2, 155.4 and 23.3 us.)  Of the 50 thousand cycles of a flat top-p row the
// histogram takes 7, the choice of its bin 7, the lists 7, their sort 8, the last sums 10: barriers of the
// cluster in each.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

#include "kv.cuh"
#include "sample.cuh"

namespace cg = cooperative_groups;

namespace mq {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048, kPer = kBins / kThreads;  // bins of a thread in a scan
constexpr int kSide = 4;                              // tokens of a lane side by side
constexpr int kGroup = 32 * kSide;                    // of a warp: a group
constexpr int kList = 1024;                           // tokens listed and sorted
constexpr int kQuick = kList / 2;                     // groups' maxima that a list's tokens are found by
constexpr int kCounted = kThreads / 2;                // listed tokens that are sorted by counting
constexpr int kFew = 4;                               // groups that a warp goes through alone
constexpr int kMaxRanks = 16;
constexpr float kBinsPerHalving = 45.f;
constexpr int kLastBin = kBins - 1;  // (2026 and up weigh nothing)
constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: added to a number, it leaves the nearest integer in the low bits
constexpr uint32_t kMagicBits = 0x4b400000u;
constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLow = 1.92596299112661746887e-8f;  // log2(e) in two parts

struct Shared {
  // the block's bins, low and high words; while a cut's tokens are sorted: its own list, all lists
  union {
    uint32_t bins[2][kBins];
    u64 list[2][kList];
  };
  static_assert(kWarps * 64 * sizeof(float) <= kList * sizeof(u64), "the warps' queues lie in the second list");
  u64 warp_sum[kWarps];
  uint32_t warp_key[kWarps];
  uint32_t rank_key[kMaxRanks], rank_n[kMaxRanks];
  u64 rank_sum[kMaxRanks];
  u64 rank_look[kMaxRanks];  // (read without a barrier behind: a block that is ahead writes rank_sum meanwhile)
  u64 above, inside;  // of the bin that was chosen: what lies before it, and in it
  uint32_t bin, listed, cut_index;
  float least;
  double floor_log;  // T ln(min_p)
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
  float top, hi, lo;  // m (finite); log2(e) / T in two parts
  // Weights are in units of 2^-unit: 44, or, in rows of 2^14 tokens or more whose groups of 128 have maxima of
  // 2^-16 or 2^-8 of the largest weight or more on average, 38 or 34 (their sums are far above that
  // one).  A weight has less than 32 bits from y = unit - 29 (`deep`) on.
  int unit;
  float deep;
};
__device__ __forceinline__ float depth(const Scale &s, float x) { return __fmul_rn(__fsub_rn(s.top, x), s.hi); }
// The bin of a logit by its y, rounded (which falls with the logit, never the other way round).
__device__ __forceinline__ int bin_of(const Scale &s, float x) {
  return (int)min(__float_as_uint(__fmaf_rn(depth(s, x), kBinsPerHalving, kMagic)) - kMagicBits, (uint32_t)kLastBin);
}
// The weight 2^-y in units of 2^-unit.  The product of the difference d with log2(e) / T is carried in two
// parts; n is y rounded and f = n - y, so that 2^-y = 2^-n 2^f.  From y = 8 on (or 4, for the smaller
// unit; most tokens of most rows) 2^f is the hardware's, and the weight right to 2^-21, with an error that is as
// often above as below (its mean over f is -8e-9).  Above it (precise) 2^f is the series of e^(f ln 2) to
// the ninth power (|f ln 2| < 0.347: the tenth is 2^-37), with the rounding of d and 1 + f ln 2 in two
// parts: 2^-27.
__device__ __noinline__ u64 precise(float top, float hi, float lo, float x, int unit) {
  const float d = __fsub_rn(top, x), y = __fmul_rn(d, hi);
  const float b = __fsub_rn(d, top);
  const float e = __fsub_rn(__fsub_rn(top, __fsub_rn(d, b)), __fadd_rn(x, b));  // top - x - d
  const float less = __fmaf_rn(d, hi, -y) + __fmaf_rn(d, lo, e * hi);           // y's second part
  const float n = rintf(y), f = __fsub_rn(n, y);
  constexpr float ln2 = 0.693147182464599609375f, ln2_lo = -1.904654323148236e-9f;
  const float t = __fmul_rn(f, ln2);
  const float t_lo = __fmaf_rn(f, ln2, -t) + __fmaf_rn(f, ln2_lo, -less * ln2);
  float q = 1.f / 362880;
  q = fmaf(q, t, 1.f / 40320), q = fmaf(q, t, 1.f / 5040), q = fmaf(q, t, 1.f / 720);
  q = fmaf(q, t, 1.f / 120), q = fmaf(q, t, 1.f / 24), q = fmaf(q, t, 1.f / 6), q = fmaf(q, t, 0.5f);
  const float rest = fmaf(t * t, q, fmaf(t, t_lo, t_lo));
  const int mantissa = (1 << 30) + __float2int_rn(t * 0x1p30f) + __float2int_rn(rest * 0x1p30f);
  return (u64(uint32_t(mantissa)) << (unit - 30)) >> (int)n;
}
// kSide tokens' weights where all are deep; where not (`any`), those that are by whole().
struct Weights {
  uint32_t w[kSide], v[kSide], by[kSide];
  bool any;
  __device__ __forceinline__ Weights(const Scale &s, const float (&x)[kSide]) {
    any = false;
#pragma unroll
    for (int q = 0; q < kSide; ++q) {
      const float d = __fsub_rn(s.top, x[q]), y = __fmul_rn(d, s.hi), m = __fadd_rn(y, kMagic);
      const float n = __fsub_rn(m, kMagic), f = __fmaf_rn(-d, s.lo, __fmaf_rn(-d, s.hi, n));
      float r;
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(f));
      // r in [0.70, 1.42] as a whole number of 2^-22, in the low bits of its sum with 2^23; to the left by 8 and
      // to the right by n - (unit - 30), rounded (cut off, 150 thousand tokens would lose half a unit each).
      // (Past 32 the shift leaves zero: all of y from unit + 1 on, infinities and NaN, whose m are larger
      // or no numbers.)
      v[q] = __float_as_uint(__fmaf_rn(r, 0x1p22f, 0x1p23f)) << 8;
      by[q] = __float_as_uint(m) - (kMagicBits + (uint32_t)(s.unit - 30));
      w[q] = (__funnelshift_rc(v[q], 0u, by[q] - 1) + 1) >> 1;
      any |= y < s.deep;
    }
  }
  __device__ __forceinline__ u64 whole(const Scale &s, const float (&x)[kSide], int q) const {
    const float y = depth(s, x[q]);
    if (y < fminf(s.deep, 8.f)) return precise(s.top, s.hi, s.lo, x[q], s.unit);
    return y < s.deep ? (u64)v[q] << 8 >> (8 + (int)by[q]) : w[q];
  }
};
__device__ __noinline__ u64 weight(const Scale &s, float x) {
  const float in[kSide] = {x, -INFINITY, -INFINITY, -INFINITY};
  return Weights(s, in).whole(s, in, 0);
}

// -(top - x) / T - ln(sum 2^-unit), rounded once: each in two parts.  The sum is the largest weight (2^unit) and what is
// beside it; its logarithm y has the second part sum 2^-unit e^-y - 1 (one step of Newton's).
__device__ __noinline__ float log_share(float top, float x, float T, u64 sum, int unit) {
  const float d = __fsub_rn(top, x), b = __fsub_rn(d, top);
  const float e = __fsub_rn(__fsub_rn(top, __fsub_rn(d, b)), __fadd_rn(x, b));  // top - x - d
  const float l = __fdiv_rn(d, T), l_lo = l > 0.f ? __fdiv_rn(__fmaf_rn(-l, T, d) + e, T) : 0.f;
  const float rest = (float)(sum - min(sum, u64(1) << unit));
  const float y = log1pf(rest * __uint_as_float((uint32_t)(127 - unit) << 23));
  const u64 one = __umul64hi(sum, precise(y, kLog2e, kLog2eLow, 0.f, 62));  // 2^(unit - 2), nearly
  const float y_lo = (float)(int64_t)(one - (u64(1) << (unit - 2))) * __uint_as_float((uint32_t)(129 - unit) << 23);
  const float s = __fadd_rn(l, y), v = __fsub_rn(s, l);
  const float s_lo = __fadd_rn(__fsub_rn(l, __fsub_rn(s, v)), __fsub_rn(y, v));
  return __fsub_rn(0.f, __fadd_rn(s, __fadd_rn(s_lo, __fadd_rn(l_lo, y_lo))));
}

// floor(x v) for 0 < x < 1, and whether x v is more than that.
__device__ __forceinline__ u64 part_of(float x, u64 v, bool &more) {
  const uint32_t bits = __float_as_uint(x), e = bits >> 23;
  const u64 m = e ? (bits & 0x7fffffu) | 0x800000u : bits;  // x = m 2^-k
  const int k = 150 - max((int)e, 1);                       // 24 .. 149
  const u64 lo = m * v, hi = __umul64hi(m, v);
  if (k < 64) {
    more = (lo & ((u64(1) << k) - 1)) != 0;
    return hi << (64 - k) | lo >> k;
  }
  more = lo || k - 64 >= 64 || (hi & ((u64(1) << (k - 64)) - 1));
  return k < 128 ? hi >> (k - 64) : 0;
}

// Adds to a 64-bit sum kept as two words (a 64-bit atomic on shared memory is a loop of exchanges).
__device__ __forceinline__ void add_to(uint32_t *lo, uint32_t *hi, u64 v) {
  const uint32_t w = (uint32_t)v, before = atomicAdd(lo, w);
  const uint32_t up = (uint32_t)(v >> 32) + (before + w < before);
  if (up) atomicAdd(hi, up);
}
__device__ __forceinline__ void add_to(uint32_t *lo, uint32_t *hi, uint32_t w) {
  const uint32_t before = atomicAdd(lo, w);
  if (before + w < before) atomicAdd(hi, 1u);
}

// What a block's threads do together.  (Functions of their own, called from several places: a row passes
// through each code only once or twice, and what it costs to fetch counts.)

// Sums over the threads up to this one; over all in sh.sum, behind a barrier.
__device__ __noinline__ u64 scan(Shared &sh, u64 v) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 upto = v;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const u64 o = __shfl_up_sync(0xffffffffu, upto, i);
    if (lane >= i) upto += o;
  }
  __syncthreads();  // (the sums before have been read)
  if (lane == 31) sh.warp_sum[warp] = upto;
  __syncthreads();
  static_assert(kWarps == 16, "half a warp adds the warps' sums up");
  const u64 own = lane < kWarps ? sh.warp_sum[lane] : 0;
  u64 sums = own;
#pragma unroll
  for (int i = 1; i < kWarps; i <<= 1) {
    const u64 o = __shfl_up_sync(0xffffffffu, sums, i);
    if (lane >= i) sums += o;
  }
  if (threadIdx.x == kWarps - 1) sh.sum = sums;
  return __shfl_sync(0xffffffffu, sums - own, warp) + upto;
}

// What a cut asks for: a number, or of the sum the share p (at least something).
struct Need {
  u64 fixed;
  float p;  // used where fixed is 0
  __device__ __forceinline__ u64 of(u64 all) const {
    if (fixed) return fixed;
    if (!(p > 0.f)) return 1;
    bool more;
    const u64 n = part_of(p, all, more) + more;
    return max(n, u64(1));
  }
};

// The block's bins added up over the cluster, and the bin at which their sum reaches what is needed
// (returned): sh.bin, sh.above, sh.inside.
__device__ __noinline__ u64 choose(Shared &sh, uint32_t *totals, bool counts, Need need) {
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), tid = threadIdx.x, run = kBins / ranks;
  // a bin's word in the rank that adds it up
  auto owner = [&](int bin) { return cluster.map_shared_rank(totals, bin / run) + bin % run; };
  __syncthreads();
  const uint32_t *low = &sh.bins[0][kPer * tid], *high = &sh.bins[1][kPer * tid];
  if (ranks > 1) {
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int i = q * kThreads + tid;
      const uint32_t lo = sh.bins[0][i], hi = counts ? 0 : sh.bins[1][i];
      if ((lo | hi) == 0) continue;
      uint32_t *const to = owner(i);
      if (counts) atomicAdd(to, lo);
      else add_to(to, to + run, (u64)hi << 32 | lo);
    }
    cluster.sync();
    low = owner(kPer * tid), high = low + run;
  }
  static_assert(kPer == 4, "a thread reads four bins at once");
  const uint4 lo = *reinterpret_cast<const uint4 *>(low), hi = *reinterpret_cast<const uint4 *>(high);
  const u64 v[kPer] = {(u64)hi.x << 32 | lo.x, (u64)hi.y << 32 | lo.y, (u64)hi.z << 32 | lo.z, (u64)hi.w << 32 | lo.w};
  const u64 mine = v[0] + v[1] + v[2] + v[3];
  u64 before = scan(sh, mine) - mine;
  __syncthreads();
  const u64 wanted = need.of(sh.sum);
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    if (before < wanted && wanted <= before + v[q]) sh.bin = kPer * tid + q, sh.above = before, sh.inside = v[q];
    before += v[q];
  }
  __syncthreads();
  return wanted;
}

// A thread's share of something about each of n <= kCounted things: `parts` threads side by side to each.
struct Share {
  int parts, at, part;
  __device__ __forceinline__ explicit Share(int n) {
    parts = 2;
    while (parts < 32 && parts * 2 * n <= kThreads) parts *= 2;
    at = threadIdx.x / parts, part = threadIdx.x % parts;
  }
};

// The lists of the cluster's blocks (sh.listed tokens in sh.list[0]), sorted in sh.list[1]: the largest key
// first, equal ones by their index.  Their number, or -1 where they are too many.
__device__ __noinline__ int sort_lists(Shared &sh, int rank) {
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), tid = threadIdx.x;
  u64 *const sorted = sh.list[1];
  __syncthreads();
  if (tid < ranks) *cluster.map_shared_rank(&sh.rank_n[rank], tid) = sh.listed;
  cluster.sync();
  int all = 0;
  for (int q = 0; q < ranks; ++q) all += (int)min(sh.rank_n[q], (uint32_t)kList + 1);
  if (tid == 0) sh.listed = 0;
  if (all > kList) return -1;
  auto listed = [&](int i) {  // the i-th of the lists one behind the other
    for (int q = 0; q < ranks; ++q) {
      const int there = (int)sh.rank_n[q];
      if (i < there) return (u64)cluster.map_shared_rank(sh.list[0], q)[i];
      i -= there;
    }
    return u64(0);
  };
  if (all <= kCounted) {  // each token's place is the number of those before it
    u64 *const unsorted = sorted + kCounted;
    for (int i = tid; i < all; i += kThreads) unsorted[i] = listed(i);
    __syncthreads();
    const Share e(all);
    const u64 own = e.at < all ? unsorted[e.at] : 0;
    int place = 0;
    for (int j = e.part; j < all; j += e.parts) place += unsorted[j] > own;
    for (int d = 1; d < e.parts; d <<= 1) place += __shfl_xor_sync(0xffffffffu, place, d);
    if (e.at < all && e.part == 0) sorted[place] = own;
    __syncthreads();
    return all;
  }
  // bitonic, a warp's 64 in registers where the places compared lie in them (a step of all threads takes
  // 400 cycles, 1024 tokens by those alone 12 us)
  int size = 64;  // a power of two
  while (size < all) size *= 2;
  const int lane = tid & 31, i0 = (tid & ~31) * 2 + lane, i1 = i0 + 32;
  u64 x = i0 < all ? listed(i0) : 0, y = i1 < all ? listed(i1) : 0;
  auto larger = [](int i, int gap, int len) { return ((i & len) == 0) == ((i & gap) == 0); };
  auto within = [&](int gap, int len) {
    for (; gap; gap /= 2) {
      const bool inner = gap == 32;
      const u64 ox = inner ? y : __shfl_xor_sync(0xffffffffu, x, gap), oy = inner ? x : __shfl_xor_sync(0xffffffffu, y, gap);
      x = larger(i0, gap, len) ? max(x, ox) : min(x, ox);
      y = larger(i1, gap, len) ? max(y, oy) : min(y, oy);
    }
  };
  for (int len = 2; len <= 64; len *= 2) within(len / 2, len);
  for (int len = 128; len <= size; len *= 2) {
    __syncthreads();
    if (i0 < size) sorted[i0] = x, sorted[i1] = y;
    __syncthreads();
    for (int gap = len / 2; gap >= 64; gap /= 2) {
      for (int t = tid; t < size / 2; t += kThreads) {
        const int i = 2 * t - (t & (gap - 1)), j = i + gap;
        const u64 u = sorted[i], v = sorted[j];
        if ((u < v) == ((i & len) == 0)) sorted[i] = v, sorted[j] = u;
      }
      __syncthreads();
    }
    if (i0 < size) x = sorted[i0], y = sorted[i1];
    within(32, len);
  }
  __syncthreads();
  if (i0 < size) sorted[i0] = x, sorted[i1] = y;
  __syncthreads();
  return all;
}

// The place in the sorted list's first `most` tokens at which their weights' sum, from `above` on,
// reaches what is needed.
__device__ __noinline__ int place_by_weight(Shared &sh, const Scale &s, int most, u64 above, Need need) {
  constexpr int N = kList / kThreads;
  u64 w[N], mine = 0;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const int i = N * threadIdx.x + q;
    w[q] = i < most ? weight(s, logit_of((uint32_t)(sh.list[1][i] >> 32))) : 0;
    mine += w[q];
  }
  u64 before = scan(sh, mine) - mine + above;
  __syncthreads();
  const u64 wanted = need.of(above + sh.sum);
#pragma unroll
  for (int q = 0; q < N; ++q) {
    if (before < wanted && wanted <= before + w[q]) sh.bin = N * threadIdx.x + q;
    before += w[q];
  }
  __syncthreads();
  return (int)sh.bin;
}

// The row of the cluster `y`: first the rows that pass over all of their logits more than once (top-p without a
// small top-k, large top-k), in their order, then the others.
__device__ __noinline__ int row_of(Shared &sh, const SampleArgs &a, int y) {
  const int r = threadIdx.x, lane = r & 31, warp = r >> 5;
  bool slow = false;
  if (r < a.B) {
    const int k = a.top_k ? a.top_k[r] : 0;
    const bool few = k > 0 && k <= kQuick;
    slow = (!a.temperature || a.temperature[r] > 0.f) && !few && ((k > 0 && k < a.V) || (a.top_p && a.top_p[r] < 1.f));
  }
  const int n = __syncthreads_count(slow);
  const bool in = r < a.B && slow == (y < n);
  const unsigned who = __ballot_sync(0xffffffffu, in);
  if (lane == 0) sh.warp_key[warp] = __popc(who);
  __syncthreads();
  int at = y < n ? y : y - n;
  for (int w = 0; w < warp; ++w) at -= (int)sh.warp_key[w];
  if (in && at == __popc(who & ((1u << lane) - 1))) sh.bin = r;
  __syncthreads();
  return (int)sh.bin;
}

// What the unit of the weights is chosen by: of a warp's groups, counted from the row's first token on, the maxima
// times `by` (rounded, in the upper bits) and their number.  The groups as they are read begin `off` tokens
// earlier: their first tokens are the group's before, and where one of those may be the maximum, the group
// is read again.
template <int IO>
__device__ __noinline__ u64 look_at(const void *from, int V, int off, int first, int groups, const float *maxima, float by) {
  const int lane = threadIdx.x & 31;
  u64 look = 0;
  for (int g0 = 0; g0 < groups; g0 += 32) {
    const int at = (first + g0 + lane) * kGroup;
    const bool on = g0 + lane < groups && at < V;
    float top = on ? maxima[g0 + lane] : -INFINITY;
    if (off) {
      bool again = false;
      for (int i = at - off; i < at; ++i)
        if (i >= 0 && top > -INFINITY) again |= load_io1(from, IO, i) >= top;
      for (unsigned todo = __ballot_sync(0xffffffffu, again); todo; todo &= todo - 1) {
        const int who = __ffs(todo) - 1, start = (first + g0 + who) * kGroup;
        float t = -INFINITY;
        for (int i = start + lane; i < min(start + kGroup, V); i += 32) t = fmaxf(t, load_io1(from, IO, i));
        t = logit_of(__reduce_max_sync(0xffffffffu, key_of(t)));
        if (lane == who) top = t;
      }
      if (on)
        for (int i = at + kGroup - off; i < min(at + kGroup, V); ++i) top = fmaxf(top, load_io1(from, IO, i));
    }
    if (top > -INFINITY) look += (u64)((int64_t)__float2int_rn(fminf(fmaxf(top * by, -1e9f), 1e9f)) << 20) + 1;
  }
  return look;
}

// groups: of a warp (their tokens are consecutive, and the warps' in a block, the blocks' in a cluster).
template <int IO>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a, int groups) {
  extern __shared__ __align__(16) uint32_t totals[];  // the cluster's bins of this rank's run; the groups' maxima
  __shared__ __align__(16) Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float *const maxima = reinterpret_cast<float *>(totals + (ranks > 1 ? 2 * kBins / ranks : 0));  // [kWarps][groups]
  float *const mine = maxima + warp * groups;
  auto zero = [&] {
    for (int i = tid; i < 2 * kBins; i += kThreads) (&sh.bins[0][0])[i] = 0;
    if (ranks > 1)
      for (int i = tid; i < 2 * kBins / ranks; i += kThreads) totals[i] = 0;
  };
  zero();
  if (tid == 0) sh.listed = 0;
  cluster.barrier_arrive();  // (every block's shared memory exists and is clear; waited for below)
  grid_dependency();
  const int64_t row = a.slow_first ? row_of(sh, a, (int)blockIdx.y) : (int)blockIdx.y;

  float T = a.temperature ? a.temperature[row] : 1.f;
  if (T > 0.f) T = fmaxf(T, 0x1p-127f);  // (so that log2(e) / T is finite)
  const int k = a.top_k ? a.top_k[row] : 0;
  const float p = a.top_p ? a.top_p[row] : 1.f, floor_p = a.min_p ? a.min_p[row] : 0.f;
  const float u = a.u[row];
  const bool greedy = !(T > 0.f), by_count = k > 0 && k < a.V, by_share = p < 1.f;
  const bool by_floor = floor_p > 0.f && T < INFINITY;

  // ---- the tokens ----
  // They are counted from the 8 or 16-byte block that the row starts in (`off` before its start), so that
  // lane i of a group has its tokens 4 i .. 4 i + 3 in one aligned load; what is none is -inf.
  using E = typename std::conditional<IO == MQ_F32, float, uint16_t>::type;
  const E *const from = static_cast<const E *>(a.logits) + row * a.ld;
  const int off = (int)(reinterpret_cast<uintptr_t>(from) % (kSide * sizeof(E)) / sizeof(E)), V = (int)a.V;
  const int first = (rank * kWarps + warp) * groups * kGroup - off + kSide * lane;  // this lane's first token
  bool infinite = false;  // a row with infinite logits, which share all weight
  struct Raw {
    uint4 v;
  };
  auto load = [&](int i) {  // four tokens as they are stored
    Raw r;
    if (IO == MQ_F32) {
      r.v = *reinterpret_cast<const uint4 *>(from + i);
    } else {
      const uint2 h = *reinterpret_cast<const uint2 *>(from + i);
      r.v = make_uint4(h.x, h.y, 0, 0);
    }
    return r;
  };
  auto convert = [&](const Raw &r, float (&x)[kSide]) {
    const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
    for (int q = 0; q < kSide; ++q) {
      const uint16_t h = (uint16_t)(w[q / 2] >> 16 * (q & 1));
      x[q] = IO == MQ_F32    ? __uint_as_float(w[q])
             : IO == MQ_BF16 ? __uint_as_float(uint32_t(h) << 16)
                             : __half2float(__ushort_as_half(h));
      if (infinite) x[q] = x[q] == INFINITY ? 0.f : -INFINITY;
    }
  };
  auto fetch = [&](int g) {  // a group's tokens of this lane, where all are in the row
    const int i = first + g * kGroup;
    return i >= 0 && i + kSide <= V ? load(i) : Raw();
  };
  auto decode = [&](const Raw &r, int g, float (&x)[kSide]) {
    const int i = first + g * kGroup;
    convert(r, x);
    if (!(i >= 0 && i + kSide <= V)) {  // (at the row's ends)
#pragma unroll
      for (int q = 0; q < kSide; ++q) {
        x[q] = i + q >= 0 && i + q < V ? load_io1(from, IO, i + q) : -INFINITY;
        if (infinite) x[q] = x[q] == INFINITY ? 0.f : -INFINITY;
      }
    }
  };
  // The groups of warp `of` (from g0 on, every `step`-th) whose maximum reaches `border`: U of them on their way
  // at a time, then what(tokens, group) each, the group as this warp counts.
  auto visit = [&](auto U, int of, int g0, int step, float border, auto what) {
    const float *const best = maxima + of * groups;
    const int shift = (of - warp) * groups;
    for (int base = g0; base < groups; base += 32 * step) {
      const int at = base + lane * step;
      const float there = at < groups ? best[at] : -INFINITY;
      unsigned todo = __ballot_sync(0xffffffffu, there >= border && there > -INFINITY);
      while (todo) {
        int g[U.value];
        Raw r[U.value];
#pragma unroll
        for (int j = 0; j < U.value; ++j) {
          g[j] = todo ? base + (__ffs(todo) - 1) * step : -1;
          todo &= todo - 1;
          if (g[j] >= 0) r[j] = fetch(g[j] + shift);
        }
#pragma unroll
        for (int j = 0; j < U.value; ++j) {
          if (g[j] < 0) break;
          float x[kSide];
          decode(r[j], g[j] + shift, x);
          what(x, g[j] + shift);
        }
      }
    }
  };
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  using Four = std::integral_constant<int, 4>;
  // All of the warp's groups in order: `side` loads on their way, without a look at the row's ends where they
  // are not near.
  auto each_group = [&](auto side, auto what) {
    constexpr int U = side.value;
    const int start = first - kSide * lane;  // the warp's first token
    for (int g0 = 0; g0 < groups; g0 += U) {
      const int at = start + g0 * kGroup;
      if (at >= V) break;
      if (at >= 0 && at + U * kGroup <= V && g0 + U <= groups) {
        Raw r[U];
#pragma unroll
        for (int j = 0; j < U; ++j) r[j] = load(first + (g0 + j) * kGroup);
#pragma unroll
        for (int j = 0; j < U; ++j) {
          float x[kSide];
          convert(r[j], x);
          what(x, g0 + j);
        }
      } else {
#pragma unroll 1
        for (int g = g0; g < min(g0 + U, groups); ++g) {
          float x[kSide];
          decode(fetch(g), g, x);
          what(x, g);
        }
      }
    }
  };
  auto each = [&](float border, auto what) { visit(Two(), warp, 0, 1, border, what); };
  auto each_at_leisure = [&](float border, auto what) { visit(One(), warp, 0, 1, border, what); };

  float top = -INFINITY;
  for (int g = lane; g < groups; g += 32) mine[g] = -INFINITY;  // (groups behind the row)
  __syncwarp();
  each_group(Four(), [&](const float (&x)[kSide], int g) {
    // (the maximum takes the number of a number and a NaN)
    const float t = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), -INFINITY);
    const float best = logit_of(__reduce_max_sync(0xffffffffu, key_of(t)));
    if (lane == 0) mine[g] = best;
    top = fmaxf(top, best);
  });
  __syncwarp();  // (lane 0's maxima are read by the others)

  // ---- the maximum ----
  uint32_t top_key = key_of(top);
  if (lane == 0) sh.warp_key[warp] = top_key;
  // log2(e) / T: the quotient, and its remainder over T
  float c = 0.f, c_lo = 0.f;
  if (!greedy) {
    c = __fdiv_rn(kLog2e, T);
    if (c > 0.f) c_lo = __fdiv_rn(__fmaf_rn(-c, T, kLog2e) + kLog2eLow, T);
  }
  // (of min-p the border is exact to 64 bits: in flat rows thousands of tokens lie near it)
  if (tid == kThreads - 1 && by_floor) sh.floor_log = (double)T * log((double)fminf(floor_p, 1.f));
  // Rows without limits and top-p read all tokens again: for the unit of their weights, the mean of the groups'
  // maxima in sixteenths of y, as a sum and a number.  (Of the groups, not the warps or blocks, so that
  // a row's results do not depend on their number, nor on where the row lies.)
  const bool looks = !greedy && !by_count && !by_floor && V >= 1 << 14;
  if (looks) scan(sh, look_at<IO>(from, V, off, (rank * kWarps + warp) * groups, groups, mine, c * 16.f));
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top_key = max(top_key, sh.warp_key[w]);
  cluster.barrier_wait();
  if (tid < ranks) {
    *cluster.map_shared_rank(&sh.rank_key[rank], tid) = top_key;
    if (looks) *cluster.map_shared_rank(&sh.rank_look[rank], tid) = sh.sum;
  }
  cluster.sync();
  int winner = 0;  // the first rank with the row's maximum
  top_key = sh.rank_key[0];
  for (int q = 1; q < ranks; ++q)
    if (sh.rank_key[q] > top_key) top_key = sh.rank_key[q], winner = q;
  Scale s = {logit_of(top_key), c, c_lo, 44, 15.f};
  if (looks) {
    u64 look = 0;
    for (int q = 0; q < ranks; ++q) look += sh.rank_look[q];
    const float mean = (float)((int64_t)look >> 20) / (float)(look & 0xfffff);
    const float y = s.top * c - mean * 0.0625f;
    if (y < 16.f) s.unit = y < 8.f ? 34 : 38, s.deep = (float)(s.unit - 29);
  }
  auto finish = [&](int token, float logprob) {
    a.token[row] = token;
    if (a.logprob) a.logprob[row] = logprob;
  };
  if (s.top == -INFINITY) {
    if (rank == 0 && tid == 0) finish(-1, -INFINITY);
    return;
  }
  if (greedy) {  // the first token with the maximum: of its rank the first warp's
    if (rank != winner) return;
    int w = 0;
    while (w < kWarps - 1 && sh.warp_key[w] != top_key) ++w;
    if (w != warp) return;
    uint32_t index = 0xffffffffu;
    each_at_leisure(s.top, [&](const float (&x)[kSide], int g) {
#pragma unroll
      for (int q = 0; q < kSide; ++q)
        if (x[q] == s.top) index = min(index, (uint32_t)(first + g * kGroup + q));
    });
    index = __reduce_min_sync(0xffffffffu, index);
    if (lane == 0) finish((int)index, 0.f);
    return;
  }
  if (s.top == INFINITY) {
    infinite = true, s.top = 0.f;
    for (int g = lane; g < groups; g += 32) mine[g] = mine[g] == INFINITY ? 0.f : -INFINITY;
    __syncthreads();
  }

  // ---- the cuts ----
  // What stays: larger logits than cut, and equal ones up to cut_index.
  float cut = -INFINITY;
  int cut_index = -1;
  auto stays = [&](float x, int i) { return x > cut || (x == cut && i <= cut_index); };
  bool fresh = true;  // the bins are clear
  auto clear = [&] {
    if (!fresh) {
      cluster.sync();  // (the totals, and what is listed in the bins' place, have been read)
      zero();
      cluster.sync();
    }
    fresh = false;
  };
  // A block's sum, to the cluster's ranks (behind their next barrier).
  auto publish = [&](u64 mine) {
    scan(sh, mine);
    __syncthreads();
    if (tid < ranks) *cluster.map_shared_rank(&sh.rank_sum[rank], tid) = sh.sum;
  };
  auto sum_of_ranks = [&](int upto) {
    u64 all = 0;
    for (int q = 0; q < upto; ++q) all += sh.rank_sum[q];
    return all;
  };
  // The sum of the weights of what stays; each of them to one(which, weight), an uint32_t or u64.
  auto kept = [&](const float (&x)[kSide], int g, auto one) {
    const Weights w(s, x);
    u64 sum = 0;
    const bool all = cut == -INFINITY;
    bool on[kSide];
#pragma unroll
    for (int q = 0; q < kSide; ++q) on[q] = all || stays(x[q], first + g * kGroup + q);
#pragma unroll
    for (int q = 0; q < kSide; ++q) {
      const uint32_t v = on[q] && !(depth(s, x[q]) < s.deep) ? w.w[q] : 0;
      one(q, v), sum += v;
    }
    if (w.any) {
#pragma unroll
      for (int q = 0; q < kSide; ++q)
        if (on[q] && depth(s, x[q]) < s.deep) {
          const u64 v = w.whole(s, x, q);
          one(q, v), sum += v;
        }
    }
    return sum;
  };
  auto nothing = [](int, auto) {};
  auto of_warp = [&](u64 v) {
#pragma unroll
    for (int q = 16; q; q >>= 1) v += __shfl_xor_sync(0xffffffffu, v, q);
    return v;
  };
  // The first token in order at which the sum of amount(), over the cluster's blocks in order, passes
  // target(sum of all): its lane calls found(token, logit, sum).  sum: this thread's share of its warp's.  The
  // block that has it narrows it down to a warp's run, then, all warps together, to a group, and one
  // warp to the token.
  auto find = [&](float border, u64 sum, auto amount, auto target, auto found) {
    publish(sum);
    u64 before = 0;  // of the block's warps
    int run = 0;
    cluster.sync();
    const u64 lead = sum_of_ranks(rank), all = sum_of_ranks(ranks), at = target(all);
    if (at < lead || at >= lead + sh.sum) return;
    before = lead;
    while (run < kWarps - 1 && at >= before + sh.warp_sum[run]) before += sh.warp_sum[run++];
    // the group: that warp alone through a few, or all warps add up a share of them each (in the bins' place)
    u64 *const sums = &sh.list[0][0];
    auto group_sum = [&](const float (&x)[kSide], int g) { return of_warp(amount(x, g, nothing)); };
    if (groups <= kFew) {
      if (warp != run) return;
      for (int g = lane; g < groups; g += 32) sums[g] = 0;
      __syncwarp();
      each_at_leisure(border, [&](const float (&x)[kSide], int g) {
        const u64 side = group_sum(x, g);
        if (lane == 0) sums[g] = side;
      });
      __syncwarp();
    } else {
      for (int i = tid; i < groups; i += kThreads) sums[i] = 0;
      __syncthreads();
      visit(One(), run, warp, kWarps, border, [&](const float (&x)[kSide], int g) {
        const u64 side = group_sum(x, g);
        if (lane == 0) sums[g - (run - warp) * groups] = side;
      });
      __syncthreads();
      if (warp) return;
    }
    auto upto_lane = [&](u64 v) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const u64 o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
      }
      return v;
    };
    int g = 0;
    for (;; g += 32) {
      if (g >= groups) return;  // (only where the logits were written to meanwhile)
      const u64 upto = upto_lane(g + lane < groups ? sums[g + lane] : 0);
      const unsigned past = __ballot_sync(0xffffffffu, at < before + upto);
      if (past) {
        const int l = __ffs(past) - 1;
        if (l) before += __shfl_sync(0xffffffffu, upto, l - 1);
        g += l + (run - warp) * groups;
        break;
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
    float x[kSide];
    u64 w[kSide];
    decode(fetch(g), g, x);
    const u64 own = amount(x, g, [&](int q, auto v) { w[q] = v; });  // (a token's last is its weight)
    u64 from = before + upto_lane(own) - own;
#pragma unroll
    for (int q = 0; q < kSide; ++q) {
      if (at >= from && at < from + w[q]) found(first + g * kGroup + q, x[q], all);
      from += w[q];
    }
  };

  // Top-k, then top-p.  Top-k is tried first on the tokens above the k-th of the groups' maxima, and if that
  // does not do, on all; top-p on all.
  const int some = min(kQuick, (V + 2 * kGroup - 1) / (2 * kGroup));
  bool share_left = by_share;
  int held = 0;  // tokens that stay, where all of them are in the sorted list
  for (int phase = by_count ? 0 : 1; phase < 2; ++phase) {
    const bool counts = phase == 0;
    if (!counts && !share_left) break;
    for (int tries = counts && k <= some ? 0 : 1; tries < 2; ++tries) {
      clear();
      const bool of_maxima = tries == 0;
      if (of_maxima) {
        for (int i = tid; i < kWarps * groups; i += kThreads) {
          const int bin = bin_of(s, maxima[i]);
          if (bin < kLastBin) atomicAdd(&sh.bins[0][bin], 1u);
        }
      } else if (counts) {
        each_group(Two(), [&](const float (&x)[kSide], int g) {
#pragma unroll
          for (int q = 0; q < kSide; ++q) {
            const int bin = bin_of(s, x[q]);
            if (bin < kLastBin) atomicAdd(&sh.bins[0][bin], 1u);
          }
        });
      } else {
        each_group(Two(), [&](const float (&x)[kSide], int g) {
          kept(x, g, [&](int q, auto w) {
            const int bin = bin_of(s, x[q]);
            if (w) add_to(&sh.bins[0][bin], &sh.bins[1][bin], w);
          });
        });
      }
      if (counts && tid == 0) sh.bins[0][kLastBin] = (uint32_t)V;  // (what is left, or more)
      u64 wanted = choose(sh, totals, counts, {counts ? (u64)k : 0, p});
      const int bin = (int)sh.bin;
      u64 above = sh.above;
      if (bin == kLastBin) continue;  // (at the second try: all that weighs something stays)
      // the list: top-k's of all tokens up to the bin where it holds them (top-p's cut is then in it too)
      const bool whole = of_maxima || (counts && above + sh.inside <= kList);
      const float border = s.top - (float)(bin + 1) / kBinsPerHalving / s.hi * 1.0001f;  // (a little below the bin)
      int sub = -1;  // the part of the bin, where the tokens of all of it are too many
      auto part = [&](float x) {  // (as bin_of: falls with the logit)
        const float t = __fmaf_rn(depth(s, x), kBinsPerHalving, 0.5f - (float)bin);
        return min(max((int)(t * (float)kBins), 0), kBins - 1);
      };
      auto inside = [&](float x, int i) {
        if (!(x >= border)) return false;
        const int b = bin_of(s, x);
        return (b == bin ? sub < 0 || part(x) == sub : whole && b < bin) && stays(x, i);
      };
      int listed;
      for (;;) {
        __syncthreads();
        each(border, [&](const float (&x)[kSide], int g) {
#pragma unroll
          for (int q = 0; q < kSide; ++q) {
            const int i = first + g * kGroup + q;
            if (!inside(x[q], i)) continue;
            const uint32_t at = atomicAdd(&sh.listed, 1u);
            if (at < kList) sh.list[0][at] = (u64)key_of(x[q]) << 32 | ~(uint32_t)i;
          }
        });
        listed = sort_lists(sh, rank);
        if (listed >= 0 || sub >= 0 || whole) break;
        wanted -= above;
        clear();
        each_at_leisure(border, [&](const float (&x)[kSide], int g) {
#pragma unroll
          for (int q = 0; q < kSide; ++q) {
            if (!inside(x[q], first + g * kGroup + q)) continue;
            const int b = part(x[q]);
            if (counts) atomicAdd(&sh.bins[0][b], 1u);
            else add_to(&sh.bins[0][b], &sh.bins[1][b], weight(s, x[q]));
          }
        });
        choose(sh, totals, counts, {wanted, 0.f});
        sub = (int)sh.bin, above = sh.above;
      }
      if (listed >= 0) {
        int at = whole ? k - 1 : (int)(wanted - above) - 1;
        if (!counts || (whole && by_share)) {
          at = place_by_weight(sh, s, counts ? k : listed, counts ? 0 : above, {counts ? 0 : wanted, p});
          share_left = false;
        }
        at = min(max(at, 0), kList - 1);  // (in the list, whatever was written to the logits meanwhile)
        cut = logit_of((uint32_t)(sh.list[1][at] >> 32)), cut_index = (int)~(uint32_t)sh.list[1][at];
        held = whole && !share_left ? at + 1 : 0;
        break;
      }
      if (whole) continue;  // (the first try's: more tokens above the maxima than a list holds)
      // still too many (equal logits among them): by the logits' bits, then by the index
      wanted -= above;
      uint32_t prefix = 0;
      for (int level = 0; level < 3; ++level) {
        const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
        clear();
        each_at_leisure(border, [&](const float (&x)[kSide], int g) {
#pragma unroll
          for (int q = 0; q < kSide; ++q) {
            if (!inside(x[q], first + g * kGroup + q)) continue;
            const uint32_t rev = ~key_of(x[q]);
            if (level && rev >> (shift + bits) != prefix) continue;
            const uint32_t digit = rev >> shift & ((1u << bits) - 1);
            if (counts) atomicAdd(&sh.bins[0][digit], 1u);
            else add_to(&sh.bins[0][digit], &sh.bins[1][digit], weight(s, x[q]));
          }
        });
        choose(sh, totals, counts, {wanted, 0.f});
        wanted -= sh.above;
        prefix = prefix << bits | sh.bin;
        __syncthreads();
      }
      const float at = logit_of(~prefix);
      if (!counts) {
        const u64 w = weight(s, at);
        wanted = (wanted + w - 1) / w;
        share_left = false;
      }
      auto equal = [&](const float (&x)[kSide], int g, auto one) {
        u64 sum = 0;
#pragma unroll
        for (int q = 0; q < kSide; ++q) {
          const uint32_t v = x[q] == at && stays(x[q], first + g * kGroup + q);
          one(q, v), sum += v;
        }
        return sum;
      };
      u64 equals = 0;
      each_at_leisure(at, [&](const float (&x)[kSide], int g) { equals += equal(x, g, nothing); });
      find(
          at, equals, equal,
          [&](u64) { return wanted - 1; },
          [&](int i, float, u64) {
            for (int q = 0; q < ranks; ++q) *cluster.map_shared_rank(&sh.cut_index, q) = i;
          });
      cluster.sync();
      cut = at, cut_index = (int)sh.cut_index;
      break;
    }
  }
  if (by_floor) {  // min-p: w < min_p is l < m + T ln(min_p)
    if (tid == 0) sh.least = __double2float_ru((double)s.top + sh.floor_log);
    __syncthreads();
    if (sh.least > cut) cut = sh.least, cut_index = 0x7fffffff;
  }

  // ---- the token ----
  auto target = [&](u64 all) {
    bool more;
    return !(u > 0.f) ? u64(0) : u < 1.f ? part_of(u, all, more) : all - 1;
  };
  auto drawn = [&](int i, float x, u64 all) {
    finish(i, log_share(s.top, x, T, all, s.unit));
  };
  if (held && held <= kCounted) {
    // every block has all that stays: each token's sum of the weights before it, by its index
    cluster.barrier_arrive();  // (the lists have been read)
    const u64 *const sorted = sh.list[1];
    u64 *const w = sh.list[1] + kCounted;
    for (int i = tid; i < held; i += kThreads) {
      const float x = logit_of((uint32_t)(sorted[i] >> 32));
      w[i] = x >= cut ? weight(s, x) : 0;  // (min-p)
    }
    __syncthreads();
    const Share e(held);
    const u64 own = e.at < held ? sorted[e.at] : 0;
    u64 before = 0, all = 0;
    for (int j = e.part; j < held; j += e.parts) {
      all += w[j];
      if (~(uint32_t)sorted[j] < ~(uint32_t)own) before += w[j];
    }
    for (int d = 1; d < e.parts; d <<= 1)
      before += __shfl_xor_sync(0xffffffffu, before, d), all += __shfl_xor_sync(0xffffffffu, all, d);
    const u64 at = target(all);
    if (rank == 0 && e.part == 0 && e.at < held && at >= before && at < before + w[e.at])
      drawn((int)~(uint32_t)own, logit_of((uint32_t)(own >> 32)), all);
    cluster.barrier_wait();
    return;
  }
  u64 sum = 0;
  if (cut == -INFINITY) {
    each_group(Four(), [&](const float (&x)[kSide], int g) { sum += kept(x, g, nothing); });
  } else if (by_floor || by_count) {
    // few tokens of a group stay, and most of them are not deep: they are put side by side for their weights
    // (256 rows of 151936 with min-p: 67 us without)
    __syncthreads();  // (the cut has been read from the list)
    float *const queue = reinterpret_cast<float *>(sh.list[1]) + warp * 64;
    int waiting = 0;
    each(cut, [&](const float (&x)[kSide], int g) {
#pragma unroll
      for (int q = 0; q < kSide; ++q) {
        const bool on = stays(x[q], first + g * kGroup + q);
        const unsigned who = __ballot_sync(0xffffffffu, on);
        if (who == 0) continue;
        if (on) queue[waiting + __popc(who & ((1u << lane) - 1))] = x[q];
        waiting += __popc(who);
        __syncwarp();
        if (waiting < 32) continue;
        sum += weight(s, queue[lane]);
        const float next = queue[32 + lane];
        __syncwarp();
        queue[lane] = next, waiting -= 32;
        __syncwarp();
      }
    });
    if (lane < waiting) sum += weight(s, queue[lane]);
  } else {
    each(cut, [&](const float (&x)[kSide], int g) { sum += kept(x, g, nothing); });
  }
  find(cut, sum, kept, target, drawn);
}

}  // namespace

namespace {
// A warp's groups of a row (a row may start inside a group's first load), and a block's shared memory.
int groups_of(int64_t V, int ranks) {
  const int64_t run = int64_t(ranks) * kWarps * kGroup;
  return (int)((V + kSide - 1 + run - 1) / run);
}
size_t smem_of(int groups, int ranks) { return (ranks > 1 ? 2 * kBins / ranks * 4 : 0) + size_t(kWarps) * groups * 4; }
}  // namespace

mq_status init_sample(DeviceState *st) {
  cudaError_t e = cudaSuccess;
  for (int &n : st->sample_clusters) n = INT_MAX;
  auto set_up = [&](auto *kernel) {
    if (e != cudaSuccess) return;
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return;
    const int most = (int)smem_of(groups_of((1 << 19) - 1, 1), 1);  // (the largest row in one block)
    if (most + (int)fa.sharedSizeBytes > st->smem_optin) {
      e = cudaErrorInvalidConfiguration;
      return;
    }
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return;
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
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 0;
      }
      st->sample_clusters[i] = std::min(st->sample_clusters[i], n);  // (what every type's kernel can have)
    }
  };
  set_up(sample_kernel<MQ_F32>);
  set_up(sample_kernel<MQ_F16>);
  set_up(sample_kernel<MQ_BF16>);
  return e == cudaSuccess ? MQ_OK : cuda_fail(e, "cudaFuncSetAttribute", "sample_kernel");
}

mq_status launch_sample(const SampleArgs &a, cudaStream_t s, const DeviceState *st) {
  // Blocks of a cluster: as many as leave all rows resident at once (one row after the other costs twice the time: 16
  // rows of 151936 with top-k and top-p 14.8 us by 8 blocks each, 27.2 by 16, of which 14 rows fit), with
  // 2048 logits or more each.  Twice as many where rows may take unlike times and the few blocks of the slow ones
  // would be left alone at the end: top-p with min-p, from 4 blocks down (64 rows with settings of their own 66 us,
  // 52 by twice as many; of the same settings 18, 35); top-p alone, from 2 down (128 rows 105, 99; 256 203,
  // 176; but 42 55, 61); min-p without it, from one (256 rows at T = 1 69, 59; of few tokens that stay 35, 44).
  // It goes by which settings are given, not by what they hold: 64 rows with all four given and none in effect take 34 us,
  // 23 by half as many blocks.  And eight blocks a row would do for a few more than 72 rows of settings of their own
  // (73 rows 57, by the rule's four 69; 80 64, 73; 96 81, 76; 128 100, 80), four for more than 144 (160 85, by
  // two 124; 256 131, 140).
  auto fits = [&](int ranks_log, int waves) {
    return ranks_log <= 4 && a.V >> ranks_log >= 2048 && a.B <= int64_t(waves) * st->sample_clusters[ranks_log];
  };
  int r = 0;
  while (fits(r + 1, 1)) ++r;
  const int most = a.top_p ? (a.min_p ? 2 : a.top_k ? -1 : 1) : a.min_p ? 0 : -1;
  if (r <= most && fits(r + 1, 2)) ++r;
  const int ranks = 1 << r, groups = groups_of(a.V, ranks);
  // Where not all clusters are resident at once and rows differ in their cuts (two settings or more are given), the
  // slow ones begin first: those 64 rows (of one draw) 57.7 us without, 52.5 with; finding its row costs a cluster 1.5 us (64
  // rows of top-p alone 73 us, 78 with it).
  SampleArgs b = a;
  b.slow_first = !!a.top_k + !!a.top_p + !!a.min_p > 1 && a.B <= kThreads && a.B > st->sample_clusters[r];
  auto *kernel = a.io == MQ_F32 ? sample_kernel<MQ_F32> : a.io == MQ_F16 ? sample_kernel<MQ_F16> : sample_kernel<MQ_BF16>;
  return launch_cluster("sample_kernel", kernel, dim3(ranks, (unsigned)a.B, 1), dim3(kThreads, 1, 1),
                        smem_of(groups, ranks),
                        s, ranks, b, groups);
}

}  // namespace mq
