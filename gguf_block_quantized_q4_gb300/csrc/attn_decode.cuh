// attn_decode.cuh -- mq_attn_decode: attention of one new token per sequence over the paged
// cache, split over the length and joined.
//
// Mathematics.  For the query heads of one kv head, s = q k / sqrt(D) and o = sum softmax(s) v
// are kept in the running form: per query row a maximum m, a sum l = sum exp2(s - m) and an
// unnormalised o, which pieces of the length join as
//     M = max m_i,  L = sum l_i exp2(m_i - M),  o = sum o_i exp2(m_i - M) / L.
//
// What bounds it: the bytes of K and V (over Q4_0 rows the issue slots, below).  A group of up to 16 query heads (8 for heads of 192 and
// 256) shares one reading of them; a larger one is several row groups, each a unit of its own that
// reads them again (38 x 8192, F16: 96/4 heads of 128 207 us, 64/4 107; 64/4 heads of 256 405, 8/4
// 206).  A group's rows share the keys, so
// both products are matrix products with 8 (or 16) columns: S^T = K Q^T and O^T = V^T P^T on
// mma.sync m16n8k16, keys (and dims of V^T) as the 16-row operand, the query rows as the 8
// columns.  (A tcgen05 tile has 64 or 128 rows and at least 8 columns of its own accumulator
// memory; here the softmax between the products lives in registers and the products take a
// fifth of the time that the bytes need.)
//
// Loads: one thread block per SM.  Each warp takes 16 or 32 keys at a time and has a ring of its
// own in shared memory, filled row by row with 16-byte asynchronous copies that follow the page
// table (a page may end anywhere; a row past the end is filled with zeros, nothing is read for
// it), so no barrier stands between the loads and the products and about 128 KB are in flight
// per SM; 44 KB cover the memory's latency.  ldmatrix, transposing for V, reads the operands;
// rows are padded by 16 bytes (those of 64 bytes have their chunks exchanged by the key), which puts
// the eight rows of a matrix on different banks.
//
// Work: (sequence, kv head, row group) units of tiles of TK keys, laid end to end; thread block b
// of the `parts` that have work takes the steps [b T / parts, (b + 1) T / parts) of all T.  The
// split is made on the device from the lengths, so unlike lengths load all SMs alike.  A unit
// whole in one block is written at once; the pieces of the others go to the workspace, and the
// last block of a unit (or of a group of its pieces) to arrive joins them in a fixed order
// (counters, back to zero afterwards), so results do not depend on the order of execution.  The
// rings run on across pieces.
//
// Precision: f16 operands are multiplied exactly and summed in binary32.  q (scaled by a power
// of two per row) and the weights are carried as two f16 parts (22 bits), against bf16 keys and
// values as three bf16 parts (24 bits); Q8_0 quants are exact in f16, the keys' scales multiply
// the 32-element block sums in binary32, the values' scales the weights (both first scaled by
// powers of two that put the largest weight at 2^15 and a tile's largest scale in [1/2, 1), so
// that the second f16 part is a normal number for all but negligible products).  Each tile's
// product is added to o by a binary32 fma (the tensor cores' own long sums may truncate).  Operands
// in parts do not follow the definition at infinities: of an infinite key's logit the first part
// alone counts, and a warp whose o holds an infinity or NaN at a piece's end sums what is infinite or
// NaN among its rows once more, in binary32 (sum_infinities).  The check at a piece's end and the
// select per logit cost nothing at 38 x 8192 (28/4 heads of 128) and up to 0.5 us where a block has
// few tiles (16 x 4096, 16/1 heads of 128, F16: 18.3 -> 18.6 us).
//
// Q4_0 rows have half the bytes of Q8_0's and as many products, so that the instructions bound them.
// A word holds the dims j and 16 + j of four keys' or dims' pairs; the query's rows (and the dims of o)
// are put in that order instead of the quants.  n - 8 is exact in f16 (a LOP3 and an addition or an fma
// per pair); the keys' scales multiply their block's sum in binary32, and the values' scales the f16
// parts of the weights, whose rest the fma keeps.  A power of two puts a tile's largest value scale between 1/2 and 1:
// downwards it divides the weights (at 2^15, f16 has no room above them), upwards it multiplies the scales.  (Only
// for tiles outside [2^-4, 1): 57.7 to 59.6 us, by where it stands, at the 64 sequences below.)  A tile
// without a logit above its row's largest so far, as most are, spares the maxima over the lanes (59.1 -> 58.2).
//
// Measured (28/4 heads of 128; from one card to another 3% apart): 38 x 8192 keys f16 104.5 to 108 us
// (5.9 to 6.1 TB/s, 88 to 91% of a plain copy's rate), bf16 104.7 to 108, Q8_0 67 (5.1 TB/s, 76%: not
// the bytes, and no pipe full: half of the issue slots stay empty, two warps per scheduler waiting
// on fixed latencies of conversions, shared memory and products; its copies alone take 55); 131072
// bf16 keys of one sequence 53 us (76%: 42 of streaming, the rest the start, the first rows and the
// join); 64 ragged sequences up to 8192, f16 97 to 100 us, Q8_0 67.5; one sequence of 37 keys, 14/2
// heads of 64, 5.1.  Q4_0: those 64 sequences 58.9 us (39% of a plain copy's rate; the copies alone take 36.5,
// all but the copies 55, without the second product 46, with half of the products' instructions
// 47.4, without the conversion of the quants 52.6, without the scales of V 55.3; 12 warps of 16 or 32
// keys 63 to 66, 16 of 16 keys 74.5); 131072 keys, bf16 activations (one part of the queries) 32.4 us (34%); 37 keys 5.4.
#pragma once

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "kv.cuh"

namespace mq {
namespace attn {

constexpr int kMaxParts = MQ_ATTN_WS_ZERO / 12;  // thread blocks with work (three counters each)
constexpr float kLog2e = 1.44269504088896340736f;

// ---- device helpers ---------------------------------------------------------------------
// 16 bytes to shared memory, of which `size` (16 or 0) are read and the others zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src, uint32_t size) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size)
               : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void *src, uint32_t size) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, uint32_t size) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the N newest groups
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Four 8 x 8 matrices of 16-bit elements; lane 8 i + r gives the address of row r of matrix i.
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
template <bool BF>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if (BF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = a b + c in f16 operands.
__device__ __forceinline__ void mma_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1, float4 c) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c.x), "f"(c.y), "f"(c.z), "f"(c.w));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (BF)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if (BF) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  return __half22float2(*reinterpret_cast<__half2 *>(&v));
}
// A pair as N parts whose sum is the pair: part i holds what the parts before it left.
template <bool BF, int N>
__device__ __forceinline__ void split2(float lo, float hi, uint32_t (&part)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    part[i] = pack2<BF>(lo, hi);
    const float2 b = unpack2<BF>(part[i]);
    lo -= b.x, hi -= b.y;
  }
}
// Two int8 (the bytes of v ^ 0x80 that SEL picks) as f16x2: 1024 + (v + 128) by bits, less 1152.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t int8_f16(uint32_t biased) {
  uint32_t u = __byte_perm(biased, 0x64646464u, SEL);
  const uint32_t c = 0x64806480u;
  __half2 r = __hsub2(*reinterpret_cast<__half2 *>(&u), *reinterpret_cast<const __half2 *>(&c));
  return *reinterpret_cast<uint32_t *>(&r);
}

// The 4-bit numbers n at the bits MASK of each half as f16x2 n - 8: 1024 + n (or 1024 + 16 n) by bits,
// then an exact subtraction (or multiplication by 1/16 and subtraction).  An instruction takes one
// immediate operand, so 0x6400 and 1/16 come in registers that the compiler does not know to be
// constants (it would make two instructions of each: 128 more for 16 keys of 128).
struct Int4Constants {
  uint32_t magic, sixteenth;
};
template <uint32_t MASK>
__device__ __forceinline__ uint32_t int4_f16(uint32_t v, Int4Constants c) {
  static_assert(MASK == 0x000f000fu || MASK == 0x00f000f0u, "bits 0-3 or 4-7");
  uint32_t u;  // v & MASK | magic
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(u) : "r"(v), "n"(MASK), "r"(c.magic));
  const uint32_t less = MASK == 0x000f000fu ? 0xe408e408u : 0xd480d480u;  // -1032, -72
  const __half2 x = *reinterpret_cast<const __half2 *>(&u), y = *reinterpret_cast<const __half2 *>(&less);
  const __half2 r = MASK == 0x000f000fu ? __hadd2_rn(x, y)
                                        : __hfma2(x, *reinterpret_cast<const __half2 *>(&c.sixteenth), y);
  return *reinterpret_cast<const uint32_t *>(&r);
}
// The two parts of a pair of weights times a pair of f16 scales, as two parts: the first part's product
// rounded, and what that leaves (exact) with the second's.
template <int N>
__device__ __forceinline__ void scale_parts(const uint32_t (&p)[N], uint32_t d, uint32_t (&to)[N]) {
  const __half2 a = *reinterpret_cast<const __half2 *>(&p[0]), b = *reinterpret_cast<const __half2 *>(&p[N - 1]);
  const __half2 x = *reinterpret_cast<const __half2 *>(&d), hi = __hmul2_rn(a, x);
  to[0] = *reinterpret_cast<const uint32_t *>(&hi);
  if (N == 1) return;
  const __half2 lo = __hfma2(b, x, __hfma2(a, x, __hneg2(hi)));
  to[N - 1] = *reinterpret_cast<const uint32_t *>(&lo);
}

// ---- the shape of a kernel ----------------------------------------------------------------
constexpr int kSmemMax = 226 * 1024;  // per thread block (of 227 KB; a little is static)

template <int TYPE, int D, int NT, int IO>
struct Shape {
  static constexpr bool kQ8 = TYPE == MQ_Q8_0, kQ4 = TYPE == MQ_Q4_0;
  static constexpr bool kScaled = kQ8 || kQ4;   // blocks of 32 dims with a scale each
  static constexpr bool kBf = TYPE == MQ_BF16;  // operands bf16, else f16
  // parts of the query and of the weights.  Q4_0: 16-bit queries are one f16 part (f16 exact, bf16 to 2^-38 of
  // the row's largest), as mma.sync holds the issue port for 8.6 cycles here and its instructions are 37%
  // of the time of a tile.
  static constexpr int kQueryParts = kBf ? 3 : kQ4 && IO != MQ_F32 ? 1 : 2;
  static constexpr int kParts = kBf ? 3 : 2;
  static constexpr int kRow = kQ4 ? D / 2 : kQ8 ? D : 2 * D;  // bytes of a key row
  static constexpr int kNG = D / 32;            // groups of 32 dims
  static constexpr int kMT = kRow <= 128 ? 2 : 1;  // 16-key groups a warp takes at a time
  static constexpr int kKeys = 16 * kMT;
  static constexpr int kRows = 8 * NT;          // query rows of a unit
  // shared memory: the rings, query parts, the warps' results
  // Rows an odd number of 16-byte steps apart; those of 64 bytes lie close, their chunks exchanged by the
  // key (64 ragged Q4_0 sequences up to 8192, 28/4 heads of 128: 57.8 -> 56.9 us, 8 x 1100 9.4 -> 9.0).
  static constexpr bool kSwizzled = kQ4 && kRow == 64;
  static constexpr int kStride = kSwizzled || kRow / 16 % 2 ? kRow : kRow + 16;
  static __device__ __forceinline__ uint32_t chunk_at(int key, int ch) {
    return key * kStride + (kSwizzled ? ch ^ (key >> 1 & 3) : ch) * 16;
  }
  // a stage: K rows, V rows, the page entries of the tile a ring's length ahead, the blocks' scales as
  // they are stored (K's keys, V's keys)
  static constexpr int kEntries = 2 * kKeys * kStride;
  static constexpr int kRaw = kEntries + kKeys * 4;
  static constexpr int kScaleRow = (kNG + 1) / 2 * 4;
  static constexpr int kStage = (kRaw + (kScaled ? 2 * kKeys * kScaleRow : 0) + 15) / 16 * 16;
  static constexpr int kLdO = D + 4;
  // the query's parts as operand words; Q8_0: and -128 times its block sums as accumulators
  static constexpr int kQuery = kQueryParts * NT * kNG * 32 * 16;
  static constexpr int kSums = kQ8 ? NT * kNG * 4 * 16 : 0;
  static constexpr int smem(int warps, int stages) {
    return warps * (stages * kStage + kRows * (kLdO + 2) * 4) + kQuery + kSums + kRows * 4;
  }
  static constexpr int kWarps = smem(8, 2) <= kSmemMax ? 8 : smem(6, 2) <= kSmemMax ? 6 : 4;
  static constexpr int kStages = smem(kWarps, 3) <= kSmemMax ? 3 : 2;
  static constexpr int kSmem = smem(kWarps, kStages), kThreads = 32 * kWarps;
  static constexpr int kTK = kKeys * kWarps;    // keys of a tile
  static_assert(smem(kWarps, kStages) <= kSmemMax, "shared memory");
  // the f16 parts hold weights in (0, 2^15], so that the second part of all but negligible weights is
  // a normal f16.  (Multiplied in after the exponential: added to its argument it would round that
  // to 2^-21 where s - m itself is nearly exact.)
  static constexpr float kUnit = kBf ? 1.f : 0x1p15f;
};

struct Params {
  AttnArgs a;
  int group, row_groups, units;  // query heads of a kv head; row groups of them; per sequence
  int logit_width;               // query rows per key in the logits (2, or whole fours)
  int *count;                    // [3][kMaxParts]: a unit's first group, its others, its groups
  // results of blocks (two each: a piece whose unit began before the block; one whose unit begins
  // in it), then of groups (by their first block, two each: a unit's others, its first)
  float *piece_o;                // [4][blocks][rows][D]
  float2 *piece_ml;              // [4][blocks][rows]: maximum, sum
  int blocks;
  float *logits;                 // [S][units][max_len][logit_width], or nullptr
  float2 *stats;                 // [S][units][rows]: maximum, weight of exp2(0)
};

// ---- the schedule -------------------------------------------------------------------------
struct Span {
  int lo, len;  // positions read: [lo, len)
  int tiles;
};
__device__ __forceinline__ Span span_of(const AttnArgs &a, int s, int tk) {
  Span r;
  r.len = clamped_len(a.len[s], a.max_len);
  r.lo = a.window && r.len > a.window ? r.len - (int)a.window : 0;
  r.tiles = (r.len - r.lo + tk - 1) / tk;
  return r;
}
// The units' tiles laid end to end, each unit `gap` steps after the one before it: a unit costs a
// block about as much beside its tiles as a tile does (its query, the join of the warps), and
// blocks of many short units are to have fewer tiles.  (32 ragged sequences of up to 4001 keys,
// 32/8 heads of 128, f16: 64 us without it, 54 with.)  Blocks of only a few tiles get no gaps.
struct Line {
  int64_t steps;        // of all sequences
  int gap;
  int64_t lane_first;   // lane i's run of the sequences: lane_n from lane_s on; its first step (in
  int lane_s, lane_n;   // steps of one unit per sequence)
};
__device__ __forceinline__ Line lay_out(const AttnArgs &a, int units, int tk, int blocks) {
  const int lane = threadIdx.x & 31, S = (int)a.S;
  const int per = (S + 31) / 32;
  Line r;
  r.lane_s = min(lane * per, S);
  r.lane_n = min(per, S - r.lane_s);
  int64_t tiles = 0;
  int live = 0;  // sequences with tiles
  for (int i = 0; i < r.lane_n; ++i) {
    const int n = span_of(a, r.lane_s + i, tk).tiles;
    tiles += n, live += n > 0;
  }
  int64_t upto = tiles;
  int live_upto = live;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, upto, k);
    const int q = __shfl_up_sync(0xffffffffu, live_upto, k);
    if (lane >= k) upto += o, live_upto += q;
  }
  const int64_t all = __shfl_sync(0xffffffffu, upto, 31);
  r.gap = all * units >= 4 * int64_t(blocks);
  r.lane_first = upto - tiles + int64_t(live_upto - live) * r.gap;
  r.steps = (all + int64_t(__shfl_sync(0xffffffffu, live_upto, 31)) * r.gap) * units;
  return r;
}

// A place on the line: tile `tile` of a unit, at step `at` (a unit's tile 0 lies behind its gap).
struct Cursor {
  int s, hk, rg, tile;  // sequence, kv head, row group, tile
  Span span;
  int64_t at;
};
// The first tile at or after a step of the line; for every lane of the warp.
__device__ __forceinline__ Cursor cursor_at(const Params &p, const Line &line, int tk, int64_t at) {
  Cursor c;
  const int64_t q = at / p.units;
  const unsigned owners = __ballot_sync(0xffffffffu, line.lane_first <= q && line.lane_n > 0);
  const int src = 31 - __clz(owners);
  int64_t first = __shfl_sync(0xffffffffu, line.lane_first, src);
  c.s = __shfl_sync(0xffffffffu, line.lane_s, src);
  c.span = span_of(p.a, c.s, tk);
  while (c.span.tiles == 0 || first + c.span.tiles + line.gap <= q) {
    if (c.span.tiles) first += c.span.tiles + line.gap;
    c.span = span_of(p.a, ++c.s, tk);
  }
  const int64_t in = at - first * p.units, unit = in / (c.span.tiles + line.gap);
  c.hk = (int)(unit / p.row_groups);
  c.rg = (int)(unit % p.row_groups);
  const int step = (int)(in - unit * (c.span.tiles + line.gap));
  c.tile = max(0, step - line.gap);
  c.at = at - step + line.gap + c.tile;
  return c;
}
// The next tile; `end` bounds the steps, from there on the sequence stays.
__device__ __forceinline__ void next_tile(Cursor &c, const Params &p, int tk, int gap, int64_t end) {
  ++c.at;
  if (++c.tile < c.span.tiles) return;
  c.tile = 0;
  c.at += gap;
  if (++c.rg < p.row_groups) return;
  c.rg = 0;
  if (++c.hk < p.a.c.hkv) return;
  c.hk = 0;
  if (c.at >= end) return;
  do {
    c.span = span_of(p.a, ++c.s, tk);
  } while (c.span.tiles == 0);
}

// A unit that several blocks share: its first query head's row of q and o, its number, its first
// and last block, its query rows; whether this block arrived last at a count.
struct Split {
  int64_t head0, unit_id, b0, b1;
  int rows, last;
  int64_t first;  // the group of this block's piece: its first block, its blocks
  int members;
};

// A result in the workspace: kind 0, 1 a block's pieces, 2, 3 a group's (Params).
struct Result {
  float *o;
  float2 *ml;
};
template <class C, int D>
__device__ __forceinline__ Result result_of(const Params &p, int kind, int64_t block) {
  const int64_t at = (int64_t(kind) * p.blocks + block) * C::kRows;
  return {p.piece_o + at * D, p.piece_ml + at};
}
__device__ __forceinline__ void store_result(const Result &to, int D, int r, int d, float4 x, float m, float l) {
  *reinterpret_cast<float4 *>(to.o + r * D + d) = x;
  if (d == 0) to.ml[r] = make_float2(m, l);
}

// Four dims of a query row's output, normalised.
template <class C>
__device__ __forceinline__ void finish(const Params &p, int64_t head0, int64_t unit_id, int r, int d,
                                       int dim, float4 x, float m, float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  store_io4(p.a.o, p.a.io, (head0 + r) * dim + d,
            make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
  if (d == 0 && p.stats)
    p.stats[unit_id * C::kRows + r] = make_float2(m == -INFINITY ? 0.f : m, inv * C::kUnit);
}

// Counts a piece in, of `others` + 1; true where it is the last.  One thread calls it, after a
// barrier behind the block's stores: the release covers them (the barrier orders them before it),
// the acquire what the other blocks stored.
__device__ __forceinline__ bool arrive(int *count, int64_t others) {
  int before;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(count) : "memory");
  const bool last = before == (int)others;
  if (last) *count = 0;
  return last;
}

// How a shared unit's pieces are joined: up to kOneJoin at once; more in groups of about the square
// root of their number, by the last block of each group, then the groups by the last of those (one
// block for all read 38 pieces in 4 us and 152 in 16: what a single SM takes in bounds it).
constexpr int kOneJoin = 12;
struct Groups {
  int size, number;
};
__device__ __forceinline__ Groups groups_of(const Split &u) {
  const int n = (int)(u.b1 - u.b0 + 1);
  const int size = n <= kOneJoin ? n : (int)ceilf(sqrtf((float)n));
  return {size, (n + size - 1) / size};
}

// Joins n results of a unit, the first at `r0`, the i-th `i * step` blocks behind `r1`: a thread
// sums I places of four dims of a row over them in their order, J results on their way at a time.
// To `to` in the workspace, or (to.o null) normalised to the output.  Out of line, and with plain
// arguments: what it keeps in registers is not the tiles' loop's.
template <class C, int D>
__device__ __noinline__ void join_results(const Params &p, const Split &u, Result r0, Result r1, int step,
                                          int n, Result to) {
  constexpr int I = (C::kRows * D / 4 + C::kThreads - 1) / C::kThreads, J = I == 1 ? 10 : I == 2 ? 6 : 4;
  float4 x[I];
  float m[I], l[I];
  int at[I];  // (a place past the rows takes the first instead, and stores nothing)
  const int places = u.rows * (D / 4);
#pragma unroll
  for (int q = 0; q < I; ++q) {
    x[q] = make_float4(0.f, 0.f, 0.f, 0.f), m[q] = -INFINITY, l[q] = 0.f;
    at[q] = threadIdx.x + q * C::kThreads < places ? threadIdx.x + q * C::kThreads : 0;
  }
  for (int c0 = 0; c0 < n; c0 += J) {
    float4 y[I][J];
    float2 ml[I][J];
#pragma unroll
    for (int i = 0; i < J; ++i) {
      const int64_t row = int64_t(c0 + i) * step * C::kRows;
      const float *const o = c0 + i ? r1.o + row * D : r0.o;
      const float2 *const s = c0 + i ? r1.ml + row : r0.ml;
#pragma unroll
      for (int q = 0; q < I; ++q) {
        ml[q][i] = make_float2(-INFINITY, 0.f), y[q][i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c0 + i < n) {
          ml[q][i] = __ldcg(s + at[q] / (D / 4));
          y[q][i] = __ldcg(reinterpret_cast<const float4 *>(o) + at[q]);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < I; ++q) {
      float top = m[q];
#pragma unroll
      for (int i = 0; i < J; ++i) top = fmaxf(top, ml[q][i].x);
      const float low = top == -INFINITY ? 0.f : top, f0 = exp2_fast(m[q] - low);
      m[q] = top;
      l[q] *= f0, x[q].x *= f0, x[q].y *= f0, x[q].z *= f0, x[q].w *= f0;
#pragma unroll
      for (int i = 0; i < J; ++i) {
        const float f = exp2_fast(ml[q][i].x - low);
        l[q] = fmaf(ml[q][i].y, f, l[q]);
        x[q].x = fmaf(y[q][i].x, f, x[q].x), x[q].y = fmaf(y[q][i].y, f, x[q].y);
        x[q].z = fmaf(y[q][i].z, f, x[q].z), x[q].w = fmaf(y[q][i].w, f, x[q].w);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < I; ++q) {
    if (threadIdx.x + q * C::kThreads >= places) continue;
    const int r = at[q] / (D / 4), d = 4 * (at[q] % (D / 4));
    if (to.o)
      store_result(to, D, r, d, x[q], m[q], l[q]);
    else
      finish<C>(p, u.head0, u.unit_id, r, d, D, x[q], m[q], l[q]);
  }
}

// Joins the results that the warps left in shared memory: so[w][row][dim], sm / sl the maxima and
// sums.  Calls put(row, dim, o, m, l) with four dims of o (not normalised) for the first `rows`.
template <class C, class Put>
__device__ __forceinline__ void join_warps(const float *so, const float *sm, const float *sl, int D,
                                           int rows, Put put) {
  for (int i = threadIdx.x; i < rows * (D / 4); i += C::kThreads) {
    const int r = i / (D / 4), d = 4 * (i % (D / 4));
    float m = sm[r], l = 0.f;
#pragma unroll
    for (int w = 1; w < C::kWarps; ++w) m = fmaxf(m, sm[w * C::kRows + r]);
    const float base = m == -INFINITY ? 0.f : m;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) {
      const float f = exp2_fast(sm[w * C::kRows + r] - base);
      const float4 y = *reinterpret_cast<const float4 *>(so + (w * C::kRows + r) * C::kLdO + d);
      l = fmaf(sl[w * C::kRows + r], f, l);
      x.x = fmaf(y.x, f, x.x), x.y = fmaf(y.y, f, x.y);
      x.z = fmaf(y.z, f, x.z), x.w = fmaf(y.w, f, x.w);
    }
    put(r, d, x, m, l);
  }
}

// A warp's sums o of a piece where they hold an infinity or NaN that its weights do not explain: a
// weight in parts does not give what the definition does (a part that is zero or of the other sign
// makes NaN of an infinite value).  A dim's sum with such a value among its rows is that of these
// values alone, each times its weight in binary32.  The warp's rows of V (of Q8_0 their scales) are
// read again for them; of a row that has one, K too.  m: the warp's maxima by row, so: its sums.  Lane
// i has the dims i, 32 + i, ...  Only calls with such values come here: a call of 38 x 8192 (28/4 heads
// of 128) takes 210 us with one of them instead of 111 (Q8_0 99 instead of 72), 3.3 ms with one in
// every row.  (Summing all of the warp's rows once more took 1.2 ms with one and 1.6 with all.)
template <class C, int TYPE, int D>
__device__ __noinline__ void sum_infinities(const Params &p, int seq, int hk, int lo, int len, int tile, int count,
                                            int64_t head0, int rows, const float *m, float *so) {
  constexpr int N = 4, E = D / 32;  // query rows at a time, dims of a lane
  const AttnArgs &a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t *const pages = a.pages + seq * a.pages_ld;
  constexpr uint32_t kTop = C::kBf ? 0x7f80u : 0x7c00u;  // the exponent of what is no number
  auto is_odd = [](uint32_t x) { return (x & kTop) == kTop; };
  auto value = [&](const uint8_t *plane, const __half *scales, uint32_t row, int e) {
    const uint64_t at = uint64_t(row) * D + 32 * e + lane;
    if (C::kQ8) return float(reinterpret_cast<const int8_t *>(plane)[at]) * __half2float(scales[uint64_t(row) * E + e]);
    if (C::kQ4) {
      const uint32_t two = plane[uint64_t(row) * C::kRow + 16 * e + (lane & 15)];
      return float(int(lane < 16 ? two & 15 : two >> 4) - 8) * __half2float(scales[uint64_t(row) * E + e]);
    }
    const uint16_t x = reinterpret_cast<const uint16_t *>(plane)[at];
    return C::kBf ? __uint_as_float(uint32_t(x) << 16) : __half2float(__ushort_as_half(x));
  };
  uint32_t seen = 0;  // this lane's dims that have had such a value
  for (int t = tile; t < tile + count; ++t) {
    const int key = lo + t * C::kTK + warp * C::kKeys + lane;
    const uint32_t my_row = lane < C::kKeys && key < len ? kv_row32(a.c, pages, hk, key) : kNoRow;
    uint32_t odd = 0;  // keys with such values
    if constexpr (C::kScaled) {
      if (my_row != kNoRow)
        for (int e = 0; e < E; ++e)
          if (is_odd(__half_as_ushort(a.c.vs[uint64_t(my_row) * E + e]))) odd = 1u << lane;
    } else {
      constexpr int CH = C::kRow / 16, STEPS = C::kKeys * CH / 32, U = STEPS % 8 == 0 ? 8 : STEPS % 6 == 0 ? 6 : 4;
      static_assert(STEPS % U == 0, "whole rounds");
      for (int i0 = 0; i0 < STEPS; i0 += U) {
        uint4 v[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int at = (i0 + i) * 32 + lane;
          const uint32_t row = __shfl_sync(0xffffffffu, my_row, at / CH);
          v[i] = make_uint4(0, 0, 0, 0);
          if (row != kNoRow)
            v[i] = *reinterpret_cast<const uint4 *>(a.c.v + uint64_t(row) * C::kRow + at % CH * 16);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (is_odd(w[q]) || is_odd(w[q] >> 16)) odd |= 1u << ((i0 + i) * 32 + lane) / CH;
        }
      }
    }
    for (odd = __reduce_or_sync(0xffffffffu, odd); odd; odd &= odd - 1) {
      const uint32_t row = __shfl_sync(0xffffffffu, my_row, __ffs(odd) - 1);
      float k[E], v[E];
      uint32_t here = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        k[e] = value(a.c.k, a.c.ks, row, e), v[e] = value(a.c.v, a.c.vs, row, e);
        if (!(fabsf(v[e]) < INFINITY)) here |= 1u << e;
      }
      for (int r0 = 0; r0 < rows; r0 += N) {
        float s[N] = {};
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (r0 + i < rows)
#pragma unroll
            for (int e = 0; e < E; ++e)
              s[i] = fmaf(load_io1(a.q, a.io, (head0 + r0 + i) * D + 32 * e + lane) * a.scale * kLog2e, k[e], s[i]);
#pragma unroll
        for (int x = 16; x; x >>= 1)
#pragma unroll
          for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], x);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (r0 + i >= rows) break;
          const float top = m[r0 + i], w = exp2_fast(s[i] - (top == -INFINITY ? 0.f : top)) * C::kUnit;
          float *const o = so + (r0 + i) * C::kLdO + lane;
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (here >> e & 1) o[32 * e] = seen >> e & 1 ? fmaf(w, v[e], o[32 * e]) : w * v[e];
        }
      }
      seen |= here;
    }
  }
}

// IO: of Q4_0 rows the activations' type, else MQ_F32 (any).
template <int TYPE, int D, int NT, int IO>
__global__ void __launch_bounds__(Shape<TYPE, D, NT, IO>::kThreads, 1)
attn_decode_kernel(const __grid_constant__ Params p) {
  using C = Shape<TYPE, D, NT, IO>;
  constexpr int NG = C::kNG, MT = C::kMT, KS = D / 16;
  constexpr uint32_t kAll = MT == 2 ? 0xffffffffu : 0xffffu;  // all keys of a warp's tile
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *const ring = smem;                                               // [warp][stage][K, V]
  uint4 *const sq = reinterpret_cast<uint4 *>(ring + C::kWarps * C::kStages * C::kStage);
  float4 *const ssum = reinterpret_cast<float4 *>(sq + C::kQuery / 16);     // [8 rows][block][t]
  float *const so = reinterpret_cast<float *>(ssum + C::kSums / 16);        // [warp][row][kLdO]
  float *const sm = so + C::kWarps * C::kRows * C::kLdO, *const sl = sm + C::kWarps * C::kRows;
  float *const sfac = sl + C::kWarps * C::kRows;  // per row: scale * log2 e * 2^-e
  __shared__ Split split[2];
  int splits = 0;
  const AttnArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  grid_dependency();

  // idle sequences: their outputs are zero; and the report of bad lengths
  for (int s = blockIdx.x; s < a.S; s += gridDim.x) {
    const int raw = a.len[s];
    if (raw != clamped_len(raw, a.max_len) && tid == 0) index_error(a.status, kIdxAttnLen, raw);
    if (raw <= 0)
      for (int i = tid; i < a.hq * (D / 4); i += C::kThreads)
        store_io4(a.o, a.io, int64_t(s) * a.hq * D + 4 * i, make_float4(0.f, 0.f, 0.f, 0.f));
  }

  const Line line = lay_out(a, p.units, C::kTK, gridDim.x);
  const int64_t T = line.steps, parts = min((int64_t)gridDim.x, T);
  const int64_t me = blockIdx.x;
  if (me >= parts) return;
  const int64_t end = T * (me + 1) / parts;                         // this block's steps end here
  Cursor cur = cursor_at(p, line, C::kTK, T * me / parts);  // the next tile whose rows are looked up

  // ---- the ring ----
  // A tile's rows are found from page entries that were copied into shared memory with the tile a
  // ring's length before it.  (No load into registers stays on its way while a tile is multiplied:
  // the few scoreboards of a warp are shared, and an operand's wait became a wait for it.)
  uint8_t *const my_ring = ring + warp * C::kStages * C::kStage;
  const uint32_t ring0 = smem_addr(my_ring);
  uint32_t valid_bits[C::kStages] = {};  // per tile in flight (oldest first): keys that are there
  uint32_t odd_bits[C::kStages] = {};    // keys of odd rows (their scales, where NG is odd)
  struct Place {
    uint32_t row;  // this lane's key: its row within the page's first
    bool there;
  } place[C::kStages];  // per tile looked up (oldest first)
  auto look_up = [&](Place &to, int32_t *entry) -> const int32_t * {  // at cur; then the next tile
    const int key = cur.span.lo + cur.tile * C::kTK + warp * C::kKeys + lane;
    to.there = cur.at < end && lane < C::kKeys && key < cur.span.len;
    const uint32_t pi = quotient((uint32_t)(to.there ? key : 0), a.c.page);
    to.row = (uint32_t)(cur.hk * a.c.head_stride) +
             ((uint32_t)key - pi * a.c.page.d) * (uint32_t)a.c.slot_stride;
    const int32_t *const from = a.pages + cur.s * a.pages_ld + pi;
    if (entry && lane < C::kKeys) copy4(smem_addr(entry + lane), from, to.there ? 4 : 0);
    next_tile(cur, p, C::kTK, line.gap, end);
    return from;
  };
  auto issue = [&](int stage, Place at, int32_t page) {  // a tile's rows into a stage
    uint32_t row = 0;
    if (at.there) {
      if (page >= 0 && page < a.c.n_pages) {
        row = (uint32_t)page * (uint32_t)a.c.page_stride + at.row;
      } else {
        index_error(a.status, kIdxAttnPage, page);
        at.there = false;
      }
    }
    const uint32_t valid = __ballot_sync(0xffffffffu, at.there);
#pragma unroll
    for (int i = 0; i + 1 < C::kStages; ++i) valid_bits[i] = valid_bits[i + 1], odd_bits[i] = odd_bits[i + 1];
    valid_bits[C::kStages - 1] = valid;
    if (NG & 1) odd_bits[C::kStages - 1] = __ballot_sync(0xffffffffu, row & 1);
    constexpr int CH = C::kRow / 16;  // 16-byte chunks of a row
    const uint32_t dst = ring0 + stage * C::kStage;
#pragma unroll
    for (int i = 0; i < C::kKeys * CH / 32; ++i) {
      const int key = (i * 32 + lane) / CH, ch = (i * 32 + lane) % CH;
      const uint64_t off = uint64_t(__shfl_sync(0xffffffffu, row, key)) * C::kRow;
      const uint32_t size = (valid >> key & 1) * 16;
      copy16(dst + C::chunk_at(key, ch), a.c.k + ch * 16 + off, size);
      copy16(dst + C::kKeys * C::kStride + C::chunk_at(key, ch), a.c.v + ch * 16 + off, size);
    }
    if (C::kScaled) {  // lane i: key i % 16 (+ 16) of K, or of V
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int key = 16 * m + (lane & 15);
        const uint32_t r = __shfl_sync(0xffffffffu, row, key), on = valid >> key & 1;
        const __half *const from = (lane < 16 ? a.c.ks : a.c.vs) + uint64_t(r) * NG;
        const uint32_t to = dst + C::kRaw + ((lane >> 4) * C::kKeys + key) * C::kScaleRow;
        if constexpr (NG == 8) {
          copy16(to, reinterpret_cast<const uint8_t *>(from), on * 16);
        } else if constexpr (NG == 4) {
          copy8(to, from, on * 8);
        } else if constexpr (NG % 2 == 0) {
#pragma unroll
          for (int j = 0; j < NG / 2; ++j) copy4(to + 4 * j, from + 2 * j, on * 4);
        } else {  // an odd row starts in the middle of a word; an even one ends there
          const __half *const word = from - (r & 1);
#pragma unroll
          for (int j = 0; j < (NG + 1) / 2; ++j)
            copy4(to + 4 * j, word + 2 * j, on * (2 * j + 2 > NG && !(r & 1) ? 2 : 4));
        }
      }
    }
  };

  Cursor now = cur;  // the tile being multiplied (its piece's unit)
  {
    // the first tiles: their page entries are read here
    int32_t first[C::kStages];
#pragma unroll
    for (int i = 0; i < C::kStages; ++i) {
      const int32_t *const from = look_up(place[i], nullptr);
      first[i] = place[i].there ? *from : 0;
    }
#pragma unroll
    for (int i = 0; i < C::kStages; ++i) {
      issue(i, place[i], first[i]);
      look_up(place[i], reinterpret_cast<int32_t *>(my_ring + i * C::kStage + C::kEntries));
      copies_commit();
    }
  }
  int stage = 0;

  // operand addresses of this lane within a stage: matrix lane >> 3, row lane & 7
  const uint32_t k_lane = ((lane & 7) + (lane & 8)) * C::kStride + (lane >> 4) * 16;
  const uint32_t v_lane = (C::kKeys + (lane & 7) + (lane >> 4) * 8) * C::kStride + (lane >> 3 & 1) * 16;
  // Q8_0: the two chunks of 16 dims side by side, keys 0-7 and 8-15 each
  const uint32_t v_lane8 = (C::kKeys + (lane & 7) + (lane & 8)) * C::kStride + (lane >> 4) * 16;

  const uint32_t nil = p.group >> 31;  // (zero)
  const Int4Constants i4 = {0x64006400u + nil, 0x2c002c00u + nil};

  // Q4_0: two blocks of 32 dims side by side, keys 0-7 and 8-15 each
  const uint32_t k_lane4 = C::chunk_at((lane & 7) + (lane & 8), lane >> 4), v_lane4 = k_lane4 + C::kKeys * C::kStride;

  // The query rows of a unit as they are read: warp w has the rows w, w + kWarps, ..., lane i the
  // dims 8 i .. 8 i + 7.
  constexpr int RPW = (C::kRows + C::kWarps - 1) / C::kWarps;
  float4 query[RPW][2];
  auto load_query = [&](const Cursor &c) {
    const int rows = min(C::kRows, p.group - c.rg * C::kRows);
    const int64_t head0 = int64_t(c.s) * a.hq + c.hk * p.group + c.rg * C::kRows;
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      const int r = warp + i * C::kWarps;
      query[i][0] = query[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows && lane < D / 8) {
        query[i][0] = load_io4(a.q, a.io, (head0 + r) * D + lane * 8);
        query[i][1] = load_io4(a.q, a.io, (head0 + r) * D + lane * 8 + 4);
      }
    }
  };
  load_query(now);

  while (now.at < end) {
    // ---- one piece: tiles of one unit ----
    const int64_t unit_first = now.at - now.tile;  // the step of the unit's first tile
    const int tiles = now.span.tiles;
    const int count = (int)min(end - now.at, int64_t(tiles - now.tile));
    const int rows = min(C::kRows, p.group - now.rg * C::kRows);  // query rows that exist
    const int64_t head0 = int64_t(now.s) * a.hq + now.hk * p.group + now.rg * C::kRows;
    const int64_t unit_id = int64_t(now.s) * p.units + now.hk * p.row_groups + now.rg;

    // the query's parts as operand words: lane 4 r + t' of (part, 8-row group, 32 dims) has the
    // words of two 16-dim steps.  f16 and bf16 rows: dims 2t', 2t' + 1 and 8 more of a step;
    // Q8_0 rows: dims 4t' .. 4t' + 3 (a chunk's four bytes); Q4_0 rows: the dims 4t', 4t' + 2; 4t' + 1,
    // 4t' + 3 (four bytes' low halves), and 16 more (their high halves)
#pragma unroll
    for (int i0 = 0; i0 < RPW; ++i0) {
      const int r = warp + i0 * C::kWarps;
      if (r >= C::kRows) break;
      const float4 u = query[i0][0], v = query[i0][1];
      const float x[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
      // a power of two that puts the row's largest element in [2^14, 2^15); bf16 has binary32's range:
      // only what its ends are near is put about 1
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
      top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
      const int power = (int)(__float_as_uint(top) >> 23) - 127;
      int e = 0;
      if (top > 0.f && top < INFINITY && (!C::kBf || abs(power) > 60))
        e = min(max((C::kBf ? 0 : 14) - power, -126), 126);
      const float up = __uint_as_float(uint32_t(127 + e) << 23);
      // (Q8_0 keys enter the product as 2^-24 (v + 128), see below; a factor past binary32 has logits
      // there or zeros, and a finite one in its place leaves their order)
      if (lane == 0) {
        const float f = a.scale * __uint_as_float(uint32_t(127 - e) << 23) * (kLog2e * (C::kQ8 ? 0x1p24f : 1.f));
        sfac[r] = fminf(fmaxf(f, -FLT_MAX), FLT_MAX);
      }
      if (lane < D / 8) {
        uint32_t w[4][C::kQueryParts];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int a = C::kQ4 ? 4 * (i >> 1) + (i & 1) : 2 * i, b = C::kQ4 ? a + 2 : a + 1;
          split2<C::kBf>(x[a] * up, x[b] * up, w[i]);
        }
        if (C::kQ8) {
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < C::kQueryParts; ++k) {
              const float2 v = unpack2<C::kBf>(w[i][k]);
              sum += v.x + v.y;
            }
          constexpr unsigned mask = D / 8 == 32 ? 0xffffffffu : (1u << D / 8 % 32) - 1;
          sum += __shfl_xor_sync(mask, sum, 1);
          sum += __shfl_xor_sync(mask, sum, 2);
          if ((lane & 3) == 0) {  // rows r & 6 and r | 1 of the accumulator's elements 0, 2 and 1, 3
            float *const to = reinterpret_cast<float *>(ssum + ((r >> 3) * NG + (lane >> 2)) * 4 + (r >> 1 & 3));
            to[r & 1] = to[(r & 1) + 2] = sum * (-128 * 0x1p-24f);
          }
        }
        // the lane's 8 dims are half `lane & 1` of step lane >> 1
        uint32_t *q = reinterpret_cast<uint32_t *>(sq + ((r >> 3) * NG + (lane >> 2)) * 32 + (r & 7) * 4);
        const int step = lane >> 1 & 1, half = lane & 1;
#pragma unroll
        for (int k = 0; k < C::kQueryParts; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t *const to = q + k * NT * NG * 128;
            if (C::kScaled)
              to[(2 * half + (i >> 1)) * 4 + 2 * step + (i & 1)] = w[i][k];
            else
              to[i * 4 + 2 * step + half] = w[i][k];
          }
      }
    }
    __syncthreads();
    float fac[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) fac[n][0] = sfac[8 * n + 2 * t], fac[n][1] = sfac[8 * n + 2 * t + 1];

    float o[KS][NT][4] = {}, mx[NT][2], ls[NT][2] = {}, unit = 1.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) mx[n][0] = mx[n][1] = -INFINITY;

    for (int i = 0; i < count; ++i) {
      copies_wait<C::kStages - 1>();
      __syncwarp();
      const uint32_t here = valid_bits[0];
      const uint32_t base = ring0 + stage * C::kStage;
      uint8_t *const my_stage = my_ring + stage * C::kStage;
      auto at4 = [&](uint32_t lane_at, int block) {  // (an even block's chunk: a bit of its own)
        return C::kSwizzled ? (base + lane_at) ^ (block * 16) : base + lane_at + block * 16;
      };
      if (here) {
        float tile_unit = 1.f, per_unit = 1.f;  // the power of two of V's scales, and its inverse
        constexpr int SW = C::kScaleRow / 4;    // words of a row's scales, two each
        // the scales of a key: of K (plane 0) or V (1)
        auto scales_of = [&](uint32_t (&w)[SW], int plane, int key) {
          const uint8_t *const from = my_stage + C::kRaw + (plane * C::kKeys + key) * C::kScaleRow;
          if constexpr (SW == 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(from);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
          } else if constexpr (SW == 2) {
            const uint2 v = *reinterpret_cast<const uint2 *>(from);
            w[0] = v.x, w[1] = v.y;
          } else {
#pragma unroll
            for (int j = 0; j < SW; ++j) w[j] = reinterpret_cast<const uint32_t *>(from)[j];
          }
          if constexpr (NG & 1) {  // (an odd row's start in the middle of its first word)
            const int shift = odd_bits[0] >> key & 1 ? 16 : 0;
#pragma unroll
            for (int j = 0; j < SW; ++j) w[j] = __funnelshift_r(w[j], j + 1 < SW ? w[(j + 1) % SW] : 0, shift);
          }
        };
        if (C::kScaled) {  // a power of two that V's largest scale of the tile is below
          // (f16 bits of magnitudes order as numbers; with 0x400 more, those of infinities and NaN are negative: beside
          // one the other products must stay numbers.  Two at a time 58.8 us of Q4_0's 64 sequences above, one by
          // one 59.5; of Q8_0's 66.4 and 65.6.)
          int top = 0;
          uint32_t tops = 0x04000400u;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            uint32_t w[SW];
            scales_of(w, 1, 16 * m + (lane & 15));
            if (NG & 1) w[SW - 1] &= 0xffffu;
#pragma unroll
            for (int j = 0; j < SW; ++j) {
              const uint32_t x = (w[j] & 0x7fff7fffu) + 0x04000400u;
              if (C::kQ4) tops = __vmaxs2(tops, x);
              else top = max(top, max((int)x >> 16, (int)(int16_t)x));
            }
          }
          if (C::kQ4) top = max(tops & 0xffffu, tops >> 16);
          top = __reduce_max_sync(0xffffffffu, max(top - 0x400, 0));
          int e = top == 0 ? 126 : (int)(__float_as_uint(__half2float(__ushort_as_half((uint16_t)top))) >> 23);
          if (C::kQ4) e = max(e, 111);  // (up by 2^15 at most: a factor in f16)
          tile_unit = __uint_as_float(uint32_t(e + 1) << 23), per_unit = __uint_as_float(uint32_t(253 - e) << 23);
        }
        // ---- S^T = K Q^T ----
        // Two groups of 32 dims at a time, so that (with two 16-key groups for narrow rows) four
        // chains of products are on their way; f16 and bf16 rows have an accumulator per chain
        // and part kind (first; others) up to the end.
        float s[MT][NT][4], acc[2][2][MT][NT][4] = {};
        uint32_t kscale[MT][2][SW];  // of the keys g, g + 8
        if (C::kScaled)
#pragma unroll
          for (int m = 0; m < MT; ++m) scales_of(kscale[m][0], 0, 16 * m + g), scales_of(kscale[m][1], 0, 16 * m + 8 + g);
#pragma unroll
        for (int j0 = 0; j0 < NG; j0 += 2) {
          uint4 b[2][C::kQueryParts][NT];
          uint32_t ka[2][MT][2][4];  // two steps of 16 dims
          float cq[2][MT][NT][4];    // Q8_0, Q4_0: the blocks' sums
          if (C::kQ4) {
            // Four bytes of a key's block, exact: as subnormals with the 8 in the accumulators' start, as
            // Q8_0's are, they save 28 operations a row of 128 and lose bits (the tensor cores align a
            // product by its factors' exponents, and a subnormal's says nothing of its leading
            // zeros): an error to 64 bits of 2e-6 at 64 ragged sequences instead of 4e-7.
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              uint32_t x[4];  // block j0: keys g, g + 8; block j0 + 1
              ldmatrix4<false>(x, at4(k_lane4 + 16 * m * C::kStride, j0));
#pragma unroll
              for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t u = x[2 * jj + h], v = u >> 8;
                  ka[jj][m][0][h] = int4_f16<0x000f000fu>(u, i4), ka[jj][m][0][2 + h] = int4_f16<0x000f000fu>(v, i4);
                  ka[jj][m][1][h] = int4_f16<0x00f000f0u>(u, i4), ka[jj][m][1][2 + h] = int4_f16<0x00f000f0u>(v, i4);
                }
            }
          }
#pragma unroll
          for (int jj = 0; jj < 2; ++jj) {
            const int j = j0 + jj;
            if (j >= NG) continue;
#pragma unroll
            for (int k = 0; k < C::kQueryParts; ++k)
#pragma unroll
              for (int n = 0; n < NT; ++n) b[jj][k][n] = sq[((k * NT + n) * NG + j) * 32 + lane];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              const uint32_t at_k = base + k_lane + 16 * m * C::kStride;
              if (C::kQ8) {
                // a byte of v ^ 0x80 alone in 16 bits is the f16 (subnormal) 2^-24 (v + 128); the
                // accumulators start at -128 * 2^-24 times the block's sum of the query
                uint32_t x[4];  // keys g (0, 2) and g + 8 (1, 3), chunks 0 and 1
                ldmatrix4<false>(x, at_k + j * 32);
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                  const uint32_t xa = x[2 * st] ^ 0x80808080u, xb = x[2 * st + 1] ^ 0x80808080u;
                  ka[jj][m][st][0] = __byte_perm(xa, 0, 0x4140), ka[jj][m][st][1] = __byte_perm(xb, 0, 0x4140);
                  ka[jj][m][st][2] = __byte_perm(xa, 0, 0x4342), ka[jj][m][st][3] = __byte_perm(xb, 0, 0x4342);
                }
              } else if (!C::kQ4) {
                ldmatrix4<false>(ka[jj][m][0], at_k + j * 64);
                ldmatrix4<false>(ka[jj][m][1], at_k + j * 64 + 32);
              }
            }
          }
#pragma unroll
          for (int k = 0; k < C::kQueryParts; ++k)
#pragma unroll
            for (int st = 0; st < 2; ++st)
#pragma unroll
              for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                  for (int n = 0; n < NT; ++n) {
                    if (j0 + jj >= NG) continue;
                    const uint32_t(&x)[4] = ka[jj][m][st];
                    const uint32_t b0 = st ? b[jj][k][n].z : b[jj][k][n].x;
                    const uint32_t b1 = st ? b[jj][k][n].w : b[jj][k][n].y;
                    if (!C::kScaled)
                      mma<C::kBf>(acc[jj][k > 0][m][n], x[0], x[1], x[2], x[3], b0, b1);
                    else if (k == 0 && st == 0)
                      mma_from(cq[jj][m][n], x[0], x[1], x[2], x[3], b0, b1,
                               C::kQ8 ? ssum[(n * NG + j0 + jj) * 4 + t] : make_float4(0.f, 0.f, 0.f, 0.f));
                    else
                      mma<false>(cq[jj][m][n], x[0], x[1], x[2], x[3], b0, b1);
                  }
          if (C::kScaled) {  // the blocks' sums times the scales of keys g, g + 8
#pragma unroll
            for (int jj = 0; jj < 2; ++jj)
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                if (j0 + jj >= NG) continue;
                const float2 d0 = unpack2<false>(kscale[m][0][j0 / 2]), d1 = unpack2<false>(kscale[m][1][j0 / 2]);
                const float da = jj ? d0.y : d0.x, db = jj ? d1.y : d1.x;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                  for (int w = 0; w < 4; ++w)
                    acc[0][0][m][n][w] = fmaf(cq[jj][m][n][w], w < 2 ? da : db, acc[0][0][m][n][w]);
              }
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              if (C::kScaled) {
                s[m][n][w] = acc[0][0][m][n][w];
              } else {
                // (an infinite key: the first parts' product has the sign, the others' may be NaN)
                const float first = acc[0][0][m][n][w] + acc[1][0][m][n][w];
                const float others = acc[0][1][m][n][w] + acc[1][1][m][n][w];
                s[m][n][w] = first + (fabsf(first) < INFINITY ? others : 0.f);
              }
            }
        // ---- softmax ----
        const int key0 = now.span.lo + (now.tile + i) * C::kTK + warp * C::kKeys;
        float al[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int w = 0; w < 4; ++w) s[m][n][w] *= fac[n][w & 1];
        // Q4_0: a tile without a logit above its row's largest so far, as most are, needs no maximum over the lanes
        // (three shuffles one after the other)
        bool renew = !C::kQ4;
        if (here != kAll) {
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const bool ga = here >> (16 * m + g) & 1, gb = here >> (16 * m + 8 + g) & 1;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int w = 0; w < 4; ++w)
                if (!(w < 2 ? ga : gb)) s[m][n][w] = -INFINITY;
          }
        }
        if (p.logits) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
              if (8 * n + 2 * t < p.logit_width) {
                const int ka = key0 + 16 * m + g;
                float *q = p.logits + (unit_id * a.max_len + ka) * p.logit_width + 8 * n + 2 * t;
                if (ka < now.span.len) *reinterpret_cast<float2 *>(q) = make_float2(s[m][n][0], s[m][n][1]);
                if (ka + 8 < now.span.len)
                  *reinterpret_cast<float2 *>(q + 8 * p.logit_width) = make_float2(s[m][n][2], s[m][n][3]);
              }
        }
        if (C::kQ4) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              float top = -INFINITY;
#pragma unroll
              for (int m = 0; m < MT; ++m) top = fmaxf(top, fmaxf(s[m][n][w], s[m][n][w + 2]));
              renew |= top > mx[n][w];
            }
          renew = __any_sync(0xffffffffu, renew);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            al[n][w] = 1.f;
            if (renew) {
              float top = mx[n][w];
#pragma unroll
              for (int m = 0; m < MT; ++m) top = fmaxf(top, fmaxf(s[m][n][w], s[m][n][w + 2]));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
              al[n][w] = exp2_fast(mx[n][w] - (top == -INFINITY ? 0.f : top));
              mx[n][w] = top;
            }
            const float low = mx[n][w] == -INFINITY ? 0.f : mx[n][w];  // no key yet: all weights 0
            float sum = 0.f;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              s[m][n][w] = exp2_fast(s[m][n][w] - low) * (C::kQ4 ? 1.f : C::kUnit);
              s[m][n][w + 2] = exp2_fast(s[m][n][w + 2] - low) * (C::kQ4 ? 1.f : C::kUnit);
              sum += s[m][n][w] + s[m][n][w + 2];
            }
            if (C::kQ4) sum *= C::kUnit;
            ls[n][w] = fmaf(ls[n][w], al[n][w], sum);
          }
        const float weight_unit = C::kUnit * fminf(per_unit, 1.f);  // Q4_0
        // the weights transposed: lane (g, t) gets row g's of the keys 2t, 2t + 1, 2t + 8, 2t + 9;
        // their parts, or for Q8_0 (whose blocks' scales come first) as binary32 in two halves
        uint32_t pw[MT][NT][2][C::kParts];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (C::kQ8) {
                const uint32_t x = __float_as_uint(s[m][n][2 * h]), y = __float_as_uint(s[m][n][2 * h + 1]);
                const uint32_t hi = transpose8x8(__byte_perm(x, y, 0x7632));
                const uint32_t lo = transpose8x8(__byte_perm(x, y, 0x5410));
                s[m][n][2 * h] = __uint_as_float(__byte_perm(lo, hi, 0x5410)) * per_unit;
                s[m][n][2 * h + 1] = __uint_as_float(__byte_perm(lo, hi, 0x7632)) * per_unit;
              } else {
                if (C::kQ4) s[m][n][2 * h] *= weight_unit, s[m][n][2 * h + 1] *= weight_unit;
                split2<C::kBf>(s[m][n][2 * h], s[m][n][2 * h + 1], pw[m][n][h]);
#pragma unroll
                for (int k = 0; k < C::kParts; ++k) pw[m][n][h][k] = transpose8x8(pw[m][n][h][k]);
              }
            }
        // ---- O^T = O^T alpha + V^T P^T ----
        if (C::kScaled) {  // o stands in units of the tile's power of two
#pragma unroll
          for (int n = 0; n < NT; ++n) al[n][0] *= unit * per_unit, al[n][1] *= unit * per_unit;
          unit = tile_unit;
        }
        uint32_t vscale[MT][4][SW];  // of the keys 2t, 2t + 1, 2t + 8, 2t + 9
        if (C::kScaled)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int q = 0; q < 4; ++q) scales_of(vscale[m][q], 1, 16 * m + 8 * (q >> 1) + 2 * t + (q & 1));
        if (C::kQ4 && per_unit > 1.f) {  // (exact)
          const __half2 up = __float2half2_rn(per_unit);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int j = 0; j < SW; ++j) {
                const __half2 d = __hmul2_rn(*reinterpret_cast<const __half2 *>(&vscale[m][q][j]), up);
                vscale[m][q][j] = *reinterpret_cast<const uint32_t *>(&d);
              }
        }
#pragma unroll
        for (int j0 = 0; j0 < NG; j0 += 2) {  // (two groups of 32 dims, four chains)
          float c[2][2][NT][4] = {};
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            uint32_t va[2][2][4];  // [group][16 dims][operand word]
            uint32_t pq[2][NT][2][C::kParts];
            if constexpr (C::kQ4) {
              uint32_t x[4];  // bytes 2g, 2g + 1 of the keys 2t, 2t + 1: block j0 of keys 0-7, 8-15, then j0 + 1
              ldmatrix4<true>(x, at4(v_lane4 + 16 * m * C::kStride, j0));
#pragma unroll
              for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  // low halves: dims 2g and 2g + 1, high halves: 16 more
                  const uint32_t u = x[2 * jj + q], v = u >> 8;
                  va[jj][0][2 * q] = int4_f16<0x000f000fu>(u, i4), va[jj][0][2 * q + 1] = int4_f16<0x000f000fu>(v, i4);
                  va[jj][1][2 * q] = int4_f16<0x00f000f0u>(u, i4), va[jj][1][2 * q + 1] = int4_f16<0x00f000f0u>(v, i4);
                  const uint32_t d = __byte_perm(vscale[m][2 * q][j0 / 2], vscale[m][2 * q + 1][j0 / 2], jj ? 0x7632 : 0x5410);
#pragma unroll
                  for (int n = 0; n < NT; ++n) scale_parts(pw[m][n][q], d, pq[jj][n][q]);
                }
            }
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
              const int j = j0 + jj;
              if (j >= NG) continue;
              if (C::kQ8) {
                uint32_t x[4];  // dims 2g, 2g + 1 of the keys 2t, 2t + 1: chunk 0, 1 of keys 0-7, 8-15
                ldmatrix4<true>(x, base + v_lane8 + 16 * m * C::kStride + j * 32);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                  for (int q = 0; q < 2; ++q) {
                    const uint32_t u = x[2 * h + q] ^ 0x80808080u;
                    va[jj][h][2 * q] = int8_f16<0x4240>(u), va[jj][h][2 * q + 1] = int8_f16<0x4341>(u);
                  }
                float d[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const float2 v = unpack2<false>(vscale[m][q][j0 / 2]);
                  d[q] = jj ? v.y : v.x;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  split2<C::kBf>(s[m][n][0] * d[0], s[m][n][1] * d[1], pq[jj][n][0]);
                  split2<C::kBf>(s[m][n][2] * d[2], s[m][n][3] * d[3], pq[jj][n][1]);
                }
              } else if (!C::kQ4) {
                ldmatrix4<true>(va[jj][0], base + v_lane + 16 * m * C::kStride + j * 64);
                ldmatrix4<true>(va[jj][1], base + v_lane + 16 * m * C::kStride + j * 64 + 32);
              }
            }
#pragma unroll
            for (int k = 0; k < C::kParts; ++k)
#pragma unroll
              for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                  for (int n = 0; n < NT; ++n) {
                    if (j0 + jj >= NG) continue;
                    const uint32_t(&v)[4] = va[jj][h];
                    mma<C::kBf>(c[jj][h][n], v[0], v[1], v[2], v[3],
                                C::kScaled ? pq[jj][n][0][k] : pw[m][n][0][k],
                                C::kScaled ? pq[jj][n][1][k] : pw[m][n][1][k]);
                  }
          }
#pragma unroll
          for (int jj = 0; jj < 2; ++jj)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                  if (j0 + jj >= NG) continue;
                  float &old = o[2 * (j0 + jj) + h][n][w];
                  old = fmaf(old, al[n][w & 1], c[jj][h][n][w]);
                }
        }
      }
      __syncwarp();  // the stage has been read
      {
        int32_t *const entry = reinterpret_cast<int32_t *>(my_stage + C::kEntries);
        const int32_t page = entry[lane & (C::kKeys - 1)];
        issue(stage, place[0], page);
#pragma unroll
        for (int q = 0; q + 1 < C::kStages; ++q) place[q] = place[q + 1];
        look_up(place[C::kStages - 1], entry);
        copies_commit();
      }
      if (++stage == C::kStages) stage = 0;
    }

    // ---- the piece's result; the next piece's query is on its way meanwhile ----
    Cursor next = now;
    next.tile += count - 1, next.at += count - 1;
    next_tile(next, p, C::kTK, line.gap, end);
    if (next.at < end) load_query(next);
    bool odd = false;  // a row whose weights are numbers has a dim that is none
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float l = ls[n][w];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int r = warp * C::kRows + 8 * n + 2 * t + w;
        if (g == 0) sm[r] = mx[n][w], sl[r] = l;
        float zero[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < KS; ++j)
          zero[0] = fmaf(o[j][n][w], 0.f, zero[0]), zero[1] = fmaf(o[j][n][w + 2], 0.f, zero[1]);
        odd |= l < INFINITY && zero[0] + zero[1] != 0.f;
#pragma unroll
        for (int j = 0; j < KS; ++j)
          if (C::kScaled) {  // dims 16 j + 2g, 2g + 1
            *reinterpret_cast<float2 *>(so + r * C::kLdO + 16 * j + 2 * g) =
                make_float2(o[j][n][w] * unit, o[j][n][w + 2] * unit);
          } else {
            so[r * C::kLdO + 16 * j + g] = o[j][n][w];
            so[r * C::kLdO + 16 * j + 8 + g] = o[j][n][w + 2];
          }
      }
    if (__any_sync(0xffffffffu, odd)) {
      __syncwarp();
      sum_infinities<C, TYPE, D>(p, now.s, now.hk, now.span.lo, now.span.len, now.tile, count, head0, rows,
                                 sm + warp * C::kRows, so + warp * C::kRows * C::kLdO);
    }
    __syncthreads();
    if (now.tile == 0 && count == tiles) {
      join_warps<C>(so, sm, sl, D, rows, [&](int r, int d, float4 x, float m, float l) {
        finish<C>(p, head0, unit_id, r, d, D, x, m, l);
      });
    } else {
      const Result mine = result_of<C, D>(p, now.tile == 0, me);  // a block leaves at most two pieces
      join_warps<C>(so, sm, sl, D, rows, [&](int r, int d, float4 x, float m, float l) {
        store_result(mine, D, r, d, x, m, l);
      });
      // blocks of the unit's first and last tile: block b has the steps from T b / parts on
      if (tid == 0)
        split[splits] = {head0, unit_id, ((unit_first + 1) * parts - 1) / T,
                         ((unit_first + tiles) * parts - 1) / T, rows, 0, 0, 0};
      ++splits;
    }
    now = next;
  }
  // Shared units, after the last piece (to count a piece in behind its stores holds a block up, at
  // the end as after the first piece, but here once).
  if (splits == 0) return;
  __syncthreads();
  if (tid < splits) {
    Split &u = split[tid];
    const Groups gr = groups_of(u);
    const int mine = (int)(me - u.b0) / gr.size;
    u.first = u.b0 + mine * gr.size;
    u.members = (int)min(int64_t(gr.size), u.b1 - u.first + 1);
    u.last = arrive(p.count + (mine ? kMaxParts : 0) + u.first, u.members - 1);
  }
  __syncthreads();
  for (int k = 0; k < splits; ++k) {
    const Split &u = split[k];
    if (!u.last) continue;
    const Groups gr = groups_of(u);
    const Result none = {nullptr, nullptr};
    const Result group = result_of<C, D>(p, 2 + (u.first == u.b0), u.first);
    join_results<C, D>(p, u, result_of<C, D>(p, u.first == u.b0, u.first), result_of<C, D>(p, 0, u.first), 1,
                       u.members, gr.number == 1 ? none : group);
    if (gr.number == 1) continue;
    __syncthreads();
    if (tid == 0) split[k].last = arrive(p.count + 2 * kMaxParts + u.b0, gr.number - 1);
    __syncthreads();
    if (u.last)
      join_results<C, D>(p, u, result_of<C, D>(p, 3, u.b0), result_of<C, D>(p, 2, u.b0), gr.size, gr.number,
                         none);
  }
}

template <int TYPE, int D, int NT, int IO>
mq_status launch_shape(const Params &p, cudaStream_t s, const DeviceState *st) {
  using C = Shape<TYPE, D, NT, IO>;
  const int64_t tiles = (p.a.max_len + C::kTK - 1) / C::kTK * p.a.S * p.units;
  const int64_t grid = std::min<int64_t>(std::min(st->sms, kMaxParts), tiles);
  return launch_dependent("attn_decode_kernel", attn_decode_kernel<TYPE, D, NT, IO>,
                          dim3((unsigned)grid, 1, 1), dim3(C::kThreads, 1, 1), C::kSmem, s, p);
}
template <int TYPE, int D, int NT, int IO>
mq_status opt_in_shape(const DeviceState *st) {
  using C = Shape<TYPE, D, NT, IO>;
  if (C::kSmem > st->smem_optin)
    return fail(MQ_ERR_LAUNCH, "attn_decode_kernel needs %d bytes of shared memory, the device allows %d",
                C::kSmem, st->smem_optin);
  const cudaError_t e = cudaFuncSetAttribute(attn_decode_kernel<TYPE, D, NT, IO>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  return e == cudaSuccess ? MQ_OK : cuda_fail(e, "cudaFuncSetAttribute", "attn_decode_kernel");
}
template <int TYPE, int D, int IO>
mq_status opt_in_rows(const DeviceState *st) {
  mq_status r = opt_in_shape<TYPE, D, 1, IO>(st);
  if constexpr (D <= 128)
    if (r == MQ_OK) r = opt_in_shape<TYPE, D, 2, IO>(st);
  return r;
}
template <int TYPE, int IO>
mq_status opt_in(const DeviceState *st) {
  mq_status r = opt_in_rows<TYPE, 64, IO>(st);
  if (r == MQ_OK) r = opt_in_rows<TYPE, 96, IO>(st);
  if (r == MQ_OK) r = opt_in_rows<TYPE, 128, IO>(st);
  if (r == MQ_OK) r = opt_in_rows<TYPE, 192, IO>(st);
  if (r == MQ_OK) r = opt_in_rows<TYPE, 256, IO>(st);
  return r;
}
template <int TYPE, int D, int IO>
mq_status launch_rows(const Params &p, int rows, cudaStream_t s, const DeviceState *st) {
  if constexpr (D <= 128)
    if (rows == 16) return launch_shape<TYPE, D, 2, IO>(p, s, st);
  return launch_shape<TYPE, D, 1, IO>(p, s, st);
}
template <int TYPE, int IO>
mq_status launch_dim(const Params &p, int rows, cudaStream_t s, const DeviceState *st) {
  switch (p.a.c.dim) {
    case 64: return launch_rows<TYPE, 64, IO>(p, rows, s, st);
    case 96: return launch_rows<TYPE, 96, IO>(p, rows, s, st);
    case 128: return launch_rows<TYPE, 128, IO>(p, rows, s, st);
    case 192: return launch_rows<TYPE, 192, IO>(p, rows, s, st);
    default: return launch_rows<TYPE, 256, IO>(p, rows, s, st);
  }
}

}  // namespace attn

// attn_decode_q4.cu: the kernels of Q4_0 rows.
mq_status init_attn_decode_q4(const DeviceState *st);
mq_status launch_attn_decode_q4(const attn::Params &p, int rows, cudaStream_t s, const DeviceState *st);

}  // namespace mq
