// rope_store.cu -- mq_rope_store and mq_norm_rope_store: bias, norms of the query and key heads, rotary
// positions with several axes, and the store of keys and values into the paged cache.
//
// Mathematics: pair i of a head turns by the angle of table[pos[axis[i]]][i] = (c, s),
//     r0 = a0 c - a1 s,   r1 = a0 s + a1 c,
// every step rounded on its own (no contraction), so that the result is defined bit for bit.  With norms
// a0 and a1 are first multiplied by g = 1 / sqrt(mean(a^2) + eps) of their head and by their weights.
//
// What bounds it: the bytes of qkv, q and the rows stored, each moved once.  A thread keeps one
// place in the head, four pairs (two groups of four dims, 16 bytes of f32 each), for all heads
// that it visits: the cosines and sines of a token are read once and stay in registers, and
// every access is 8 or 16 bytes wide.  A thread block takes one token after another, its threads
// as many heads at a time as divide the heads evenly (a block per token pays the threads' places,
// axes and divisions for each: 652 instructions a warp, 131 us for 16384 bf16 tokens); few tokens
// are spread over more blocks, a round of heads each.  Q8_0 rows: the largest magnitude of a
// 32-element block meets in shared memory as an integer maximum (the halves of a partial rotation
// may end inside a block, so no fixed lanes share one), then the quants as in quant_row.cuh.  Q4_0 rows:
// the largest element keeps its sign, and a block's 32 numbers meet in shared memory, from which every thread
// packs four bytes of the row.  A norm's two sums (`squares`) are added over the lanes of a head where they are a
// power of two, else in shared memory by fours; the kernels with norms are made for each head size
// and go round by round (NP = 1), so that five blocks of 256 threads are on an SM: they are bound by their
// instructions, not by the bytes.
// Measured (28/4 heads of 128): 16384 tokens f32 to f16 98 us (5.9 TB/s, 89% of a plain copy's
// rate), to Q8_0 93 us (90%; three rounds at once spill 8 bytes a thread), bf16 to f16 64 us (72%: one
// token's loads are in flight per block, fewer bytes than cover the latency); 4096 tokens f32 to
// f16, three axes, 25.2 us (86%); 1023 tokens bf16 to Q8_0, 32/8 heads, half of a head rotated, 9.9 us
// (2.8 times its bytes' time: a block has one or two whole tokens, so the shares are uneven); 8
// tokens 2.1 us.  4096 tokens, 32/8 heads of 128, f32 to Q4_0: 31.7 us without norms, 44.4 with them (58% of a
// plain copy's rate; with pairs of sums 63, by whole numbers 50.7, by rounds 47.9, by head size 45.0,
// magnitudes compared as numbers instead of bits 44.4; four blocks an SM 49.0, six 44.8); 1023 of 12/12
// heads of 96, bf16 to bf16, with norms 8.9 us (5.6 without); 8 of 16/8 heads of 128 2.8 us.
#include <algorithm>
#include <type_traits>

#include "kv.cuh"
#include "quant_row.cuh"

namespace mq {
namespace {

constexpr int kThreads = 256;  // at most
constexpr int kNormBlocks = 5;  // of 256 threads per SM, of the kernels with norms

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y), __fadd_rn(a.z, b.z),
                     __fadd_rn(a.w, b.w));
}
__device__ __forceinline__ float4 normed4(float4 x, float by, float4 w) {
  return make_float4(__fmul_rn(__fmul_rn(x.x, by), w.x), __fmul_rn(__fmul_rn(x.y, by), w.y),
                     __fmul_rn(__fmul_rn(x.z, by), w.z), __fmul_rn(__fmul_rn(x.w, by), w.w));
}
__device__ __forceinline__ void turn(float &a, float &b, float2 cs) {
  const float x = a, y = b;
  a = __fsub_rn(__fmul_rn(x, cs.x), __fmul_rn(y, cs.y));
  b = __fadd_rn(__fmul_rn(x, cs.y), __fmul_rn(y, cs.x));
}
__device__ __forceinline__ uint32_t top4(float4 v) {  // (a NaN's bits exceed every number's)
  return max(max(__float_as_uint(v.x) & 0x7fffffffu, __float_as_uint(v.y) & 0x7fffffffu),
             max(__float_as_uint(v.z) & 0x7fffffffu, __float_as_uint(v.w) & 0x7fffffffu));
}
// The largest magnitude, a NaN if there is one.
__device__ __forceinline__ float magnitude4(float4 v) {
  return max_nan(max_nan(fabsf(v.x), fabsf(v.y)), max_nan(fabsf(v.z), fabsf(v.w)));
}
// The scale of a block whose largest magnitude has the bits `top`, and the quants of four of its
// elements.
__device__ __forceinline__ __half block_scale(uint32_t top) {
  const float d = div127(__uint_as_float(top));
  return __float2half_rn(d > 65504.f ? 65504.f : d);
}
__device__ __forceinline__ uint32_t quants4(float4 v, float d) {
  float t[4] = {kQuantMagic, kQuantMagic, kQuantMagic, kQuantMagic}, q[4];
  if (d != 0.f) quant_codes4(v, d, __frcp_rn(d), t, q);
  return __byte_perm(__byte_perm(__float_as_uint(t[0]), __float_as_uint(t[1]), 0x0040),
                     __byte_perm(__float_as_uint(t[2]), __float_as_uint(t[3]), 0x0040), 0x5410);
}

// Q4_0 rows: a block's scale has the sign that its largest element has not, so that element is -8 or near
// it.  The largest meets as its magnitude's bits with the sign below them (of two alike the positive one).
__device__ __forceinline__ uint32_t signed_top4(float4 v) {
  auto key = [](float x) {
    const uint32_t b = __float_as_uint(x);
    return b << 1 | (b >> 31 ^ 1);
  };
  return max(max(key(v.x), key(v.y)), max(key(v.z), key(v.w)));
}
__device__ __forceinline__ __half block_scale4(uint32_t top) {
  const float d = __uint_as_float(top >> 1 | (top << 31 ^ 0x80000000u)) * -0.125f;
  return __float2half_rn(d > 65504.f ? 65504.f : d < -65504.f ? -65504.f : d);
}
// The numbers n of four elements, a byte each.
__device__ __forceinline__ uint32_t numbers4(float4 v, float d) {
  float t[4], q[4] = {0.f, 0.f, 0.f, 0.f};
  if (d != 0.f) quant_codes4(v, d, __frcp_rn(d), t, q);
#pragma unroll
  for (int k = 0; k < 4; ++k) t[k] = __fadd_rn(fminf(fmaxf(q[k], -8.f), 7.f), kQuantMagic + 8.f);
  return __byte_perm(__byte_perm(__float_as_uint(t[0]), __float_as_uint(t[1]), 0x0040),
                     __byte_perm(__float_as_uint(t[2]), __float_as_uint(t[3]), 0x0040), 0x5410);
}

// The norm's factor g = 1 / sqrt(mean(a^2) + eps), to the nearest binary32 number but for values very near the
// middle of two: a stored row is rounded to few bits, so a last place of g would show in them.  In units
// of a power of two q, 2^-7 of the head's largest element or so, an element is h + l, h a whole number of
// at most 2^8 and |l| <= 1/2.  Then sum h^2 is exact (a whole number below 2^24), and sum (2 h + l) l is
// 2^-8 of it and keeps 2^-31 of the whole in binary32.  (Sums of squares and what they round off as pairs
// took half as many operations again.)  One step of Newton's from the approximate root, with its residual in
// parts, does the rest.
struct Unit {
  float q, inv;  // and 1 / q
};
// top: the bits of the largest magnitude; least: the exponent that q has at least (elements that small beside
// sqrt(eps) do not count).
__device__ __forceinline__ Unit unit_of(uint32_t top, int least) {
  const int e = min(max((int)(top >> 23) - 7, least), 247);
  return {__uint_as_float((uint32_t)e << 23), __uint_as_float((uint32_t)(254 - e) << 23)};
}
// The two sums of a thread's elements.
__device__ __forceinline__ float2 squares(float4 x, float4 y, Unit u) {
  const float2 inv = make_float2(u.inv, u.inv), up = make_float2(kQuantMagic, kQuantMagic);
  const float2 down = make_float2(-kQuantMagic, -kQuantMagic), neg = make_float2(-1.f, -1.f);
  const float2 v[4] = {make_float2(x.x, x.y), make_float2(x.z, x.w), make_float2(y.x, y.y), make_float2(y.z, y.w)};
  float2 a = make_float2(0.f, 0.f), b = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // (pairs side by side)
    const float2 t = __fmul2_rn(v[i], inv), h = __fadd2_rn(__fadd2_rn(t, up), down), l = __ffma2_rn(h, neg, t);
    a = __ffma2_rn(h, h, a);
    b = __ffma2_rn(__fadd2_rn(__fadd2_rn(h, h), l), l, b);
  }
  return make_float2(__fadd_rn(a.x, a.y), __fadd_rn(b.x, b.y));
}
// 1 / (q sqrt(S / dim + eps / q^2)), S = s.x + s.y.
__device__ __forceinline__ float inverse_rms(float2 s, uint32_t top, Unit u, float dim, float eps) {
  const float w = eps * u.inv * u.inv, p = __fmul_rn(dim, w), p_lo = __fmaf_rn(dim, w, -p);
  // M = S + dim eps / q^2 as hi + lo (Knuth's two-sum of s.x and p; s.y is small beside the first)
  const float c = __fadd_rn(s.x, p), v = __fsub_rn(c, s.x);
  const float c_lo = __fadd_rn(__fsub_rn(s.x, __fsub_rn(c, v)), __fsub_rn(p, v));
  const float hi = __fadd_rn(c, s.y), z = __fsub_rn(hi, c);
  const float lo = __fadd_rn(__fadd_rn(__fadd_rn(__fsub_rn(c, __fsub_rn(hi, z)), __fsub_rn(s.y, z)), c_lo), p_lo);
  const float y = rsqrtf(__fdividef(hi, dim));
  // the residual dim - y^2 M
  const float a = __fmul_rn(y, y), b = __fmaf_rn(y, y, -a);
  const float d = __fmul_rn(a, hi), d_lo = __fmaf_rn(a, hi, -d);
  const float e = __fsub_rn(__fsub_rn(__fsub_rn(dim, d), d_lo), __fmaf_rn(a, lo, __fmul_rn(b, hi)));
  const float r = __fmaf_rn(y, __fmul_rn(e, __fdividef(0.5f, dim)), y);
  return top < 0x7f800000u ? r * u.inv : top == 0x7f800000u ? 0.f : __uint_as_float(0x7fffffffu);
}

// How a cache's rows are stored.
enum Store : int { kStore16, kStoreQ8, kStoreQ4 };

// per_pass: heads that the block's threads take at once; passes: the rounds of a token, of which NP
// are loaded at a time; gridDim.y blocks share them.  A token's first loads need nothing but its
// number, its positions and slot were read with the token before, so one latency covers a token.
// D: the heads' size, with their norms; 0: no norms, any size.
template <int STORE, int D, int NP, int IO>
__global__ void __launch_bounds__(kThreads, D ? kNormBlocks : 4)
rope_store_kernel(const __grid_constant__ RopeArgs a, int per_pass, int passes) {
  constexpr bool NORM = D > 0;
  constexpr bool Q8 = STORE == kStoreQ8, Q4 = STORE == kStoreQ4, QUANT = Q8 || Q4;
  __shared__ uint32_t amax[QUANT ? NP : 1][kThreads];  // [round][head of the round][32-element block]
  __shared__ uint32_t numbers[Q4 ? NP : 1][Q4 ? 2 * kThreads : 1];  // [round][head of the round][dim], a byte each
  // what four threads have, where a head's threads are no power of two
  __shared__ uint32_t quad_top[NORM ? NP : 1][NORM ? kThreads / 4 : 1];
  __shared__ float2 quad_sum[NORM ? NP : 1][NORM ? kThreads / 4 : 1];
  const int dim = NORM ? D : a.c.dim, units = dim / 8, hkv = a.c.hkv, heads = a.hq + 2 * hkv, nb = dim / 32;
  const int u = threadIdx.x % units, sub = threadIdx.x / units;
  const int half = a.rope.rot_dim / 2;
  const bool turns = 4 * u < half;
  const bool apart = turns && !a.rope.pairs;
  const int d0 = apart ? 4 * u : 8 * u, d1 = apart ? half + 4 * u : 8 * u + 4;
  const uint32_t axes = turns && a.rope.n_axes > 1 ? *reinterpret_cast<const uint32_t *>(a.rope.axis + 4 * u) : 0;
  grid_dependency();

  // this thread's places: the element offset of its first group in a row of qkv (and of q), its
  // kv head's rows from the token's first, by round of a group
  using E = typename std::conditional<IO == MQ_F32, float, uint16_t>::type;
  const int gap = d1 - d0;
  auto head_of = [&](int pass) { return sub < per_pass ? pass * per_pass + sub : heads; };

  float4 x[NP], y[NP];
  auto load = [&](const E *row, int pass0) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int head = head_of(pass0 + k);
      x[k] = y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (head < heads) {
        const E *const from = row + (head * dim + d0);
        x[k] = load_io4(from, IO, 0);
        y[k] = load_io4(from + gap, IO, 0);
      }
    }
  };
  int next_pos[4] = {};
  int64_t next_slot = -1;
  auto look_up = [&](int64_t t) {
    next_pos[0] = a.pos[t];
    if (a.rope.n_axes > 1) {
#pragma unroll
      for (int ax = 1; ax < 4; ++ax)
        if (ax < a.rope.n_axes) next_pos[ax] = a.pos[ax * a.T + t];
    }
    next_slot = a.slot[t];
  };
  const uint32_t max_pos = (uint32_t)a.rope.max_pos;  // (<= 2^31)
  look_up(blockIdx.x);

  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const E *const row = static_cast<const E *>(a.qkv) + t * a.ld;
    load(row, blockIdx.y * NP);
    bool known = true;  // every position of the token lies in the table
#pragma unroll
    for (int ax = 0; ax < 4; ++ax)
      if ((uint32_t)next_pos[ax] >= max_pos) {
        known = false;
        if (blockIdx.y == 0 && threadIdx.x == 0) index_error(a.status, kIdxPosition, next_pos[ax]);
      }
    float2 cs[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) cs[k] = make_float2(1.f, 0.f);
    if (turns && known) {
      const float2 *const table = reinterpret_cast<const float2 *>(a.rope.table) + 4 * u;
      if (a.rope.n_axes == 1) {
        const float4 *const from = reinterpret_cast<const float4 *>(table + (uint64_t)(uint32_t)next_pos[0] * half);
        const float4 v = from[0], w = from[1];
        cs[0] = make_float2(v.x, v.y), cs[1] = make_float2(v.z, v.w);
        cs[2] = make_float2(w.x, w.y), cs[3] = make_float2(w.z, w.w);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t ax = axes >> 8 * k & 3;
          const int p = ax & 2 ? (ax & 1 ? next_pos[3] : next_pos[2]) : (ax & 1 ? next_pos[1] : next_pos[0]);
          cs[k] = table[(uint64_t)(uint32_t)p * half + k];
        }
      }
    }
    const int64_t slot = next_slot;
    bool stores = known && slot >= 0;
    uint32_t row0 = 0;  // the row of kv head 0 (the cache spans less than 2^32 rows)
    if (stores) {
      const int64_t page = slot < (int64_t(1) << 31) ? quotient((uint32_t)slot, a.c.page) : slot / a.c.page.d;
      stores = page < a.c.n_pages;
      if (stores)
        row0 = (uint32_t)page * (uint32_t)a.c.page_stride +
               (uint32_t)(slot - page * a.c.page.d) * (uint32_t)a.c.slot_stride;
      else if (blockIdx.y == 0 && threadIdx.x == 0)
        index_error(a.status, kIdxSlot, slot);
    }
    if (t + gridDim.x < a.T) look_up(t + gridDim.x);
    E *const q = static_cast<E *>(a.q) + t * (a.hq * dim);

    for (int pass0 = blockIdx.y * NP; pass0 < passes; pass0 += gridDim.y * NP) {
      if (pass0 != blockIdx.y * NP) load(row, pass0);
      if constexpr (NORM) {
        // bias, then the norm of the rounds' query and key heads
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const int head = head_of(pass0 + k);
          if (a.bias && head < heads) {
            x[k] = add4(x[k], *reinterpret_cast<const float4 *>(a.bias + head * dim + d0));
            y[k] = add4(y[k], *reinterpret_cast<const float4 *>(a.bias + head * dim + d0 + gap));
          }
        }
        auto apply = [&](int k, uint32_t top, Unit unit, float2 sum) {
          const int head = head_of(pass0 + k);
          if (head >= a.hq + hkv) return;
          const float by = inverse_rms(sum, top, unit, (float)dim, a.eps);
          const float *const w = (head < a.hq ? a.norm_q : a.norm_k) + d0;
          x[k] = normed4(x[k], by, *reinterpret_cast<const float4 *>(w));
          y[k] = normed4(y[k], by, *reinterpret_cast<const float4 *>(w + gap));
        };
        const int least = ((int)(__float_as_uint(a.eps) >> 23) - 127) / 2 + 127 - 30;
        constexpr int W = D / 8;  // threads of a head
        if constexpr ((W & (W - 1)) == 0) {
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            uint32_t top = __float_as_uint(max_nan(magnitude4(x[k]), magnitude4(y[k])));
#pragma unroll
            for (int i = 1; i < W; i <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, i));
            const Unit unit = unit_of(top, least);
            float2 sum = squares(x[k], y[k], unit);
#pragma unroll
            for (int i = 1; i < W; i <<= 1) {
              sum.x += __shfl_xor_sync(0xffffffffu, sum.x, i);
              sum.y += __shfl_xor_sync(0xffffffffu, sum.y, i);
            }
            apply(k, top, unit, sum);
          }
        } else {  // heads of 96 and 192: their threads' fours meet in shared memory
          const int first = min(sub, per_pass - 1) * (W / 4);
          uint32_t top[NP];
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            top[k] = __float_as_uint(max_nan(magnitude4(x[k]), magnitude4(y[k])));
            for (int i = 1; i < 4; i <<= 1) top[k] = max(top[k], __shfl_xor_sync(0xffffffffu, top[k], i));
            if (threadIdx.x % 4 == 0) quad_top[NORM ? k : 0][threadIdx.x / 4] = top[k];
          }
          __syncthreads();
          Unit unit[NP];
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            for (int i = 0; i < W / 4; ++i) top[k] = max(top[k], quad_top[NORM ? k : 0][first + i]);
            unit[k] = unit_of(top[k], least);
            float2 sum = squares(x[k], y[k], unit[k]);
#pragma unroll
            for (int i = 1; i < 4; i <<= 1) {
              sum.x += __shfl_xor_sync(0xffffffffu, sum.x, i);
              sum.y += __shfl_xor_sync(0xffffffffu, sum.y, i);
            }
            if (threadIdx.x % 4 == 0) quad_sum[NORM ? k : 0][threadIdx.x / 4] = sum;
          }
          __syncthreads();
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            float2 sum = make_float2(0.f, 0.f);
            for (int i = 0; i < W / 4; ++i) {
              const float2 v = quad_sum[NORM ? k : 0][first + i];
              sum.x += v.x, sum.y += v.y;
            }
            apply(k, top[k], unit[k], sum);
          }
        }
      }
      const bool quantises = QUANT && (pass0 + NP) * per_pass > a.hq;  // (the same for the whole block)
      if (quantises) {
#pragma unroll
        for (int k = 0; k < NP; ++k) amax[QUANT ? k : 0][threadIdx.x] = 0;
        __syncthreads();
      }
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int head = head_of(pass0 + k);
        if (head >= heads) continue;
        const int at = head * dim + d0;
        if (!NORM && a.bias) {
          x[k] = add4(x[k], *reinterpret_cast<const float4 *>(a.bias + at));
          y[k] = add4(y[k], *reinterpret_cast<const float4 *>(a.bias + at + gap));
        }
        if (turns && head < a.hq + hkv) {
          if (apart) {
            turn(x[k].x, y[k].x, cs[0]), turn(x[k].y, y[k].y, cs[1]);
            turn(x[k].z, y[k].z, cs[2]), turn(x[k].w, y[k].w, cs[3]);
          } else {
            turn(x[k].x, x[k].y, cs[0]), turn(x[k].z, x[k].w, cs[1]);
            turn(y[k].x, y[k].y, cs[2]), turn(y[k].z, y[k].w, cs[3]);
          }
        }
        if (head < a.hq) {
          if (!known) x[k] = y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          store_io4(q + at, IO, 0, x[k]);
          store_io4(q + at + gap, IO, 0, y[k]);
          continue;
        }
        if (!stores) continue;
        const bool key = head < a.hq + hkv;
        const uint32_t r = row0 + (uint32_t)(key ? head - a.hq : head - a.hq - hkv) * (uint32_t)a.c.head_stride;
        if (key && a.c.sums && u == 0) a.c.sums[r] = 0.f;
        if (Q8) {
          atomicMax(&amax[Q8 ? k : 0][sub * nb + d0 / 32], top4(x[k]));
          atomicMax(&amax[Q8 ? k : 0][sub * nb + d1 / 32], top4(y[k]));
        } else if (Q4) {
          atomicMax(&amax[QUANT ? k : 0][sub * nb + d0 / 32], signed_top4(x[k]));
          atomicMax(&amax[QUANT ? k : 0][sub * nb + d1 / 32], signed_top4(y[k]));
        } else {
          uint16_t *const to = reinterpret_cast<uint16_t *>(key ? a.c.k : a.c.v) + ((uint64_t)r * dim + d0);
          *reinterpret_cast<uint2 *>(to) = pack4(x[k], a.c.type == MQ_BF16);
          *reinterpret_cast<uint2 *>(to + gap) = pack4(y[k], a.c.type == MQ_BF16);
        }
      }
      if (!quantises) continue;
      __syncthreads();
      if constexpr (Q4) {  // the numbers meet in shared memory: a byte of a row has two, 16 dims apart
        auto wanted = [&](int head) { return head < heads && head >= a.hq && stores; };
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          if (!wanted(head_of(pass0 + k))) continue;
          const uint32_t *const top = &amax[QUANT ? k : 0][sub * nb];
          numbers[k][(sub * dim + d0) / 4] = numbers4(x[k], __half2float(block_scale4(top[d0 / 32])));
          numbers[k][(sub * dim + d1) / 4] = numbers4(y[k], __half2float(block_scale4(top[d1 / 32])));
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const int head = head_of(pass0 + k);
          if (!wanted(head)) continue;
          const bool key = head < a.hq + hkv;
          const uint32_t r = row0 + (uint32_t)(key ? head - a.hq : head - a.hq - hkv) * (uint32_t)a.c.head_stride;
          // thread u: bytes 4u .. 4u + 3 of the row, block u / 4
          const uint32_t *const from = &numbers[k][sub * (dim / 4) + u / 4 * 8 + u % 4];
          *reinterpret_cast<uint32_t *>((key ? a.c.k : a.c.v) + ((uint64_t)r * (dim / 2) + 4 * u)) =
              from[0] | from[4] << 4;
          if (u < nb)
            ((key ? a.c.ks : a.c.vs) + (uint64_t)r * nb)[u] = block_scale4(amax[QUANT ? k : 0][sub * nb + u]);
        }
        __syncthreads();
        continue;
      }
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int head = head_of(pass0 + k);
        if (head >= heads || head < a.hq || !stores) continue;
        const bool key = head < a.hq + hkv;
        const uint32_t r = row0 + (uint32_t)(key ? head - a.hq : head - a.hq - hkv) * (uint32_t)a.c.head_stride;
        const __half s0 = block_scale(amax[Q8 ? k : 0][sub * nb + d0 / 32]);
        const __half s1 = block_scale(amax[Q8 ? k : 0][sub * nb + d1 / 32]);
        uint8_t *const to = (key ? a.c.k : a.c.v) + ((uint64_t)r * dim + d0);
        *reinterpret_cast<uint32_t *>(to) = quants4(x[k], __half2float(s0));
        *reinterpret_cast<uint32_t *>(to + gap) = quants4(y[k], __half2float(s1));
        // the thread that holds a block's first dims writes its scale
        __half *const scale = (key ? a.c.ks : a.c.vs) + (uint64_t)r * nb;
        if (d0 % 32 == 0) scale[d0 / 32] = s0;
        if (d1 % 32 == 0) scale[d1 / 32] = s1;
      }
      __syncthreads();
    }
  }
}

// (IO is a template argument so that the loads of a group stand together, without a branch on the
// type at each)
template <int STORE, int D, int NP>
mq_status launch_io(const RopeArgs &a, dim3 grid, dim3 block, int per_pass, int passes, cudaStream_t s) {
  auto *kernel = a.io == MQ_F32   ? rope_store_kernel<STORE, D, NP, MQ_F32>
                 : a.io == MQ_F16 ? rope_store_kernel<STORE, D, NP, MQ_F16>
                                  : rope_store_kernel<STORE, D, NP, MQ_BF16>;
  return launch_dependent("rope_store_kernel", kernel, grid, block, 0, s, a, per_pass, passes);
}
template <int STORE>
mq_status launch_store(const RopeArgs &a, int np, dim3 grid, dim3 block, int per_pass, int passes, cudaStream_t s) {
  if (a.norm_q) switch (a.c.dim) {
      case 64: return launch_io<STORE, 64, 1>(a, grid, block, per_pass, passes, s);
      case 96: return launch_io<STORE, 96, 1>(a, grid, block, per_pass, passes, s);
      case 128: return launch_io<STORE, 128, 1>(a, grid, block, per_pass, passes, s);
      case 192: return launch_io<STORE, 192, 1>(a, grid, block, per_pass, passes, s);
      default: return launch_io<STORE, 256, 1>(a, grid, block, per_pass, passes, s);
    }
  switch (np) {
    case 1: return launch_io<STORE, 0, 1>(a, grid, block, per_pass, passes, s);
    case 2: return launch_io<STORE, 0, 2>(a, grid, block, per_pass, passes, s);
    default: return launch_io<STORE, 0, 3>(a, grid, block, per_pass, passes, s);
  }
}

}  // namespace

mq_status launch_rope_store(const RopeArgs &a, cudaStream_t s, const DeviceState *st) {
  const int units = a.c.dim / 8, heads = a.hq + 2 * a.c.hkv;
  const int most = kThreads / units;
  const int passes = (heads + most - 1) / most, per_pass = (heads + passes - 1) / passes;
  const unsigned threads = (per_pass * units + 31) / 32 * 32;
  // fewer tokens than fill the SMs: the rounds go to blocks of their own
  const bool split = a.T * passes <= 8 * st->sms;
  const int np = split ? 1 : std::min(passes, 3);
  // blocks of up to 256 threads with 64 registers (48 with norms): as many as are resident at once
  const int registers = a.norm_q ? 65536 / (kThreads * kNormBlocks) / 8 * 8 : 64;
  const int64_t resident =
      int64_t(st->sms) * std::max(1, std::min(2048 / (int)threads, 65536 / (registers * (int)threads)));
  const dim3 grid((unsigned)std::min(a.T, resident), split ? passes : 1, 1), block(threads, 1, 1);
  switch (a.c.type) {
    case MQ_Q8_0: return launch_store<kStoreQ8>(a, np, grid, block, per_pass, passes, s);
    case MQ_Q4_0: return launch_store<kStoreQ4>(a, np, grid, block, per_pass, passes, s);
    default: return launch_store<kStore16>(a, np, grid, block, per_pass, passes, s);
  }
}

}  // namespace mq
