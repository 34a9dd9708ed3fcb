// rope_store.cu -- mq_rope_store: bias, rotary positions with several axes, and the store of
// keys and values into the paged cache.
//
// Mathematics: pair i of a head turns by the angle of table[pos[axis[i]]][i] = (c, s),
//     r0 = a0 c - a1 s,   r1 = a0 s + a1 c,
// every step rounded on its own (no contraction), so that the result is defined bit for bit.
//
// What bounds it: the bytes of qkv, q and the rows stored, each moved once.  A thread keeps one
// place in the head, four pairs (two groups of four dims, 16 bytes of f32 each), for all heads
// that it visits: the cosines and sines of a token are read once and stay in registers, and
// every access is 8 or 16 bytes wide.  A thread block takes one token after another, its threads
// as many heads at a time as divide the heads evenly (a block per token pays the threads' places,
// axes and divisions for each: 652 instructions a warp, 131 us for 16384 bf16 tokens); few tokens
// are spread over more blocks, a round of heads each.  Q8_0 rows: the largest magnitude of a
// 32-element block meets in shared memory as an integer maximum (the halves of a partial rotation
// may end inside a block, so no fixed lanes share one), then the quants as in quant_row.cuh.
// Measured (28/4 heads of 128): 16384 tokens f32 to f16 98 us (5.9 TB/s, 89% of a plain copy's
// rate), to Q8_0 93 us (90%; three rounds at once spill 8 bytes a thread), bf16 to f16 64 us (72%: one
// token's loads are in flight per block, fewer bytes than cover the latency); 4096 tokens f32 to
// f16, three axes, 25.2 us (86%); 1023 tokens bf16 to Q8_0, 32/8 heads, half of a head rotated, 9.9 us
// (2.8 times its bytes' time: a block has one or two whole tokens, so the shares are uneven); 8
// tokens 2.1 us.
#include <algorithm>
#include <type_traits>

#include "kv.cuh"
#include "quant_row.cuh"

namespace mq {
namespace {

constexpr int kThreads = 256;  // at most

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y), __fadd_rn(a.z, b.z),
                     __fadd_rn(a.w, b.w));
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

// per_pass: heads that the block's threads take at once; passes: the rounds of a token, of which NP
// are loaded at a time; gridDim.y blocks share them.  A token's first loads need nothing but its
// number, its positions and slot were read with the token before, so one latency covers a token.
template <bool Q8, int NP, int IO>
__global__ void __launch_bounds__(kThreads, 4) rope_store_kernel(const __grid_constant__ RopeArgs a,
                                                              int per_pass, int passes) {
  __shared__ uint32_t amax[Q8 ? NP : 1][kThreads];  // [round][head of the round][32-element block]
  const int dim = a.c.dim, units = dim / 8, hkv = a.c.hkv, heads = a.hq + 2 * hkv, nb = dim / 32;
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
      const bool quantises = Q8 && (pass0 + NP) * per_pass > a.hq;  // (the same for the whole block)
      if (quantises) {
#pragma unroll
        for (int k = 0; k < NP; ++k) amax[Q8 ? k : 0][threadIdx.x] = 0;
        __syncthreads();
      }
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        const int head = head_of(pass0 + k);
        if (head >= heads) continue;
        const int at = head * dim + d0;
        if (a.bias) {
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
        } else {
          uint16_t *const to = reinterpret_cast<uint16_t *>(key ? a.c.k : a.c.v) + ((uint64_t)r * dim + d0);
          *reinterpret_cast<uint2 *>(to) = pack4(x[k], a.c.type == MQ_BF16);
          *reinterpret_cast<uint2 *>(to + gap) = pack4(y[k], a.c.type == MQ_BF16);
        }
      }
      if (!quantises) continue;
      __syncthreads();
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
template <bool Q8, int NP>
mq_status launch_io(const RopeArgs &a, dim3 grid, dim3 block, int per_pass, int passes, cudaStream_t s) {
  auto *kernel = a.io == MQ_F32   ? rope_store_kernel<Q8, NP, MQ_F32>
                 : a.io == MQ_F16 ? rope_store_kernel<Q8, NP, MQ_F16>
                                  : rope_store_kernel<Q8, NP, MQ_BF16>;
  return launch_dependent("rope_store_kernel", kernel, grid, block, 0, s, a, per_pass, passes);
}
template <bool Q8>
mq_status launch_rounds(const RopeArgs &a, int np, dim3 grid, dim3 block, int per_pass, int passes,
                        cudaStream_t s) {
  switch (np) {
    case 1: return launch_io<Q8, 1>(a, grid, block, per_pass, passes, s);
    case 2: return launch_io<Q8, 2>(a, grid, block, per_pass, passes, s);
    default: return launch_io<Q8, 3>(a, grid, block, per_pass, passes, s);
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
  // blocks of up to 256 threads with 64 registers: as many as are resident at once
  const int64_t resident = int64_t(st->sms) * std::max(1, std::min(2048 / (int)threads, 65536 / (64 * (int)threads)));
  const dim3 grid((unsigned)std::min(a.T, resident), split ? passes : 1, 1), block(threads, 1, 1);
  return a.c.type == MQ_Q8_0 ? launch_rounds<true>(a, np, grid, block, per_pass, passes, s)
                             : launch_rounds<false>(a, np, grid, block, per_pass, passes, s);
}

}  // namespace mq
