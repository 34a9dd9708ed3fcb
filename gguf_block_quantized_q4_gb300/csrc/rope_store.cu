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
// every access is 8 or 16 bytes wide.  A thread block takes a token, its threads as many heads
// at a time as divide the heads evenly; few tokens are spread over more blocks, a round of heads
// each.  Q8_0 rows: the largest magnitude of a 32-element block meets in shared memory as an
// integer maximum (the halves of a partial rotation may end inside a block, so no fixed lanes
// share one), then the quants as in quant_row.cuh.
#include <algorithm>

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

// per_pass: heads that the block's threads take at once; passes: their rounds; gridDim.y blocks
// share the rounds of a token.
template <bool Q8>
__global__ void __launch_bounds__(kThreads) rope_store_kernel(const __grid_constant__ RopeArgs a,
                                                              int per_pass, int passes) {
  __shared__ uint32_t amax[kThreads];  // [head of the round][32-element block]
  grid_dependency();
  const int64_t t = blockIdx.x;
  const int dim = a.c.dim, units = dim / 8, hkv = a.c.hkv, heads = a.hq + 2 * hkv;
  const int u = threadIdx.x % units, sub = threadIdx.x / units;
  const int half = a.rope.rot_dim / 2;
  const bool turns = 4 * u < half;
  const bool apart = turns && !a.rope.pairs;
  const int d0 = apart ? 4 * u : 8 * u, d1 = apart ? half + 4 * u : 8 * u + 4;

  bool known = true;  // every position of the token lies in the table
  for (int ax = 0; ax < a.rope.n_axes; ++ax) {
    const int p = a.pos[ax * a.T + t];
    if (p < 0 || p >= a.rope.max_pos) {
      known = false;
      if (blockIdx.y == 0 && threadIdx.x == 0) index_error(a.status, kIdxPosition, p);
    }
  }
  float2 cs[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    cs[k] = make_float2(1.f, 0.f);
    if (turns && known) {
      const int64_t p = a.pos[a.rope.axis[4 * u + k] * a.T + t];
      cs[k] = reinterpret_cast<const float2 *>(a.rope.table)[p * half + 4 * u + k];
    }
  }
  int64_t slot = a.slot[t], row0 = -1;  // the row of kv head 0, or -1: nothing is stored
  if (known && slot >= 0) {
    const int64_t page = slot / a.c.page.d;
    if (page < a.c.n_pages)
      row0 = page * a.c.page_stride + (slot - page * a.c.page.d) * a.c.slot_stride;
    else if (blockIdx.y == 0 && threadIdx.x == 0)
      index_error(a.status, kIdxSlot, slot);
  }

  for (int pass = blockIdx.y; pass < passes; pass += gridDim.y) {
    const int head = pass * per_pass + sub;
    const bool on = sub < per_pass && head < heads;
    const int64_t col = int64_t(head) * dim;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    if (on) {
      x = load_io4(a.qkv, a.io, t * a.ld + col + d0);
      y = load_io4(a.qkv, a.io, t * a.ld + col + d1);
      if (a.bias) {
        x = add4(x, *reinterpret_cast<const float4 *>(a.bias + col + d0));
        y = add4(y, *reinterpret_cast<const float4 *>(a.bias + col + d1));
      }
      if (turns && head < a.hq + hkv) {
        if (apart) {
          turn(x.x, y.x, cs[0]), turn(x.y, y.y, cs[1]), turn(x.z, y.z, cs[2]), turn(x.w, y.w, cs[3]);
        } else {
          turn(x.x, x.y, cs[0]), turn(x.z, x.w, cs[1]), turn(y.x, y.y, cs[2]), turn(y.z, y.w, cs[3]);
        }
      }
    }
    if (on && head < a.hq) {
      if (!known) x = y = make_float4(0.f, 0.f, 0.f, 0.f);
      store_io4(a.q, a.io, t * a.hq * dim + col + d0, x);
      store_io4(a.q, a.io, t * a.hq * dim + col + d1, y);
    }
    // keys and values
    const bool stores = on && head >= a.hq && row0 >= 0;
    const bool key = head < a.hq + hkv;
    const int64_t r = row0 + (key ? head - a.hq : head - a.hq - hkv) * a.c.head_stride;
    uint8_t *const plane = key ? a.c.k : a.c.v;
    if (stores && key && a.c.sums && u == 0) a.c.sums[r] = 0.f;
    if (!Q8) {
      if (stores) {
        *reinterpret_cast<uint2 *>(plane + (r * dim + d0) * 2) = pack4(x, a.c.type == MQ_BF16);
        *reinterpret_cast<uint2 *>(plane + (r * dim + d1) * 2) = pack4(y, a.c.type == MQ_BF16);
      }
    } else if ((pass + 1) * per_pass > a.hq) {  // (the same for the whole block)
      const int nb = dim / 32;
      amax[threadIdx.x] = 0;
      __syncthreads();
      if (stores) {
        atomicMax(&amax[sub * nb + d0 / 32], top4(x));
        atomicMax(&amax[sub * nb + d1 / 32], top4(y));
      }
      __syncthreads();
      if (stores) {
        const __half s0 = block_scale(amax[sub * nb + d0 / 32]);
        const __half s1 = d1 / 32 == d0 / 32 ? s0 : block_scale(amax[sub * nb + d1 / 32]);
        *reinterpret_cast<uint32_t *>(plane + r * dim + d0) = quants4(x, __half2float(s0));
        *reinterpret_cast<uint32_t *>(plane + r * dim + d1) = quants4(y, __half2float(s1));
        // the thread that holds a block's first dims writes its scale
        __half *const scale = (key ? a.c.ks : a.c.vs) + r * nb;
        if (d0 % 32 == 0) scale[d0 / 32] = s0;
        if (d1 % 32 == 0) scale[d1 / 32] = s1;
      }
      __syncthreads();
    }
  }
}

}  // namespace

mq_status launch_rope_store(const RopeArgs &a, cudaStream_t s, const DeviceState *st) {
  const int units = a.c.dim / 8, heads = a.hq + 2 * a.c.hkv;
  const int most = kThreads / units;
  const int passes = (heads + most - 1) / most, per_pass = (heads + passes - 1) / passes;
  const unsigned threads = (per_pass * units + 31) / 32 * 32;
  // fewer tokens than fill the SMs: the rounds go to blocks of their own
  const unsigned split = a.T * passes <= 8 * st->sms ? passes : 1;
  const dim3 grid((unsigned)a.T, split, 1), block(threads, 1, 1);
  return a.c.type == MQ_Q8_0
             ? launch_dependent("rope_store_kernel", rope_store_kernel<true>, grid, block, 0, s, a,
                                per_pass, passes)
             : launch_dependent("rope_store_kernel", rope_store_kernel<false>, grid, block, 0, s, a,
                                per_pass, passes);
}

}  // namespace mq
