// rope_store.cu -- mq_rope_store: bias, rotary positions with several axes, and the store of
// keys and values into the paged cache.
//
// One CTA per (token, head), one thread per dim, so that a warp is one 32-element Q8_0 block.
// Every step is rounded on its own (no contraction), so that the stored bytes can be compared
// exactly.
#include "kv.cuh"

namespace mq {
namespace {

__device__ __forceinline__ float load_io(const void *p, int io, int64_t i) {
  if (io == MQ_F32) return static_cast<const float *>(p)[i];
  if (io == MQ_F16) return __half2float(static_cast<const __half *>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void store_io(void *p, int io, int64_t i, float v) {
  if (io == MQ_F32)
    static_cast<float *>(p)[i] = v;
  else if (io == MQ_F16)
    static_cast<__half *>(p)[i] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

__global__ void __launch_bounds__(256) rope_store_kernel(RopeArgs a) {
  __shared__ float row[256];
  grid_dependency();
  const int64_t t = blockIdx.x;
  const int head = blockIdx.y, d = threadIdx.x, dim = a.c.dim, hkv = a.c.hkv;
  const int64_t col = int64_t(head) * dim + d;
  float x = load_io(a.qkv, a.io, t * a.ld + col);
  if (a.bias) x = __fadd_rn(x, a.bias[col]);
  row[d] = x;
  __syncthreads();
  bool known = true;  // every position of the token lies in the table
  for (int ax = 0; ax < a.rope.n_axes; ++ax) {
    const int p = a.pos[ax * a.T + t];
    if (p < 0 || p >= a.rope.max_pos) {
      known = false;
      if (head == 0 && d == 0) index_error(a.status, kIdxPosition, p);
    }
  }
  const int half = a.rope.rot_dim / 2;
  if (known && head < a.hq + hkv && d < 2 * half) {
    const int i = a.rope.pairs ? d >> 1 : d % half;
    const bool second = a.rope.pairs ? d & 1 : d >= half;
    const float x0 = row[a.rope.pairs ? 2 * i : i], x1 = row[a.rope.pairs ? 2 * i + 1 : i + half];
    const int64_t p = a.pos[a.rope.axis[i] * a.T + t];
    const float c = a.rope.table[(p * half + i) * 2], s = a.rope.table[(p * half + i) * 2 + 1];
    x = second ? __fadd_rn(__fmul_rn(x0, s), __fmul_rn(x1, c))
               : __fsub_rn(__fmul_rn(x0, c), __fmul_rn(x1, s));
  }
  if (head < a.hq) {
    store_io(a.q, a.io, t * a.hq * dim + col, known ? x : 0.f);
    return;
  }
  const int64_t slot = a.slot[t];
  if (!known || slot < 0) return;
  const int64_t page = slot / a.c.page.d;
  if (page >= a.c.n_pages) {
    if (head == a.hq && d == 0) index_error(a.status, kIdxSlot, slot);
    return;
  }
  const bool key = head < a.hq + hkv;
  const int h = key ? head - a.hq : head - a.hq - hkv;
  const int64_t r = page * a.c.page_stride + h * a.c.head_stride +
                    (slot - page * a.c.page.d) * a.c.slot_stride;
  uint8_t *plane = key ? a.c.k : a.c.v;
  if (key && a.c.sums && d == 0) a.c.sums[r] = 0.f;
  if (a.c.type == MQ_F16) {
    reinterpret_cast<__half *>(plane)[r * dim + d] = __float2half_rn(x);
  } else if (a.c.type == MQ_BF16) {
    reinterpret_cast<__nv_bfloat16 *>(plane)[r * dim + d] = __float2bfloat16_rn(x);
  } else {
    float amax = fabsf(x);
    for (int m = 16; m; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
    const __half dh = __float2half_rn(fminf(__fdiv_rn(amax, 127.f), 65504.f));
    const float ds = __half2float(dh);
    const float q = ds == 0.f ? 0.f : rintf(__fdiv_rn(x, ds));
    reinterpret_cast<int8_t *>(plane)[r * dim + d] = (int8_t)fminf(fmaxf(q, -127.f), 127.f);
    if ((d & 31) == 0) (key ? a.c.ks : a.c.vs)[r * (dim / 32) + d / 32] = dh;
  }
}

}  // namespace

mq_status launch_rope_store(const RopeArgs &a, cudaStream_t s, const DeviceState *) {
  return launch_dependent("rope_store_kernel", rope_store_kernel,
                          dim3((unsigned)a.T, a.hq + 2 * a.c.hkv, 1), dim3(a.c.dim, 1, 1), 0, s, a);
}

}  // namespace mq
