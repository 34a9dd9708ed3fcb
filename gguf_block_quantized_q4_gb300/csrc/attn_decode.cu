// attn_decode.cu -- mq_attn_decode: attention of one new token per sequence over the paged
// cache.
//
// One warp per (sequence, query head): lane l holds the dims l, l + 32, ... of the query and of
// the output; the keys are taken one after the other with the running maximum and sum of the
// softmax.  For the weight sums the logits go to the workspace, and a second kernel adds
// exp(s - m) / l of the group's heads per row.
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
__device__ __forceinline__ float load_row(const uint8_t *plane, const __half *scale, int type,
                                          int64_t r, int dim, int d) {
  if (type == MQ_F16) return __half2float(reinterpret_cast<const __half *>(plane)[r * dim + d]);
  if (type == MQ_BF16)
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(plane)[r * dim + d]);
  return __half2float(scale[r * (dim / 32) + d / 32]) *
         (float)reinterpret_cast<const int8_t *>(plane)[r * dim + d];
}

struct Stat {
  float m, l;
};

__global__ void __launch_bounds__(32) attn_decode_kernel(AttnArgs a) {
  grid_dependency();
  const int s = blockIdx.x, head = blockIdx.y, lane = threadIdx.x, dim = a.c.dim, n = dim / 32;
  const int h = head / (a.hq / a.c.hkv);
  const int raw = a.len[s], len = clamped_len(raw, a.max_len);
  if (raw != len && head == 0 && lane == 0) index_error(a.status, kIdxAttnLen, raw);
  const int lo = a.window ? (int)max((int64_t)0, len - a.window) : 0;
  const int64_t at = (int64_t(s) * a.hq + head) * dim;
  float *logit = reinterpret_cast<float *>(a.ws) + (int64_t(s) * a.hq + head) * a.max_len;
  float q[8], o[8];
  for (int i = 0; i < n; ++i) q[i] = load_io(a.q, a.io, at + lane + 32 * i) * a.scale, o[i] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int j = lo; j < len; ++j) {
    const int64_t r = kv_row(a.c, a.pages + s * a.pages_ld, h, j);
    if (r < 0) {
      if (lane == 0) index_error(a.status, kIdxAttnPage, a.pages[s * a.pages_ld + j / a.c.page.d]);
      if (a.track && lane == 0) logit[j] = -INFINITY;
      continue;
    }
    float x = 0.f;
    for (int i = 0; i < n; ++i) x += q[i] * load_row(a.c.k, a.c.ks, a.c.type, r, dim, lane + 32 * i);
    for (int k = 16; k; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
    const float mn = fmaxf(m, x), p = expf(x - mn), al = expf(m - mn);
    l = l * al + p;
    m = mn;
    for (int i = 0; i < n; ++i)
      o[i] = o[i] * al + p * load_row(a.c.v, a.c.vs, a.c.type, r, dim, lane + 32 * i);
    if (a.track && lane == 0) logit[j] = x;
  }
  for (int i = 0; i < n; ++i) store_io(a.o, a.io, at + lane + 32 * i, l > 0.f ? o[i] / l : 0.f);
  if (a.track && lane == 0) {
    Stat *st = reinterpret_cast<Stat *>(reinterpret_cast<float *>(a.ws) + a.S * a.hq * a.max_len);
    st[int64_t(s) * a.hq + head] = {m, l};
  }
}

__global__ void __launch_bounds__(256) attn_track_kernel(AttnArgs a) {
  grid_dependency();
  const int s = blockIdx.x, h = blockIdx.y, group = a.hq / a.c.hkv;
  const int len = clamped_len(a.len[s], a.max_len);
  const int lo = a.window ? (int)max((int64_t)0, len - a.window) : 0;
  const Stat *st = reinterpret_cast<const Stat *>(reinterpret_cast<float *>(a.ws) + a.S * a.hq * a.max_len);
  for (int j = lo + threadIdx.x; j < len; j += blockDim.x) {
    const int64_t r = kv_row(a.c, a.pages + s * a.pages_ld, h, j);
    if (r < 0) continue;
    float w = 0.f;
    for (int g = 0; g < group; ++g) {
      const int64_t sh = int64_t(s) * a.hq + h * group + g;
      const float x = reinterpret_cast<const float *>(a.ws)[sh * a.max_len + j];
      w += expf(x - st[sh].m) / st[sh].l;
    }
    a.c.sums[r] += w;
  }
}

}  // namespace

size_t attn_ws_bytes(int64_t S, int hq, int, int, int64_t max_len, bool track,
                     const DeviceState *) {
  return 256 + (track ? align256(size_t(S) * hq * (size_t(max_len) * 4 + sizeof(Stat))) : 0);
}

mq_status launch_attn_decode(const AttnArgs &a, cudaStream_t s, const DeviceState *) {
  mq_status r = launch_dependent("attn_decode_kernel", attn_decode_kernel,
                                 dim3((unsigned)a.S, a.hq, 1), dim3(32, 1, 1), 0, s, a);
  if (r == MQ_OK && a.track)
    r = launch_dependent("attn_track_kernel", attn_track_kernel,
                         dim3((unsigned)a.S, a.c.hkv, 1), dim3(256, 1, 1), 0, s, a);
  return r;
}

}  // namespace mq
