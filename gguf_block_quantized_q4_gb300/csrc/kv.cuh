// kv.cuh -- the paged key-value cache as the kernels see it: row addressing, the checks of
// indexes that only the device knows, and the launchers of rope_store.cu, attn_decode.cu and
// kv_evict.cu.
#pragma once

#include <cuda_bf16.h>

#include "mq_common.cuh"

namespace mq {

// What an index error names (status word kStatusIndexWord).
enum IndexError : int {
  kIdxNone = 0,
  kIdxPosition = 1,  // mq_rope_store: a token's position
  kIdxSlot = 2,      // mq_rope_store: a token's slot
  kIdxAttnLen = 3,   // mq_attn_decode: a sequence's length
  kIdxAttnPage = 4,  // mq_attn_decode: a page
  kIdxEvictLen = 5,  // mq_kv_evict: a sequence's length
  kIdxEvictPage = 6  // mq_kv_evict: an old or new page
};
inline const char *index_error_name(int code) {
  switch (code) {
    case kIdxPosition: return "mq_rope_store: position";
    case kIdxSlot: return "mq_rope_store: slot";
    case kIdxAttnLen: return "mq_attn_decode: length";
    case kIdxAttnPage: return "mq_attn_decode: page";
    case kIdxEvictLen: return "mq_kv_evict: length";
    case kIdxEvictPage: return "mq_kv_evict: page";
    default: return "index";
  }
}

// Quotients by a page size: n / d = (umulhi(n, mul) + n) >> shift for 0 <= n < 2^31, with
// shift = ceil(log2 d) and mul = floor(2^32 (2^shift - d) / d) + 1 (division by an invariant
// through a rounded-up reciprocal, Granlund and Montgomery 1994).
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  while ((uint64_t(1) << f.shift) < d) ++f.shift;
  f.mul = uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << f.shift) - d)) / d + 1);
  return f;
}
__device__ __forceinline__ uint32_t quotient(uint32_t n, const FastDiv &f) {
  return (__umulhi(n, f.mul) + n) >> f.shift;
}

// The cache, by value in the kernels' parameters.
struct KvView {
  uint8_t *k, *v;
  __half *ks, *vs;  // scales of Q8_0 and Q4_0
  float *sums;
  int64_t n_pages, page_stride, head_stride, slot_stride;  // strides in rows
  int type, hkv, dim;
  FastDiv page;  // page size
};
// Whether rows have scales (in planes of their own).
inline bool kv_scaled(int type) { return type == MQ_Q8_0 || type == MQ_Q4_0; }

// The first error's thread alone writes the value.  (By a store: an atomic exchange here, on a path
// that no valid call takes, cost mq_rope_store 5 us of 64 at 16384 bf16 tokens, out of line 4.)
__device__ __forceinline__ void index_error(int *status, int code, int64_t value) {
  if (atomicCAS(status + kStatusIndexWord, 0, code) == 0)
    *reinterpret_cast<int64_t *>(status + kStatusIndexWord + 2) = value;
}

// A sequence's length, clamped to [0, max_len].
__device__ __forceinline__ int clamped_len(int len, int max_len) {
  return min(max(len, 0), max_len);
}

// The row of (head, position), kNoRow where its page lies outside the cache.  In 32 bits: a cache
// spans at most 2^32 - 2 rows.
constexpr uint32_t kNoRow = 0xffffffffu;
__device__ __forceinline__ uint32_t kv_row32(const KvView &c, const int32_t *pages, int head, int pos) {
  const uint32_t pi = quotient((uint32_t)pos, c.page);
  const int page = pages[pi];
  const uint32_t row = (uint32_t)page * (uint32_t)c.page_stride + (uint32_t)head * (uint32_t)c.head_stride +
                       ((uint32_t)pos - pi * c.page.d) * (uint32_t)c.slot_stride;
  return (uint32_t)page < (uint32_t)c.n_pages ? row : kNoRow;
}

// Kernels are launched with programmatic stream serialisation: they may become resident while
// the previous kernel of the stream runs, and wait for it before their first global access (the
// weight sums' kernel of a call: before its first access to what the attention writes).
__device__ __forceinline__ void grid_dependency() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// cluster: thread blocks of a cluster, along x (grid.x a multiple of it).
template <class... P, class... A>
mq_status launch_cluster(const char *name, void (*kernel)(P...), dim3 grid, dim3 block,
                         size_t smem, cudaStream_t s, unsigned cluster, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = test_fail_launch() ? dim3(0, 1, 1) : grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(MQ_ERR_LAUNCH, "launch of %s (grid %u x %u x %u, %u threads) failed: %s", name,
                grid.x, grid.y, grid.z, block.x, cudaGetErrorName(e));
  }
  return MQ_OK;
}

template <class... P, class... A>
mq_status launch_dependent(const char *name, void (*kernel)(P...), dim3 grid, dim3 block,
                           size_t smem, cudaStream_t s, A... args) {
  return launch_cluster(name, kernel, grid, block, smem, s, 1, args...);
}

// Four elements of an activation row of type io (MQ_F32, MQ_F16, MQ_BF16), as binary32.
__device__ __forceinline__ float4 load_io4(const void *p, int io, int64_t i) {
  if (io == MQ_F32) return *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
  const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
  if (io == MQ_BF16)
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&v.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&v.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float load_io1(const void *p, int io, int64_t i) {
  if (io == MQ_F32) return static_cast<const float *>(p)[i];
  const uint16_t v = static_cast<const uint16_t *>(p)[i];
  return io == MQ_BF16 ? __uint_as_float(uint32_t(v) << 16) : __half2float(__ushort_as_half(v));
}
__device__ __forceinline__ uint2 pack4(float4 v, bool bf16) {  // rounded to nearest even
  uint2 u;
  if (bf16) {
    *reinterpret_cast<__nv_bfloat162 *>(&u.x) = __floats2bfloat162_rn(v.x, v.y);
    *reinterpret_cast<__nv_bfloat162 *>(&u.y) = __floats2bfloat162_rn(v.z, v.w);
  } else {
    *reinterpret_cast<__half2 *>(&u.x) = __floats2half2_rn(v.x, v.y);
    *reinterpret_cast<__half2 *>(&u.y) = __floats2half2_rn(v.z, v.w);
  }
  return u;
}
__device__ __forceinline__ void store_io4(void *p, int io, int64_t i, float4 v) {
  if (io == MQ_F32)
    *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) = v;
  else
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + i) = pack4(v, io == MQ_BF16);
}

// ---- rope_store.cu ----
struct RopeArgs {
  KvView c;
  mq_rope rope;
  int io;
  const void *qkv;
  int64_t ld;
  const float *bias;
  const float *norm_q, *norm_k;  // weights of the heads' norms; null: no norms
  float eps;
  const int32_t *pos;
  const int64_t *slot;
  void *q;
  int64_t T;
  int hq;
  int *status;
};
mq_status launch_rope_store(const RopeArgs &a, cudaStream_t s, const DeviceState *st);

// ---- attn_decode.cu ----
struct AttnArgs {
  KvView c;
  int io;
  const void *q;
  void *o;
  const int32_t *pages;
  int64_t pages_ld;
  const int32_t *len;
  int64_t S;
  int hq, max_len;
  float scale;
  int64_t window;  // 0: none
  bool track;
  uint8_t *ws;
  int *status;
};
size_t attn_ws_bytes(int64_t S, int hq, int hkv, int dim, int64_t max_len, bool track,
                     const DeviceState *st);
mq_status launch_attn_decode(const AttnArgs &a, cudaStream_t s, const DeviceState *st);
mq_status init_attn_decode(const DeviceState *st);  // shared-memory opt-ins

// ---- kv_evict.cu ----
struct EvictArgs {
  KvView c;
  const int32_t *pages;
  int64_t pages_ld;
  const int32_t *len;
  int64_t S;
  int max_len;
  const int32_t *new_pages;
  int64_t new_pages_ld;
  int keep, sink, recent;
  int32_t *kept, *new_len;
  int *status;
};
mq_status launch_kv_evict(const EvictArgs &a, cudaStream_t s, const DeviceState *st);
mq_status init_kv_evict(DeviceState *st);  // shared-memory opt-in, resident clusters

}  // namespace mq
