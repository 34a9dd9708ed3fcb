// sample_host.cpp -- mq_sample's kernel on the host: sample.cu as it stands, but for its shared memory's
// declarations and one instruction (SAMPLE_CU is the file with those replaced).
#include "device.h"

enum { MQ_F32 = 0, MQ_F16 = 1, MQ_BF16 = 30 };
enum mq_status { MQ_OK, MQ_ERR };
using cudaStream_t = void *;
enum cudaError_t { cudaSuccess, cudaErrorInvalidConfiguration };
enum { cudaFuncAttributeMaxDynamicSharedMemorySize, cudaFuncAttributeNonPortableClusterSizeAllowed, cudaLaunchAttributeClusterDimension };
struct cudaFuncAttributes { size_t sharedSizeBytes = 0; };
struct cudaLaunchAttribute { int id; struct { dim3 clusterDim; } val; };
struct cudaLaunchConfig_t {
  dim3 gridDim, blockDim;
  size_t dynamicSmemBytes;
  cudaLaunchAttribute *attrs;
  int numAttrs;
};
template <class K> cudaError_t cudaFuncGetAttributes(cudaFuncAttributes *, K *) { return cudaSuccess; }
template <class K> cudaError_t cudaFuncSetAttribute(K *, int, int) { return cudaSuccess; }
inline const int *resident = nullptr;  // of each kernel's set-up, size by size: clusters, or -1 for one that cannot run
template <class K> cudaError_t cudaOccupancyMaxActiveClusters(int *n, K *, cudaLaunchConfig_t *) {
  *n = *resident++;
  return *n < 0 ? cudaErrorInvalidConfiguration : cudaSuccess;
}
inline cudaError_t cudaGetLastError() { return cudaSuccess; }

namespace mq {
struct DeviceState {
  int smem_optin = 227 << 10, sample_clusters[5] = {};
};
inline mq_status cuda_fail(cudaError_t, const char *, const char *) { return MQ_ERR; }
inline void grid_dependency() {}
inline float load_io1(const void *p, int io, int64_t i) {
  if (io == MQ_F32) return static_cast<const float *>(p)[i];
  const uint16_t v = static_cast<const uint16_t *>(p)[i];
  return io == MQ_BF16 ? __uint_as_float(uint32_t(v) << 16) : __half2float(v);
}
inline size_t fixed_bytes = 0;
template <class Args>
mq_status launch_cluster(const char *, void (*kernel)(Args, int), dim3 grid, dim3 block, size_t smem, cudaStream_t, int ranks,
                         const Args &a, int groups) {
  struct Call {
    void (*kernel)(Args, int);
    Args a;
    int groups;
  } call = {kernel, a, groups};
  for (unsigned y = 0; y < grid.y; ++y)
    threads::run_cluster(ranks, (int)block.x, dim3(0, y, 0), fixed_bytes, smem,
                         threads::order_of(ranks, (int)block.x, threads::which_order, threads::order_seed),
                         [](void *p) {
                           Call &c = *static_cast<Call *>(p);
                           c.kernel(c.a, c.groups);
                         },
                         &call);
  return MQ_OK;
}
}  // namespace mq

#include SAMPLE_CU

// clusters[i]: of 2^i blocks that are resident at once.
extern "C" int sample_host(int io, const void *logits, int64_t ld, int64_t B, int64_t V, const float *u, const float *temperature,
                           const int32_t *top_k, const float *top_p, const float *min_p, int32_t *token, float *logprob,
                           const int *clusters, int order, unsigned seed) {
  mq::SampleArgs a = {};
  a.io = io, a.logits = logits, a.ld = ld, a.B = B, a.V = V, a.u = u, a.temperature = temperature;
  a.top_k = top_k, a.top_p = top_p, a.min_p = min_p, a.token = token, a.logprob = logprob;
  mq::DeviceState st;
  for (int i = 0; i < 5; ++i) st.sample_clusters[i] = clusters[i];
  threads::which_order = order, threads::order_seed = seed;
  mq::fixed_bytes = sizeof(mq::Shared);
  return mq::launch_sample(a, nullptr, &st);
}

extern "C" int sample_host_init(const int *clusters, int *out) {
  mq::DeviceState st;
  resident = clusters;
  const int r = mq::init_sample(&st);
  for (int i = 0; i < 5; ++i) out[i] = st.sample_clusters[i];
  return r;
}
