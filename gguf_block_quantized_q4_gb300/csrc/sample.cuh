// sample.cuh -- the launcher of sample.cu.
#pragma once

#include "mq_common.cuh"

namespace mq {

struct SampleArgs {
  int io;
  const void *logits;
  int64_t ld, B, V;
  const float *u, *temperature;
  const int32_t *top_k;
  const float *top_p, *min_p;
  int32_t *token;
  float *logprob;
  bool slow_first;  // the launcher's: the order of the rows
};
mq_status launch_sample(const SampleArgs &a, cudaStream_t s, const DeviceState *st);
mq_status init_sample(DeviceState *st);  // shared-memory opt-in, cluster sizes

}  // namespace mq
