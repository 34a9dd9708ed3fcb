// attn_decode_q4.cu -- mq_attn_decode's kernels over Q4_0 rows (attn_decode.cuh), by the activations' type, which
// says in how many parts the operands are.
#include "attn_decode.cuh"

namespace mq {
using namespace attn;

mq_status init_attn_decode_q4(const DeviceState *st) {
  mq_status r = opt_in<MQ_Q4_0, MQ_F32>(st);
  if (r == MQ_OK) r = opt_in<MQ_Q4_0, MQ_F16>(st);
  if (r == MQ_OK) r = opt_in<MQ_Q4_0, MQ_BF16>(st);
  return r;
}

mq_status launch_attn_decode_q4(const Params &p, int rows, cudaStream_t s, const DeviceState *st) {
  switch (p.a.io) {
    case MQ_F32: return launch_dim<MQ_Q4_0, MQ_F32>(p, rows, s, st);
    case MQ_F16: return launch_dim<MQ_Q4_0, MQ_F16>(p, rows, s, st);
    default: return launch_dim<MQ_Q4_0, MQ_BF16>(p, rows, s, st);
  }
}

}  // namespace mq
