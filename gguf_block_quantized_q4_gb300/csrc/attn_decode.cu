// attn_decode.cu -- mq_attn_decode: its kernels over F16, BF16 and Q8_0 rows, the weight sums' kernel, the
// workspace and the launches (the mathematics and the measurements stand in attn_decode.cuh).
#include "attn_decode.cuh"

namespace mq {
using namespace attn;
namespace {

// The weight sums: w = exp2(s - m) / l per query row, summed over the rows of the kv
// head in their order.  Bounded by latency (a few bytes a row): a thread has four keys of a kv
// head side by side, and finds their rows and reads their sums before it waits for the attention,
// which writes neither (nor the tables: what came before the attention has ended when all of its
// blocks have begun, and only then do these start).  Then the logits, four rows of a key at once,
// and each row's maximum and sum for the four keys.  It and the logits add 8 us to the 54.5 of 32
// ragged sequences of up to 4001 keys (32/8 heads of 128, f16), 2.3 to the 9 of 8 of up to 1100
// (28/4); waiting first and with a place of every kv head per thread, 10 and 6.
constexpr int kTrackThreads = 128, kTrackKeys = 4;  // keys of a thread
template <int W>  // logits at a time
__global__ void __launch_bounds__(kTrackThreads) attn_track_kernel(const __grid_constant__ Params p,
                                                                   int rows, int keys) {
  constexpr int N = kTrackKeys;
  using Logits = typename std::conditional<W == 4, float4, float2>::type;
  const AttnArgs &a = p.a;
  const int s = blockIdx.y, hkv = a.c.hkv;
  const Span sp = span_of(a, s, 1);
  const int first = sp.lo + blockIdx.x * keys, n = min(keys, sp.len - first);
  bool waiting = true;
  if (n <= 0) {
    grid_dependency();  // (so that this kernel's end is the attention's, too)
    return;
  }
  const int32_t *const pages = a.pages + s * a.pages_ld;
  const int apart = keys / N;  // a thread's keys
  for (int i = threadIdx.x; i < apart * hkv; i += kTrackThreads) {
    const int h = i / apart, j = i - h * apart;
    const int64_t unit = (int64_t(s) * hkv + h) * p.row_groups;
    const float *x = p.logits + (unit * a.max_len + first + j) * p.logit_width;
    const float2 *stats = p.stats + unit * rows;
    uint32_t r[N];
    int step[N];  // (a key that is not there: the thread's first)
    float w[N] = {}, old[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const bool on = j + k * apart < n;
      r[k] = on ? kv_row32(a.c, pages, h, first + j + k * apart) : kNoRow;
      step[k] = on ? k * apart * p.logit_width : 0;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) old[k] = r[k] == kNoRow ? 0.f : a.c.sums[r[k]];
    if (waiting) grid_dependency();
    waiting = false;
    if (j >= n) continue;
    for (int rg = 0; rg < p.row_groups; ++rg) {
      const int group = min(rows, p.group - rg * rows);
      for (int q = 0; q < group; q += W) {  // (the last ones' rows may not be there)
        __align__(16) float v[N][W];
#pragma unroll
        for (int k = 0; k < N; ++k)
          *reinterpret_cast<Logits *>(v[k]) = *reinterpret_cast<const Logits *>(x + step[k] + q);
#pragma unroll
        for (int e = 0; e < W; ++e) {
          if (q + e >= group) break;
          const float2 st = stats[q + e];
#pragma unroll
          for (int k = 0; k < N; ++k) w[k] += exp2_fast(v[k][e] - st.x) * st.y;
        }
      }
      x += a.max_len * int64_t(p.logit_width), stats += rows;
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (r[k] != kNoRow) a.c.sums[r[k]] = old[k] + w[k];
  }
}

// Query rows of a unit: 8 columns of the products, or 16 where the group fills more than 8 of
// them and the accumulators (D/8 registers per 8 columns) leave room for K and V in flight.
int rows_of(int group, int dim) { return group > 8 && dim <= 128 ? 16 : 8; }

struct Workspace {
  size_t piece_o, piece_ml, stats, logits, total;
  int logit_width, blocks;
};
Workspace workspace_of(int64_t S, int hq, int hkv, int dim, int64_t max_len, bool track,
                       const DeviceState *st) {
  const int group = hq / hkv, rows = rows_of(group, dim), grid = std::min(st->sms, kMaxParts);
  const size_t units = size_t(hkv) * ((group + rows - 1) / rows);
  Workspace w;
  w.logit_width = std::min(rows, group <= 2 ? 2 : (group + 3) & ~3);  // (whole float2 or float4)
  w.blocks = grid;
  w.piece_ml = MQ_ATTN_WS_ZERO;
  w.piece_o = align256(w.piece_ml + size_t(grid) * 4 * rows * sizeof(float2));
  w.stats = align256(w.piece_o + size_t(grid) * 4 * rows * dim * 4);
  w.logits = align256(w.stats + (track ? size_t(S) * units * rows * 8 : 0));
  w.total = align256(w.logits + (track ? size_t(S) * units * size_t(max_len) * w.logit_width * 4 : 0));
  return w;
}

}  // namespace

mq_status init_attn_decode(const DeviceState *st) {
  mq_status r = opt_in<MQ_F16, MQ_F32>(st);
  if (r == MQ_OK) r = opt_in<MQ_BF16, MQ_F32>(st);
  if (r == MQ_OK) r = opt_in<MQ_Q8_0, MQ_F32>(st);
  if (r == MQ_OK) r = init_attn_decode_q4(st);
  return r;
}

size_t attn_ws_bytes(int64_t S, int hq, int hkv, int dim, int64_t max_len, bool track,
                     const DeviceState *st) {
  return workspace_of(S, hq, hkv, dim, max_len, track, st).total;
}

mq_status launch_attn_decode(const AttnArgs &a, cudaStream_t s, const DeviceState *st) {
  const Workspace w = workspace_of(a.S, a.hq, a.c.hkv, a.c.dim, a.max_len, a.track, st);
  Params p;
  p.a = a;
  p.group = a.hq / a.c.hkv;
  const int rows = rows_of(p.group, a.c.dim);
  p.row_groups = (p.group + rows - 1) / rows;
  p.units = a.c.hkv * p.row_groups;
  p.logit_width = w.logit_width;
  p.count = reinterpret_cast<int *>(a.ws);
  p.blocks = w.blocks;
  p.piece_ml = reinterpret_cast<float2 *>(a.ws + w.piece_ml);
  p.piece_o = reinterpret_cast<float *>(a.ws + w.piece_o);
  p.stats = a.track ? reinterpret_cast<float2 *>(a.ws + w.stats) : nullptr;
  p.logits = a.track ? reinterpret_cast<float *>(a.ws + w.logits) : nullptr;
  mq_status r;
  switch (a.c.type) {
    case MQ_F16: r = launch_dim<MQ_F16, MQ_F32>(p, rows, s, st); break;
    case MQ_BF16: r = launch_dim<MQ_BF16, MQ_F32>(p, rows, s, st); break;
    case MQ_Q8_0: r = launch_dim<MQ_Q8_0, MQ_F32>(p, rows, s, st); break;
    default: r = launch_attn_decode_q4(p, rows, s, st); break;
  }
  if (r == MQ_OK && a.track) {
    const int keys = std::max(32, kTrackThreads * kTrackKeys / a.c.hkv / 32 * 32);
    r = launch_dependent("attn_track_kernel",
                         w.logit_width == 2 ? attn_track_kernel<2> : attn_track_kernel<4>,
                         dim3((a.max_len + keys - 1) / keys, (unsigned)a.S, 1),
                         dim3(kTrackThreads, 1, 1), 0, s, p, rows, keys);
  }
  return r;
}

}  // namespace mq
