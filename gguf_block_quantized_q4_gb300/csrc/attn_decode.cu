// attn_decode.cu -- mq_attn_decode: attention of one new token per sequence over the paged
// cache, split over the length and joined.
//
// Mathematics.  For the query heads of one kv head, s = q k / sqrt(D) and o = sum softmax(s) v
// are kept in the running form: per query row a maximum m, a sum l = sum exp2(s - m) and an
// unnormalised o, which pieces of the length join as
//     M = max m_i,  L = sum l_i exp2(m_i - M),  o = sum o_i exp2(m_i - M) / L.
//
// What bounds it: the bytes of K and V, each read once.  A group of query heads shares them, so
// both products are matrix products with 8 (or 16) columns: S^T = K Q^T and O^T = V^T P^T on
// mma.sync m16n8k16, the rows of K (keys) and of V^T (dims) as the 16-row operand, the query
// rows as the 8 columns.  (A tcgen05 tile has 64 or 128 rows and its operands in shared memory;
// eight columns leave it idle, and the products take a fifth of the tensor time here anyway.)
// Because a key is used by one warp only, K and V go from global memory straight into the
// operand registers: the order of the dims in a product is free, so a lane's 16 bytes of a key
// row are its operand words, and V's pairs of keys are put together by byte permutes.  No
// shared memory, no alignment of pages to tiles, and a row past the end is simply not loaded.
//
// Work: (sequence, kv head, row group) units of tiles of TK keys, laid end to end; thread block b
// of the `parts` that have work takes the tiles [b T / parts, (b + 1) T / parts) of all T.  The
// split is made on the device from the lengths, so unlike lengths load all SMs alike.  A unit
// whole in one block is written at once; the pieces of the others go to the workspace, and the
// last block of a unit to arrive joins them in the order of the blocks (a counter per unit's
// first block, back to zero afterwards), so results do not depend on the order of execution.
//
// Precision: f16 operands are multiplied exactly and summed in binary32.  q (scaled by a power
// of two per row) and the weights are carried as two f16 parts (22 bits), against bf16 keys and
// values as three bf16 parts (24 bits); Q8_0 quants are exact in f16 and bf16, the keys' scales
// multiply the 32-element block sums in binary32, the values' scales the weights.  Each tile's
// product is added to o by a binary32 fma (the tensor cores' own long sums may truncate).
#include <algorithm>

#include "kv.cuh"

namespace mq {
namespace {

constexpr int kWarps = 4;           // per thread block
constexpr int kMaxParts = 1024;     // thread blocks with work (counters in the workspace)
constexpr uint32_t kNoRow = 0xffffffffu;
constexpr float kLog2e = 1.44269504088896340736f;

// ---- device helpers ---------------------------------------------------------------------
__device__ __forceinline__ uint4 load16(const uint8_t *p, bool on) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (on)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load8(const uint8_t *p, bool on) {
  uint2 v = make_uint2(0, 0);
  if (on)
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t load4(const uint8_t *p, bool on) {
  uint32_t v = 0;
  if (on) asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
template <bool BF>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if (BF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (BF)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if (BF) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  return __half22float2(*reinterpret_cast<__half2 *>(&v));
}
// A pair as N parts whose sum is the pair: part i holds what the parts before it left.
template <bool BF, int N>
__device__ __forceinline__ void split2(float lo, float hi, uint32_t (&part)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    part[i] = pack2<BF>(lo, hi);
    const float2 b = unpack2<BF>(part[i]);
    lo -= b.x, hi -= b.y;
  }
}
// Two int8 (the bytes that SEL picks) as f16x2: 1024 + (v + 128) by bits, less 1152.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t int8_f16(uint32_t biased) {
  uint32_t u = __byte_perm(biased, 0x64646464u, SEL);
  const uint32_t c = 0x64806480u;
  __half2 r = __hsub2(*reinterpret_cast<__half2 *>(&u), *reinterpret_cast<const __half2 *>(&c));
  return *reinterpret_cast<uint32_t *>(&r);
}
// Two int8 in the low bytes of 0x43vv 0x43vv as bf16x2: (128 + low seven bits) less (128, or
// 256 where the sign bit is set).
__device__ __forceinline__ uint32_t int8_bf16(uint32_t u) {
  uint32_t a = u & 0x437f437fu, b = u & 0x43804380u;
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&a),
                             *reinterpret_cast<__nv_bfloat162 *>(&b));
  return *reinterpret_cast<uint32_t *>(&r);
}
// 4 elements of an activation row.
__device__ __forceinline__ float4 load_io4(const void *p, int io, int64_t i) {
  if (io == MQ_F32) return *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
  const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
  const float2 a = io == MQ_F16 ? unpack2<false>(v.x) : unpack2<true>(v.x);
  const float2 b = io == MQ_F16 ? unpack2<false>(v.y) : unpack2<true>(v.y);
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store_io4(void *p, int io, int64_t i, float4 v) {
  if (io == MQ_F32) {
    *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) = v;
  } else {
    const uint2 u = io == MQ_F16 ? make_uint2(pack2<false>(v.x, v.y), pack2<false>(v.z, v.w))
                                 : make_uint2(pack2<true>(v.x, v.y), pack2<true>(v.z, v.w));
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + i) = u;
  }
}

// ---- the shape of a kernel ----------------------------------------------------------------
template <int TYPE, int D, int NT>
struct Shape {
  static constexpr bool kQ8 = TYPE == MQ_Q8_0;
  static constexpr bool kBfK = TYPE == MQ_BF16;                   // operand type of K Q^T
  static constexpr bool kBfV = TYPE == MQ_BF16 || TYPE == MQ_Q8_0;  // of V^T P^T
  static constexpr int kPartsK = kBfK ? 3 : 2, kPartsV = kBfV ? 3 : 2;
  static constexpr int kRow = kQ8 ? D : 2 * D;  // bytes of a key row
  static constexpr int kNG = D / 32;            // groups of 32 dims
  // 16-key groups a warp takes at a time: about 4 KB of K (and of V) in flight per warp
  static constexpr int kMT = kRow * 16 >= 3072 ? 1 : 2;
  static constexpr int kKeys = 16 * kMT, kTK = kKeys * kWarps;
  static constexpr int kRows = 8 * NT;          // query rows of a unit
  static constexpr int kKWords = kQ8 ? 2 : 4;   // a lane's words of a key row, per group
  static constexpr int kVWords = kQ8 ? 1 : 2;
  // exp2 of a weight's exponent in the f16 parts: weights in (0, 2^15], so that the second part
  // of all but negligible weights is a normal f16
  static constexpr float kBias = kBfV ? 0.f : 15.f;
};
// thread blocks per SM that the registers are sized for
template <int TYPE, int D, int NT>
constexpr int blocks_per_sm() {
  return D * NT <= 64 ? 4 : D * NT <= 128 ? 3 : 2;
}

struct Params {
  AttnArgs a;
  int group, row_groups, units;  // query heads of a kv head; row groups of them; per sequence
  int logit_width;               // query rows per key in the logits (even)
  float scale_log2;
  int *count;                    // [kMaxParts]
  float *piece_o, *piece_ml;     // [block][2][rows][D], [block][2][rows][2]
  float *logits;                 // [S][units][max_len][logit_width], or nullptr
  float2 *stats;                 // [S][units][rows]: (m - bias, 1 / l)
};

// ---- the schedule -------------------------------------------------------------------------
struct Span {
  int lo, len;  // positions read: [lo, len)
  int tiles;
};
__device__ __forceinline__ Span span_of(const AttnArgs &a, int s, int tk) {
  Span r;
  r.len = clamped_len(a.len[s], a.max_len);
  r.lo = a.window && r.len > a.window ? r.len - (int)a.window : 0;
  r.tiles = (r.len - r.lo + tk - 1) / tk;
  return r;
}
// Tiles of all sequences (in units of one unit per sequence), and the sequence in which tile
// `at` of that order lies with its first tile; every lane of the warp gets them.
__device__ __forceinline__ int64_t all_tiles(const AttnArgs &a, int tk, int64_t *lane_first,
                                             int *lane_s, int *lane_n) {
  const int lane = threadIdx.x & 31, S = (int)a.S;
  const int per = (S + 31) / 32;
  *lane_s = min(lane * per, S);
  *lane_n = min(per, S - *lane_s);
  int64_t sum = 0;
  for (int i = 0; i < *lane_n; ++i) sum += span_of(a, *lane_s + i, tk).tiles;
  int64_t inc = sum;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, inc, k);
    if (lane >= k) inc += o;
  }
  *lane_first = inc - sum;
  return __shfl_sync(0xffffffffu, inc, 31);
}

// Where a warp's next tile lies.
struct Cursor {
  int s, unit, tile;  // sequence, (kv head, row group), tile
  Span span;
  int64_t left;       // tiles of this block from here on
};
__device__ __forceinline__ void next_tile(Cursor &c, const AttnArgs &a, int units, int tk) {
  --c.left;
  if (++c.tile < c.span.tiles) return;
  c.tile = 0;
  if (++c.unit < units) return;
  c.unit = 0;
  if (c.left <= 0) return;
  do {
    c.span = span_of(a, ++c.s, tk);
  } while (c.span.tiles == 0);
}

template <int TYPE, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, blocks_per_sm<TYPE, D, NT>())
attn_decode_kernel(const __grid_constant__ Params p) {
  using C = Shape<TYPE, D, NT>;
  constexpr int NG = C::kNG, MT = C::kMT, LDO = D + 4;
  __shared__ uint4 sq[C::kPartsK][NT][NG][32];          // query parts as operand words
  __shared__ float sfac[C::kRows];                      // per row: scale * log2 e * 2^-e
  __shared__ float sm[kWarps][C::kRows], sl[kWarps][C::kRows];
  __shared__ __align__(16) float so[kWarps][C::kRows][LDO];
  __shared__ int slast;
  const AttnArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  grid_dependency();

  // idle sequences: their outputs are zero; and the report of bad lengths
  for (int s = blockIdx.x; s < a.S; s += gridDim.x) {
    const int raw = a.len[s];
    if (raw != clamped_len(raw, a.max_len) && tid == 0) index_error(a.status, kIdxAttnLen, raw);
    if (raw <= 0)
      for (int i = tid; i < a.hq * (D / 4); i += kWarps * 32)
        store_io4(a.o, a.io, int64_t(s) * a.hq * D + 4 * i, make_float4(0.f, 0.f, 0.f, 0.f));
  }

  int64_t lane_first;
  int lane_s, lane_n;
  const int64_t T = all_tiles(a, C::kTK, &lane_first, &lane_s, &lane_n) * p.units;
  const int64_t parts = min((int64_t)gridDim.x, T);
  const int64_t me = blockIdx.x;
  if (me >= parts) return;
  int64_t at = T * me / parts;  // this block's next tile, of all
  const int64_t end = T * (me + 1) / parts;

  Cursor cur;  // the next tile whose rows are looked up
  {
    const unsigned owners = __ballot_sync(0xffffffffu, lane_first * p.units <= at && lane_n > 0);
    const int src = 31 - __clz(owners);
    int64_t first = __shfl_sync(0xffffffffu, lane_first, src) * p.units;
    int s = __shfl_sync(0xffffffffu, lane_s, src);
    cur.span = span_of(a, s, C::kTK);
    while (first + int64_t(cur.span.tiles) * p.units <= at) {
      first += int64_t(cur.span.tiles) * p.units;
      cur.span = span_of(a, ++s, C::kTK);
    }
    cur.s = s;
    cur.unit = (int)((at - first) / cur.span.tiles);
    cur.tile = (int)((at - first) % cur.span.tiles);
    cur.left = end - at;
  }

  // Rows of a tile's keys: lane i holds key i's.  Its page entry is read one tile ahead.
  int32_t page = -1;
  uint32_t slot = 0;
  int page_unit = 0;
  auto look_up = [&]() {  // at cur
    const int key = cur.span.lo + cur.tile * C::kTK + warp * C::kKeys + lane;
    page = -1;
    page_unit = cur.unit;
    if (cur.left > 0 && lane < C::kKeys && key < cur.span.len) {
      const uint32_t pi = quotient((uint32_t)key, a.c.page);
      slot = (uint32_t)key - pi * a.c.page.d;
      page = a.pages[cur.s * a.pages_ld + pi];
      if (page < 0 || page >= a.c.n_pages) {
        index_error(a.status, kIdxAttnPage, page);
        page = -1;
      }
    }
  };
  auto row_of_lane = [&]() -> uint32_t {
    if (page < 0) return kNoRow;
    return (uint32_t)(page * a.c.page_stride + (page_unit / p.row_groups) * a.c.head_stride +
                      slot * a.c.slot_stride);
  };

  uint32_t kr[MT][2][NG][C::kKWords], vr[MT][4][NG][C::kVWords];  // K, V in flight
  uint32_t kscale[MT][2][(NG + 1) / 2], vscale[MT][4][(NG + 1) / 2];  // Q8_0 scales, two a word
  uint32_t row = kNoRow;                                            // lane i: key i's row
  uint32_t valid = 0;                                               // bit i: key i is there
  auto load_scales = [&](const __half *plane, uint32_t r, bool on, uint32_t (&w)[(NG + 1) / 2]) {
    const uint8_t *q = reinterpret_cast<const uint8_t *>(plane) + size_t(r) * (NG * 2);
    if (NG == 8) {
      const uint4 v = load16(q, on);
      w[0] = v.x, w[1 % ((NG + 1) / 2)] = v.y, w[2 % ((NG + 1) / 2)] = v.z, w[3 % ((NG + 1) / 2)] = v.w;
    } else if (NG == 4) {
      const uint2 v = load8(q, on);
      w[0] = v.x, w[1 % ((NG + 1) / 2)] = v.y;
    } else if (NG % 2 == 0) {
#pragma unroll
      for (int i = 0; i < NG / 2; ++i) w[i] = load4(q + 4 * i, on);
    } else {  // rows of an odd number of scales are 2-byte aligned
#pragma unroll
      for (int i = 0; i < (NG + 1) / 2; ++i) {
        uint16_t x = 0, y = 0;
        if (on) {
          x = *reinterpret_cast<const uint16_t *>(q + 4 * i);
          if (2 * i + 1 < NG) y = *reinterpret_cast<const uint16_t *>(q + 4 * i + 2);
        }
        w[i] = x | uint32_t(y) << 16;
      }
    }
  };
  auto load_k = [&]() {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t r = __shfl_sync(0xffffffffu, row, 16 * m + 8 * i + g);
        const bool on = r != kNoRow;
        const uint8_t *q = a.c.k + size_t(r) * C::kRow + t * (C::kKWords * 4);
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          if (C::kQ8) {
            const uint2 v = load8(q + 32 * j, on);
            kr[m][i][j][0] = v.x, kr[m][i][j][1] = v.y;
          } else {
            const uint4 v = load16(q + 64 * j, on);
            kr[m][i][j][0] = v.x, kr[m][i][j][1] = v.y;
            kr[m][i][j][2 % C::kKWords] = v.z, kr[m][i][j][3 % C::kKWords] = v.w;
          }
        }
        if (C::kQ8) load_scales(a.c.ks, r, on, kscale[m][i]);
      }
  };
  auto load_v = [&]() {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t r = __shfl_sync(0xffffffffu, row, 16 * m + 8 * (i >> 1) + 2 * t + (i & 1));
        const bool on = r != kNoRow;
        const uint8_t *q = a.c.v + size_t(r) * C::kRow + g * (C::kVWords * 4);
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          if (C::kQ8) {
            vr[m][i][j][0] = load4(q + 32 * j, on);
          } else {
            const uint2 v = load8(q + 64 * j, on);
            vr[m][i][j][0] = v.x, vr[m][i][j][1 % C::kVWords] = v.y;
          }
        }
        if (C::kQ8) load_scales(a.c.vs, r, on, vscale[m][i]);
      }
  };

  Cursor now = cur;  // the tile being multiplied (its piece's unit)
  look_up();
  row = row_of_lane();
  valid = __ballot_sync(0xffffffffu, row != kNoRow);
  load_k();
  load_v();
  next_tile(cur, a, p.units, C::kTK);
  look_up();

  while (at < end) {
    // ---- one piece: tiles of one unit ----
    const int64_t unit_first = at - now.tile;  // the unit's first tile, of all
    const int tiles = now.span.tiles;
    const int count = (int)min(end - at, int64_t(tiles - now.tile));
    const int hk = now.unit / p.row_groups, rg = now.unit % p.row_groups;
    const int rows = min(C::kRows, p.group - rg * C::kRows);  // query rows that exist
    const int64_t head0 = int64_t(now.s) * a.hq + hk * p.group + rg * C::kRows;
    const int64_t unit_id = int64_t(now.s) * p.units + now.unit;

    // the query's parts
    for (int r = warp; r < C::kRows; r += kWarps) {
      float x[8];
      float top = 0.f;
      const bool on = r < rows && lane < D / 8;
      const float4 u = on ? load_io4(a.q, a.io, (head0 + r) * D + lane * 8) : make_float4(0, 0, 0, 0);
      const float4 v = on ? load_io4(a.q, a.io, (head0 + r) * D + lane * 8 + 4) : make_float4(0, 0, 0, 0);
      x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
      int e = 0;
      if (!C::kBfK) {  // a power of two that puts the row's largest element in [2^14, 2^15)
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
        top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
        if (top > 0.f && top < INFINITY) e = min(max(141 - (int)(__float_as_uint(top) >> 23), -100), 100);
      }
      const float up = __uint_as_float(uint32_t(127 + e) << 23);
      if (lane == 0) sfac[r] = p.scale_log2 * __uint_as_float(uint32_t(127 - e) << 23);
      if (lane < D / 8) {
        uint32_t w[4][C::kPartsK];
#pragma unroll
        for (int i = 0; i < 4; ++i) split2<C::kBfK>(x[2 * i] * up, x[2 * i + 1] * up, w[i]);
#pragma unroll
        for (int k = 0; k < C::kPartsK; ++k)
          sq[k][r >> 3][lane >> 2][(r & 7) * 4 + (lane & 3)] =
              make_uint4(w[0][k], w[1][k], w[2][k], w[3][k]);
      }
    }
    __syncthreads();
    float fac[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) fac[n][0] = sfac[8 * n + 2 * t], fac[n][1] = sfac[8 * n + 2 * t + 1];

    float o[NG][2][NT][4] = {}, mx[NT][2], ls[NT][2] = {};
#pragma unroll
    for (int n = 0; n < NT; ++n) mx[n][0] = mx[n][1] = -INFINITY;

    for (int i = 0; i < count; ++i) {
      const uint32_t here = valid;
      const int key0 = now.span.lo + (now.tile + i) * C::kTK + warp * C::kKeys;
      // ---- S^T = K Q^T ----
      float s[MT][NT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float c0[4] = {}, c1[4] = {}, total[4] = {};
#pragma unroll
          for (int j = 0; j < NG; ++j) {
            uint32_t ka[4], kb[4];
            if (C::kQ8) {
              const uint32_t x0 = kr[m][0][j][0] ^ 0x80808080u, x1 = kr[m][0][j][1] ^ 0x80808080u;
              const uint32_t y0 = kr[m][1][j][0] ^ 0x80808080u, y1 = kr[m][1][j][1] ^ 0x80808080u;
              ka[0] = int8_f16<0x4140>(x0), ka[1] = int8_f16<0x4342>(x0);
              ka[2] = int8_f16<0x4140>(x1), ka[3] = int8_f16<0x4342>(x1);
              kb[0] = int8_f16<0x4140>(y0), kb[1] = int8_f16<0x4342>(y0);
              kb[2] = int8_f16<0x4140>(y1), kb[3] = int8_f16<0x4342>(y1);
            } else {
#pragma unroll
              for (int w = 0; w < 4; ++w)
                ka[w] = kr[m][0][j][w % C::kKWords], kb[w] = kr[m][1][j][w % C::kKWords];
            }
#pragma unroll
            for (int k = 0; k < C::kPartsK; ++k) {
              const uint4 b = sq[k][n][j][lane];
              mma<C::kBfK>(k ? c1 : c0, ka[0], kb[0], ka[1], kb[1], b.x, b.y);
              mma<C::kBfK>(k ? c1 : c0, ka[2], kb[2], ka[3], kb[3], b.z, b.w);
            }
            if (C::kQ8) {  // the block's scales: keys g (elements 0, 1) and g + 8 (2, 3)
              const float2 d0 = unpack2<false>(kscale[m][0][j / 2]);
              const float2 d1 = unpack2<false>(kscale[m][1][j / 2]);
              const float da = j & 1 ? d0.y : d0.x, db = j & 1 ? d1.y : d1.x;
              total[0] = fmaf(c0[0] + c1[0], da, total[0]);
              total[1] = fmaf(c0[1] + c1[1], da, total[1]);
              total[2] = fmaf(c0[2] + c1[2], db, total[2]);
              total[3] = fmaf(c0[3] + c1[3], db, total[3]);
#pragma unroll
              for (int w = 0; w < 4; ++w) c0[w] = c1[w] = 0.f;
            }
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) s[m][n][w] = C::kQ8 ? total[w] : c0[w] + c1[w];
        }
      // the next tile's rows; K's registers are free
      const bool more = at + i + 1 < end;
      if (more) {
        row = row_of_lane();
        valid = __ballot_sync(0xffffffffu, row != kNoRow);
        load_k();
      }
      // ---- softmax ----
      float al[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float top[2] = {mx[n][0], mx[n][1]};
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const bool ga = here >> (16 * m + g) & 1, gb = here >> (16 * m + 8 + g) & 1;
          s[m][n][0] = ga ? s[m][n][0] * fac[n][0] : -INFINITY;
          s[m][n][1] = ga ? s[m][n][1] * fac[n][1] : -INFINITY;
          s[m][n][2] = gb ? s[m][n][2] * fac[n][0] : -INFINITY;
          s[m][n][3] = gb ? s[m][n][3] * fac[n][1] : -INFINITY;
          top[0] = fmaxf(top[0], fmaxf(s[m][n][0], s[m][n][2]));
          top[1] = fmaxf(top[1], fmaxf(s[m][n][1], s[m][n][3]));
          if (p.logits && 8 * n + 2 * t < p.logit_width) {
            float *q = p.logits + (unit_id * a.max_len + key0 + 16 * m + g) * p.logit_width + 8 * n + 2 * t;
            const int ka = key0 + 16 * m + g;
            if (ka < now.span.len) *reinterpret_cast<float2 *>(q) = make_float2(s[m][n][0], s[m][n][1]);
            if (ka + 8 < now.span.len)
              *reinterpret_cast<float2 *>(q + 8 * p.logit_width) = make_float2(s[m][n][2], s[m][n][3]);
          }
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          top[w] = fmaxf(top[w], __shfl_xor_sync(0xffffffffu, top[w], 4));
          top[w] = fmaxf(top[w], __shfl_xor_sync(0xffffffffu, top[w], 8));
          top[w] = fmaxf(top[w], __shfl_xor_sync(0xffffffffu, top[w], 16));
          const float base = top[w] == -INFINITY ? 0.f : top[w];  // no key yet: all weights 0
          al[n][w] = exp2_fast(mx[n][w] - base);
          mx[n][w] = top[w];
          float sum = 0.f;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            s[m][n][w] = exp2_fast(s[m][n][w] - base + C::kBias);
            s[m][n][w + 2] = exp2_fast(s[m][n][w + 2] - base + C::kBias);
            sum += s[m][n][w] + s[m][n][w + 2];
          }
          ls[n][w] = fmaf(ls[n][w], al[n][w], sum);
        }
      }
      // the weights transposed, as binary32 in two halves: lane (g, t) gets row g's weights of
      // the keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int w = 0; w < 4; w += 2) {
            const uint32_t x = __float_as_uint(s[m][n][w]), y = __float_as_uint(s[m][n][w + 1]);
            const uint32_t hi = transpose8x8(__byte_perm(x, y, 0x7632));
            const uint32_t lo = transpose8x8(__byte_perm(x, y, 0x5410));
            s[m][n][w] = __uint_as_float(__byte_perm(lo, hi, 0x5410));
            s[m][n][w + 1] = __uint_as_float(__byte_perm(lo, hi, 0x7632));
          }
      uint32_t pw[MT][NT][2][C::kPartsV];  // the weights' parts (for Q8_0: made per block)
      if (!C::kQ8)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            split2<C::kBfV>(s[m][n][0], s[m][n][1], pw[m][n][0]);
            split2<C::kBfV>(s[m][n][2], s[m][n][3], pw[m][n][1]);
          }
      // ---- O^T = O^T alpha + V^T P^T ----
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        float c[2][NT][4] = {};
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint32_t va[2][4];  // [16 dims][operand word]
          if (C::kQ8) {
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2) {  // keys 2t, 2t + 1; then 2t + 8, 2t + 9
              const uint32_t x = vr[m][2 * i2][j][0], y = vr[m][2 * i2 + 1][j][0];
              const uint32_t d01 = __byte_perm(x, y, 0x5140), d23 = __byte_perm(x, y, 0x7362);
              va[0][2 * i2] = int8_bf16(__byte_perm(d01, 0x43434343u, 0x4140));
              va[0][2 * i2 + 1] = int8_bf16(__byte_perm(d01, 0x43434343u, 0x4342));
              va[1][2 * i2] = int8_bf16(__byte_perm(d23, 0x43434343u, 0x4140));
              va[1][2 * i2 + 1] = int8_bf16(__byte_perm(d23, 0x43434343u, 0x4342));
            }
            float dv[4];  // the four keys' scales of this block
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 d = unpack2<false>(vscale[m][k][j / 2]);
              dv[k] = j & 1 ? d.y : d.x;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              split2<C::kBfV>(s[m][n][0] * dv[0], s[m][n][1] * dv[1], pw[m][n][0]);
              split2<C::kBfV>(s[m][n][2] * dv[2], s[m][n][3] * dv[3], pw[m][n][1]);
            }
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i2 = 0; i2 < 2; ++i2) {
                const uint32_t x = vr[m][2 * i2][j][h % C::kVWords], y = vr[m][2 * i2 + 1][j][h % C::kVWords];
                va[h][2 * i2] = __byte_perm(x, y, 0x5410);
                va[h][2 * i2 + 1] = __byte_perm(x, y, 0x7632);
              }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int k = 0; k < C::kPartsV; ++k)
                mma<C::kBfV>(c[h][n], va[h][0], va[h][1], va[h][2], va[h][3], pw[m][n][0][k],
                             pw[m][n][1][k]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int w = 0; w < 4; ++w) o[j][h][n][w] = fmaf(o[j][h][n][w], al[n][w & 1], c[h][n][w]);
      }
      if (more) {
        load_v();
        next_tile(cur, a, p.units, C::kTK);
        look_up();
      }
    }

    // ---- the warps' parts of the piece joined ----
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float l = ls[n][w];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int r = 8 * n + 2 * t + w;
        if (g == 0) sm[warp][r] = mx[n][w], sl[warp][r] = l;
#pragma unroll
        for (int j = 0; j < NG; ++j)
          *reinterpret_cast<float4 *>(&so[warp][r][32 * j + 4 * g]) =
              make_float4(o[j][0][n][w], o[j][0][n][w + 2], o[j][1][n][w], o[j][1][n][w + 2]);
      }
    __syncthreads();
    const bool whole = now.tile == 0 && count == tiles;
    const int64_t slot_id = me * 2 + (now.tile == 0);
    for (int i = tid; i < rows * (D / 4); i += kWarps * 32) {
      const int r = i / (D / 4), d = 4 * (i % (D / 4));
      float m = sm[0][r], l = 0.f;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) m = fmaxf(m, sm[w][r]);
      const float base = m == -INFINITY ? 0.f : m;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2_fast(sm[w][r] - base);
        const float4 y = *reinterpret_cast<const float4 *>(&so[w][r][d]);
        l = fmaf(sl[w][r], f, l);
        x.x = fmaf(y.x, f, x.x), x.y = fmaf(y.y, f, x.y), x.z = fmaf(y.z, f, x.z), x.w = fmaf(y.w, f, x.w);
      }
      if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        store_io4(a.o, a.io, (head0 + r) * D + d,
                  make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
        if (d == 0 && p.stats) p.stats[unit_id * C::kRows + r] = make_float2(base - C::kBias, inv);
      } else {
        *reinterpret_cast<float4 *>(p.piece_o + (slot_id * C::kRows + r) * D + d) = x;
        if (d == 0)
          *reinterpret_cast<float2 *>(p.piece_ml + (slot_id * C::kRows + r) * 2) = make_float2(m, l);
      }
    }
    if (!whole) {
      // blocks of the unit's first and last tile: block b has the tiles from T b / parts on
      const int64_t b0 = ((unit_first + 1) * parts - 1) / T;
      const int64_t b1 = ((unit_first + tiles) * parts - 1) / T;
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int before = atomicAdd(p.count + b0, 1);
        slast = before == (int)(b1 - b0);
        if (slast) p.count[b0] = 0;
      }
      __syncthreads();
      if (slast) {
        __threadfence();
        for (int i = tid; i < rows * (D / 4); i += kWarps * 32) {
          const int r = i / (D / 4), d = 4 * (i % (D / 4));
          float m = -INFINITY, l = 0.f;
          auto ml = [&](int64_t b) {
            return __ldcg(reinterpret_cast<const float2 *>(
                p.piece_ml + ((b * 2 + (b == b0)) * C::kRows + r) * 2));
          };
#pragma unroll 4
          for (int64_t b = b0; b <= b1; ++b) m = fmaxf(m, ml(b).x);
          const float base = m == -INFINITY ? 0.f : m;
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int64_t b = b0; b <= b1; ++b) {
            const float2 v = ml(b);
            const float f = exp2_fast(v.x - base);
            const float4 y = __ldcg(reinterpret_cast<const float4 *>(
                p.piece_o + ((b * 2 + (b == b0)) * C::kRows + r) * D + d));
            l = fmaf(v.y, f, l);
            x.x = fmaf(y.x, f, x.x), x.y = fmaf(y.y, f, x.y), x.z = fmaf(y.z, f, x.z), x.w = fmaf(y.w, f, x.w);
          }
          const float inv = l == 0.f ? 0.f : 1.f / l;
          store_io4(a.o, a.io, (head0 + r) * D + d,
                    make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
          if (d == 0 && p.stats) p.stats[unit_id * C::kRows + r] = make_float2(base - C::kBias, inv);
        }
      }
    }
    // the next piece
    at += count;
    now.left = end - at + 1;
    now.tile += count - 1;
    next_tile(now, a, p.units, C::kTK);
  }
}

// The weight sums: w = exp2(s - (m - bias)) / l per query row, summed over the rows of the kv
// head in their order.
constexpr int kTrackKeys = 1024;
__global__ void __launch_bounds__(256) attn_track_kernel(const __grid_constant__ Params p, int rows) {
  grid_dependency();
  const AttnArgs &a = p.a;
  const int s = blockIdx.z, h = blockIdx.y;
  const Span sp = span_of(a, s, 1);
  for (int j = sp.lo + blockIdx.x * kTrackKeys + threadIdx.x, k = 0; k < kTrackKeys && j < sp.len;
       j += 256, k += 256) {
    const int64_t r = kv_row(a.c, a.pages + s * a.pages_ld, h, j);
    if (r < 0) continue;
    float w = 0.f;
    for (int rg = 0; rg < p.row_groups; ++rg) {
      const int64_t unit = int64_t(s) * p.units + h * p.row_groups + rg;
      const float *x = p.logits + (unit * a.max_len + j) * p.logit_width;
      const int n = min(rows, p.group - rg * rows);
      for (int i = 0; i < n; ++i) {
        const float2 st = p.stats[unit * rows + i];
        w += exp2_fast(x[i] - st.x) * st.y;
      }
    }
    a.c.sums[r] += w;
  }
}

// Query rows of a unit: 8 columns of the products, or 16 where the group fills more than 8 of
// them and the accumulators (D/8 registers per 8 columns) leave room for K and V in flight.
int rows_of(int group, int dim) { return group > 8 && dim <= 128 ? 16 : 8; }

int grid_of(int dim, int rows, const DeviceState *st) {
  const int per_sm = dim * (rows / 8) <= 64 ? 4 : dim * (rows / 8) <= 128 ? 3 : 2;
  return std::min(st->sms * per_sm, kMaxParts);
}
struct Workspace {
  size_t piece_o, piece_ml, stats, logits, total;
  int logit_width;
};
Workspace workspace_of(int64_t S, int hq, int hkv, int dim, int64_t max_len, bool track,
                       const DeviceState *st) {
  const int group = hq / hkv, rows = rows_of(group, dim), grid = grid_of(dim, rows, st);
  const size_t units = size_t(hkv) * ((group + rows - 1) / rows);
  Workspace w;
  w.logit_width = std::min(rows, (group + 1) & ~1);
  w.piece_ml = align256(kMaxParts * sizeof(int));
  w.piece_o = align256(w.piece_ml + size_t(grid) * 2 * rows * 2 * 4);
  w.stats = align256(w.piece_o + size_t(grid) * 2 * rows * dim * 4);
  w.logits = align256(w.stats + (track ? size_t(S) * units * rows * 8 : 0));
  w.total = align256(w.logits + (track ? size_t(S) * units * size_t(max_len) * w.logit_width * 4 : 0));
  return w;
}

template <int TYPE, int D, int NT>
mq_status launch_shape(Params p, cudaStream_t s, const DeviceState *st) {
  using C = Shape<TYPE, D, NT>;
  static_assert(blocks_per_sm<TYPE, D, NT>() * 152 <= kMaxParts, "counters");
  const int64_t tiles = (p.a.max_len + C::kTK - 1) / C::kTK * p.a.S * p.units;
  const int64_t grid = std::min<int64_t>(grid_of(D, C::kRows, st), tiles);
  return launch_dependent("attn_decode_kernel", attn_decode_kernel<TYPE, D, NT>,
                          dim3((unsigned)grid, 1, 1), dim3(kWarps * 32, 1, 1), 0, s, p);
}
template <int TYPE, int D>
mq_status launch_rows(const Params &p, int rows, cudaStream_t s, const DeviceState *st) {
  if constexpr (D <= 128)
    if (rows == 16) return launch_shape<TYPE, D, 2>(p, s, st);
  return launch_shape<TYPE, D, 1>(p, s, st);
}
template <int TYPE>
mq_status launch_dim(const Params &p, int rows, cudaStream_t s, const DeviceState *st) {
  switch (p.a.c.dim) {
    case 64: return launch_rows<TYPE, 64>(p, rows, s, st);
    case 96: return launch_rows<TYPE, 96>(p, rows, s, st);
    case 128: return launch_rows<TYPE, 128>(p, rows, s, st);
    case 192: return launch_rows<TYPE, 192>(p, rows, s, st);
    default: return launch_rows<TYPE, 256>(p, rows, s, st);
  }
}

}  // namespace

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
  p.scale_log2 = a.scale * kLog2e;
  p.count = reinterpret_cast<int *>(a.ws);
  p.piece_ml = reinterpret_cast<float *>(a.ws + w.piece_ml);
  p.piece_o = reinterpret_cast<float *>(a.ws + w.piece_o);
  p.stats = a.track ? reinterpret_cast<float2 *>(a.ws + w.stats) : nullptr;
  p.logits = a.track ? reinterpret_cast<float *>(a.ws + w.logits) : nullptr;
  mq_status r;
  switch (a.c.type) {
    case MQ_F16: r = launch_dim<MQ_F16>(p, rows, s, st); break;
    case MQ_BF16: r = launch_dim<MQ_BF16>(p, rows, s, st); break;
    default: r = launch_dim<MQ_Q8_0>(p, rows, s, st); break;
  }
  if (r == MQ_OK && a.track)
    r = launch_dependent("attn_track_kernel", attn_track_kernel,
                         dim3((a.max_len + kTrackKeys - 1) / kTrackKeys, a.c.hkv, (unsigned)a.S),
                         dim3(256, 1, 1), 0, s, p, rows);
  return r;
}

}  // namespace mq
