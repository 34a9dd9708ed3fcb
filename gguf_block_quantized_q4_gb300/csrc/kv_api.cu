// kv_api.cu -- the C ABI entry points of the paged cache and its decode attention: argument
// validation ("minfer CUDA Backend Design" §4.9 rule 1: every violation returns a status and a
// message that names it, before anything is launched).  Indexes that lie in device memory
// (positions, slots, lengths, pages) are checked by the kernels.
#include <algorithm>

#include "kv.cuh"

using namespace mq;

namespace {

mq_status check_cache(const char *site, const mq_kv_cache *c) {
  if (!c) return fail(MQ_ERR_ARG, "%s: cache is NULL", site);
  if (c->type != MQ_F16 && c->type != MQ_BF16 && c->type != MQ_Q8_0)
    return fail(MQ_ERR_TYPE, "%s: cache type %d (supported: 1 F16, 8 Q8_0, 30 BF16)", site,
                (int)c->type);
  const int d = c->head_dim;
  if (d != 64 && d != 96 && d != 128 && d != 192 && d != 256)
    return fail(MQ_ERR_SHAPE, "%s: head_dim=%d is not one of 64, 96, 128, 192, 256", site, d);
  if (c->n_kv_heads < 1 || c->n_kv_heads > 1024)
    return fail(MQ_ERR_SHAPE, "%s: n_kv_heads=%d outside [1, 1024]", site, c->n_kv_heads);
  if (c->page_size < 1 || c->page_size > 65536)
    return fail(MQ_ERR_SHAPE, "%s: page_size=%d outside [1, 65536]", site, c->page_size);
  if (c->n_pages < 1 || c->n_pages > 0x7fffffff)
    return fail(MQ_ERR_SHAPE, "%s: n_pages=%lld outside [1, 2^31)", site, (long long)c->n_pages);
  // the rows of different (page, head, slot) must not meet: each stride clears the extent of
  // the next smaller one
  struct Axis {
    int64_t stride, n;
    const char *name;
  } ax[3] = {{c->page_stride, c->n_pages, "page_stride"},
             {c->head_stride, c->n_kv_heads, "head_stride"},
             {c->slot_stride, c->page_size, "slot_stride"}};
  for (const Axis &a : ax)
    if (a.stride < 1 || a.stride > (int64_t(1) << 40) / a.n)
      return fail(MQ_ERR_SHAPE, "%s: %s=%lld rows is out of range for an extent of %lld", site,
                  a.name, (long long)a.stride, (long long)a.n);
  std::sort(ax, ax + 3, [](const Axis &a, const Axis &b) {
    return a.stride != b.stride ? a.stride < b.stride : a.n < b.n;
  });
  int64_t extent = 1;  // rows that the axes so far span
  for (const Axis &a : ax) {
    if (a.n == 1) continue;
    if (a.stride < extent)
      return fail(MQ_ERR_SHAPE, "%s: %s=%lld lets rows overlap (the inner axes span %lld rows)",
                  site, a.name, (long long)a.stride, (long long)extent);
    extent = a.stride * (a.n - 1) + extent;
  }
  if (extent > int64_t(0xfffffffe))  // the kernels keep row indexes in 32 bits
    return fail(MQ_ERR_SHAPE, "%s: the strides span %lld rows; at most 2^32 - 2 are supported", site,
                (long long)extent);
  return MQ_OK;
}

mq_status check_io(const char *site, int io) {
  if (io != MQ_F32 && io != MQ_F16 && io != MQ_BF16)
    return fail(MQ_ERR_TYPE, "%s: io type %d (supported: 0 F32, 1 F16, 30 BF16)", site, io);
  return MQ_OK;
}

mq_status check_heads(const char *site, const mq_kv_cache *c, int n_heads) {
  if (n_heads < 1 || n_heads > 4096 || n_heads % c->n_kv_heads)
    return fail(MQ_ERR_SHAPE, "%s: n_heads=%d is not a multiple of n_kv_heads=%d in [1, 4096]",
                site, n_heads, c->n_kv_heads);
  return MQ_OK;
}

// The planes' pointers, and the view of the cache.
mq_status cache_view(const char *site, const mq_kv_cache *c, bool sums, int dev, KvView *v) {
  mq_status s;
  if ((s = check_dev_ptr(site, "cache.k", c->k, dev, 16)) != MQ_OK) return s;
  if ((s = check_dev_ptr(site, "cache.v", c->v, dev, 16)) != MQ_OK) return s;
  if (c->type == MQ_Q8_0) {
    if ((s = check_dev_ptr(site, "cache.k_scale", c->k_scale, dev, 16)) != MQ_OK) return s;
    if ((s = check_dev_ptr(site, "cache.v_scale", c->v_scale, dev, 16)) != MQ_OK) return s;
  }
  if (sums && (s = check_dev_ptr(site, "cache.weight_sum", c->weight_sum, dev, 16)) != MQ_OK)
    return s;
  v->k = static_cast<uint8_t *>(c->k);
  v->v = static_cast<uint8_t *>(c->v);
  v->ks = static_cast<__half *>(c->k_scale);
  v->vs = static_cast<__half *>(c->v_scale);
  v->sums = c->weight_sum;
  v->n_pages = c->n_pages;
  v->page_stride = c->page_stride;
  v->head_stride = c->head_stride;
  v->slot_stride = c->slot_stride;
  v->type = c->type;
  v->hkv = c->n_kv_heads;
  v->dim = c->head_dim;
  v->page = fast_div((uint32_t)c->page_size);
  return MQ_OK;
}

// Whether two ranges of bytes share any.
bool overlap(const void *a, uint64_t a_bytes, const void *b, uint64_t b_bytes) {
  const auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a_bytes && b_bytes && (x < y ? y - x < a_bytes : x - y < b_bytes);
}

mq_status check_lengths(const char *site, const mq_kv_cache *c, int64_t S, int64_t max_len,
                        int64_t pages_ld) {
  if (S < 0 || S > 65535) return fail(MQ_ERR_ARG, "%s: S=%lld outside [0, 65535]", site, (long long)S);
  if (pages_ld < 1 || pages_ld > 0x7fffffff)
    return fail(MQ_ERR_ARG, "%s: pages_ld=%lld outside [1, 2^31)", site, (long long)pages_ld);
  if (max_len < 1 || max_len > 0x7fff0000 || max_len > pages_ld * c->page_size)
    return fail(MQ_ERR_ARG, "%s: max_len=%lld outside [1, min(2^31 - 65536, pages_ld*page_size=%lld)]",
                site, (long long)max_len, (long long)(pages_ld * c->page_size));
  return MQ_OK;
}

}  // namespace

extern "C" mq_status mq_rope_store(const mq_kv_cache *cache, const mq_rope *rope, mq_type io,
                                   const void *qkv, int64_t ld, const float *bias,
                                   const int32_t *pos, const int64_t *slot, void *q, int64_t T,
                                   int n_heads, mq_stream stream) {
  const char *site = "mq_rope_store";
  mq_status s;
  if ((s = check_cache(site, cache)) != MQ_OK) return s;
  if ((s = check_io(site, io)) != MQ_OK) return s;
  if ((s = check_heads(site, cache, n_heads)) != MQ_OK) return s;
  if (!rope) return fail(MQ_ERR_ARG, "%s: rope is NULL", site);
  if (rope->rot_dim < 8 || rope->rot_dim % 8 || rope->rot_dim > cache->head_dim)
    return fail(MQ_ERR_SHAPE, "%s: rot_dim=%d is not a multiple of 8 in [8, head_dim=%d]", site,
                rope->rot_dim, cache->head_dim);
  if (rope->n_axes < 1 || rope->n_axes > 4)
    return fail(MQ_ERR_ARG, "%s: n_axes=%d outside [1, 4]", site, rope->n_axes);
  if (rope->pairs != 0 && rope->pairs != 1)
    return fail(MQ_ERR_ARG, "%s: pairs=%d is neither 0 nor 1", site, rope->pairs);
  for (int i = 0; i < rope->rot_dim / 2; ++i)
    if (rope->axis[i] >= rope->n_axes)
      return fail(MQ_ERR_ARG, "%s: axis[%d]=%d but n_axes=%d", site, i, rope->axis[i],
                  rope->n_axes);
  if (rope->max_pos < 1 || rope->max_pos > (int64_t(1) << 31))
    return fail(MQ_ERR_ARG, "%s: max_pos=%lld outside [1, 2^31]", site, (long long)rope->max_pos);
  if (T < 0 || T > 0x7fffffff)
    return fail(MQ_ERR_ARG, "%s: T=%lld outside [0, 2^31)", site, (long long)T);
  const int64_t width = int64_t(n_heads + 2 * cache->n_kv_heads) * cache->head_dim;
  const int esize = io == MQ_F32 ? 4 : 2;
  if (ld < width || ld > (int64_t(1) << 31))
    return fail(MQ_ERR_SHAPE, "%s: ld=%lld is less than the %lld elements of a row, or beyond 2^31",
                site, (long long)ld, (long long)width);
  if (ld * esize % 16)
    return fail(MQ_ERR_ALIGN, "%s: rows of ld=%lld elements are not 16-byte aligned", site,
                (long long)ld);
  // a thread writes the queries where it read them only if there is one row and q begins with it
  if (T && !(T == 1 && q == qkv) &&
      overlap(q, T * n_heads * cache->head_dim * esize, qkv, uint64_t((T - 1) * ld + width) * esize))
    return fail(MQ_ERR_ARG, "%s: q=%p overlaps qkv=%p (only one token's may, from the row's start)", site, q, qkv);
  DeviceState *st = nullptr;
  if ((s = current_state(&st, site)) != MQ_OK) return s;
  if (T == 0) return MQ_OK;
  int dev = 0;
  cudaGetDevice(&dev);
  RopeArgs a;
  if ((s = cache_view(site, cache, cache->weight_sum != nullptr, dev, &a.c)) != MQ_OK) return s;
  if ((s = check_dev_ptr(site, "rope.table", rope->table, dev, 16)) != MQ_OK) return s;
  if ((s = check_dev_ptr(site, "qkv", qkv, dev, 16)) != MQ_OK) return s;
  if (bias && (s = check_dev_ptr(site, "bias", bias, dev, 16)) != MQ_OK) return s;
  if ((s = check_dev_ptr(site, "pos", pos, dev, 4)) != MQ_OK) return s;
  if ((s = check_dev_ptr(site, "slot", slot, dev, 8)) != MQ_OK) return s;
  if ((s = check_dev_ptr(site, "q", q, dev, 16)) != MQ_OK) return s;
  a.rope = *rope;
  a.io = io;
  a.qkv = qkv;
  a.ld = ld;
  a.bias = bias;
  a.pos = pos;
  a.slot = slot;
  a.q = q;
  a.T = T;
  a.hq = n_heads;
  a.status = st->status;
  return launch_rope_store(a, (cudaStream_t)stream, st);
}

extern "C" size_t mq_attn_workspace_bytes(const mq_kv_cache *cache, int64_t S, int n_heads,
                                          int64_t max_len, uint32_t flags) {
  const char *site = "mq_attn_workspace_bytes";
  DeviceState *st = nullptr;
  if (check_cache(site, cache) != MQ_OK || check_heads(site, cache, n_heads) != MQ_OK ||
      current_state(&st, site) != MQ_OK)
    return 0;
  if (S < 0 || S > 65535 || max_len < 1 || max_len > 0x7fff0000 || (flags & ~MQ_ATTN_TRACK)) {
    fail(MQ_ERR_ARG, "%s: S=%lld, max_len=%lld or flags=0x%x out of range", site, (long long)S,
         (long long)max_len, flags);
    return 0;
  }
  return attn_ws_bytes(S, n_heads, cache->n_kv_heads, cache->head_dim, max_len,
                       flags & MQ_ATTN_TRACK, st);
}

extern "C" mq_status mq_attn_decode(const mq_kv_cache *cache, mq_type io, const void *q, void *o,
                                    const int32_t *pages, int64_t pages_ld, const int32_t *len,
                                    int64_t S, int n_heads, int64_t max_len, float scale,
                                    int64_t window, uint32_t flags, void *ws, size_t ws_bytes,
                                    mq_stream stream) {
  const char *site = "mq_attn_decode";
  mq_status s;
  if ((s = check_cache(site, cache)) != MQ_OK) return s;
  if ((s = check_io(site, io)) != MQ_OK) return s;
  if ((s = check_heads(site, cache, n_heads)) != MQ_OK) return s;
  if ((s = check_lengths(site, cache, S, max_len, pages_ld)) != MQ_OK) return s;
  if (flags & ~MQ_ATTN_TRACK)
    return fail(MQ_ERR_ARG, "%s: unknown flag bits 0x%x", site, flags & ~MQ_ATTN_TRACK);
  if (window < 0) return fail(MQ_ERR_ARG, "%s: window=%lld is negative", site, (long long)window);
  if (!(scale - scale == 0.0f))
    return fail(MQ_ERR_ARG, "%s: scale=%g is not finite", site, (double)scale);
  // a row of o is written when every block that reads the same row of q has done so: in place, but
  // not shifted
  const uint64_t bytes = uint64_t(S) * n_heads * cache->head_dim * (io == MQ_F32 ? 4 : 2);
  if (o != q && overlap(o, bytes, q, bytes))
    return fail(MQ_ERR_ARG, "%s: o=%p overlaps q=%p (it may only be the same array)", site, o, q);
  const bool track = flags & MQ_ATTN_TRACK;
  DeviceState *st = nullptr;
  if ((s = current_state(&st, site)) != MQ_OK) return s;
  if (S == 0) return MQ_OK;
  int dev = 0;
  cudaGetDevice(&dev);
  AttnArgs a;
  if ((s = cache_view(site, cache, track, dev, &a.c)) != MQ_OK) return s;
  if ((s = check_dev_ptr(site, "q", q, dev, 16)) != MQ_OK) return s;
  if ((s = check_dev_ptr(site, "o", o, dev, 16)) != MQ_OK) return s;
  if ((s = check_dev_ptr(site, "pages", pages, dev, 4)) != MQ_OK) return s;
  if ((s = check_dev_ptr(site, "len", len, dev, 4)) != MQ_OK) return s;
  const size_t need =
      attn_ws_bytes(S, n_heads, cache->n_kv_heads, cache->head_dim, max_len, track, st);
  if (ws_bytes < need)
    return fail(MQ_ERR_ARG, "%s: ws_bytes=%zu but the call needs %zu (mq_attn_workspace_bytes)",
                site, ws_bytes, need);
  if ((s = check_dev_ptr(site, "ws", ws, dev, 256)) != MQ_OK) return s;
  a.io = io;
  a.q = q;
  a.o = o;
  a.pages = pages;
  a.pages_ld = pages_ld;
  a.len = len;
  a.S = S;
  a.hq = n_heads;
  a.max_len = (int)max_len;
  a.scale = scale;
  a.window = window;
  a.track = track;
  a.ws = static_cast<uint8_t *>(ws);
  a.status = st->status;
  return launch_attn_decode(a, (cudaStream_t)stream, st);
}

extern "C" mq_status mq_kv_evict(const mq_kv_cache *cache, const int32_t *pages, int64_t pages_ld,
                                 const int32_t *len, int64_t S, int64_t max_len,
                                 const int32_t *new_pages, int64_t new_pages_ld, int64_t keep,
                                 int64_t sink, int64_t recent, int32_t *kept, int32_t *new_len,
                                 mq_stream stream) {
  const char *site = "mq_kv_evict";
  mq_status s;
  if ((s = check_cache(site, cache)) != MQ_OK) return s;
  if ((s = check_lengths(site, cache, S, max_len, pages_ld)) != MQ_OK) return s;
  if (new_pages_ld < 1 || new_pages_ld > 0x7fffffff)
    return fail(MQ_ERR_ARG, "%s: new_pages_ld=%lld outside [1, 2^31)", site,
                (long long)new_pages_ld);
  if (keep < 1 || keep > 0x7fff0000 || keep > new_pages_ld * cache->page_size)
    return fail(MQ_ERR_ARG,
                "%s: keep=%lld outside [1, min(2^31 - 65536, new_pages_ld*page_size=%lld)]", site,
                (long long)keep, (long long)(new_pages_ld * cache->page_size));
  if (sink < 0 || recent < 0 || sink > keep || recent > keep || sink + recent > keep)
    return fail(MQ_ERR_ARG, "%s: sink=%lld and recent=%lld must be >= 0 and together <= keep=%lld",
                site, (long long)sink, (long long)recent, (long long)keep);
  // one length is read and written by one thread: in place, but not shifted
  if (len != new_len && overlap(len, 4 * S, new_len, 4 * S))
    return fail(MQ_ERR_ARG, "%s: new_len=%p overlaps len=%p (it may only be the same array)", site,
                (void *)new_len, (const void *)len);
  DeviceState *st = nullptr;
  if ((s = current_state(&st, site)) != MQ_OK) return s;
  if (S == 0) return MQ_OK;
  int dev = 0;
  cudaGetDevice(&dev);
  EvictArgs a;
  if ((s = cache_view(site, cache, true, dev, &a.c)) != MQ_OK) return s;
  if ((s = check_dev_ptr(site, "pages", pages, dev, 4)) != MQ_OK) return s;
  if ((s = check_dev_ptr(site, "len", len, dev, 4)) != MQ_OK) return s;
  if ((s = check_dev_ptr(site, "new_pages", new_pages, dev, 4)) != MQ_OK) return s;
  if ((s = check_dev_ptr(site, "kept", kept, dev, 4)) != MQ_OK) return s;
  if ((s = check_dev_ptr(site, "new_len", new_len, dev, 4)) != MQ_OK) return s;
  a.pages = pages;
  a.pages_ld = pages_ld;
  a.len = len;
  a.S = S;
  a.max_len = (int)max_len;
  a.new_pages = new_pages;
  a.new_pages_ld = new_pages_ld;
  a.keep = (int)keep;
  a.sink = (int)sink;
  a.recent = (int)recent;
  a.kept = kept;
  a.new_len = new_len;
  a.status = st->status;
  return launch_kv_evict(a, (cudaStream_t)stream, st);
}
