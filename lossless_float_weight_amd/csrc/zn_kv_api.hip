// zn_kv_api.hip -- the C ABI of the key-value cache (include/zn.h): argument
// checks and the launch; nothing here allocates or synchronises.
#include "../../include/zn.h"
#include "zn_kv.h"

using namespace zn;

namespace {

constexpr uint64_t kMost = 0x7FFFFFFFull;
constexpr uint64_t kMostStride = 1ull << 40;

bool plain(int dt) { return dt == ZN_BF16 || dt == ZN_FP32; }
// elements are read and written whole
bool at(const void *p, int dt) { return p && uintptr_t(p) % (dt == ZN_FP32 ? 4 : 2) == 0; }
bool at4(const void *p) { return p && uintptr_t(p) % 4 == 0; }
bool at16(const void *p) { return p && uintptr_t(p) % 16 == 0; }
bool power(uint64_t v, uint64_t least, uint64_t most) { return v >= least && v <= most && (v & (v - 1)) == 0; }
uint32_t log2_of(uint32_t v) { return uint32_t(__builtin_ctz(v)); }

zn_status done(hipError_t e) { return e == hipSuccess ? ZN_OK : ZN_ERR_HIP; }

// The cache's description, checked (its addresses where `used`).
bool good_cache(const zn_mx_cache *c, bool used, KvCache *out) {
  if (!c || c->reserved || !power(c->page_size, 16, kKvMaxPage)) return false;
  if (c->head_dim < kMxBlock || c->head_dim > kKvMaxDim || c->head_dim % kMxBlock) return false;
  if (c->kv_heads < 1 || c->kv_heads > kKvMaxHeads) return false;
  if (c->n_pages < 1 || c->n_pages > kMost / c->page_size) return false;
  if (c->page_stride > kKvMaxPageStride || c->head_stride > kMostStride || c->place_stride > kKvMaxPlaceStride) return false;
  if (used && (!at16(c->k) || !c->k_scales || !at16(c->v) || !c->v_scales)) return false;
  out->k = static_cast<uint8_t *>(c->k);
  out->ks = static_cast<uint8_t *>(c->k_scales);
  out->v = static_cast<uint8_t *>(c->v);
  out->vs = static_cast<uint8_t *>(c->v_scales);
  out->n_pages = uint32_t(c->n_pages);
  out->shift = log2_of(c->page_size);
  out->heads = c->kv_heads;
  out->blocks = c->head_dim / kMxBlock;
  out->page_stride = c->page_stride;
  out->head_stride = c->head_stride;
  out->place_stride = c->place_stride;
  return true;
}

// What an extension and a release check alike.
bool good_step(const void *lens, const void *flags, uint32_t batch, const void *table, uint64_t table_stride,
               uint32_t width, const void *free, uint64_t free_cap, const void *n_free, uint32_t page_size,
               const void *new_lens, const void *n_left) {
  if (!power(page_size, 1, kKvMaxPage) || batch > kKvMaxBatch) return false;
  if (uint64_t(width) * page_size > kMost || free_cap > kMost || table_stride > kMostStride) return false;
  if (!at4(n_free) || !at4(n_left) || n_left == n_free || (free_cap && !at4(free))) return false;
  if (batch == 0) return true;
  if (batch > 1 && table_stride < width) return false;
  return at4(lens) && flags && at4(new_lens) && new_lens != lens && (width == 0 || at4(table));
}

// Rows of `row` elements, m by n of them at two strides (at most 2^40), do not run into each other.
bool apart(uint64_t m, uint64_t m_stride, uint64_t n, uint64_t n_stride, uint64_t row) {
  if (m < 2 || n < 2) return (m < 2 || m_stride >= row) && (n < 2 || n_stride >= row);
  const bool m_first = m_stride <= n_stride;
  const uint64_t low = m_first ? m_stride : n_stride, high = m_first ? n_stride : m_stride;
  // steps of the shorter stride fit the longer one, which holds for every layout of a dense axis order
  return low >= row && high >= row && (high - row) / low >= (m_first ? m : n) - 1;
}

bool attention_of(const zn_mx_cache *cache, const zn_mx_attention_args *g, bool used, AttnArgs *a) {
  *a = AttnArgs{};
  if (!g || !good_cache(cache, used, &a->c) || !plain(g->dtype)) return false;
  if (g->heads < 1 || g->heads % a->c.heads || g->batch > kKvMaxBatch) return false;
  const uint64_t group = g->heads / a->c.heads;
  // workgroups of 256 threads, one for 128 rows and one more for every request and key head, fit a grid
  if (g->tokens > (1ull << 29) / g->heads) return false;
  if (uint64_t(g->width) * cache->page_size > kMost || g->window > kMost || (g->window && !g->causal)) return false;
  if (!(g->scale > 0.0f) || g->scale > 0x1p127f) return false;   // times log2(e) it is finite
  if (!g->starts && g->tokens != g->batch) return false;
  if (g->table_stride > kMostStride || (g->batch > 1 && g->table_stride < g->width)) return false;
  for (uint64_t s : {g->q_token_stride, g->q_head_stride, g->out_token_stride, g->out_head_stride})
    if (s > kMostStride) return false;
  if (!apart(g->heads, g->out_head_stride, g->tokens, g->out_token_stride, cache->head_dim)) return false;
  a->q = static_cast<const uint8_t *>(g->q);
  a->q_token = g->q_token_stride;
  a->q_head = g->q_head_stride;
  a->out = static_cast<uint8_t *>(g->out);
  a->out_token = g->out_token_stride;
  a->out_head = g->out_head_stride;
  a->lse = g->lse;
  a->table = g->table;
  a->lens = g->lens;
  a->starts = g->starts;
  a->table_stride = g->table_stride;
  a->width = g->width;
  a->batch = g->batch;
  a->tokens = uint32_t(g->tokens);
  a->heads = g->heads;
  a->group = uint32_t(group);
  a->scale = g->scale;
  a->causal = g->causal != 0;
  a->window = g->window;
  a->max_new = uint32_t(g->max_new < g->tokens ? g->max_new : g->tokens);
  return true;
}

}  // namespace

extern "C" zn_status zn_kv_extend(const int32_t *d_lens, const int32_t *d_add, uint32_t batch, int32_t *d_table,
                                  uint64_t table_stride, uint32_t width, const int32_t *d_free, uint64_t free_cap,
                                  const int32_t *d_n_free, uint32_t page_size, uint64_t n_pages, uint64_t tokens,
                                  int32_t *d_new_lens, int32_t *d_starts, int32_t *d_slots, int32_t *d_positions,
                                  int32_t *d_n_left, hipStream_t stream) {
  if (!good_step(d_lens, d_add, batch, d_table, table_stride, width, d_free, free_cap, d_n_free, page_size,
                 d_new_lens, d_n_left))
    return ZN_ERR_ARG;
  if (tokens > kMost || n_pages > kMost / page_size || !at4(d_starts)) return ZN_ERR_ARG;
  if (batch && (!at4(d_add) || d_new_lens == d_add)) return ZN_ERR_ARG;
  if (tokens && (!at4(d_slots) || !at4(d_positions))) return ZN_ERR_ARG;
  KvStepArgs a = {};
  a.lens = d_lens;
  a.add = d_add;
  a.batch = batch;
  a.width = width;
  a.shift = log2_of(page_size);
  a.table = d_table;
  a.table_stride = table_stride;
  a.free = const_cast<int32_t *>(d_free);
  a.free_cap = uint32_t(free_cap);
  a.n_pages = uint32_t(n_pages);
  a.tokens = uint32_t(tokens);
  a.n_free = d_n_free;
  a.new_lens = d_new_lens;
  a.starts = d_starts;
  a.slots = d_slots;
  a.positions = d_positions;
  a.n_left = d_n_left;
  return done(launch_kv_extend(a, stream));
}

extern "C" zn_status zn_kv_release(const int32_t *d_lens, const uint8_t *d_done, uint32_t batch,
                                   const int32_t *d_table, uint64_t table_stride, uint32_t width, int32_t *d_free,
                                   uint64_t free_cap, const int32_t *d_n_free, uint32_t page_size,
                                   int32_t *d_new_lens, int32_t *d_n_left, hipStream_t stream) {
  if (!good_step(d_lens, d_done, batch, d_table, table_stride, width, d_free, free_cap, d_n_free, page_size,
                 d_new_lens, d_n_left))
    return ZN_ERR_ARG;
  KvStepArgs a = {};
  a.lens = d_lens;
  a.done = d_done;
  a.batch = batch;
  a.width = width;
  a.shift = log2_of(page_size);
  a.table = const_cast<int32_t *>(d_table);
  a.table_stride = table_stride;
  a.free = d_free;
  a.free_cap = uint32_t(free_cap);
  a.n_free = d_n_free;
  a.new_lens = d_new_lens;
  a.n_left = d_n_left;
  return done(launch_kv_release(a, stream));
}

extern "C" zn_status zn_mx_kv_write(zn_dtype dtype, const void *d_k, uint64_t k_token_stride, uint64_t k_head_stride,
                                    const void *d_v, uint64_t v_token_stride, uint64_t v_head_stride,
                                    const int32_t *d_slots, uint64_t tokens, const zn_mx_cache *cache,
                                    hipStream_t stream) {
  KvRowsArgs a = {};
  if (!plain(dtype) || tokens > kMost || !good_cache(cache, tokens != 0, &a.c)) return ZN_ERR_ARG;
  for (uint64_t s : {k_token_stride, k_head_stride, v_token_stride, v_head_stride})
    if (s > kMostStride) return ZN_ERR_ARG;
  if (tokens == 0) return ZN_OK;
  if (!at(d_k, dtype) || !at(d_v, dtype) || !at4(d_slots)) return ZN_ERR_ARG;
  a.k = static_cast<const uint8_t *>(d_k);
  a.v = static_cast<const uint8_t *>(d_v);
  a.k_token = k_token_stride;
  a.k_head = k_head_stride;
  a.v_token = v_token_stride;
  a.v_head = v_head_stride;
  a.slots = d_slots;
  a.tokens = tokens;
  return done(launch_kv_write(dtype, a, stream));
}

extern "C" zn_status zn_mx_kv_read(const zn_mx_cache *cache, const int32_t *d_slots, uint64_t tokens, zn_dtype dtype,
                                   void *d_k, void *d_v, hipStream_t stream) {
  KvRowsArgs a = {};
  if (!plain(dtype) || tokens > kMost || !good_cache(cache, tokens != 0, &a.c)) return ZN_ERR_ARG;
  if (tokens == 0) return ZN_OK;
  if (!at(d_k, dtype) || !at(d_v, dtype) || !at4(d_slots)) return ZN_ERR_ARG;
  a.k_out = static_cast<uint8_t *>(d_k);
  a.v_out = static_cast<uint8_t *>(d_v);
  a.slots = d_slots;
  a.tokens = tokens;
  return done(launch_kv_read(dtype, a, stream));
}

extern "C" zn_status zn_mx_attention_scratch_bytes(const zn_mx_cache *cache, const zn_mx_attention_args *args,
                                                   uint64_t *bytes) {
  AttnArgs a;
  if (!bytes || !attention_of(cache, args, false, &a)) return ZN_ERR_ARG;
  *bytes = a.tokens && a.batch ? attention_scratch(args->dtype, a) : 0;
  return ZN_OK;
}

extern "C" zn_status zn_debug_attention_kernel(const zn_mx_cache *cache, const zn_mx_attention_args *args, int *kernel) {
  AttnArgs a;
  if (!kernel || !attention_of(cache, args, false, &a)) return ZN_ERR_ARG;
  *kernel = a.tokens && a.batch ? attention_kernel(args->dtype, a) : -1;
  return ZN_OK;
}

extern "C" zn_status zn_mx_attention(const zn_mx_cache *cache, const zn_mx_attention_args *args, void *d_scratch,
                                     uint64_t scratch_bytes, hipStream_t stream) {
  return zn_mx_attention2(cache, args, 0, d_scratch, scratch_bytes, stream);
}

extern "C" zn_status zn_mx_attention2(const zn_mx_cache *cache, const zn_mx_attention_args *args, uint32_t flags,
                                      void *d_scratch, uint64_t scratch_bytes, hipStream_t stream) {
  AttnArgs a;
  if (flags & ~uint32_t(ZN_MX_FAST_WEIGHTS) || (flags && args && args->dtype != ZN_BF16)) return ZN_ERR_ARG;
  if (!attention_of(cache, args, args && args->tokens && args->batch, &a)) return ZN_ERR_ARG;
  if (a.tokens == 0 || a.batch == 0) return ZN_OK;
  if (!at(a.q, args->dtype) || !at(a.out, args->dtype) || (a.lse && !at4(a.lse))) return ZN_ERR_ARG;
  if (!at4(a.lens) || (a.starts && !at4(a.starts)) || (a.width && !at4(a.table))) return ZN_ERR_ARG;
  const uint64_t need = attention_scratch(args->dtype, a);
  if (need && !at16(d_scratch)) return ZN_ERR_ARG;
  if (scratch_bytes < need) return ZN_ERR_CAPACITY;
  a.scratch = static_cast<uint8_t *>(d_scratch);
  a.fast_weights = flags & ZN_MX_FAST_WEIGHTS;
  return done(launch_attention(args->dtype, a, stream));
}
