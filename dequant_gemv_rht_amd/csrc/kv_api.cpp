// C ABI of the paged key-value cache, the attention over it and rotary
// positions: argument checks on the host, before any HIP call.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstring>

#include "wq_internal.h"

namespace {

using wq::set_error;

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

wq_status hip_status(hipError_t e, const char *who) {
  return e == hipSuccess ? WQ_OK : set_error(WQ_E_HIP, "%s: %s", who, hipGetErrorString(e));
}

wq_status check_cache(const wq_kv_cache *c, const char *who) {
  if (!c) return set_error(WQ_E_ARG, "%s: cache descriptor is NULL", who);
  if (c->bits != 4 && c->bits != 8 && c->bits != 16)
    return set_error(WQ_E_UNSUPPORTED, "%s: bits=%d (supported: 4, 8, 16)", who, c->bits);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return set_error(WQ_E_UNSUPPORTED, "%s: head_dim=%d (supported: 64, 128, 256)", who, c->head_dim);
  if (c->kv_heads <= 0) return set_error(WQ_E_ARG, "%s: kv_heads=%d must be positive", who, c->kv_heads);
  if (c->kv_heads > INT32_MAX / c->head_dim)
    return set_error(WQ_E_UNSUPPORTED, "%s: kv_heads * head_dim above 2^31-1", who);
  if (c->page_size < 16 || (c->page_size & (c->page_size - 1)))
    return set_error(WQ_E_UNSUPPORTED, "%s: page_size=%d (a power of two, at least 16)", who, c->page_size);
  if (c->pages <= 0) return set_error(WQ_E_ARG, "%s: pages=%lld must be positive", who, (long long)c->pages);
  if (c->pages > (int64_t)INT32_MAX / c->page_size)
    return set_error(WQ_E_UNSUPPORTED, "%s: pages * page_size above 2^31-1", who);
  if (!c->k || !c->v) return set_error(WQ_E_ARG, "%s: cache k and v must be non-NULL", who);
  if (!aligned(c->k, 16) || !aligned(c->v, 16))
    return set_error(WQ_E_ALIGN, "%s: cache k and v must be 16-byte aligned", who);
  if (c->bits != 16) {
    if (!c->k_params || !c->v_params)
      return set_error(WQ_E_ARG, "%s: k_params and v_params must be non-NULL for %d bits", who, c->bits);
    if (!aligned(c->k_params, 16) || !aligned(c->v_params, 16))
      return set_error(WQ_E_ALIGN, "%s: k_params and v_params must be 16-byte aligned", who);
  }
  if (c->rht_signs) {
    if (c->rht_block != WQ_RHT_BLOCK)
      return set_error(WQ_E_UNSUPPORTED, "%s: rht_block=%d (only 128)", who, c->rht_block);
    if (c->head_dim % WQ_RHT_BLOCK)
      return set_error(WQ_E_UNSUPPORTED, "%s: a rotated cache needs head_dim to be a multiple of 128 (got %d)", who,
                       c->head_dim);
    if (!aligned(c->rht_signs, 16)) return set_error(WQ_E_ALIGN, "%s: rht_signs must be 16-byte aligned", who);
  }
  return WQ_OK;
}

wq_status check_rows(const wq_kv_cache *c, const void *k, int64_t ldk, const void *v, int64_t ldv,
                     const int32_t *slots, int64_t tokens, wq::RowPlan *plan, const char *who) {
  const wq_status st = check_cache(c, who);
  if (st != WQ_OK) return st;
  if (tokens < 0) return set_error(WQ_E_ARG, "%s: tokens=%lld", who, (long long)tokens);
  if (tokens > (int64_t)INT32_MAX / 2 / c->kv_heads)
    return set_error(WQ_E_UNSUPPORTED, "%s: tokens * kv_heads of 2^30 or more", who);
  if (tokens == 0) return WQ_OK;
  *plan = wq::kv_row_plan(c->head_dim, tokens, c->kv_heads);
  if (plan->groups > wq::kMaxGroups256)
    return set_error(WQ_E_UNSUPPORTED, "%s: tokens * kv_heads of %lld heads of %d too many for one launch", who,
                     (long long)(tokens * c->kv_heads), c->head_dim);
  if (!k || !v || !slots) return set_error(WQ_E_ARG, "%s: k, v and slots must be non-NULL", who);
  const int64_t row = (int64_t)c->kv_heads * c->head_dim;
  if (ldk < row || ldv < row)
    return set_error(WQ_E_ARG, "%s: ldk=%lld, ldv=%lld below kv_heads * head_dim=%lld", who, (long long)ldk,
                     (long long)ldv, (long long)row);
  if (ldk % 8 || ldv % 8) return set_error(WQ_E_ALIGN, "%s: ldk and ldv must be multiples of 8", who);
  if (ldk > INT64_MAX / 2 / tokens || ldv > INT64_MAX / 2 / tokens)
    return set_error(WQ_E_UNSUPPORTED, "%s: tokens * ld past the address range", who);
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4))
    return set_error(WQ_E_ALIGN, "%s: k and v 16-byte, slots 4-byte aligned", who);
  return WQ_OK;
}

wq_status check_attn(const wq_kv_cache *c, int64_t seqs, int32_t q_heads, int64_t max_len, int64_t window,
                     const char *who) {
  const wq_status st = check_cache(c, who);
  if (st != WQ_OK) return st;
  if (seqs < 0) return set_error(WQ_E_ARG, "%s: seqs=%lld", who, (long long)seqs);
  if (q_heads <= 0 || q_heads % c->kv_heads)
    return set_error(WQ_E_ARG, "%s: q_heads=%d must be a positive multiple of kv_heads=%d", who, q_heads, c->kv_heads);
  if (max_len < 0 || window < 0)
    return set_error(WQ_E_ARG, "%s: max_len=%lld and window=%lld must not be negative", who, (long long)max_len,
                     (long long)window);
  if (max_len > (int64_t)INT32_MAX - 16384)   // positions past the last run stay in 32 bits
    return set_error(WQ_E_UNSUPPORTED, "%s: max_len above 2^31-16385", who);
  if (q_heads > INT32_MAX / c->head_dim || seqs > (int64_t)INT32_MAX / q_heads)
    return set_error(WQ_E_UNSUPPORTED, "%s: q_heads * head_dim or seqs * q_heads above 2^31-1", who);
  return WQ_OK;
}

}  // namespace

extern "C" {

wq_status wq_kv_write(const wq_kv_cache *cache, const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv,
                      const int32_t *slots, int64_t tokens, void *stream) {
  wq::clear_error();
  wq::RowPlan plan;
  const wq_status st = check_rows(cache, k, ldk, v, ldv, slots, tokens, &plan, "wq_kv_write");
  if (st != WQ_OK || tokens == 0) return st;
  return hip_status(wq::launch_kv_write(*cache, plan, k, ldk, v, ldv, slots, tokens, (hipStream_t)stream), "wq_kv_write");
}

wq_status wq_kv_read(const wq_kv_cache *cache, const int32_t *slots, int64_t tokens, uint16_t *k, int64_t ldk,
                     uint16_t *v, int64_t ldv, void *stream) {
  wq::clear_error();
  wq::RowPlan plan;
  const wq_status st = check_rows(cache, k, ldk, v, ldv, slots, tokens, &plan, "wq_kv_read");
  if (st != WQ_OK || tokens == 0) return st;
  return hip_status(wq::launch_kv_read(*cache, plan, slots, tokens, k, ldk, v, ldv, (hipStream_t)stream), "wq_kv_read");
}

size_t wq_attn_decode_workspace(const wq_kv_cache *cache, int64_t seqs, int32_t q_heads, int64_t max_len,
                                int64_t window) {
  wq::clear_error();
  if (check_attn(cache, seqs, q_heads, max_len, window, "wq_attn_decode_workspace") != WQ_OK) return (size_t)-1;
  return seqs ? wq::attn_workspace(*cache, seqs, q_heads, max_len, window) : 0;
}

wq_status wq_attn_decode(const wq_kv_cache *cache, const uint16_t *q, int64_t ldq, int32_t q_heads, int64_t seqs,
                         const int32_t *table, int64_t ld_table, const int32_t *lens, int64_t max_len, int64_t window,
                         float scale, uint16_t *out, int64_t ldo, void *workspace, size_t workspace_bytes,
                         void *stream) {
  const char *who = "wq_attn_decode";
  wq::clear_error();
  const wq_status st = check_attn(cache, seqs, q_heads, max_len, window, who);
  if (st != WQ_OK || seqs == 0) return st;
  if (!q || !lens || !out || (max_len && !table))
    return set_error(WQ_E_ARG, "%s: q, table, lens and out must be non-NULL", who);
  const int64_t row = (int64_t)q_heads * cache->head_dim;
  if (ldq < row || ldo < row)
    return set_error(WQ_E_ARG, "%s: ldq=%lld, ldo=%lld below q_heads * head_dim=%lld", who, (long long)ldq,
                     (long long)ldo, (long long)row);
  if (ld_table < 0 || ld_table < (max_len + cache->page_size - 1) / cache->page_size)
    return set_error(WQ_E_ARG, "%s: ld_table=%lld pages of %d tokens hold fewer than max_len=%lld", who,
                     (long long)ld_table, cache->page_size, (long long)max_len);
  if (!(scale - scale == 0.0f)) return set_error(WQ_E_ARG, "%s: scale is not finite", who);
  if (ldq % 8 || ldo % 8) return set_error(WQ_E_ALIGN, "%s: ldq and ldo must be multiples of 8", who);
  if (ldq > INT64_MAX / 2 / seqs || ldo > INT64_MAX / 2 / seqs || ld_table > INT64_MAX / 4 / seqs)
    return set_error(WQ_E_UNSUPPORTED, "%s: seqs * ld past the address range", who);
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(table, 4) || !aligned(lens, 4))
    return set_error(WQ_E_ALIGN, "%s: q and out 16-byte, table and lens 4-byte aligned", who);
  const wq::SplitPlan plan =
      wq::attn_plan(cache->bits, cache->head_dim, seqs, cache->kv_heads, q_heads / cache->kv_heads, max_len, window);
  if (plan.groups > wq::kMaxGroups256 || plan.join_groups > wq::kMaxGroups256)
    return set_error(WQ_E_UNSUPPORTED, "%s: %lld sequences of %d heads up to %lld tokens are too many workgroups for one launch",
                     who, (long long)seqs, q_heads, (long long)max_len);
  const size_t need = wq::attn_workspace(*cache, seqs, q_heads, max_len, window);
  if (need > workspace_bytes || (need && !workspace))
    return set_error(WQ_E_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", who, need, workspace_bytes);
  if (need && !aligned(workspace, 16)) return set_error(WQ_E_ALIGN, "%s: workspace must be 16-byte aligned", who);
  wq::AttnArgs a;
  memset(&a, 0, sizeof a);
  a.k = cache->k;
  a.v = cache->v;
  a.k_params = reinterpret_cast<const uint32_t *>(cache->k_params);
  a.v_params = reinterpret_cast<const uint32_t *>(cache->v_params);
  a.signs = cache->rht_signs;
  a.q = q;
  a.out = out;
  a.table = table;
  a.lens = lens;
  a.partial = static_cast<float *>(workspace);
  a.ldq = ldq;
  a.ldo = ldo;
  a.ld_table = ld_table;
  a.seqs = seqs;
  a.pages = (int32_t)cache->pages;
  a.kv_heads = cache->kv_heads;
  a.group = q_heads / cache->kv_heads;
  while ((1 << a.page_shift) < cache->page_size) ++a.page_shift;
  a.max_len = (int32_t)max_len;
  a.window = (int32_t)(window < max_len ? window : 0);   // a window of max_len or more hides nothing
  a.scale = scale;
  return hip_status(wq::launch_attn_decode(cache->bits, cache->head_dim, a, plan, (hipStream_t)stream), who);
}

wq_status wq_rope(int32_t count, const uint16_t *const *x, const int64_t *ldx, uint16_t *const *y, const int64_t *ldy,
                  const int32_t *heads, int64_t tokens, int32_t head_dim, int32_t rot, const float *cos,
                  const float *sin, int64_t table_rows, const int32_t *positions, int64_t ld_pos, int32_t axes,
                  const uint8_t *pair_axis, uint32_t flags, void *stream) {
  const char *who = "wq_rope";
  wq::clear_error();
  if (count <= 0 || count > WQ_MAX_BATCH)
    return set_error(WQ_E_ARG, "%s: count=%d (1 to %d)", who, count, WQ_MAX_BATCH);
  if (!x || !ldx || !y || !ldy || !heads) return set_error(WQ_E_ARG, "%s: NULL argument array", who);
  if (head_dim <= 0 || head_dim > 256 || head_dim % 8)
    return set_error(WQ_E_UNSUPPORTED, "%s: head_dim=%d (a multiple of 8 up to 256)", who, head_dim);
  if (rot <= 0 || rot > head_dim || rot % 16)
    return set_error(WQ_E_UNSUPPORTED, "%s: rot=%d (a multiple of 16 up to head_dim)", who, rot);
  if (axes < 1 || axes > WQ_ROPE_MAX_AXES)
    return set_error(WQ_E_UNSUPPORTED, "%s: axes=%d (1 to %d)", who, axes, WQ_ROPE_MAX_AXES);
  if (flags & ~WQ_ROPE_ADJACENT) return set_error(WQ_E_ARG, "%s: unknown flags 0x%x", who, flags);
  if (tokens < 0) return set_error(WQ_E_ARG, "%s: tokens=%lld", who, (long long)tokens);
  if (table_rows <= 0 || table_rows > INT32_MAX)
    return set_error(WQ_E_ARG, "%s: table_rows=%lld (1 to 2^31-1)", who, (long long)table_rows);
  wq::RopeArgs a;
  memset(&a, 0, sizeof a);
  if (pair_axis)
    for (int i = 0; i < rot / 2; ++i) {
      if (pair_axis[i] >= axes)
        return set_error(WQ_E_ARG, "%s: pair_axis[%d]=%d (below axes=%d)", who, i, (int)pair_axis[i], axes);
      a.pair_axis[i] = pair_axis[i];
    }
  int64_t all = 0;
  int32_t most = 0;
  for (int i = 0; i < count; ++i) {
    if (heads[i] > most) most = heads[i];
    if (heads[i] <= 0) return set_error(WQ_E_ARG, "%s: heads[%d]=%d must be positive", who, i, heads[i]);
    all += heads[i];
    const int64_t row = (int64_t)heads[i] * head_dim;
    if (ldx[i] < row || ldy[i] < row)
      return set_error(WQ_E_ARG, "%s: ldx[%d]=%lld, ldy=%lld below heads * head_dim=%lld", who, i, (long long)ldx[i],
                       (long long)ldy[i], (long long)row);
    if (ldx[i] % 8 || ldy[i] % 8) return set_error(WQ_E_ALIGN, "%s: ldx and ldy must be multiples of 8", who);
    if (tokens && (ldx[i] > INT64_MAX / 2 / tokens || ldy[i] > INT64_MAX / 2 / tokens))
      return set_error(WQ_E_UNSUPPORTED, "%s: tokens * ld past the address range", who);
    if (tokens && (!x[i] || !y[i])) return set_error(WQ_E_ARG, "%s: x[%d] and y must be non-NULL", who, i);
    if (!aligned(x[i], 16) || !aligned(y[i], 16))
      return set_error(WQ_E_ALIGN, "%s: x[%d] and y must be 16-byte aligned", who, i);
    if (tokens && x[i] == y[i] && ldx[i] != ldy[i])
      return set_error(WQ_E_ARG, "%s: in place needs ldx == ldy", who);
    a.arr[i] = {x[i], y[i], ldx[i], ldy[i], heads[i]};
  }
  if (tokens > INT32_MAX / 64 || most > 65535)
    return set_error(WQ_E_UNSUPPORTED, "%s: tokens=%lld, heads=%lld too many for one call", who, (long long)tokens,
                     (long long)all);
  if (tokens == 0) return WQ_OK;
  if (!cos || !sin || !positions) return set_error(WQ_E_ARG, "%s: cos, sin and positions must be non-NULL", who);
  if (ld_pos < tokens && axes > 1)
    return set_error(WQ_E_ARG, "%s: ld_pos=%lld < tokens=%lld", who, (long long)ld_pos, (long long)tokens);
  if (ld_pos > INT64_MAX / 16) return set_error(WQ_E_UNSUPPORTED, "%s: ld_pos past the address range", who);
  if (!aligned(cos, 16) || !aligned(sin, 16) || !aligned(positions, 4))
    return set_error(WQ_E_ALIGN, "%s: cos and sin 16-byte, positions 4-byte aligned", who);
  a.cos = cos;
  a.sin = sin;
  a.positions = positions;
  a.ld_pos = axes > 1 ? ld_pos : 0;
  a.tokens = tokens;
  a.count = count;
  a.head_dim = head_dim;
  a.rot = rot;
  a.axes = axes;
  a.table_rows = (int32_t)table_rows;
  a.adjacent = (flags & WQ_ROPE_ADJACENT) ? 1 : 0;
  return hip_status(wq::launch_rope(a, (hipStream_t)stream), who);
}

}  // extern "C"
