// C ABI of a serving step's slots, adapters and sampling: argument checks on
// the host, before any HIP call.
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

// bytes [begin, end) of an array; empty ones overlap nothing.  Of rows, their
// distance and their own bytes.
struct Range {
  uintptr_t begin, end, pitch, width;
};

Range range(const void *p, int64_t bytes) { return {(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, 0, 0}; }

// rows of `cols` elements, `ld` apart
Range rows(const void *p, int64_t n, int64_t ld, int64_t cols, int size) {
  Range r = range(p, n && cols ? ((n - 1) * ld + cols) * size : 0);
  r.pitch = (uintptr_t)ld * size;
  r.width = (uintptr_t)cols * size;
  return r;
}

bool overlap(const Range &a, const Range &b) {
  if (a.begin == a.end || b.begin == b.end || a.begin >= b.end || b.begin >= a.end) return false;
  if (!a.pitch || a.pitch != b.pitch) return true;
  // rows at one distance: other columns of one wider array
  const uintptr_t off = a.begin <= b.begin ? (b.begin - a.begin) % a.pitch : (a.pitch - (a.begin - b.begin) % a.pitch) % a.pitch;
  return off < a.width || off + b.width > a.pitch;
}

wq_status check_adapters(int32_t count, const wq_adapters *w, int64_t m, const char *who) {
  if (count <= 0 || count > WQ_MAX_BATCH)
    return set_error(WQ_E_ARG, "%s: count=%d (1 to %d)", who, count, WQ_MAX_BATCH);
  if (!w) return set_error(WQ_E_ARG, "%s: adapters are NULL", who);
  if (m < 0) return set_error(WQ_E_ARG, "%s: m=%lld", who, (long long)m);
  if (m >= 1 << 24) return set_error(WQ_E_UNSUPPORTED, "%s: m of 2^24 or more", who);
  for (int i = 0; i < count; ++i) {
    if (w[i].rank < 8 || w[i].rank > 128 || w[i].rank % 8)
      return set_error(WQ_E_UNSUPPORTED, "%s: rank[%d]=%d (a multiple of 8, 8 to 128)", who, i, w[i].rank);
    if (w[i].k <= 0 || w[i].n <= 0 || w[i].count <= 0)
      return set_error(WQ_E_ARG, "%s: adapters[%d]: n=%lld, k=%lld and count=%d must be positive", who, i,
                       (long long)w[i].n, (long long)w[i].k, w[i].count);
    if (w[i].k % 128) return set_error(WQ_E_ARG, "%s: k[%d]=%lld is not a multiple of 128", who, i, (long long)w[i].k);
    if (w[i].n >= 1 << 30 || w[i].k >= 1 << 27)
      return set_error(WQ_E_UNSUPPORTED, "%s: n[%d] of 2^30 or k of 2^27 or more", who, i);
    if ((int64_t)w[i].count * w[i].rank > INT64_MAX / 8 / (w[i].k > w[i].n ? w[i].k : w[i].n))
      return set_error(WQ_E_UNSUPPORTED, "%s: adapters[%d] past the address range", who, i);
  }
  return WQ_OK;
}

}  // namespace

extern "C" {

wq_status wq_kv_slots(int32_t page_size, int64_t pages, int32_t *table, int64_t ld_table, int64_t table_pages,
                      const int32_t *lens, const int32_t *new_tokens, int64_t seqs, const int32_t *free_pages,
                      int64_t free_count, const int32_t *used, int64_t tokens, int32_t *slots, int32_t *positions,
                      int32_t *seq_of, int32_t *lens_out, int32_t *last, int32_t *used_out, void *stream) {
  const char *who = "wq_kv_slots";
  wq::clear_error();
  if (page_size < 16 || (page_size & (page_size - 1)))
    return set_error(WQ_E_UNSUPPORTED, "%s: page_size=%d (a power of two, at least 16)", who, page_size);
  if (pages <= 0) return set_error(WQ_E_ARG, "%s: pages=%lld must be positive", who, (long long)pages);
  if (pages > (int64_t)INT32_MAX / page_size)
    return set_error(WQ_E_UNSUPPORTED, "%s: pages * page_size above 2^31-1", who);
  if (seqs < 0 || tokens < 0 || free_count < 0 || table_pages < 0)
    return set_error(WQ_E_ARG, "%s: seqs=%lld, tokens=%lld, free_count=%lld and table_pages=%lld must not be negative", who,
                     (long long)seqs, (long long)tokens, (long long)free_count, (long long)table_pages);
  if (seqs > 1 << 20 || tokens > 1 << 30 || free_count > INT32_MAX)
    return set_error(WQ_E_UNSUPPORTED, "%s: seqs above 2^20, tokens above 2^30 or free_count above 2^31-1", who);
  if (ld_table < table_pages)
    return set_error(WQ_E_ARG, "%s: ld_table=%lld < table_pages=%lld", who, (long long)ld_table, (long long)table_pages);
  if (seqs && ld_table > INT64_MAX / 8 / seqs)
    return set_error(WQ_E_UNSUPPORTED, "%s: seqs * ld_table past the address range", who);
  if (!used || !used_out || (seqs && (!lens || !new_tokens || !lens_out || !last)) ||
      (seqs && table_pages && !table) || (free_count && !free_pages) || (tokens && (!slots || !positions || !seq_of)))
    return set_error(WQ_E_ARG, "%s: every array must be non-NULL", who);
  const void *all[] = {table, lens, new_tokens, free_pages, used, slots, positions, seq_of, lens_out, last, used_out};
  for (const void *p : all)
    if (!aligned(p, 4)) return set_error(WQ_E_ALIGN, "%s: arrays must be 4-byte aligned", who);
  const Range in[] = {range(lens, 4 * seqs), range(new_tokens, 4 * seqs), range(free_pages, 4 * free_count), range(used, 4)};
  const Range out[] = {rows(table, seqs, ld_table, table_pages, 4), range(slots, 4 * tokens), range(positions, 4 * tokens),
                       range(seq_of, 4 * tokens), range(lens_out, 4 * seqs), range(last, 4 * seqs), range(used_out, 4)};
  for (int i = 0; i < 7; ++i) {
    for (const Range &r : in)
      if (overlap(out[i], r)) return set_error(WQ_E_ARG, "%s: an output overlaps an input", who);
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return set_error(WQ_E_ARG, "%s: outputs overlap", who);
  }
  wq::SlotsArgs a;
  memset(&a, 0, sizeof a);
  a.table = table;
  a.lens = lens;
  a.new_tokens = new_tokens;
  a.free_pages = free_pages;
  a.used = used;
  a.slots = slots;
  a.positions = positions;
  a.seq_of = seq_of;
  a.lens_out = lens_out;
  a.last = last;
  a.used_out = used_out;
  a.ld_table = ld_table;
  while ((1 << a.page_shift) < page_size) ++a.page_shift;
  // positions stay in 32 bits
  const int64_t most = (int64_t)INT32_MAX >> a.page_shift;
  a.table_pages = (int32_t)(table_pages < most ? table_pages : most);
  a.seqs = (int32_t)seqs;
  a.free_count = (int32_t)free_count;
  a.tokens = (int32_t)tokens;
  a.pages = (int32_t)pages;
  return hip_status(wq::launch_kv_slots(a, (hipStream_t)stream), who);
}

size_t wq_lora_workspace(int32_t count, const wq_adapters *w, int64_t m) {
  wq::clear_error();
  if (check_adapters(count, w, m, "wq_lora_workspace") != WQ_OK) return (size_t)-1;
  size_t bytes = 0;
  for (int i = 0; i < count; ++i) bytes += wq::lora_workspace(w[i], m);
  return bytes;
}

wq_status wq_lora(int32_t count, const wq_adapters *w, const uint16_t *const *x, const int64_t *ldx, int64_t m,
                  const int32_t *ids, const void *const *base, const int64_t *ldb, void *const *y,
                  const int64_t *ldy, const wq_dtype *dtype, void *workspace, size_t workspace_bytes, void *stream) {
  const char *who = "wq_lora";
  wq::clear_error();
  const wq_status st = check_adapters(count, w, m, who);
  if (st != WQ_OK) return st;
  if (!x || !ldx || !base || !ldb || !y || !ldy || !dtype) return set_error(WQ_E_ARG, "%s: NULL argument array", who);
  if (m == 0) return WQ_OK;
  if (!ids) return set_error(WQ_E_ARG, "%s: ids must be non-NULL", who);
  if (!aligned(ids, 4)) return set_error(WQ_E_ALIGN, "%s: ids must be 4-byte aligned", who);
  wq::LoraArgs a;
  memset(&a, 0, sizeof a);
  Range in[5 * WQ_MAX_BATCH + 1], out[WQ_MAX_BATCH];
  int ins = 0;
  in[ins++] = range(ids, 4 * m);
  size_t need = 0;
  for (int i = 0; i < count; ++i) {
    if (!w[i].a || !w[i].b || !x[i] || !base[i] || !y[i])
      return set_error(WQ_E_ARG, "%s: a, b, x, base and y of linear %d must be non-NULL", who, i);
    if (dtype[i] != WQ_F16 && dtype[i] != WQ_F32) return set_error(WQ_E_ARG, "%s: dtype[%d]=%d", who, i, dtype[i]);
    if (ldx[i] < w[i].k || ldb[i] < w[i].n || ldy[i] < w[i].n)
      return set_error(WQ_E_ARG, "%s: linear %d: ldx=%lld < k, or ldb=%lld or ldy=%lld < n", who, i, (long long)ldx[i],
                       (long long)ldb[i], (long long)ldy[i]);
    if (ldx[i] > INT64_MAX / 8 / m || ldb[i] > INT64_MAX / 8 / m || ldy[i] > INT64_MAX / 8 / m)
      return set_error(WQ_E_UNSUPPORTED, "%s: linear %d: m * ld past the address range", who, i);
    if (ldx[i] % 8) return set_error(WQ_E_ALIGN, "%s: ldx[%d]=%lld is not a multiple of 8", who, i, (long long)ldx[i]);
    if (!aligned(w[i].a, 16) || !aligned(w[i].b, 16) || !aligned(w[i].scales, 4) || !aligned(x[i], 16) ||
        !aligned(base[i], 16) || !aligned(y[i], 16))
      return set_error(WQ_E_ALIGN, "%s: linear %d: a, b, x, base and y 16-byte, scales 4-byte aligned", who, i);
    const int size = dtype[i] == WQ_F32 ? 4 : 2;
    in[ins++] = rows(x[i], m, ldx[i], w[i].k, 2);
    in[ins++] = range(w[i].scales, w[i].scales ? 4 * (int64_t)w[i].count : 0);
    in[ins++] = rows(base[i], m, ldb[i], w[i].n, size);
    in[ins++] = range(w[i].a, (int64_t)w[i].count * w[i].rank * w[i].k * 2);
    in[ins++] = range(w[i].b, (int64_t)w[i].count * w[i].rank * w[i].n * 2);
    out[i] = rows(y[i], m, ldy[i], w[i].n, size);
    a.lin[i] = {w[i].a, w[i].b, w[i].scales, x[i], base[i], y[i], nullptr, ldx[i], ldb[i], ldy[i],
                (int32_t)w[i].n, (int32_t)w[i].k, w[i].count, w[i].rank, dtype[i] == WQ_F32};
    need += wq::lora_workspace(w[i], m);
  }
  for (int i = 0; i < count; ++i) {
    for (int j = 0; j < ins; ++j) {
      const bool in_place = j == 5 * i + 3 && y[i] == base[i] && ldy[i] == ldb[i];
      if (!in_place && overlap(out[i], in[j])) return set_error(WQ_E_ARG, "%s: y[%d] overlaps an input", who, i);
    }
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return set_error(WQ_E_ARG, "%s: y[%d] and y[%d] overlap", who, j, i);
  }
  if (workspace_bytes < need || !workspace)
    return set_error(WQ_E_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", who, need, workspace_bytes);
  if (!aligned(workspace, 16)) return set_error(WQ_E_ALIGN, "%s: workspace must be 16-byte aligned", who);
  const Range scratch = range(workspace, (int64_t)need);
  for (int j = 0; j < ins; ++j)
    if (overlap(scratch, in[j])) return set_error(WQ_E_ARG, "%s: the workspace overlaps an input", who);
  for (int i = 0; i < count; ++i)
    if (overlap(scratch, out[i])) return set_error(WQ_E_ARG, "%s: the workspace overlaps y[%d]", who, i);
  char *at = static_cast<char *>(workspace);
  for (int i = 0; i < count; ++i) {
    a.lin[i].t = reinterpret_cast<float *>(at);
    at += wq::lora_workspace(w[i], m);
  }
  a.ids = ids;
  a.count = count;
  a.m = (int32_t)m;
  const wq::LoraPlan plan = wq::lora_plan(count, w, m);
  a.steps = plan.steps;
  a.slots = plan.slots;
  a.near = plan.near;
  memcpy(a.splits_to, plan.splits_to, sizeof a.splits_to);
  memcpy(a.chunks_to, plan.chunks_to, sizeof a.chunks_to);
  a.chunk = plan.chunk;
  return hip_status(wq::launch_lora(a, plan, (hipStream_t)stream), who);
}

size_t wq_sample_workspace(int64_t rows, int64_t vocab) {
  wq::clear_error();
  if (rows < 0 || rows > 1 << 20 || vocab <= 0 || vocab > 1 << 20) {
    set_error(WQ_E_ARG, "wq_sample_workspace: rows=%lld, vocab=%lld (up to 2^20 each)", (long long)rows, (long long)vocab);
    return (size_t)-1;
  }
  return wq::sample_workspace(rows, vocab, nullptr, nullptr);
}

wq_status wq_sample(const void *logits, wq_dtype dtype, int64_t rows, int64_t vocab, int64_t ldl, const float *u,
                    const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                    int32_t *ids, float *logprobs, void *workspace, size_t workspace_bytes, void *stream) {
  const char *who = "wq_sample";
  wq::clear_error();
  if (rows < 0 || vocab <= 0)
    return set_error(WQ_E_ARG, "%s: rows=%lld and vocab=%lld must be positive", who, (long long)rows, (long long)vocab);
  if (rows > 1 << 20 || vocab > 1 << 20) return set_error(WQ_E_UNSUPPORTED, "%s: rows or vocab above 2^20", who);
  if (dtype != WQ_F16 && dtype != WQ_F32) return set_error(WQ_E_ARG, "%s: dtype=%d", who, dtype);
  if (ldl < vocab) return set_error(WQ_E_ARG, "%s: ldl=%lld < vocab=%lld", who, (long long)ldl, (long long)vocab);
  if (rows == 0) return WQ_OK;
  if (ldl > INT64_MAX / 8 / rows) return set_error(WQ_E_UNSUPPORTED, "%s: rows * ldl past the address range", who);
  if (!logits || !u || !ids) return set_error(WQ_E_ARG, "%s: logits, u and ids must be non-NULL", who);
  if (!aligned(logits, 16) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) ||
      !aligned(min_p, 4) || !aligned(ids, 4) || !aligned(logprobs, 4))
    return set_error(WQ_E_ALIGN, "%s: logits 16-byte, the other arrays 4-byte aligned", who);
  size_t sums_at, counts_at;
  const size_t need = wq::sample_workspace(rows, vocab, &sums_at, &counts_at);
  if (workspace_bytes < need || (need && !workspace))
    return set_error(WQ_E_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", who, need, workspace_bytes);
  if (need && !aligned(workspace, 16)) return set_error(WQ_E_ALIGN, "%s: workspace must be 16-byte aligned", who);
  const Range in[] = {::rows(logits, rows, ldl, vocab, dtype == WQ_F32 ? 4 : 2),
                      range(u, 4 * rows),
                      range(temperature, temperature ? 4 * rows : 0),
                      range(top_k, top_k ? 4 * rows : 0),
                      range(top_p, top_p ? 4 * rows : 0),
                      range(min_p, min_p ? 4 * rows : 0)};
  const Range out[] = {range(ids, 4 * rows), range(logprobs, logprobs ? 4 * rows : 0)};
  for (const Range &o : out)
    for (const Range &r : in)
      if (overlap(o, r)) return set_error(WQ_E_ARG, "%s: an output overlaps an input", who);
  if (overlap(out[0], out[1])) return set_error(WQ_E_ARG, "%s: outputs overlap", who);
  const Range scratch = range(workspace, (int64_t)need);
  for (const Range &r : in)
    if (overlap(scratch, r)) return set_error(WQ_E_ARG, "%s: the workspace overlaps an input", who);
  if (overlap(scratch, out[0]) || overlap(scratch, out[1]))
    return set_error(WQ_E_ARG, "%s: the workspace overlaps an output", who);
  wq::SampleArgs a;
  memset(&a, 0, sizeof a);
  a.logits = logits;
  a.ldl = ldl;
  a.u = u;
  a.given = (temperature ? wq::kGivenHeat : 0) | (top_k ? wq::kGivenTopK : 0) | (top_p ? wq::kGivenTopP : 0) |
            (min_p ? wq::kGivenMinP : 0);
  a.temperature = temperature ? temperature : u;
  a.top_k = top_k ? top_k : reinterpret_cast<const int32_t *>(u);
  a.top_p = top_p ? top_p : u;
  a.min_p = min_p ? min_p : u;
  a.ids = ids;
  a.logprobs = logprobs;
  a.rows = (int32_t)rows;
  a.vocab = (int32_t)vocab;
  a.f32 = dtype == WQ_F32;
  a.parts = (int32_t)((vocab + wq::kSamplePart - 1) / wq::kSamplePart);
  a.heads = static_cast<wq::SamplePart *>(workspace);
  a.sums = reinterpret_cast<uint64_t *>(static_cast<char *>(workspace) + sums_at);
  a.counts = reinterpret_cast<uint32_t *>(static_cast<char *>(workspace) + counts_at);
  // the sum of vocab weights, each below 2, stays below 2^63
  a.unit = 44;
  while (((int64_t)1 << (62 - a.unit)) < vocab) --a.unit;
  return hip_status(wq::launch_sample(a, (hipStream_t)stream), who);
}

}  // extern "C"
