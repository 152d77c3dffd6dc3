// How the adapters' and sampling calls are cut into workgroups, and the
// workspaces that follow: host arithmetic only, known before any launch.
#include "wq_internal.h"

namespace wq {

namespace {

constexpr int64_t kWork = 2048;   // workgroups that K and the outputs of up to kWholeRows rows are cut for
constexpr int64_t kLongWork = 768, kLongSplits = 4;

// the smallest multiple of `unit` in which `pieces`, cut, make at most kWork
// workgroups for each `tiles`, and at most `most` of the longest piece
int64_t cut(int32_t count, const wq_adapters *w, int64_t wq_adapters::*length, int64_t tiles, int64_t unit, int64_t most) {
  int64_t sum = 0, longest = 0;
  for (int32_t i = 0; i < count; ++i) {
    sum += w[i].*length;
    longest = w[i].*length > longest ? w[i].*length : longest;
  }
  int64_t piece = (sum * tiles + kWork - 1) / kWork;
  if (piece > longest) piece = longest;
  const int64_t least = (longest + most - 1) / most;
  if (piece < least) piece = least;
  return (piece + unit - 1) / unit * unit;
}

// splits of K in a long call, for three workgroups a CU (their LDS fits): 4001
// rows, three projections, rank 64: 30 us with one, 27 with two
int32_t splits_for(int64_t tiles) {
  const int64_t s = kLongWork / tiles;
  return (int32_t)(s < 1 ? 1 : s > kLongSplits ? kLongSplits : s);
}

}  // namespace

LoraPlan lora_plan(int32_t count, const wq_adapters *w, int64_t m) {
  LoraPlan p;
  p.whole = m <= kWholeRows;
  p.inner_tiles = p.whole ? m : (m + 31) / 32;
  p.outer_tiles = p.whole ? m : (m + 63) / 64;
  int64_t n = 0, k = 0;
  p.rank = 0;
  for (int32_t i = 0; i < count; ++i) {
    n = w[i].n > n ? w[i].n : n;
    k = w[i].k > k ? w[i].k : k;
    p.rank = w[i].rank > p.rank ? w[i].rank : p.rank;
  }
  int64_t piece;
  if (p.whole) {
    piece = cut(count, w, &wq_adapters::k, m, 128, kLoraSplits);
  } else {
    const int64_t splits = splits_for(p.inner_tiles * count);
    piece = ((k + splits - 1) / splits + 255) / 256 * 256;
  }
  p.steps = (int32_t)(piece / 32);
  p.splits = (int32_t)((k + piece - 1) / piece);
  p.chunk = (int32_t)cut(count, w, &wq_adapters::n, p.outer_tiles, 256, INT32_MAX);
  p.chunks = (n + p.chunk - 1) / p.chunk;
  return p;
}

size_t lora_workspace(const wq_adapters &w, int64_t m) {
  // a bound of splits * m that grows with m: in a long call splits is at most
  // kLongSplits, and at most kLongWork over a 32nd of m
  const int64_t whole = (m <= kWholeRows ? m : kWholeRows) * kLoraSplits;
  const int64_t most = kLongSplits * m, filled = m + 32 * kLongWork, longer = most < filled ? most : filled;
  const size_t bytes = (size_t)(m <= kWholeRows || whole > longer ? whole : longer) * (size_t)w.rank * sizeof(float);
  return (bytes + 255) / 256 * 256;
}

// heads, then bins' sums, then their counts
size_t sample_workspace(int64_t rows, int64_t vocab, size_t *sums_at, size_t *counts_at) {
  const size_t parts = (size_t)rows * (size_t)((vocab + kSamplePart - 1) / kSamplePart);
  const size_t heads = (parts * sizeof(SamplePart) + 255) / 256 * 256, sums = parts * kSampleBins * sizeof(uint64_t);
  if (sums_at) *sums_at = heads;
  if (counts_at) *counts_at = heads + sums;
  return heads + sums + parts * kSampleBins * sizeof(uint32_t);
}

}  // namespace wq
