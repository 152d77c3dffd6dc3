// How the adapters' and sampling calls are cut into workgroups, and the
// workspaces that follow: host arithmetic only, known before any launch.
#include "wq_internal.h"

namespace wq {

namespace {

constexpr int64_t kLongWork = 768, kLongSplits = 4, kNearRows = 2048, kMostNearRows = 1 << 20;

// Workgroups that the outputs of rows in succession are cut for, about four a
// CU: 4001 rows of the projections below, rank 64, 62 us a call, with twice as
// many 67 (9728 outputs from 1100 rows 44 and 51; half as many 9728 from 2700
// rows 85 instead of 77).
constexpr int64_t kBlockWork = 1024;
constexpr int64_t kFewAdapters = 8, kShared = 4096, kMostSlots = 16;

// Workgroups that K and the outputs are cut for where one stands for each row:
// most of them find no group, so they are few, but eight of a row at least,
// one group's work being divided by that.  Projections 2560 to 4096, 1024 and
// 1024, rank 16, a call in us:
//              64 rows, 32 adapters  256 rows, 32 adapters
//   1024 all            10.9                  21.4
//   2048 all            13.7                  17.7
int64_t work(int64_t rows) { return rows <= 128 ? 1024 : 8 * rows; }

// the smallest multiple of `unit` in which the linears' lengths, cut, make at
// most `work` workgroups for `tiles`, and at most `most` of the longest
int64_t cut(int32_t count, const wq_adapters *w, int64_t wq_adapters::*length, int64_t tiles, int64_t unit, int64_t work,
            int64_t most) {
  int64_t sum = 0, longest = 0;
  for (int32_t i = 0; i < count; ++i) {
    sum += w[i].*length;
    longest = w[i].*length > longest ? w[i].*length : longest;
  }
  int64_t piece = (sum * tiles + work - 1) / work;
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

// Workgroups that share the groups of some rows in succession.  Every row may
// have an adapter of its own: one workgroup takes 205 us for 257 rows of the
// projections above with 256 adapters, fifteen 71 (32 adapters: 119 and 42, in
// runs 35 and 18; one adapter: 11 both).  With more rows the blocks are enough:
// 4001 rows 67 us both; twice as many at 512 rows 122 us instead of 102.
int32_t slots_for(int64_t rows, int32_t adapters) {
  int64_t s = kShared / rows;
  s = s < 1 ? 1 : s > kMostSlots ? kMostSlots : s;
  return (int32_t)(s > adapters + 1 ? adapters + 1 : s);
}

}  // namespace

LoraPlan lora_plan(int32_t count, const wq_adapters *w, int64_t m) {
  LoraPlan p = {};
  int32_t adapters = 0;
  for (int32_t i = 0; i < count; ++i) adapters = w[i].count > adapters ? w[i].count : adapters;
  // A workgroup for each row or for rows in succession: the projections above,
  // rows with ids in any order, a call in us:
  //   rows, adapters  32, 8  64, 1  64, 16  128, 4  128, 16  256, 8  256, 16
  //   each row          9.6   11.7    10.9    15.6     14.0    18.9     19.2
  //   in succession    10.2   10.8    12.8    10.1     17.3    15.8     27.7
  p.whole = m <= 32 || (m <= kWholeRows && adapters > kFewAdapters);
  p.inner_tiles = p.whole ? m : (m + 31) / 32;
  p.outer_tiles = p.whole ? m : (m + 63) / 64;
  int64_t k = 0;
  for (int32_t i = 0; i < count; ++i) {
    k = w[i].k > k ? w[i].k : k;
    p.rank = w[i].rank > p.rank ? w[i].rank : p.rank;
  }
  int64_t piece;
  if (p.whole) {
    piece = cut(count, w, &wq_adapters::k, m, 128, work(m), kLoraSplits);
    p.slots = 1;
  } else {
    const int64_t splits = splits_for(p.inner_tiles * count);
    piece = ((k + splits - 1) / splits + 255) / 256 * 256;
    p.slots = slots_for(m, adapters);
    // Rows' pieces next to each other on one XCD: of many rows, x, read for
    // each linear, and t, for each piece of the outputs, come from its L2 then.
    // The projections above, rank 64, 4001 rows 60 -> 56 us, one linear 4096 to
    // 2560 41 -> 36; below that many rows the XCDs get uneven shares: 1500 rows
    // of the one linear 21 -> 25.
    p.near = m >= kNearRows && m <= kMostNearRows;
  }
  p.steps = (int32_t)(piece / 32);
  p.chunk = (int32_t)cut(count, w, &wq_adapters::n, p.outer_tiles, 256, p.whole ? work(m) : kBlockWork, INT32_MAX);
  for (int32_t i = 0; i < count; ++i) {
    p.splits += (uint32_t)((w[i].k + piece - 1) / piece);
    p.chunks += (uint32_t)((w[i].n + p.chunk - 1) / p.chunk);
    p.splits_to[i] = p.splits;
    p.chunks_to[i] = p.chunks;
  }
  return p;
}

size_t lora_workspace(const wq_adapters &w, int64_t m) {
  // a bound of splits * m that grows with m: where workgroups stand for rows in
  // succession, splits is at most kLongSplits, and at most kLongWork over a 32nd of m
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
