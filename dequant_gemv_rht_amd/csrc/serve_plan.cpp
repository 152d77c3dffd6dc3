// How the adapters' and sampling calls are cut into workgroups, and the
// workspaces that follow: host arithmetic only, known before any launch.
#include "wq_internal.h"

namespace wq {

namespace {

constexpr int64_t kInnerWork = 512;     // workgroups that the first kernel's K is split for
constexpr int64_t kOuterWork = 1024;    // and the second's outputs

// K splits of a call of `tiles` groups at least
int32_t splits_for(int64_t tiles, int64_t k) {
  int64_t s = (kInnerWork + tiles - 1) / tiles;
  if (s > kLoraSplits) s = kLoraSplits;
  if (s > k / 128) s = k / 128;
  return (int32_t)(s < 1 ? 1 : s);
}

}  // namespace

LoraPlan lora_plan(int32_t count, const wq_adapters *w, int64_t m) {
  LoraPlan p;
  p.whole = m <= kWholeRows;
  p.narrow = m <= 16;
  p.tiles = p.whole ? m : (m + 63) / 64;
  int64_t n = 0, k = 0;
  p.rank = 0;
  for (int32_t i = 0; i < count; ++i) {
    n = w[i].n > n ? w[i].n : n;
    k = w[i].k > k ? w[i].k : k;
    p.rank = w[i].rank > p.rank ? w[i].rank : p.rank;
  }
  const int64_t groups = (p.whole ? (m + 15) / 16 : p.tiles) * count;
  p.splits = splits_for(groups, k);
  int64_t chunks = (kOuterWork + groups - 1) / groups;
  if (chunks > (n + 255) / 256) chunks = (n + 255) / 256;
  p.chunk = (int32_t)(((n + chunks - 1) / chunks + 255) / 256 * 256);
  p.chunks = (n + p.chunk - 1) / p.chunk;
  return p;
}

size_t lora_workspace(const wq_adapters &w, int64_t m) {
  // a bound of splits * m that grows with m: ceil(work / tiles) m with tiles
  // of at least m / 64 rows
  const int64_t most = kLoraSplits * m, filled = m + 64 * kInnerWork;
  const size_t bytes = (size_t)(most < filled ? most : filled) * (size_t)w.rank * sizeof(float);
  return (bytes + 255) / 256 * 256;
}

}  // namespace wq
