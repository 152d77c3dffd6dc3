// Host-only exercise of the attention side's plans (kv_plan.cpp), built with
// AddressSanitizer and UndefinedBehaviorSanitizer.  Without arguments: plans
// over ordinary and extreme arguments keep inside their workspace, cover
// every position a sequence may attend to, and never overflow (exit status 0:
// every answer was as expected).  With "-": reads cases from standard input,
// one a line, and prints their plans:
//   attn bits head_dim seqs kv_heads group max_len window -> splits split_len join_waves
//   rows head_dim tokens kv_heads -> quads groups
//   rope tokens rot heads -> rounds
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../dequant_gemv_rht_amd/csrc/wq_internal.h"

namespace {

int failures = 0;
long checked = 0;

void expect(bool ok, const char *what, long long a, long long b, long long c) {
  ++checked;
  if (!ok && ++failures < 20) std::fprintf(stderr, "FAIL %s (%lld, %lld, %lld)\n", what, a, b, c);
}

void check(int bits, int d, int64_t seqs, int kv_heads, int group, int64_t max_len, int64_t window) {
  const wq::SplitPlan p = wq::attn_plan(bits, d, seqs, kv_heads, group, max_len, window);
  const int64_t qtiles = (group + 15) / 16;
  expect(p.splits >= 1 && p.split_len >= wq::kMinSplit && p.split_len % wq::kMinSplit == 0 &&
             p.split_len <= wq::kMaxSplit && p.qtiles == qtiles,
         "run", max_len, window, p.split_len);
  expect(p.groups == seqs * kv_heads * qtiles * p.splits, "split grid", seqs, max_len, p.groups);
  const int64_t rows = seqs * kv_heads * group;
  if (p.splits == 1) {
    expect(p.join_waves == 0 && p.join_groups == 0, "no join", max_len, window, p.join_groups);
  } else {
    expect(p.join_waves == 1 || p.join_waves == wq::kAttnWaves, "join", max_len, window, p.join_waves);
    expect(p.join_groups * (wq::kAttnWaves / p.join_waves) >= rows, "join grid", rows, max_len, p.join_groups);
    wq_kv_cache c;
    std::memset(&c, 0, sizeof c);
    c.bits = bits;
    c.head_dim = d;
    c.kv_heads = kv_heads;
    const unsigned __int128 bytes = (unsigned __int128)rows * p.splits * (d + 4) * sizeof(float);
    expect(bytes <= wq::attn_workspace(c, seqs, kv_heads * group, max_len, window), "workspace", seqs, max_len, window);
  }
  // the kernels' arithmetic: a sequence's runs, from the 16-token boundary
  // at or before its first position, are no more than the plan's
  const int64_t win = window < max_len ? window : 0;   // as wq_attn_decode hands it on
  for (int64_t len : {max_len, max_len - 1, max_len / 2, win, win + 1, win + 15, win + 16}) {
    if (len < 0 || len > max_len) continue;
    const int64_t begin = (win && len > win ? len - win : 0) & ~(int64_t)15;
    expect((len - begin + p.split_len - 1) / p.split_len <= p.splits, "runs", len, max_len, window);
  }
}

int query() {
  char kind[8];
  while (std::scanf("%7s", kind) == 1) {
    long long v[7];
    const int want = std::strcmp(kind, "attn") ? 3 : 7;
    for (int i = 0; i < want; ++i)
      if (std::scanf("%lld", v + i) != 1) return 2;
    if (want == 7) {
      const wq::SplitPlan p = wq::attn_plan((int)v[0], (int)v[1], v[2], (int)v[3], (int)v[4], v[5], v[6]);
      std::printf("%d %d %d\n", p.splits, p.split_len, p.join_waves);
    } else if (!std::strcmp(kind, "rope")) {
      const int32_t heads = (int32_t)v[2];
      std::printf("%d\n", wq::rope_rounds(v[0], (int)v[1], 1, &heads));
    } else {
      const wq::RowPlan p = wq::kv_row_plan((int)v[0], v[1], (int)v[2]);
      std::printf("%d %lld\n", p.quads, (long long)p.groups);
    }
  }
  return 0;
}

}  // namespace

int main(int argc, char **argv) {
  if (argc > 1) return query();
  const int64_t most = (int64_t)INT32_MAX - 16384;
  const int64_t lens[] = {0,    1,     127,   128,   129,  255,  256,   257,    1000,     4096,    5119,
                          5120, 5121, 10239, 10241, 16381, 32001, 65537, 1000003, 1 << 30, most - 1, most};
  for (int bits : {4, 8, 16})
    for (int d : {64, 128, 256})
      for (int kv_heads : {1, 2, 3, 8, 100, INT32_MAX / 256})
        for (int group : {1, 2, 8, 9, 16, 17, 40, 1000})
          for (int64_t seqs : {1LL, 2LL, 3LL, 24LL, 64LL, 513LL, 100000LL, 2147483647LL}) {
            if ((int64_t)kv_heads * group > INT32_MAX / d || seqs > (int64_t)INT32_MAX / (kv_heads * group)) continue;
            for (int64_t max_len : lens)
              for (int64_t window : {(int64_t)0, (int64_t)1, (int64_t)15, (int64_t)16, (int64_t)17, (int64_t)500,
                                     (int64_t)5000, max_len - 16, max_len - 15, max_len - 1, max_len, max_len + 1,
                                     INT64_MAX - 16, INT64_MAX - 15, INT64_MAX - 14, INT64_MAX})
                if (window >= 0) check(bits, d, seqs, kv_heads, group, max_len, window);
          }
  for (int d : {64, 128, 256})
    for (int64_t heads : {1LL, 2LL, 3LL, 8LL, 77LL, 1000000LL})
      for (int64_t tokens = 1; tokens <= INT32_MAX / 2 / heads; tokens += 1 + tokens / 3) {
        const wq::RowPlan p = wq::kv_row_plan(d, tokens, (int)heads);
        const int64_t rows = 4 * p.groups * 4 * p.quads * (d == 64 ? 2 : 1);   // of keys and values
        expect(p.quads == 1 || p.quads == wq::kv_most_quads(d), "quads", d, tokens, heads);
        expect(rows >= 2 * tokens * heads, "row grid", d, tokens, heads);
      }
  for (int rot = 16; rot <= 256; rot += 16)
    for (int heads : {1, 8, 65535})
      for (int64_t tokens : {1LL, 100LL, 33554431LL}) {
        const int32_t all[wq::kMaxBatch] = {heads, heads, heads, heads, heads, heads, heads, heads};
        const int r = wq::rope_rounds(tokens, rot, wq::kMaxBatch, all);
        expect(r == 1 || r == wq::kRopeRounds, "rope", tokens, rot, heads);
      }
  std::printf("checked %ld answers\n", checked);
  return failures ? 1 : 0;
}
