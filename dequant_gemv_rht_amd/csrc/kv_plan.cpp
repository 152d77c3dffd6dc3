// How the calls of the attention side are cut into workgroups, and the
// workspace that follows: host arithmetic only, known before any launch.
#include "wq_internal.h"

namespace wq {

namespace {

// Workgroups that a call is split into where its sequences and heads alone
// make fewer: one a CU where a row is 256 bytes or more (such a workgroup
// keeps enough bytes on the way: 42 MB of 8-bit heads of 256 take 16.8 us
// with 256 workgroups, 18.5 with 512), two a CU below that (33 MB of 4-bit
// heads of 128: 16.5 and 15.2 us; four a CU 18.6).
int64_t workgroups(int bits, int d) { return d * bits / 8 >= 256 ? 256 : 512; }

// (the window is any number up to INT64_MAX: nothing is added to it before
// it is known to be below max_len)
int64_t seen_at_most(int64_t max_len, int64_t window) {
  return window > 0 && window < max_len - 15 ? window + 15 : max_len;
}

}  // namespace

// How a call is split: enough workgroups to fill the card, in runs of one
// length from kMinSplit (a step of each wave) to kMaxSplit tokens.
// kMaxSplit: short runs cost a workgroup's start and end each and more to
// join, long ones leave uneven sequences uneven.  Time over that of the
// traffic alone, geometric means over 64 x 8 heads of 128, 4 and 8 bits, 1500
// to 16381 tokens and five batches of 40 to 128 sequences:
//   runs of at most      1024  2048  4096  8192  16384
//   up to that length    1.41  1.37  1.36  1.39  1.39
//   all of that length   1.21  1.15  1.14  1.11  1.10
// 4096, the best where lengths differ, also bounds what one long sequence
// among short ones waits for.
// kMinSplit: two runs and their join are slower than one run up to about 512
// tokens (one sequence of 8 heads, 8 bits: 256 tokens 8.9 us, 6.6 as one run;
// 512 8.9 and 7.9) and faster from 1024 (9.2 and 11.3).
SplitPlan attn_plan(int bits, int d, int64_t seqs, int kv_heads, int group, int64_t max_len, int64_t window) {
  SplitPlan p;
  p.qtiles = (group + 15) / 16;
  const int64_t seen = seen_at_most(max_len, window);
  const int64_t units = seqs * kv_heads * p.qtiles;
  const int64_t want = (workgroups(bits, d) + units - 1) / units;
  int64_t splits = (seen + kMinSplit - 1) / kMinSplit;
  if (splits > want) splits = want;
  if (splits < (seen + kMaxSplit - 1) / kMaxSplit) splits = (seen + kMaxSplit - 1) / kMaxSplit;
  if (splits < 1) splits = 1;
  int64_t len = (seen + splits - 1) / splits;   // runs of one length
  len = (len + kMinSplit - 1) / kMinSplit * kMinSplit;
  if (len < kMinSplit) len = kMinSplit;
  p.split_len = (int32_t)len;
  p.splits = (int32_t)((seen + len - 1) / len);
  if (p.splits < 1) p.splits = 1;
  p.join_waves = p.splits == 1 ? 0 : p.splits <= 64 / (d / 8) * kJoinAhead ? 1 : kAttnWaves;
  const int64_t rows = seqs * kv_heads * group;
  p.groups = units * p.splits;
  p.join_groups = p.join_waves == 1 ? (rows + kAttnWaves - 1) / kAttnWaves : p.join_waves ? rows : 0;
  return p;
}

size_t attn_workspace(const wq_kv_cache &c, int64_t seqs, int32_t q_heads, int64_t max_len, int64_t window) {
  // A bound that grows with seqs and max_len: attn_plan splits a unit (a
  // sequence and up to 16 heads) at most once for every workgroups() / units
  // units, unless runs are of kMaxSplit tokens, and makes none shorter than
  // kMinSplit.
  const int64_t seen = seen_at_most(max_len, window), heads = seqs * q_heads, group = q_heads / c.kv_heads;
  if (seen <= kMinSplit) return 0;
  const int64_t fill = heads + workgroups(c.bits, c.head_dim) * (group < 16 ? group : 16);
  const int64_t few = heads * ((seen + kMinSplit - 1) / kMinSplit), many = heads * ((seen + kMaxSplit - 1) / kMaxSplit);
  const int64_t filled = fill > many ? fill : many, rows = few < filled ? few : filled;
  return (size_t)rows * (size_t)(c.head_dim + 4) * sizeof(float);
}

RowPlan kv_row_plan(int d, int64_t tokens, int kv_heads) {
  RowPlan p;
  const int heads = d == 64 ? 2 : 1;   // heads in a wave
  auto waves = [&](int quads) {
    return (tokens + 4 * quads - 1) / (4 * quads) * ((kv_heads + heads - 1) / heads) * 2;   // keys, values
  };
  // several quads a wave once that still gives every SIMD two waves
  p.quads = waves(1) >= kManyRowWaves * kv_most_quads(d) ? kv_most_quads(d) : 1;
  p.groups = (waves(p.quads) + 3) / 4;
  return p;
}

int32_t rope_rounds(int64_t tokens, int32_t rot, int32_t count, const int32_t *heads) {
  constexpr int64_t kManyWaves = 8192;   // 8 a SIMD
  const int32_t slots = 64 / (rot / 16);
  int64_t waves = 0;   // with one round each
  for (int32_t i = 0; i < count; ++i) waves += tokens * ((heads[i] + (int64_t)slots - 1) / slots);
  return waves >= kManyWaves ? kRopeRounds : 1;
}

}  // namespace wq
