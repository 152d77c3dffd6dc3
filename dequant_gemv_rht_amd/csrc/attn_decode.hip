// Attention of one new token per sequence over a paged, coded key-value
// cache (gfx950):  out = R^T sum_t softmax_t(scale (R q).k_t) v_t.
//
// A workgroup takes one (sequence, key-value head) and a run of its tokens
// (a split); its four waves take 32 tokens at a time in turn, each with its
// own running softmax, and join in LDS at the end.  Where a sequence has
// more than one split, the splits' sums go to the workspace and a second
// kernel joins them.
//
// Both products run on the matrix cores with the tokens' side as the first
// operand, so that the query heads that share the key-value head (padded to
// 16) are the columns everywhere:
//   S^T = K Q^T   16 tokens x 16 heads per v_mfma_f32_16x16x32_f16
//   O^T = V^T P^T 16 channels x 16 heads, 32 tokens deep
// A lane then holds scores of one head (its column) for tokens 4 g + i of
// each 16 (g = lane / 16), which is what the second product wants of P as
// its own operand, in the token order {4 g + i, 16 + 4 g + i}: the weights
// never leave their lane.  The cache's layout gives V in that order (quads
// of tokens side by side) and K as panels, both in whole 16-byte loads.
//
// Codes enter the products as they are: 16 bits whose value c is below 2^10
// are fp16's subnormal c 2^-24, which the matrix instructions take without
// loss, so 8-bit codes only have their bytes spread and 4-bit codes are
// masked out of their words.  Zeros come off in fp32, after the products:
//   s (dot(q, c) - z sum(q))   and   sum(w c) - sum(w z).
// The instructions line terms up by their exponents, a subnormal's being
// that of 2^10 codes, and cut them 24 bits or so below the largest; 4-bit
// values are therefore all brought to the upper half of a byte, as 16 c
// (left as c, half of the channels were off by 5e-4 of 16000 tokens' sum,
// now by 2.3e-4 as the others).  Keys' scores do not need that: their lower
// nibbles have sums of their own, taken 16-fold.
// The values' scale goes into the weight, p s, before it is rounded to
// fp16; the running reference m therefore tracks max(u + log2 |s|), so that
// p s of the largest term stays near 2^kGain and weights down to 2^-20 of
// it keep fp16's 11 bits whatever the scales are.  m moves only when a term
// exceeds 2^kSlack above it, which after the first steps is rare: the
// cross-lane maximum and the rescaling of the sums run only then.
//
// What bounds it: traffic where there is enough of it (64 sequences of 16381
// tokens, 8 key-value heads of 128, 8 bits: 2.21 GB in 339 us, 6.5 TB/s,
// what a plain read reaches); the longest sequences' last workgroups in a
// ragged batch (64 up to 4099 tokens, 4 bits: 146 MB in 38 us); the way from
// the arguments over page table and cache to the join for few tokens (77
// tokens: 5.6 us, an empty kernel 2.2).  A step of 128 tokens takes a
// workgroup 0.76 us with 4 bits and 1.3 us with 8 where three share a CU.
// Three waves a SIMD with one set of registers for the codes, asked for
// again as soon as a half is used, were faster than two waves with two sets
// (64 ragged sequences: 42.6 against 63 us), and four spill (64 of 16384
// tokens, 4 bits: 206 against 195 us).
#include "wq_internal.h"

#include <cmath>

namespace wq {
using namespace dev;

namespace {

typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef const __attribute__((address_space(4))) int32_t *const_i32;   // scalar loads

constexpr int kWaves = kAttnWaves, kAttnThreads = 64 * kWaves, kStep = kAttnStep;
constexpr float kInvSqrt128 = 0.08838834764831845f;
constexpr float kNone = -1e30f;      // no term seen yet
constexpr int kGain = 8, kSlack = 6; // 2^(kGain + kSlack) < 65504
constexpr int kQueryTop = 15;        // a rotated query's largest value is 2^14 to 2^15
constexpr float kMaxSum = 8.0f * (float)(1ull << (kGain + kSlack + 24));   // of a lane's 8 weights before the values' scales

// waves per SIMD that the registers are kept for without spilling
constexpr int occupancy(int bits, int d, bool low) {
  return d <= 128 ? (low ? 2 : 3) : bits == 16 || low ? 1 : 2;
}

template <int BITS, int D>
struct Fmt {
  static constexpr int kRow = D * BITS / 8;        // bytes of a row
  static constexpr int kWords = kRow / 16;         // 32-bit words a lane holds of 16 tokens (keys; values)
  static constexpr int kPiece = kWords < 4 ? kWords : 4;   // words per load
  static constexpr int kKeyMfma = D / 32, kOutMfma = D / 16;
  static constexpr float kUnit = BITS == 16 ? 1.0f : BITS == 8 ? 0x1p24f : 0x1p20f;   // 1 / a code of 1 in the products
  // first of the 8 channels of key operand m (4 bits: of word m) in lane group g
  __device__ static constexpr int key_channel(int m, int g) {
    if (BITS == 16) return 32 * m + 8 * g;
    if (BITS == 8) return 64 * (m >> 1) + 16 * g + 8 * (m & 1);
    return D == 64 ? 16 * g + 8 * m : 128 * (m >> 2) + 32 * g + 8 * (m & 3);
  }
  // the channel of output row r = 4 g + i of product n
  __device__ static constexpr int out_channel(int n, int r) {
    if (BITS == 16) return 32 * (n >> 1) + 2 * r + (n & 1);
    if (BITS == 8) return 64 * (n >> 2) + 4 * r + (n & 3);
    return D == 64 ? 4 * r + n : 128 * (n >> 3) + 8 * r + (n & 7);
  }
};

// What a lane holds of 32 tokens: keys or values, and their (scale, zero) pairs.
template <int BITS, int D>
struct Side {
  uint32_t w[2][Fmt<BITS, D>::kWords];
  u32x4 par[2];
};

__device__ __forceinline__ half2_t as_half2(uint32_t w) { return __builtin_bit_cast(half2_t, w); }
__device__ __forceinline__ uint32_t as_u32(half2_t h) { return __builtin_bit_cast(uint32_t, h); }
struct Quad {
  uint32_t w[4];
};
__device__ __forceinline__ half8_t as_half8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(half8_t, Quad{{a, b, c, d}});
}

__device__ __forceinline__ uint32_t bytes01(uint32_t w) { return __builtin_amdgcn_perm(w, w, 0x0C010C00u); }
__device__ __forceinline__ uint32_t bytes23(uint32_t w) { return __builtin_amdgcn_perm(w, w, 0x0C030C02u); }
constexpr uint32_t kLowNibbles = 0x000F000Fu, kHighNibbles = 0x00F000F0u;

// Key operand m of a block.  4 bits: the lower (even m) or upper nibbles of
// words m & ~1 and the next, in channel order 0, 4, 2, 6 (1, 5, 3, 7) of
// each.
template <int BITS, int D>
__device__ __forceinline__ half8_t key_operand(const uint32_t (&k)[Fmt<BITS, D>::kWords], int m) {
  if constexpr (BITS == 16) {
    return as_half8(k[4 * m], k[4 * m + 1], k[4 * m + 2], k[4 * m + 3]);
  } else if constexpr (BITS == 8) {
    return as_half8(bytes01(k[2 * m]), bytes23(k[2 * m]), bytes01(k[2 * m + 1]), bytes23(k[2 * m + 1]));
  } else {
    const uint32_t a = k[m & ~1], b = k[m | 1], mask = m & 1 ? kHighNibbles : kLowNibbles;
    return as_half8(a & mask, (a >> 8) & mask, b & mask, (b >> 8) & mask);
  }
}

// A maximum over the four lanes that share a column (head).
__device__ __forceinline__ float column_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float column_sum(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// A maximum of positive numbers over the D / 8 lanes of a row.
template <int D>
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp<kQuadXor1>(v));
  v = fmaxf(v, dpp<kQuadXor2>(v));
  v = fmaxf(v, dpp<kRowHalfMirror>(v));
  v = fmaxf(v, dpp<kRowMirror>(v));
  return D == 256 ? fmaxf(v, __shfl_xor(v, 16)) : v;
}

template <int BITS>
__device__ __forceinline__ uint4 pack_query(const float (&v)[8]) {
  if (BITS == 4)
    return make_uint4(pack_half2(v[0], v[4]), pack_half2(v[2], v[6]), pack_half2(v[1], v[5]), pack_half2(v[3], v[7]));
  return make_uint4(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]), pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
}

// One row's 8 channels in a 16-lane DPP row, rotated back and stored.
template <int D>
__device__ __forceinline__ void store_row(const AttnArgs &a, float (&v)[8], int64_t seq, uint32_t sb, int head, int c0) {
  if (D >= 128 && a.signs) {
    const int jj = threadIdx.x & 15;
    fwht128_row16_signed(v, jj);
    const float sc = fwht_lane_sign(jj) * kInvSqrt128;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= ((sb >> e) & 1u) ? -sc : sc;
  }
  *reinterpret_cast<uint4 *>(a.out + seq * a.ldo + (int64_t)head * D + c0) =
      make_uint4(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]), pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
}

// The positions a sequence attends to, from the last 16-token boundary at
// or before the first one.
struct Range {
  int start, begin, len;
  __device__ int splits(int split_len) const { return len > begin ? (len - begin + split_len - 1) / split_len : 0; }
};
__device__ __forceinline__ Range range_of(const AttnArgs &a, int64_t seq) {
  Range r;
  r.len = min(((const_i32)a.lens)[seq], a.max_len);
  r.start = a.window && r.len > a.window ? r.len - a.window : 0;
  r.begin = r.start & ~15;
  return r;
}

// LOW: the low parts of rotated queries are operands of their own (more than
// 8 heads, no columns left for them).
template <int BITS, int D, bool LOW>
__global__ __launch_bounds__(kAttnThreads, occupancy(BITS, D, LOW)) void attn_split_kernel(AttnArgs a, SplitPlan plan) {
  using F = Fmt<BITS, D>;
  constexpr int kQStride = D + 8, kOStride = D + 4;
  __shared__ union {
    _Float16 q[LOW ? 32 : 16][kQStride];
    float o[kWaves][16][kOStride];
  } sh;
  __shared__ float sh_m[kWaves][16], sh_l[kWaves][16], sh_unit[16];

  int id = blockIdx.x;
  // the sequences' first splits first: the empty ones of short sequences last
  const int kvh = id % a.kv_heads;
  id /= a.kv_heads;
  const int qt = id % plan.qtiles;
  id /= plan.qtiles;
  const int64_t seq = id % (int)a.seqs;
  const int split = id / (int)a.seqs;
  const int head0 = kvh * a.group + 16 * qt, heads = min(16, a.group - 16 * qt);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, g = lane >> 4;

  // The chain to the first scores is: launch arguments, then the length,
  // the first pages and the queries at once, then the first keys and
  // values, which travel while the queries are prepared.
  constexpr int kRows = 16 * (D / 8), kPasses = (kRows + kAttnThreads - 1) / kAttnThreads;
  uint4 raw[kPasses];
  const int ch = kvh * D + 8 * (tid % (D / 8));   // this thread's channels in every pass
  const uint32_t flips = D >= 128 && a.signs ? a.signs[ch >> 5] : 0u;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int h = (tid + i * kAttnThreads) / (D / 8), c0 = 8 * (tid % (D / 8));
    raw[i] = make_uint4(0, 0, 0, 0);
    if (h < heads) raw[i] = *reinterpret_cast<const uint4 *>(a.q + seq * a.ldq + (int64_t)(head0 + h) * D + c0);
  }
  const_i32 table = (const_i32)(a.table + seq * a.ld_table);
  const int page_mask = (1 << a.page_shift) - 1;
  // the table's entry for the 16 tokens from t, not yet looked at (the
  // scalar load is waited for where it is); past max_len any entry
  auto entry_at = [&](int t) -> int { return table[max(min(t, a.max_len - 1), 0) >> a.page_shift]; };
  const Range rg = range_of(a, seq);
  const int begin = (a.window ? rg.begin : 0) + split * plan.split_len;
  int t = begin + wave * kStep;
  int e0 = 0, e1 = 0;
  if (a.max_len > 0) {
    e0 = entry_at(t);
    e1 = entry_at(t + 16);
  }
  const int my_splits = rg.splits(plan.split_len);
  if (split >= my_splits && split > 0) return;
  const int end = min(begin + plan.split_len, rg.len);   // at or below begin: nothing to attend to

  const char *kbase = static_cast<const char *>(a.k), *vbase = static_cast<const char *>(a.v);
  const int k_lane = F::kRow >= 64 ? col * 64 + g * 16 : col * 32 + g * 8;
  const int v_lane = g * 4 * F::kRow + col * 4 * F::kPiece;
  auto takes_part = [&](int t, int entry) { return t < end && (uint32_t)entry < (uint32_t)a.pages; };
  // 16 tokens that take no part get empty resources: their loads return
  // zeros without touching memory, so every load is issued unconditionally
  auto load = [&](Side<BITS, D> &s, const char *base, const uint32_t *params, int at, int stride, int t, int e0, int e1) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int e = b ? e1 : e0;
      const bool ok = takes_part(t + 16 * b, e);
      const int64_t token = (((int64_t)(ok ? e : 0) * a.kv_heads + kvh) << a.page_shift) + ((t + 16 * b) & page_mask);
      const rsrc_t rs = make_rsrc(base + token * F::kRow, ok ? 16 * F::kRow : 0);
#pragma unroll
      for (int i = 0; i < F::kWords / F::kPiece; ++i) {
        if constexpr (F::kPiece == 4) {
          const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rs, at + i * stride, 0, kNT);
#pragma unroll
          for (int x = 0; x < 4; ++x) s.w[b][4 * i + x] = v[x];
        } else {
          const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(rs, at, 0, kNT);
          s.w[b][0] = v[0]; s.w[b][1] = v[1];
        }
      }
      if constexpr (BITS != 16)
        s.par[b] = __builtin_amdgcn_raw_buffer_load_b128(make_rsrc(params + token, ok ? 64 : 0), 16 * g, 0, kNT);
    }
  };
  auto load_k = [&](Side<BITS, D> &s, int t, int e0, int e1) { load(s, kbase, a.k_params, k_lane, 1024, t, e0, e1); };
  auto load_v = [&](Side<BITS, D> &s, int t, int e0, int e1) { load(s, vbase, a.v_params, v_lane, 256, t, e0, e1); };

  constexpr int kStride = kWaves * kStep;
  Side<BITS, D> ks, vs;
  int n0 = 0, n1 = 0;
  if (t < end) {
    load_k(ks, t, e0, e1);
    load_v(vs, t, e0, e1);
    n0 = entry_at(t + kStride);
    n1 = entry_at(t + kStride + 16);
  }

  // The queries, rotated as the cache is, rounded to fp16, in the keys'
  // channel order.  A rotated query is no longer an fp16 value: each head is
  // brought to 2^kQueryTop by a power of two (rotated it may be past fp16's
  // largest number, or need bits below its smallest), what the rounding
  // leaves goes to columns 8 to 15 where there are at most 8 heads, else to
  // operands of its own, and its scores are added to the heads' own.
  const bool split_q = !LOW && D >= 128 && a.signs && heads <= 8;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int h = (tid + i * kAttnThreads) / (D / 8), c0 = 8 * (tid % (D / 8));
    if (kRows < kAttnThreads && h >= 16) break;
    float v[8];
    v[0] = half_bits_to_float(raw[i].x & 0xFFFF); v[1] = half_bits_to_float(raw[i].x >> 16);
    v[2] = half_bits_to_float(raw[i].y & 0xFFFF); v[3] = half_bits_to_float(raw[i].y >> 16);
    v[4] = half_bits_to_float(raw[i].z & 0xFFFF); v[5] = half_bits_to_float(raw[i].z >> 16);
    v[6] = half_bits_to_float(raw[i].w & 0xFFFF); v[7] = half_bits_to_float(raw[i].w >> 16);
    if (D >= 128 && a.signs) {
      const int jj = tid & 15;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = ((flips >> ((ch + e) & 31)) & 1u) ? -v[e] : v[e];
      fwht128_row16_signed(v, jj);
      float top = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
      const int shift = kQueryTop - __builtin_amdgcn_frexp_expf(row_max<D>(top) * kInvSqrt128);
      if (c0 == 0) sh_unit[h] = ldexpf(1.0f, -shift);
      const float sc = ldexpf(fwht_lane_sign(jj) * kInvSqrt128, shift);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= sc;
    }
    const uint4 w = pack_query<BITS>(v);
    if (split_q && h >= 8) continue;
    *reinterpret_cast<uint4 *>(&sh.q[h][c0]) = w;
    if (split_q || LOW) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] -= (float)(_Float16)v[e];
      *reinterpret_cast<uint4 *>(&sh.q[h + (LOW ? 16 : 8)][c0]) = pack_query<BITS>(v);
    }
  }
  __syncthreads();
  half8_t q[F::kKeyMfma], ql[LOW ? F::kKeyMfma : 1];
  float qsum = 0.0f;
  auto operand = [&](int row, int m) {
    half8_t h;
    if constexpr (BITS == 4) {
      const half4_t a = *reinterpret_cast<const half4_t *>(&sh.q[row][F::key_channel(m & ~1, g) + 4 * (m & 1)]);
      const half4_t b = *reinterpret_cast<const half4_t *>(&sh.q[row][F::key_channel(m | 1, g) + 4 * (m & 1)]);
      h = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      h = *reinterpret_cast<const half8_t *>(&sh.q[row][F::key_channel(m, g)]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) qsum += (float)h[e];
    return h;
  };
#pragma unroll
  for (int m = 0; m < F::kKeyMfma; ++m) {
    q[m] = operand(col, m);
    if constexpr (LOW) ql[m] = operand(16 + col, m);
  }
  qsum = column_sum(qsum);
  const float unit = D >= 128 && a.signs ? sh_unit[split_q ? col & 7 : col] : 1.0f;
  __syncthreads();   // sh.q is free for sh.o

  float m = kNone, l = 0.0f, lz = 0.0f;   // lz: sum of w z
  f32x4 o[F::kOutMfma];
#pragma unroll
  for (int n = 0; n < F::kOutMfma; ++n) o[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  const float to_log2 = a.scale * 1.4426950408889634f * F::kUnit * unit, zero_sum = -qsum / F::kUnit;
  for (; t < end; t += kStride) {
    // scores before the keys' scale, in units of log2
    float x[8];
    uint32_t kp[4];   // the keys' scales, two to a word
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f}, low = acc;   // low: 4 bits' lower nibbles
      if constexpr (BITS != 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = (float)as_half2(ks.par[b][i])[1] * zero_sum;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          kp[2 * b + i] = __builtin_amdgcn_perm(ks.par[b][2 * i + 1], ks.par[b][2 * i], 0x05040100u);
          // here, and not where it is used: the pairs' registers are about to be loaded again
          asm volatile("" : "+v"(kp[2 * b + i]));
        }
      }
#pragma unroll
      for (int mm = 0; mm < F::kKeyMfma; ++mm) {
        const half8_t k = key_operand<BITS, D>(ks.w[b], mm);
        f32x4 &sum = BITS == 4 && mm % 2 == 0 ? low : acc;
        sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[mm], sum, 0, 0, 0);
        if constexpr (LOW) sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, ql[mm], sum, 0, 0, 0);
      }
      if constexpr (BITS == 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(low[i], 16.0f, acc[i]);
      if (split_q) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += dpp<kRowRor8>(acc[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[4 * b + i] = acc[i] * to_log2;
    }
    __builtin_amdgcn_sched_barrier(0);
    load_k(ks, t + kStride, n0, n1);
    const int f0 = entry_at(t + 2 * kStride), f1 = entry_at(t + 2 * kStride + 16);
    __builtin_amdgcn_sched_barrier(0);
    // the first and the last step of a sequence, pages outside the cache
    const bool in0 = takes_part(t, e0), in1 = takes_part(t + 16, e1);
    if (t < rg.start || t + kStep > end || !in0 || !in1) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        bool ok[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = t + 16 * b + 4 * g + i;
          ok[i] = at >= rg.start && at < end && (b ? in1 : in0);
          x[4 * b + i] = ok[i] ? x[4 * b + i] : -INFINITY;
          if (BITS != 16) {
            // keys: scale 1 (a NaN there must not undo the mask); values: scale and zero 0
            const uint32_t half = 0xFFFFu << (16 * (i & 1));
            kp[2 * b + (i >> 1)] = ok[i] ? kp[2 * b + (i >> 1)] : (kp[2 * b + (i >> 1)] & ~half) | (0x3C003C00u & half);
            vs.par[b][i] = ok[i] ? vs.par[b][i] : 0u;
          }
        }
        if constexpr (BITS == 16) {
          const uint32_t lo = (ok[0] ? 0xFFFFu : 0u) | (ok[1] ? 0xFFFF0000u : 0u);
          const uint32_t hi = (ok[2] ? 0xFFFFu : 0u) | (ok[3] ? 0xFFFF0000u : 0u);
#pragma unroll
          for (int i = 0; i < F::kWords; ++i) vs.w[b][i] &= (i & 1) ? hi : lo;
        }
      }
    }
    // p = 2^(u - m), w = fp16(p s); both from one fused step each
    float p[8];
    _Float16 w[8];
    auto weigh = [&]() {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = __builtin_amdgcn_exp2f(BITS == 16 ? x[i] - m : fmaf((float)as_half2(kp[i >> 1])[i & 1], x[i], -m));
        w[i] = BITS == 16 ? (_Float16)p[i] : (_Float16)fmaf(p[i], (float)as_half2(vs.par[i >> 2][i & 3])[0], 0.0f);
      }
    };
    weigh();
    // (absolute values: a scale may be negative)
    _Float16 top = __builtin_fabsf16(w[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) top = __builtin_fmaxf16(top, __builtin_fabsf16(w[i]));
    float sum = ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
    // (the sum: rows of scale 0 do not show in the w.  Other scales are 2^-24
    // or more, so while the w are in range the other rows' p stay below
    // 2^(kGain + kSlack + 24); a larger sum is theirs and moves the reference
    // too, so that no number of them makes l infinite)
    if (__any(!(top <= (_Float16)(1 << (kGain + kSlack))) || !(sum <= kMaxSum))) {
      // move the reference: the largest term so far becomes 2^kGain (2^-24:
      // the smallest positive scale, so that rows of scale 0 do not leave
      // it unset)
      float high = m + (float)kGain;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        high = fmaxf(high, BITS == 16 ? x[i]
                                      : (float)as_half2(kp[i >> 1])[i & 1] * x[i] +
                                            fmaxf(__builtin_amdgcn_logf(fabsf((float)as_half2(vs.par[i >> 2][i & 3])[0])), -24.0f));
      high = column_max(high) - (float)kGain;
      const float keep = __builtin_amdgcn_exp2f(m - high);
      m = high;
      l *= keep;
      lz *= keep;
#pragma unroll
      for (int n = 0; n < F::kOutMfma; ++n) o[n] *= keep;
      weigh();
      sum = ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
    }
    l += sum;
    // weights as the second operand, in the values' token order: 4-bit
    // codes of tokens 0, 2 and 1, 3 come out of a word together
    constexpr int o1 = BITS == 4 ? 2 : 1, o2 = BITS == 4 ? 1 : 2;
    const half8_t pw = {w[0], w[o1], w[o2], w[3], w[4], w[4 + o1], w[4 + o2], w[7]};
    if constexpr (BITS != 16)
#pragma unroll
      for (int i = 0; i < 8; ++i) lz = fmaf((float)w[i], (float)as_half2(vs.par[i >> 2][i & 3])[1], lz);
    if constexpr (BITS == 16) {
#pragma unroll
      for (int n = 0; n < F::kOutMfma; ++n)
        o[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
            as_half8(vs.w[0][2 * n], vs.w[0][2 * n + 1], vs.w[1][2 * n], vs.w[1][2 * n + 1]), pw, o[n], 0, 0, 0);
    } else if constexpr (BITS == 8) {
#pragma unroll
      for (int n = 0; n < F::kOutMfma; ++n)
        o[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
            as_half8(bytes01(vs.w[0][n]), bytes23(vs.w[0][n]), bytes01(vs.w[1][n]), bytes23(vs.w[1][n])), pw, o[n], 0, 0, 0);
    } else {
#pragma unroll
      for (int n = 0; n < F::kOutMfma; ++n) {
        const uint32_t a = vs.w[0][n / 2], b = vs.w[1][n / 2], m = kHighNibbles;
        o[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
            n & 1 ? as_half8(a & m, (a >> 8) & m, b & m, (b >> 8) & m)
                  : as_half8((a << 4) & m, (a >> 4) & m, (b << 4) & m, (b >> 4) & m), pw, o[n], 0, 0, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    load_v(vs, t + kStride, n0, n1);
    e0 = n0; e1 = n1;
    n0 = f0; n1 = f1;
  }

  // join the four waves
  l = column_sum(l);
  lz = column_sum(lz);
  if (g == 0) {
    sh_m[wave][col] = m;
    sh_l[wave][col] = l;
  }
  if (col < heads) {
#pragma unroll
    for (int n = 0; n < F::kOutMfma; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) sh.o[wave][col][F::out_channel(n, 4 * g + i)] = fmaf(o[n][i], F::kUnit, -lz);
  }
  __syncthreads();
  for (int i = tid; i < heads * (D / 8); i += kAttnThreads) {
    const int h = i / (D / 8), c0 = 8 * (i % (D / 8)), head = head0 + h;
    float high = sh_m[0][h];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) high = fmaxf(high, sh_m[w][h]);
    float total = 0.0f, v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(sh_m[w][h] - high);
      total += f * sh_l[w][h];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += f * sh.o[w][h][c0 + e];
    }
    if (my_splits <= 1) {
      const float inv = total > 0.0f || total != total ? 1.0f / total : 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= inv;
      store_row<D>(a, v, seq, flips >> (ch & 31), head, c0);
    } else {
      const int64_t at = ((seq * a.kv_heads * a.group + head) * plan.splits + split);
      float *part = a.partial + at * (D + 4);
      f32x4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
      *reinterpret_cast<f32x4 *>(part + 4 + c0) = lo;
      *reinterpret_cast<f32x4 *>(part + 8 + c0) = hi;
      if (c0 == 0) {
        part[0] = high;
        part[1] = total;
      }
    }
  }
}

// Joins the splits of a (sequence, head).  D / 8 lanes x 8 channels hold a
// split's sum, so a wave takes 64 / (D / 8) splits at a time, and each lane
// asks for kAhead of them before it looks at the first: the kernel is one
// round trip to the partial sums long.  HW waves share a head: one where it
// holds all the plan's splits that way, else four that meet in LDS.  Latency
// bound: 3.9 us for 63 splits of 32 heads (0.6 MB) as for 8 of 256, about 2
// of it what any kernel takes.
constexpr int kAhead = kJoinAhead;
template <int D, int HW>
__global__ __launch_bounds__(kAttnThreads) void attn_join_kernel(AttnArgs a, SplitPlan plan) {
  constexpr int kLanes = D / 8, kParts = 64 * HW / kLanes;
  __shared__ float sh[kWaves][D + 4], sh_m[kWaves], sh_l[kWaves];
  const int all = a.kv_heads * a.group;
  const int tid = threadIdx.x, wave = tid >> 6;
  const int64_t id = HW == 1 ? (int64_t)blockIdx.x * kWaves + wave : blockIdx.x;
  if (id >= a.seqs * all) return;
  const int head = (int)(id % all);
  const int64_t seq = id / all;
  const int part = (tid & (64 * HW - 1)) / kLanes, c0 = 8 * (tid % kLanes);
  const int ch = head / a.group * D + c0;
  const uint32_t flips = D >= 128 && a.signs ? a.signs[ch >> 5] : 0u;
  const float *in = a.partial + id * plan.splits * (D + 4);
  const int n = range_of(a, seq).splits(plan.split_len);
  float m = kNone, l = 0.0f, v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  for (int s0 = part; s0 < plan.splits; s0 += kParts * kAhead) {
    f32x4 lo[kAhead], hi[kAhead];
    float ms[kAhead], ls[kAhead];
    // up to the plan's splits: inside the workspace, whatever n turns out to be
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int s = min(s0 + i * kParts, plan.splits - 1);
      const float *p = in + (int64_t)s * (D + 4);
      ms[i] = p[0];
      ls[i] = p[1];
      lo[i] = *reinterpret_cast<const f32x4 *>(p + 4 + c0);
      hi[i] = *reinterpret_cast<const f32x4 *>(p + 8 + c0);
    }
    if (n <= 1) return;   // written by its one workgroup
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (s0 + i * kParts >= n) continue;
      const float high = fmaxf(m, ms[i]);
      const float f = __builtin_amdgcn_exp2f(m - high), fs = __builtin_amdgcn_exp2f(ms[i] - high);
      m = high;
      l = l * f + ls[i] * fs;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = v[e] * f + lo[i][e] * fs;
        v[e + 4] = v[e + 4] * f + hi[i][e] * fs;
      }
    }
    if (s0 - part + kParts * kAhead >= n) break;
  }
  if (n <= 1) return;
#pragma unroll
  for (int o = kLanes; o < 64; o <<= 1) {
    const float mo = __shfl_xor(m, o), lx = __shfl_xor(l, o), high = fmaxf(m, mo);
    const float f = __builtin_amdgcn_exp2f(m - high), fo = __builtin_amdgcn_exp2f(mo - high);
    m = high;
    l = l * f + lx * fo;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] * f + __shfl_xor(v[e], o) * fo;
  }
  if (HW > 1) {
    if ((tid & 63) < kLanes) {
      if (c0 == 0) {
        sh_m[wave] = m;
        sh_l[wave] = l;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sh[wave][c0 + e] = v[e];
    }
    __syncthreads();
    m = kNone;
    l = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) m = fmaxf(m, sh_m[i]);
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      const float f = __builtin_amdgcn_exp2f(sh_m[i] - m);
      l += f * sh_l[i];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += f * sh[i][c0 + e];
    }
  }
  if ((tid & (64 * HW - 1)) >= kLanes) return;
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= inv;
  store_row<D>(a, v, seq, flips >> (ch & 31), head, c0);
}

// (the caller has checked that both grids fit a launch)
template <int BITS, int D>
hipError_t launch(const AttnArgs &a, const SplitPlan &p, hipStream_t s) {
  const dim3 grid((unsigned)p.groups), block(kAttnThreads);
  if constexpr (D >= 128) {
    if (a.signs && a.group > 8)
      hipLaunchKernelGGL((attn_split_kernel<BITS, D, true>), grid, block, 0, s, a, p);
    else
      hipLaunchKernelGGL((attn_split_kernel<BITS, D, false>), grid, block, 0, s, a, p);
  } else {
    hipLaunchKernelGGL((attn_split_kernel<BITS, D, false>), grid, block, 0, s, a, p);
  }
  if (p.join_waves == 1)
    hipLaunchKernelGGL((attn_join_kernel<D, 1>), dim3((unsigned)p.join_groups), block, 0, s, a, p);
  else if (p.join_waves)
    hipLaunchKernelGGL((attn_join_kernel<D, kWaves>), dim3((unsigned)p.join_groups), block, 0, s, a, p);
  return hipGetLastError();
}

template <int BITS>
hipError_t launch_bits(int d, const AttnArgs &a, const SplitPlan &p, hipStream_t s) {
  switch (d) {
    case 64: return launch<BITS, 64>(a, p, s);
    case 128: return launch<BITS, 128>(a, p, s);
    case 256: return launch<BITS, 256>(a, p, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_attn_decode(int bits, int head_dim, const AttnArgs &a, const SplitPlan &p, hipStream_t s) {
  switch (bits) {
    case 4: return launch_bits<4>(head_dim, a, p, s);
    case 8: return launch_bits<8>(head_dim, a, p, s);
    case 16: return launch_bits<16>(head_dim, a, p, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace wq
