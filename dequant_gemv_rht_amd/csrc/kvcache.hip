// The paged key-value cache: new rows coded as they are written, and read
// back (gfx950).  Layouts and rules: include/wq.h.
//
// A wave takes four tokens of one head (two heads of 64 channels), keys or
// values: lane 16 t + c holds 8 channels of token t (two sets of 8 for 256),
// so a 128-block is the 16 lanes of a DPP row and its rotation is
// fwht128_row16_signed.  Everything is fp32, in the order the definition
// gives it; no product feeds a sum, so no fused multiply-add can change a
// code.
//
// Values lie in quads, the four tokens of a channel side by side.  Where the
// four tokens fill a quad, the wave transposes it in registers (the two
// lane swaps of gfx950) and moves it in whole 4- to 16-byte pieces;
// otherwise, as in a decode step, each token's units go one by one.  The
// tokens' slots may start anywhere in a quad, so waves look for quads among
// the slots rather than at multiples of four.
//
// What bounds it: vector instructions when coding (about 190 for 8 channels
// of a lane, one every 4 cycles on every SIMD: 8191 tokens of 8 heads of 128
// to 8 bits move 51 MB in 17 us, 3 TB/s), so whatever does not depend on the
// token is kept out of the loop over a wave's quads: the signs, the lane's
// offsets, the head (22 us before).  Reading takes about 110 and meets the
// traffic: the same tokens back in 11.9 us, 30011 tokens from 4 bits (156 MB)
// in 31, 5 TB/s.  Few tokens are launch bound: 64 tokens 3.5 us either way.
#include "wq_internal.h"

namespace wq {
using namespace dev;

namespace {

constexpr int kRowThreads = 256;
constexpr float kInvSqrt128 = 0.08838834764831845f;

// unit u of token t of a block of 16 (keys) / a quad of 4 (values)
template <int BITS, int D>
struct Layout {
  static constexpr int kUnits = BITS == 4 ? D / 2 : D;          // units of a row
  static constexpr int kUnitBytes = BITS == 16 ? 2 : 1;
  static constexpr int kPanel = kUnits * kUnitBytes < 64 ? kUnits : 64 / kUnitBytes;   // units
  static constexpr int kSets = D == 256 ? 2 : 1;                // sets of 8 channels in a lane
  static constexpr int kHeads = D == 64 ? 2 : 1;                // heads in a wave
  static constexpr int kWords = 8 * BITS / 32;                  // 32-bit words of 8 channels
  __device__ static int64_t key_unit(int t, int u) {
    return (int64_t)(t >> 4) * 16 * kUnits + (u / kPanel) * 16 * kPanel + (t & 15) * kPanel + u % kPanel;
  }
  __device__ static int64_t value_unit(int t, int u) { return (int64_t)(t >> 2) * 4 * kUnits + 4 * u + (t & 3); }
};

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_bits(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

// The extreme of numbers of one sign over the 16 lanes of a DPP row, or (D =
// 64) each 8 of them, by their bits: T int32_t, the largest of positive
// ones; uint32_t, the smallest of negative ones (zeros of either sign among
// them lose).  One instruction a step, where floats take three.
template <int D, class T>
__device__ __forceinline__ float row_extreme(float f) {
  T v = __builtin_bit_cast(T, f);
  v = max(v, (T)dpp_bits<kQuadXor1>((uint32_t)v));
  v = max(v, (T)dpp_bits<kQuadXor2>((uint32_t)v));
  v = max(v, (T)dpp_bits<kRowHalfMirror>((uint32_t)v));
  if (D != 64) v = max(v, (T)dpp_bits<kRowMirror>((uint32_t)v));
  return __builtin_bit_cast(float, v);
}

__device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b) {   // a's upper 32 lanes with b's lower 32
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b) {   // a's odd rows of 16 with b's even rows
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ uint32_t bytes(uint32_t hi, uint32_t lo, uint32_t sel) {
  return __builtin_amdgcn_perm(hi, lo, sel);
}

__device__ __forceinline__ half2_t as_half2(uint32_t w) { return __builtin_bit_cast(half2_t, w); }

// 8 codes less their zero, as pairs (2 i, 2 i + 1) of fp16: whole numbers,
// exact (0x6400 | c is 1024 + c).
template <int BITS>
__device__ __forceinline__ void codes_to_pairs(const uint32_t (&w)[8 * BITS / 32], _Float16 z, half2_t (&p)[4]) {
  const half2_t bias = half2_t{(_Float16)1024.0f, (_Float16)1024.0f} + half2_t{z, z};
  if constexpr (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = as_half2(bytes(0x64646464u, w[i / 2], i & 1 ? 0x04030402u : 0x04010400u)) - bias;
  } else {
    const uint32_t even = w[0] & 0x0F0F0F0Fu, odd = (w[0] >> 4) & 0x0F0F0F0Fu;   // channels 0, 2, 4, 6 and 1, 3, 5, 7
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = as_half2(bytes(odd, even, 0x0C000C00u + 0x00040000u + 0x00010001u * i) | 0x64006400u) - bias;
  }
}

template <int BITS>
__device__ __forceinline__ void codes_to_float(const uint32_t (&w)[8 * BITS / 32], _Float16 z, float (&v)[8]) {
  half2_t p[4];
  if constexpr (BITS == 16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = as_half2(w[i]);
  } else {
    codes_to_pairs<BITS>(w, z, p);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)p[e / 2][e & 1];
}

// One butterfly stage between lanes on pairs of fp16: partner + beta * mine
template <int CTRL>
__device__ __forceinline__ void pair_stage(half2_t (&p)[4], half2_t beta) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t mine = __builtin_bit_cast(uint32_t, p[i]);
    uint32_t other = dpp_bits<CTRL>(mine);
    if (CTRL == kRowHalfMirror) other = dpp_bits<kQuadRev>(other);   // lane ^ 4
    p[i] = __builtin_elementwise_fma(p[i], beta, as_half2(other));
  }
}

// The 128-point transform of code - zero (fp16 values for 16 bits); 8 and 16
// bits times (-1)^popcount(lane), which fwht128_row16_signed leaves to the
// caller's scale (lane_sign below).  Sums of whole
// numbers stay whole: up to 2048 they are exact in fp16 pairs, half the
// instructions of fp32.  That holds for all 128 codes of 4 bits (1920 at
// most), and for 8 bits through the three stages inside a lane (2040).
template <int BITS>
__device__ __forceinline__ void hadamard_codes(const uint32_t (&w)[8 * BITS / 32], _Float16 z, int jj, float (&v)[8]) {
  if constexpr (BITS == 16) {
    codes_to_float<16>(w, z, v);
    fwht128_row16_signed(v, jj);
  } else {
    half2_t p[4];
    codes_to_pairs<BITS>(w, z, p);
    const half2_t one_minus = {(_Float16)1.0f, (_Float16)-1.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = __builtin_elementwise_fma(half2_t{p[i][1], p[i][1]}, one_minus, half2_t{p[i][0], p[i][0]});
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const half2_t a = p[i], b = p[i + 1];
      p[i] = a + b;
      p[i + 1] = a - b;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const half2_t a = p[i], b = p[i + 2];
      p[i] = a + b;
      p[i + 2] = a - b;
    }
    if constexpr (BITS == 4) {
      // stored = partner + beta mine, beta = -1 on the lane of the pair's
      // second element: the transform itself
      const half2_t b1 = half2_t{(_Float16)1.0f, (_Float16)1.0f};
      pair_stage<kQuadXor1>(p, jj & 1 ? -b1 : b1);
      pair_stage<kQuadXor2>(p, jj & 2 ? -b1 : b1);
      pair_stage<kRowHalfMirror>(p, jj & 4 ? -b1 : b1);
      pair_stage<kRowRor8>(p, jj & 8 ? -b1 : b1);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (float)p[e / 2][e & 1];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (float)p[e / 2][e & 1];
#if defined(__HIP_DEVICE_COMPILE__)
      fwht_xstages_dpp(v, (jj & 1) ? -1.0f : 1.0f, (jj & 2) ? -1.0f : 1.0f, (jj & 4) ? -1.0f : 1.0f,
                       (jj & 8) ? -1.0f : 1.0f);
#endif
    }
  }
}

// Lane 16 t + c: 8 channels of token t as packed codes  <->  a quarter of the
// quad, units 2 t' .. (8 bits, fp16) or t' (4 bits) of lane c's 8 channels,
// the four tokens of each side by side.  Both directions are the transpose
// of a 4 x 4 matrix whose rows are the four DPP rows of the wave.
template <int BITS>
__device__ __forceinline__ void rows_to_quad(uint32_t (&w)[8 * BITS / 32]) {
  if constexpr (BITS == 16) {
    swap32(w[0], w[2]);
    swap32(w[1], w[3]);
    swap16(w[0], w[1]);
    swap16(w[2], w[3]);
    // w[t]: channels 2 t', 2 t' + 1 of token t
    const uint32_t a = w[0], b = w[1], c = w[2], d = w[3];
    w[0] = bytes(b, a, 0x05040100u);
    w[1] = bytes(d, c, 0x05040100u);
    w[2] = bytes(b, a, 0x07060302u);
    w[3] = bytes(d, c, 0x07060302u);
  } else if constexpr (BITS == 8) {
    swap32(w[0], w[1]);
    // 16-bit units: even ones of both words, odd ones of both
    uint32_t a = bytes(w[1], w[0], 0x05040100u), b = bytes(w[1], w[0], 0x07060302u);
    swap16(a, b);
    // a: tokens 0, 2 (one unit each); b: tokens 1, 3
    w[0] = bytes(b, a, 0x06020400u);
    w[1] = bytes(b, a, 0x07030501u);
  } else {
    uint32_t x = w[0] & 0xFFFFu, y = w[0] >> 16;
    swap32(x, y);
    uint32_t a = bytes(y, x, 0x0C040C00u), b = bytes(y, x, 0x0C050C01u);   // even and odd bytes, spread
    swap16(a, b);
    w[0] = a | (b << 8);   // a: tokens 0, 2; b: tokens 1, 3
  }
}

template <int BITS>
__device__ __forceinline__ void quad_to_rows(uint32_t (&w)[8 * BITS / 32]) {
  if constexpr (BITS == 16) {
    const uint32_t a = w[0], b = w[1], c = w[2], d = w[3];
    w[0] = bytes(c, a, 0x05040100u);
    w[1] = bytes(c, a, 0x07060302u);
    w[2] = bytes(d, b, 0x05040100u);
    w[3] = bytes(d, b, 0x07060302u);
    swap16(w[0], w[1]);
    swap16(w[2], w[3]);
    swap32(w[0], w[2]);
    swap32(w[1], w[3]);
  } else if constexpr (BITS == 8) {
    uint32_t a = bytes(w[1], w[0], 0x06020400u), b = bytes(w[1], w[0], 0x07030501u);
    swap16(a, b);
    w[0] = bytes(b, a, 0x05040100u);
    w[1] = bytes(b, a, 0x07060302u);
    swap32(w[0], w[1]);
  } else {
    uint32_t a = w[0] & 0x00FF00FFu, b = (w[0] >> 8) & 0x00FF00FFu;
    swap16(a, b);
    uint32_t x = bytes(b, a, 0x0C0C0400u), y = bytes(b, a, 0x0C0C0602u);
    swap32(x, y);
    w[0] = x | (y << 16);
  }
}

// The rotation's signs of a lane's 8 channels as sign bits of packed fp16
// pairs (an exclusive or turns them).
__device__ __forceinline__ void sign_masks(uint32_t bits8, uint32_t (&m)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m[i] = (((bits8 >> (2 * i)) & 1u) << 15) | (((bits8 >> (2 * i + 1)) & 1u) << 31);
}

// A product rounded to fp32 where it stands: without this the compiler may
// fold it into a following conversion to fp16, which then rounds once.
__device__ __forceinline__ float rounded(float v) {
  asm("" : "+v"(v));
  return v;
}

__device__ __forceinline__ void unpack8(uint4 raw, float (&v)[8]) {
  v[0] = half_bits_to_float(raw.x & 0xFFFF); v[1] = half_bits_to_float(raw.x >> 16);
  v[2] = half_bits_to_float(raw.y & 0xFFFF); v[3] = half_bits_to_float(raw.y >> 16);
  v[4] = half_bits_to_float(raw.z & 0xFFFF); v[5] = half_bits_to_float(raw.z >> 16);
  v[6] = half_bits_to_float(raw.w & 0xFFFF); v[7] = half_bits_to_float(raw.w >> 16);
}

struct RowArgs {
  void *k, *v;
  uint32_t *k_params, *v_params;
  const uint32_t *signs;
  uint16_t *xk, *xv;            // the caller's rows: read by write, written by read
  int64_t ldk, ldv;
  const int32_t *slots;
  int64_t tokens;
  int32_t kv_heads, page_shift, capacity;   // capacity: pages * page_size
};

// A wave's span: 4 NW tokens of the call from `first`.  Bit t stands for
// token first + t: `quads`, a full quad of slots starts there; `rest`, its
// slot is one of the cache's and in no full quad of the call; `outside`, its
// slot is not one of the cache's.
template <int NW>
struct Span {
  static constexpr int kLanes = NW == 1 ? 16 : 32;
  int64_t first;
  int32_t slot;                 // lane i: the slot of token first - 3 + i
  uint32_t quads, rest, outside;
  __device__ Span(const RowArgs &a, int64_t span) {
    static_assert(4 * NW + 6 <= kLanes, "three tokens on either side of the span");
    first = 4 * NW * span;
    const int i = threadIdx.x & (kLanes - 1);
    const int64_t token = first - 3 + i;
    const bool real = token >= 0 && token < a.tokens && i < 4 * NW + 6;
    slot = real ? a.slots[token] : -1;
    const bool in = slot >= 0 && slot < a.capacity;
    // every lane takes part in the shuffles
    const int32_t s1 = __shfl_down(slot, 1, kLanes), s2 = __shfl_down(slot, 2, kLanes), s3 = __shfl_down(slot, 3, kLanes);
    const bool start = in && (slot & 3) == 0 && s1 == slot + 1 && s2 == slot + 2 && s3 == slot + 3;
    constexpr uint32_t kMine = (1u << (4 * NW)) - 1u;
    const uint32_t starts = (uint32_t)__ballot(start) & ((kMine << 3) | 7u);
    const uint32_t covered = starts | (starts << 1) | (starts << 2) | (starts << 3);
    quads = (starts >> 3) & kMine;
    rest = (((uint32_t)__ballot(in) & ~covered) >> 3) & kMine;
    outside = ((uint32_t)__ballot(!in && real) >> 3) & kMine;
  }
  __device__ int32_t slot_of(int t) const { return __builtin_amdgcn_readlane(slot, t + 3); }
};

// A wave's work: a span of tokens, keys or values, one head (a pair of heads
// of 64 channels), and what a lane keeps over the span.
template <int BITS, int D, int NW>
struct Item {
  using L = Layout<BITS, D>;
  int64_t span;
  int head, c0, t;              // t: the lane's token of four
  bool is_v, live;
  char *codes;                  // the head's first page
  uint32_t *par;
  uint16_t *x;                  // the caller's row of token 0
  int64_t ld, page_codes, page_par;
  uint32_t signs[L::kSets][4];
  bool rotated;
  __device__ explicit Item(const RowArgs &a) {
    const int64_t id = (int64_t)blockIdx.x * (kRowThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int groups = (a.kv_heads + L::kHeads - 1) / L::kHeads;
    is_v = id & 1;
    span = (id >> 1) / groups;
    head = (int)((id >> 1) % groups) * L::kHeads;
    const int lane = threadIdx.x & 15;
    t = (threadIdx.x >> 4) & 3;
    c0 = 8 * lane;
    if (L::kHeads == 2) {
      head += lane >> 3;
      c0 = 8 * (lane & 7);
    }
    live = head < a.kv_heads;
    const int h = live ? head : 0;
    const int64_t head_codes = ((int64_t)L::kUnits * L::kUnitBytes) << a.page_shift, head_par = (int64_t)1 << a.page_shift;
    codes = static_cast<char *>(is_v ? a.v : a.k) + h * head_codes;
    par = (is_v ? a.v_params : a.k_params) + h * head_par;
    page_codes = head_codes * a.kv_heads;
    page_par = head_par * a.kv_heads;
    x = (is_v ? a.xv : a.xk) + (int64_t)h * D + c0;
    ld = is_v ? a.ldv : a.ldk;
    rotated = D >= 128 && a.signs;
#pragma unroll
    for (int b = 0; b < L::kSets; ++b) {
      const int ch = h * D + c0 + 128 * b;
      sign_masks(rotated ? a.signs[ch >> 5] >> (ch & 31) : 0u, signs[b]);
    }
  }
  // byte offset, in the lane's head and page, of its channels of set b of
  // token `at`, or of its quarter of the quad that starts there
  __device__ int64_t piece(int at, bool quad, int b) const {
    const int u = (c0 + 128 * b) / (BITS == 4 ? 2 : 1);
    if (!is_v) return L::kUnitBytes * L::key_unit(at, u);
    if (quad) return L::kUnitBytes * L::value_unit(at, u + (BITS == 4 ? 1 : 2) * t);
    return L::kUnitBytes * L::value_unit(at, u);
  }
};

template <int BITS>
__device__ __forceinline__ void store_piece(char *out, const uint32_t (&w)[8 * BITS / 32]) {
  if constexpr (BITS == 16) *reinterpret_cast<uint4 *>(out) = make_uint4(w[0], w[1], w[2], w[3]);
  if constexpr (BITS == 8) *reinterpret_cast<uint2 *>(out) = make_uint2(w[0], w[1]);
  if constexpr (BITS == 4) *reinterpret_cast<uint32_t *>(out) = w[0];
}
template <int BITS>
__device__ __forceinline__ void load_piece(const char *in, uint32_t (&w)[8 * BITS / 32]) {
  if constexpr (BITS == 16) {
    const uint4 r = *reinterpret_cast<const uint4 *>(in);
    w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
  }
  if constexpr (BITS == 8) {
    const uint2 r = *reinterpret_cast<const uint2 *>(in);
    w[0] = r.x; w[1] = r.y;
  }
  if constexpr (BITS == 4) w[0] = *reinterpret_cast<const uint32_t *>(in);
}

// a / b from r, the reciprocal of b, rounded as a division rounds it: one
// correction by the remainder (Markstein's division), three operations
// instead of a dozen.  b here is an fp16 value or a small whole number, so
// neither the product nor the remainder leaves the normal range where the
// quotient matters (below 2^-20 it rounds to the zero code either way).
__device__ __forceinline__ float divide(float a, float b, float r) {
  const float q = a * r;
  return fmaf(fmaf(-q, b, a), r, q);
}

// Codes of a lane's channels, the row's scale and zero: the rule of
// wq_kv_write.
template <int BITS, int D, int SETS>
__device__ __forceinline__ uint32_t code_row(const float (&v)[SETS][8], uint32_t (&w)[SETS][8 * BITS / 32]) {
  float lo = 0.0f, hi = 0.0f;
#pragma unroll
  for (int b = 0; b < SETS; ++b)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo = fminf(lo, v[b][e]);
      hi = fmaxf(hi, v[b][e]);
    }
  lo = row_extreme<D, uint32_t>(lo);
  hi = row_extreme<D, int32_t>(hi);
  const float qmax = (float)((1 << BITS) - 1);
  _Float16 s16 = (_Float16)fminf(divide(hi - lo, qmax, 1.0f / qmax), 65504.0f);
  if (s16 == (_Float16)0.0f) s16 = (_Float16)1.0f;
  const float s = (float)s16;
  float r = __builtin_amdgcn_rcpf(s);
  r = fmaf(fmaf(-s, r, 1.0f), r, r);
  const float z = __builtin_amdgcn_fmed3f(rintf(divide(0.0f - lo, s, r)), 0.0f, qmax);
#pragma unroll
  for (int b = 0; b < SETS; ++b) {
    float c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = divide(v[b][e], s, r) + z;
    // the conversion to a byte rounds half to even and clamps to 0 .. 255
#pragma unroll
    for (int e = 0; e < 8 * BITS / 32; ++e) w[b][e] = 0;
    if constexpr (BITS == 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[b][e / 4] = __builtin_amdgcn_cvt_pk_u8_f32(c[e], e & 3, w[b][e / 4]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] = __builtin_amdgcn_fmed3f(rintf(c[e]), 0.0f, 15.0f);
#pragma unroll
      for (int e = 0; e < 8; e += 2) w[b][0] = __builtin_amdgcn_cvt_pk_u8_f32(fmaf(c[e + 1], 16.0f, c[e]), e / 2, w[b][0]);
    }
  }
  return cvt_pk_half2(s, z);
}

// The lane's 8 channels (or two sets of them): given fp16 -> codes and the
// row's scale and zero.
template <int BITS, int D, int NW>
__device__ __forceinline__ uint32_t code_lane(const Item<BITS, D, NW> &it, const uint4 (&raw)[Layout<BITS, D>::kSets],
                                              uint32_t (&w)[Layout<BITS, D>::kSets][Layout<BITS, D>::kWords]) {
  using L = Layout<BITS, D>;
  float v[L::kSets][8];
#pragma unroll
  for (int b = 0; b < L::kSets; ++b) {
    const uint32_t(&m)[4] = it.signs[b];
    unpack8(make_uint4(raw[b].x ^ m[0], raw[b].y ^ m[1], raw[b].z ^ m[2], raw[b].w ^ m[3]), v[b]);
    if (it.rotated) {
      const int jj = threadIdx.x & 15;
      fwht128_row16_signed(v[b], jj);
      const float sc = fwht_lane_sign(jj) * kInvSqrt128;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[b][e] = BITS == 16 ? rounded(v[b][e] * sc) : v[b][e] * sc;
    }
  }
  if constexpr (BITS == 16) {
#pragma unroll
    for (int b = 0; b < L::kSets; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) w[b][e] = cvt_pk_half2(v[b][2 * e], v[b][2 * e + 1]);
    return 0;
  } else {
    return code_row<BITS, D, L::kSets>(v, w);
  }
}

// codes -> fp16 rows
template <int BITS, int D, int NW>
__device__ __forceinline__ u32x4 decode_lane(const Item<BITS, D, NW> &it, const uint32_t (&w)[Layout<BITS, D>::kWords],
                                             uint32_t par, int b) {
  float v[8];
  const float s = half_bits_to_float(par & 0xFFFF);
  float sc = s;
  if (it.rotated) {
    // x = D H (code - zero) (scale / sqrt(128)); H is symmetric
    const int jj = threadIdx.x & 15;
    hadamard_codes<BITS>(w, as_half2(par)[1], jj, v);
    sc = BITS == 16 ? kInvSqrt128 : rounded(s * kInvSqrt128);
    if (BITS != 4) sc *= fwht_lane_sign(jj);
  } else {
    codes_to_float<BITS>(w, as_half2(par)[1], v);
  }
  if (BITS != 16 || it.rotated)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = rounded(v[e] * sc);
  u32x4 y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = cvt_pk_half2(v[2 * e], v[2 * e + 1]) ^ it.signs[b][e];
  return y;
}

template <int BITS, int D, int NW>
__global__ __launch_bounds__(kRowThreads) void kv_write_kernel(RowArgs a) {
  using L = Layout<BITS, D>;
  const Item<BITS, D, NW> it(a);
  if (4 * NW * it.span >= a.tokens) return;   // whole waves leave together
  const Span<NW> sp(a, it.span);
  const int mask = (1 << a.page_shift) - 1;

  // the quads: all rows asked for before the first is coded
  int at[NW];
  uint4 raw[NW][L::kSets];
  const int count = __builtin_popcount(sp.quads);
  uint32_t left = sp.quads;
  if (count) {
#pragma unroll
    for (int n = 0; n < NW; ++n) {
      at[n] = left ? __builtin_ctz(left) : at[n ? n - 1 : 0];   // past the last: the last again
      left &= left - 1;
#pragma unroll
      for (int b = 0; b < L::kSets; ++b)
        raw[n][b] = *reinterpret_cast<const uint4 *>(it.x + (sp.first + at[n] + it.t) * it.ld + 128 * b);
    }
  }
#pragma unroll
  for (int n = 0; n < NW; ++n) {
    if (n >= count) break;
    const int32_t slot = sp.slot_of(at[n]);
    const int64_t page = slot >> a.page_shift;
    const int t0 = slot & mask;
    uint32_t w[L::kSets][L::kWords];
    const uint32_t par = code_lane<BITS, D, NW>(it, raw[n], w);
    if (BITS != 16 && it.live && it.c0 == 0) it.par[page * it.page_par + t0 + it.t] = par;
    char *to = it.codes + page * it.page_codes;
#pragma unroll
    for (int b = 0; b < L::kSets; ++b) {
      if (it.is_v) rows_to_quad<BITS>(w[b]);
      if (it.live) store_piece<BITS>(to + it.piece(it.is_v ? t0 : t0 + it.t, true, b), w[b]);
    }
  }

  // tokens in no quad, four at a time
#pragma unroll 1
  for (int n = 0; n < NW; ++n) {
    const uint32_t four = (sp.rest >> (4 * n)) & 0xFu;
    if (!four) continue;
    const bool mine = ((four >> it.t) & 1u) && it.live;
    const int64_t token = sp.first + 4 * n + it.t;
    const int32_t slot = mine ? a.slots[token] : 0;
    uint4 one[L::kSets];
#pragma unroll
    for (int b = 0; b < L::kSets; ++b) {
      one[b] = make_uint4(0, 0, 0, 0);
      if (mine) one[b] = *reinterpret_cast<const uint4 *>(it.x + token * it.ld + 128 * b);
    }
    uint32_t w[L::kSets][L::kWords];
    const uint32_t par = code_lane<BITS, D, NW>(it, one, w);
    if (!mine) continue;
    const int64_t page = slot >> a.page_shift;
    const int t0 = slot & mask;
    if (BITS != 16 && it.c0 == 0) it.par[page * it.page_par + t0] = par;
#pragma unroll
    for (int b = 0; b < L::kSets; ++b) {
      char *to = it.codes + page * it.page_codes + it.piece(t0, false, b);
      if (!it.is_v) {
        store_piece<BITS>(to, w[b]);
        continue;
      }
#pragma unroll
      for (int e = 0; e < (BITS == 4 ? 4 : 8); ++e) {   // a unit each, the quad's other tokens between them
        if constexpr (BITS == 16)
          reinterpret_cast<uint16_t *>(to)[4 * e] = (uint16_t)(w[b][e / 2] >> (16 * (e & 1)));
        else
          to[4 * e] = (char)(w[b][e / 4] >> (8 * (e & 3)));
      }
    }
  }
}

template <int BITS, int D, int NW>
__global__ __launch_bounds__(kRowThreads) void kv_read_kernel(RowArgs a) {
  using L = Layout<BITS, D>;
  const Item<BITS, D, NW> it(a);
  if (4 * NW * it.span >= a.tokens) return;
  const Span<NW> sp(a, it.span);
  const int mask = (1 << a.page_shift) - 1;
  auto give = [&](int64_t token, const u32x4 &y, int b) {
    u32x4 *to = reinterpret_cast<u32x4 *>(it.x + token * it.ld + 128 * b);
    // many rows: streamed past the caches (30011 4-bit rows read again and again: 38 us a pass, 45 without)
    if constexpr (NW > 1)
      __builtin_nontemporal_store(y, to);
    else
      *to = y;
  };

  int at[NW];
  uint32_t w[NW][L::kSets][L::kWords], par[NW];
  const int count = __builtin_popcount(sp.quads);
  uint32_t left = sp.quads;
  if (count) {
#pragma unroll
    for (int n = 0; n < NW; ++n) {
      at[n] = left ? __builtin_ctz(left) : at[n ? n - 1 : 0];
      left &= left - 1;
      const int32_t slot = sp.slot_of(at[n]);
      const int64_t page = slot >> a.page_shift;
      const int t0 = slot & mask;
      const char *from = it.codes + page * it.page_codes;
      par[n] = BITS == 16 ? 0 : it.par[page * it.page_par + t0 + it.t];
#pragma unroll
      for (int b = 0; b < L::kSets; ++b) load_piece<BITS>(from + it.piece(it.is_v ? t0 : t0 + it.t, true, b), w[n][b]);
    }
  }
#pragma unroll
  for (int n = 0; n < NW; ++n) {
    if (n >= count) break;
#pragma unroll
    for (int b = 0; b < L::kSets; ++b) {
      if (it.is_v) quad_to_rows<BITS>(w[n][b]);
      const u32x4 y = decode_lane<BITS, D, NW>(it, w[n][b], par[n], b);
      if (it.live) give(sp.first + at[n] + it.t, y, b);
    }
  }

  // tokens in no quad, those outside the cache (zeros) among them
#pragma unroll 1
  for (int n = 0; n < NW; ++n) {
    const uint32_t four = (sp.rest >> (4 * n)) & 0xFu, none = (sp.outside >> (4 * n)) & 0xFu;
    if (!(four | none)) continue;
    const bool mine = ((four >> it.t) & 1u) && it.live;
    const int64_t token = sp.first + 4 * n + it.t;
    const int32_t slot = mine ? a.slots[token] : 0;
    const int64_t page = slot >> a.page_shift;
    const int t0 = slot & mask;
    const uint32_t one = BITS != 16 && mine ? it.par[page * it.page_par + t0] : 0u;
#pragma unroll
    for (int b = 0; b < L::kSets; ++b) {
      const char *from = it.codes + page * it.page_codes + it.piece(t0, false, b);
      uint32_t c[L::kWords];
#pragma unroll
      for (int e = 0; e < L::kWords; ++e) c[e] = 0;
      if (mine && !it.is_v) load_piece<BITS>(from, c);
      if (mine && it.is_v) {
#pragma unroll
        for (int e = 0; e < (BITS == 4 ? 4 : 8); ++e) {
          if constexpr (BITS == 16)
            c[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(from)[4 * e] << (16 * (e & 1));
          else
            c[e / 4] |= (uint32_t)(uint8_t)from[4 * e] << (8 * (e & 3));
        }
      }
      const u32x4 y = decode_lane<BITS, D, NW>(it, c, one, b);
      if (it.live && (((four | none) >> it.t) & 1u)) give(token, y, b);
    }
  }
}

RowArgs row_args(const wq_kv_cache &c, const int32_t *slots, int64_t tokens, const uint16_t *k, int64_t ldk,
                 const uint16_t *v, int64_t ldv) {
  RowArgs a;
  a.k = c.k;
  a.v = c.v;
  a.k_params = reinterpret_cast<uint32_t *>(c.k_params);
  a.v_params = reinterpret_cast<uint32_t *>(c.v_params);
  a.signs = c.rht_signs;
  a.xk = const_cast<uint16_t *>(k);
  a.xv = const_cast<uint16_t *>(v);
  a.ldk = ldk;
  a.ldv = ldv;
  a.slots = slots;
  a.tokens = tokens;
  a.kv_heads = c.kv_heads;
  a.page_shift = 0;
  while ((1 << a.page_shift) < c.page_size) ++a.page_shift;
  a.capacity = (int32_t)(c.pages * c.page_size);
  return a;
}

// (the caller has checked that the grid fits a launch)
template <int BITS, int D, int NW>
hipError_t launch_rows(const RowArgs &a, const RowPlan &p, bool write, hipStream_t s) {
  const dim3 grid((unsigned)p.groups), block(kRowThreads);
  if (write)
    hipLaunchKernelGGL((kv_write_kernel<BITS, D, NW>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((kv_read_kernel<BITS, D, NW>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <int BITS, int D>
hipError_t launch_rows_quads(const RowArgs &a, const RowPlan &p, bool write, hipStream_t s) {
  return p.quads == 1 ? launch_rows<BITS, D, 1>(a, p, write, s) : launch_rows<BITS, D, kv_most_quads(D)>(a, p, write, s);
}

template <int BITS>
hipError_t launch_rows_bits(int d, const RowArgs &a, const RowPlan &p, bool write, hipStream_t s) {
  switch (d) {
    case 64: return launch_rows_quads<BITS, 64>(a, p, write, s);
    case 128: return launch_rows_quads<BITS, 128>(a, p, write, s);
    case 256: return launch_rows_quads<BITS, 256>(a, p, write, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_rows_any(const wq_kv_cache &c, const RowArgs &a, const RowPlan &p, bool write, hipStream_t s) {
  switch (c.bits) {
    case 4: return launch_rows_bits<4>(c.head_dim, a, p, write, s);
    case 8: return launch_rows_bits<8>(c.head_dim, a, p, write, s);
    case 16: return launch_rows_bits<16>(c.head_dim, a, p, write, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_kv_write(const wq_kv_cache &c, const RowPlan &p, const uint16_t *k, int64_t ldk, const uint16_t *v,
                           int64_t ldv, const int32_t *slots, int64_t tokens, hipStream_t s) {
  return launch_rows_any(c, row_args(c, slots, tokens, k, ldk, v, ldv), p, true, s);
}

hipError_t launch_kv_read(const wq_kv_cache &c, const RowPlan &p, const int32_t *slots, int64_t tokens, uint16_t *k,
                          int64_t ldk, uint16_t *v, int64_t ldv, hipStream_t s) {
  return launch_rows_any(c, row_args(c, slots, tokens, k, ldk, v, ldv), p, false, s);
}

}  // namespace wq
