// Rotary positions with one or several axes (gfx950): (a, b) ->
// (a c - b s, b c + a s) per pair of channels, c and s looked up at the
// token's position on the pair's axis.
//
// A lane turns 8 pairs (16 channels), a head is rot / 16 lanes, and a wave
// takes several heads of one token side by side: one such round where there
// are few waves, four with many, for one look-up of the cosines and sines.
// Traffic bound: every value is read and written once, in 16-byte pieces:
// 6001 tokens of 40 heads of 128 with three axes (126 MB) in 24 us, 5.2 TB/s
// (54 us with a look-up for each head).  16 tokens: 3.4 us, launch and
// latency.
#include "wq_internal.h"

#include <climits>
#include <cstring>

namespace wq {
using namespace dev;

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRounds = kRopeRounds;

__device__ __forceinline__ void unpack8(uint4 r, float (&v)[8]) {
  v[0] = half_bits_to_float(r.x & 0xFFFF); v[1] = half_bits_to_float(r.x >> 16);
  v[2] = half_bits_to_float(r.y & 0xFFFF); v[3] = half_bits_to_float(r.y >> 16);
  v[4] = half_bits_to_float(r.z & 0xFFFF); v[5] = half_bits_to_float(r.z >> 16);
  v[6] = half_bits_to_float(r.w & 0xFFFF); v[7] = half_bits_to_float(r.w >> 16);
}

__device__ __forceinline__ void store8(uint16_t *p, const float (&v)[8]) {
  *reinterpret_cast<uint4 *>(p) =
      make_uint4(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]), pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
}

struct RopeShape {
  uint32_t axis[WQ_ROPE_MAX_AXES][4];   // the pairs of each axis, one bit each
  int32_t turns, slots;         // lanes of a head; heads side by side in a wave
  uint32_t inv;                 // ceil(2^16 / turns)
  int32_t rounds;               // times `slots` heads a wave takes: 1 or kRounds
};

template <bool ADJACENT>
__device__ __forceinline__ void turn(const float (&lo)[8], const float (&hi)[8], const float (&c)[8], const float (&s)[8],
                                     float (&out_lo)[8], float (&out_hi)[8]) {
  if (ADJACENT) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      out_lo[2 * e] = lo[2 * e] * c[e] - lo[2 * e + 1] * s[e];
      out_lo[2 * e + 1] = lo[2 * e + 1] * c[e] + lo[2 * e] * s[e];
      out_hi[2 * e] = hi[2 * e] * c[e + 4] - hi[2 * e + 1] * s[e + 4];
      out_hi[2 * e + 1] = hi[2 * e + 1] * c[e + 4] + hi[2 * e] * s[e + 4];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      out_lo[e] = lo[e] * c[e] - hi[e] * s[e];
      out_hi[e] = hi[e] * c[e] + lo[e] * s[e];
    }
  }
}

template <bool ADJACENT>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a, RopeShape sh) {
  const int64_t token = (int64_t)blockIdx.x * (kRopeThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const RopeArray arr = a.arr[blockIdx.z];
  const int first = blockIdx.y * sh.slots * sh.rounds;   // head
  if (token >= a.tokens || first >= arr.heads) return;
  const int last = min(first + sh.slots * sh.rounds, arr.heads);
  const int lane = threadIdx.x & 63;
  const uint16_t *x = arr.x + token * arr.ldx;
  uint16_t *y = arr.y + token * arr.ldy;

  const int slot = (int)((lane * sh.inv) >> 16), part = lane - slot * sh.turns, p0 = 8 * part;
  if (slot < sh.slots) {
    const int half = a.rot / 2;
    // the 16 channels as two groups of 8: pairs (lo[e], hi[e]), or neighbours within each
    const int at = ADJACENT ? 2 * p0 : p0, to = ADJACENT ? 2 * p0 + 8 : p0 + half;
    uint4 rl[kRounds], rh[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int h = first + r * sh.slots + slot;
      if (h >= last) continue;
      rl[r] = *reinterpret_cast<const uint4 *>(x + (int64_t)h * a.head_dim + at);
      rh[r] = *reinterpret_cast<const uint4 *>(x + (int64_t)h * a.head_dim + to);
    }
    float c[8], s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = 1.0f;
      s[e] = 0.0f;
    }
    for (int ax = 0; ax < a.axes; ++ax) {
      const int32_t pos = a.positions[ax * a.ld_pos + token];
      if (pos < 0 || pos >= a.table_rows) continue;   // outside the table: unchanged
      const uint32_t lo2 = p0 & 64 ? sh.axis[ax][2] : sh.axis[ax][0], hi2 = p0 & 64 ? sh.axis[ax][3] : sh.axis[ax][1];
      const uint32_t mine = ((p0 & 32 ? hi2 : lo2) >> (p0 & 31)) & 0xFFu;
      if (!mine) continue;
      const float4 *ct = reinterpret_cast<const float4 *>(a.cos + (int64_t)pos * half + p0);
      const float4 *st = reinterpret_cast<const float4 *>(a.sin + (int64_t)pos * half + p0);
      const float4 c0 = ct[0], c1 = ct[1], s0 = st[0], s1 = st[1];
      const float cv[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
      const float sv[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = (mine >> e) & 1u ? cv[e] : c[e];
        s[e] = (mine >> e) & 1u ? sv[e] : s[e];
      }
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int h = first + r * sh.slots + slot;
      if (h >= last) continue;
      float lo[8], hi[8], out_lo[8], out_hi[8];
      unpack8(rl[r], lo);
      unpack8(rh[r], hi);
      turn<ADJACENT>(lo, hi, c, s, out_lo, out_hi);
      store8(y + (int64_t)h * a.head_dim + at, out_lo);
      store8(y + (int64_t)h * a.head_dim + to, out_hi);
    }
  }
  // channels past `rot`
  if (a.rot < a.head_dim && x != y) {
    const int per = (a.head_dim - a.rot) / 8;
    for (int i = lane; i < (last - first) * per; i += 64) {
      const int64_t ch = (int64_t)(first + i / per) * a.head_dim + a.rot + 8 * (i % per);
      *reinterpret_cast<uint4 *>(y + ch) = *reinterpret_cast<const uint4 *>(x + ch);
    }
  }
}

}  // namespace

hipError_t launch_rope(const RopeArgs &a, hipStream_t s) {
  RopeShape sh;
  memset(&sh, 0, sizeof sh);
  for (int i = 0; i < a.rot / 2; ++i) sh.axis[a.pair_axis[i]][i >> 5] |= 1u << (i & 31);
  sh.turns = a.rot / 16;
  sh.slots = 64 / sh.turns;
  sh.inv = (65536 + sh.turns - 1) / sh.turns;
  int32_t heads[kMaxBatch], most = 0;
  for (int i = 0; i < a.count; ++i) {
    heads[i] = a.arr[i].heads;
    if (heads[i] > most) most = heads[i];
  }
  sh.rounds = rope_rounds(a.tokens, a.rot, a.count, heads);
  const int64_t x = (a.tokens + kRopeThreads / 64 - 1) / (kRopeThreads / 64);
  const int64_t y = ((int64_t)most + (int64_t)sh.slots * sh.rounds - 1) / ((int64_t)sh.slots * sh.rounds);
  if (x > INT32_MAX || y > 65535) return hipErrorInvalidValue;
  const dim3 grid((unsigned)x, (unsigned)y, (unsigned)a.count);
  if (a.adjacent)
    hipLaunchKernelGGL(rope_kernel<true>, grid, dim3(kRopeThreads), 0, s, a, sh);
  else
    hipLaunchKernelGGL(rope_kernel<false>, grid, dim3(kRopeThreads), 0, s, a, sh);
  return hipGetLastError();
}

}  // namespace wq
