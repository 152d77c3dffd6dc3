// Rotary positions with one or several axes (gfx950): (a, b) ->
// (a c - b s, b c + a s) per pair of channels, c and s looked up at the
// token's position on the pair's axis.
//
// One thread turns 8 pairs (16 channels) of one head, or copies 8 of the
// channels past `rot`; a head is rot / 16 + (head_dim - rot) / 8 threads.
#include "wq_internal.h"

namespace wq {
using namespace dev;

namespace {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ void load8(const uint16_t *p, float (&v)[8]) {
  const uint4 r = *reinterpret_cast<const uint4 *>(p);
  v[0] = half_bits_to_float(r.x & 0xFFFF); v[1] = half_bits_to_float(r.x >> 16);
  v[2] = half_bits_to_float(r.y & 0xFFFF); v[3] = half_bits_to_float(r.y >> 16);
  v[4] = half_bits_to_float(r.z & 0xFFFF); v[5] = half_bits_to_float(r.z >> 16);
  v[6] = half_bits_to_float(r.w & 0xFFFF); v[7] = half_bits_to_float(r.w >> 16);
}

__device__ __forceinline__ void store8(uint16_t *p, const float (&v)[8]) {
  *reinterpret_cast<uint4 *>(p) =
      make_uint4(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]), pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
}

__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a, int32_t all_heads) {
  const int half = a.rot / 2;
  const int turns = half / 8, per_head = turns + (a.head_dim - a.rot) / 8;
  const int64_t gid = (int64_t)blockIdx.x * kRopeThreads + threadIdx.x;
  const int part = (int)(gid % per_head);
  int64_t r = gid / per_head;
  int head = (int)(r % all_heads);
  const int64_t token = r / all_heads;
  if (token >= a.tokens) return;
  int i = 0;
  while (head >= a.arr[i].heads) head -= a.arr[i++].heads;
  const uint16_t *x = a.arr[i].x + token * a.arr[i].ldx + (int64_t)head * a.head_dim;
  uint16_t *y = a.arr[i].y + token * a.arr[i].ldy + (int64_t)head * a.head_dim;
  if (part >= turns) {   // channels past `rot`
    const int c = a.rot + 8 * (part - turns);
    if (x != y) *reinterpret_cast<uint4 *>(y + c) = *reinterpret_cast<const uint4 *>(x + c);
    return;
  }
  const int p0 = 8 * part;
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int32_t pos = a.positions[a.pair_axis[p0 + e] * a.ld_pos + token];
    const bool in = pos >= 0 && pos < a.table_rows;
    c[e] = in ? a.cos[(int64_t)pos * half + p0 + e] : 1.0f;
    s[e] = in ? a.sin[(int64_t)pos * half + p0 + e] : 0.0f;
  }
  // lo, hi: the 16 channels as two groups of 8; pairs (lo[e], hi[e]), or
  // neighbours within each
  const int at = a.adjacent ? 2 * p0 : p0, to = a.adjacent ? 2 * p0 + 8 : p0 + half;
  float lo[8], hi[8];
  load8(x + at, lo);
  load8(x + to, hi);
  float out_lo[8], out_hi[8];
  if (a.adjacent) {
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
  store8(y + at, out_lo);
  store8(y + to, out_hi);
}

}  // namespace

hipError_t launch_rope(const RopeArgs &a, hipStream_t s) {
  int64_t heads = 0;
  for (int i = 0; i < a.count; ++i) heads += a.arr[i].heads;
  const int per_head = a.rot / 16 + (a.head_dim - a.rot) / 8;
  const int64_t wgs = (a.tokens * heads * per_head + kRopeThreads - 1) / kRopeThreads;
  if (wgs > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL(rope_kernel, dim3((unsigned)wgs), dim3(kRopeThreads), 0, s, a, (int32_t)heads);
  return hipGetLastError();
}

}  // namespace wq
