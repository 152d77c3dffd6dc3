// Attention of one new token per sequence over a paged, coded key-value
// cache (gfx950):  out = R^T sum_t softmax_t(scale (R q).k_t) v_t.
//
// One workgroup per (sequence, query head), 256 tokens at a time: a thread
// scores one token, the tile's largest score and sum update the running
// softmax (m, l), and thread d adds up channel d of the values.
#include "wq_internal.h"

#include <cmath>

namespace wq {
using namespace dev;

namespace {

constexpr int kAttnThreads = 256;

template <int BITS, int D>
__device__ __forceinline__ float code_at(const void *base, int64_t unit, int ch) {
  if constexpr (BITS == 16) return half_bits_to_float(static_cast<const uint16_t *>(base)[unit]);
  const uint32_t b = static_cast<const uint8_t *>(base)[unit];
  return (float)(BITS == 4 ? (b >> (4 * (ch & 1))) & 15u : b);
}

template <int BITS, int D>
__global__ __launch_bounds__(kAttnThreads) void attn_simple_kernel(AttnArgs a) {
  constexpr int U = BITS == 4 ? D / 2 : D, P = BITS == 16 ? 32 : (U < 64 ? U : 64);
  constexpr float kMasked = -INFINITY;
  __shared__ float qs[D], prob[kAttnThreads], red[kAttnThreads];
  __shared__ int32_t page_of[kAttnThreads];
  const int heads = a.kv_heads * a.group;
  const int head = blockIdx.x % heads, kvh = head / a.group;
  const int64_t seq = blockIdx.x / heads;
  const int tid = threadIdx.x;
  const int len = min(a.lens[seq], a.max_len);
  const int start = a.window && len > a.window ? len - a.window : 0;
  // the query, rotated as the cache is, rounded to fp16
  if (tid < D / 8) {
    const uint16_t *q = a.q + seq * a.ldq + (int64_t)head * D + 8 * tid;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = half_bits_to_float(q[e]);
    if (D >= 128 && a.signs) {
      const int ch = kvh * D + 8 * tid;
      const uint32_t sb = a.signs[ch >> 5] >> (ch & 31);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = ((sb >> e) & 1u) ? -v[e] : v[e];
      fwht128_row16_signed(v, tid & 15);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= fwht_lane_sign(tid & 15) * 0.08838834764831845f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) qs[8 * tid + e] = (float)(_Float16)v[e];
  }
  float m = kMasked, l = 0.0f, acc = 0.0f;
  const int mask = (1 << a.page_shift) - 1;
  for (int t0 = start; t0 < len; t0 += kAttnThreads) {
    __syncthreads();
    const int t = t0 + tid;
    float score = kMasked;
    int32_t page = -1;
    if (t < len) {
      page = a.table[seq * a.ld_table + (t >> a.page_shift)];
      if (page < 0 || page >= a.pages) page = -1;
    }
    page_of[tid] = page;
    const int64_t ph = (int64_t)page * a.kv_heads + kvh;
    if (page >= 0) {
      const int at = t & mask;
      const int64_t base = ph * ((int64_t)U << a.page_shift) + (int64_t)(at >> 4) * 16 * U + (at & 15) * P;
      float s = 1.0f, z = 0.0f;
      if (BITS != 16) {
        const uint32_t par = a.k_params[(ph << a.page_shift) + at];
        s = half_bits_to_float(par & 0xFFFF);
        z = half_bits_to_float(par >> 16);
      }
      float dot = 0.0f;
      for (int d = 0; d < D; ++d) {
        const int u = BITS == 4 ? d / 2 : d;
        dot += qs[d] * (code_at<BITS, D>(a.k, base + (u / P) * 16 * P + u % P, d) - z);
      }
      score = dot * s * a.scale;
    }
    red[tid] = score;
    __syncthreads();
    for (int o = kAttnThreads / 2; o; o >>= 1) {
      if (tid < o) red[tid] = fmaxf(red[tid], red[tid + o]);
      __syncthreads();
    }
    const float top = fmaxf(m, red[0]);
    __syncthreads();
    const float p = page >= 0 ? __expf(score - top) : 0.0f;
    prob[tid] = p;
    red[tid] = p;
    __syncthreads();
    for (int o = kAttnThreads / 2; o; o >>= 1) {
      if (tid < o) red[tid] += red[tid + o];
      __syncthreads();
    }
    const float keep = m == kMasked ? 0.0f : __expf(m - top);
    l = l * keep + red[0];
    m = top;
    acc *= keep;
    if (tid < D) {
      const int n = min(kAttnThreads, len - t0);
      for (int i = 0; i < n; ++i) {
        if (page_of[i] < 0) continue;
        const int at = (t0 + i) & mask;
        const int64_t ph2 = (int64_t)page_of[i] * a.kv_heads + kvh;
        const int u = BITS == 4 ? tid / 2 : tid;
        float v = code_at<BITS, D>(a.v, ph2 * ((int64_t)U << a.page_shift) + (int64_t)(at >> 2) * 4 * U + 4 * u + (at & 3), tid);
        if (BITS != 16) {
          const uint32_t par = a.v_params[(ph2 << a.page_shift) + at];
          v = (v - half_bits_to_float(par >> 16)) * half_bits_to_float(par & 0xFFFF);
        }
        acc += prob[i] * v;
      }
    }
  }
  __syncthreads();
  if (tid < D) qs[tid] = l > 0.0f ? acc / l : 0.0f;
  __syncthreads();
  if (tid < D / 8) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = qs[8 * tid + e];
    if (D >= 128 && a.signs) {
      fwht128_row16_signed(v, tid & 15);
      const int ch = kvh * D + 8 * tid;
      const uint32_t sb = a.signs[ch >> 5] >> (ch & 31);
      const float sc = fwht_lane_sign(tid & 15) * 0.08838834764831845f;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= ((sb >> e) & 1u) ? -sc : sc;
    }
    *reinterpret_cast<uint4 *>(a.out + seq * a.ldo + (int64_t)head * D + 8 * tid) = make_uint4(
        pack_half2(v[0], v[1]), pack_half2(v[2], v[3]), pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
  }
}

template <int BITS>
hipError_t launch_bits(int d, const AttnArgs &a, hipStream_t s) {
  const dim3 grid((unsigned)(a.seqs * a.kv_heads * a.group));
  switch (d) {
    case 64: hipLaunchKernelGGL((attn_simple_kernel<BITS, 64>), grid, dim3(kAttnThreads), 0, s, a); break;
    case 128: hipLaunchKernelGGL((attn_simple_kernel<BITS, 128>), grid, dim3(kAttnThreads), 0, s, a); break;
    case 256: hipLaunchKernelGGL((attn_simple_kernel<BITS, 256>), grid, dim3(kAttnThreads), 0, s, a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

size_t attn_workspace(const wq_kv_cache &, int64_t, int32_t, int64_t, int64_t) { return 0; }

hipError_t launch_attn_decode(int bits, int head_dim, const AttnArgs &a, hipStream_t s) {
  switch (bits) {
    case 4: return launch_bits<4>(head_dim, a, s);
    case 8: return launch_bits<8>(head_dim, a, s);
    case 16: return launch_bits<16>(head_dim, a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace wq
