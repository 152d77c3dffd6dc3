// The paged key-value cache: new rows coded as they are written, and read
// back (gfx950).  Layouts and rules: include/wq.h.
//
// A row of D = 64, 128 or 256 values is D / 8 lanes with 8 channels each, so
// a 128-block is the 16 lanes of a DPP row and its rotation is
// fwht128_row16_signed.  Everything is fp32, in the order the definition
// gives it; no product feeds a sum, so no fused multiply-add can change a
// code.
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
  __device__ static int64_t key_unit(int t, int u) {
    return (int64_t)(t >> 4) * 16 * kUnits + (u / kPanel) * 16 * kPanel + (t & 15) * kPanel + u % kPanel;
  }
  __device__ static int64_t value_unit(int t, int u) { return (int64_t)(t >> 2) * 4 * kUnits + 4 * u + (t & 3); }
};

template <int D>
__device__ __forceinline__ float row_min(float v) {
#pragma unroll
  for (int o = 1; o < D / 8; o <<= 1) v = fminf(v, __shfl_xor(v, o));
  return v;
}

template <int D>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = 1; o < D / 8; o <<= 1) v = fmaxf(v, __shfl_xor(v, o));
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

// One row (token, head, key or value) per D / 8 lanes.
template <int BITS, int D>
__global__ __launch_bounds__(kRowThreads) void kv_write_kernel(RowArgs a) {
  using L = Layout<BITS, D>;
  const int64_t gid = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  const int c0 = 8 * (int)(gid % (D / 8));
  const int64_t row = gid / (D / 8);
  const bool is_v = row & 1;
  const int64_t token = (row >> 1) / a.kv_heads;
  const int head = (int)((row >> 1) % a.kv_heads);
  if (token >= a.tokens) return;   // whole rows of lanes leave together
  const int32_t slot = a.slots[token];
  if (slot < 0 || slot >= a.capacity) return;
  const uint16_t *x = (is_v ? a.xv + token * a.ldv : a.xk + token * a.ldk) + (int64_t)head * D + c0;
  float v[8];
  unpack8(*reinterpret_cast<const uint4 *>(x), v);
  if (D >= 128 && a.signs) {
    const int ch = head * D + c0;
    const uint32_t sb = a.signs[ch >> 5] >> (ch & 31);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = ((sb >> e) & 1u) ? -v[e] : v[e];
    const int jj = threadIdx.x & 15;
    fwht128_row16_signed(v, jj);
    const float sc = fwht_lane_sign(jj) * kInvSqrt128;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= sc;
  }
  const int t = slot & ((1 << a.page_shift) - 1);
  const int64_t ph = (int64_t)(slot >> a.page_shift) * a.kv_heads + head;
  const int64_t base = ph * ((int64_t)L::kUnits << a.page_shift);
  if constexpr (BITS == 16) {
    uint16_t *out = static_cast<uint16_t *>(is_v ? a.v : a.k) + base;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      out[is_v ? L::value_unit(t, c0 + e) : L::key_unit(t, c0 + e)] =
          __builtin_bit_cast(uint16_t, (_Float16)v[e]);
  } else {
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo = fminf(lo, v[e]);
      hi = fmaxf(hi, v[e]);
    }
    lo = row_min<D>(lo);
    hi = row_max<D>(hi);
    const float qmax = (float)((1 << BITS) - 1);
    _Float16 s16 = (_Float16)fminf((hi - lo) / qmax, 65504.0f);
    if (s16 == (_Float16)0.0f) s16 = (_Float16)1.0f;
    const float s = (float)s16;
    const float z = fminf(fmaxf(rintf((0.0f - lo) / s), 0.0f), qmax);
    uint32_t code[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) code[e] = (uint32_t)fminf(fmaxf(rintf(v[e] / s + z), 0.0f), qmax);
    uint8_t *out = static_cast<uint8_t *>(is_v ? a.v : a.k) + base;
    constexpr int kStep = BITS == 4 ? 2 : 1;
#pragma unroll
    for (int e = 0; e < 8; e += kStep) {
      const uint32_t b = BITS == 4 ? code[e] | (code[e + 1] << 4) : code[e];
      const int u = (c0 + e) / kStep;
      out[is_v ? L::value_unit(t, u) : L::key_unit(t, u)] = (uint8_t)b;
    }
    if (c0 == 0) (is_v ? a.v_params : a.k_params)[(ph << a.page_shift) + t] = pack_half2(s, z);
  }
}

template <int BITS, int D>
__global__ __launch_bounds__(kRowThreads) void kv_read_kernel(RowArgs a) {
  using L = Layout<BITS, D>;
  const int64_t gid = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  const int c0 = 8 * (int)(gid % (D / 8));
  const int64_t row = gid / (D / 8);
  const bool is_v = row & 1;
  const int64_t token = (row >> 1) / a.kv_heads;
  const int head = (int)((row >> 1) % a.kv_heads);
  if (token >= a.tokens) return;
  const int32_t slot = a.slots[token];
  float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (slot >= 0 && slot < a.capacity) {
    const int t = slot & ((1 << a.page_shift) - 1);
    const int64_t ph = (int64_t)(slot >> a.page_shift) * a.kv_heads + head;
    const int64_t base = ph * ((int64_t)L::kUnits << a.page_shift);
    if constexpr (BITS == 16) {
      const uint16_t *in = static_cast<const uint16_t *>(is_v ? a.v : a.k) + base;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = half_bits_to_float(in[is_v ? L::value_unit(t, c0 + e) : L::key_unit(t, c0 + e)]);
    } else {
      const uint8_t *in = static_cast<const uint8_t *>(is_v ? a.v : a.k) + base;
      const uint32_t par = (is_v ? a.v_params : a.k_params)[(ph << a.page_shift) + t];
      const float s = half_bits_to_float(par & 0xFFFF), z = half_bits_to_float(par >> 16);
      constexpr int kStep = BITS == 4 ? 2 : 1;
#pragma unroll
      for (int e = 0; e < 8; e += kStep) {
        const int u = (c0 + e) / kStep;
        const uint32_t b = in[is_v ? L::value_unit(t, u) : L::key_unit(t, u)];
        if (BITS == 4) {
          v[e] = ((float)(b & 15u) - z) * s;
          v[e + 1] = ((float)(b >> 4) - z) * s;
        } else {
          v[e] = ((float)b - z) * s;
        }
      }
    }
  }
  // rotated back: x = D H x' / sqrt(128) (H is symmetric)
  if (D >= 128 && a.signs) {
    const int jj = threadIdx.x & 15;
    fwht128_row16_signed(v, jj);
    const float sc = fwht_lane_sign(jj) * kInvSqrt128;
    const int ch = head * D + c0;
    const uint32_t sb = a.signs[ch >> 5] >> (ch & 31);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= ((sb >> e) & 1u) ? -sc : sc;
  }
  uint16_t *x = (is_v ? a.xv + token * a.ldv : a.xk + token * a.ldk) + (int64_t)head * D + c0;
  *reinterpret_cast<uint4 *>(x) = make_uint4(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]), pack_half2(v[4], v[5]),
                                             pack_half2(v[6], v[7]));
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

template <int BITS, int D>
hipError_t launch_rows(const RowArgs &a, bool write, hipStream_t s) {
  const int64_t threads = a.tokens * a.kv_heads * 2 * (D / 8);
  const int64_t wgs = (threads + kRowThreads - 1) / kRowThreads;
  if (wgs > INT32_MAX) return hipErrorInvalidValue;
  if (write)
    hipLaunchKernelGGL((kv_write_kernel<BITS, D>), dim3((unsigned)wgs), dim3(kRowThreads), 0, s, a);
  else
    hipLaunchKernelGGL((kv_read_kernel<BITS, D>), dim3((unsigned)wgs), dim3(kRowThreads), 0, s, a);
  return hipGetLastError();
}

template <int BITS>
hipError_t launch_rows_bits(int d, const RowArgs &a, bool write, hipStream_t s) {
  switch (d) {
    case 64: return launch_rows<BITS, 64>(a, write, s);
    case 128: return launch_rows<BITS, 128>(a, write, s);
    case 256: return launch_rows<BITS, 256>(a, write, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_rows_any(const wq_kv_cache &c, const RowArgs &a, bool write, hipStream_t s) {
  switch (c.bits) {
    case 4: return launch_rows_bits<4>(c.head_dim, a, write, s);
    case 8: return launch_rows_bits<8>(c.head_dim, a, write, s);
    case 16: return launch_rows_bits<16>(c.head_dim, a, write, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_kv_write(const wq_kv_cache &c, const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv,
                           const int32_t *slots, int64_t tokens, hipStream_t s) {
  return launch_rows_any(c, row_args(c, slots, tokens, k, ldk, v, ldv), true, s);
}

hipError_t launch_kv_read(const wq_kv_cache &c, const int32_t *slots, int64_t tokens, uint16_t *k, int64_t ldk,
                          uint16_t *v, int64_t ldv, hipStream_t s) {
  return launch_rows_any(c, row_args(c, slots, tokens, k, ldk, v, ldv), false, s);
}

}  // namespace wq
