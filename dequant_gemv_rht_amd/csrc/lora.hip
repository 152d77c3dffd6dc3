// Low-rank adapters of many requests beside shared projections (gfx950):
// y = base + scale B (A x), each row with the adapter its id names.
#include "wq_internal.h"

namespace wq {
using namespace dev;

namespace {

constexpr int kLoraThreads = 256;

// t[row][r] = scale * sum_k a[id][r][k] x[row][k]: a wave a rank
__global__ __launch_bounds__(kLoraThreads) void lora_inner_kernel(LoraArgs g) {
  const LoraDesc L = g.lin[blockIdx.y];
  const int64_t row = blockIdx.x;
  const int32_t id = g.ids[row];
  if (id < 0 || id >= L.count) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const _Float16 *x = reinterpret_cast<const _Float16 *>(L.x) + row * L.ldx;
  const float scale = L.scales ? L.scales[id] : 1.0f;
  for (int r = wave; r < L.rank; r += kLoraThreads / 64) {
    const _Float16 *a = reinterpret_cast<const _Float16 *>(L.a) + ((int64_t)id * L.rank + r) * L.k;
    float sum = 0.0f;
    for (int k = lane; k < L.k; k += 64) sum += (float)a[k] * (float)x[k];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    if (lane == 0) L.t[row * L.rank + r] = sum * scale;
  }
}

__global__ __launch_bounds__(kLoraThreads) void lora_outer_kernel(LoraArgs g) {
  const LoraDesc L = g.lin[blockIdx.z];
  const int64_t row = blockIdx.x, n = (int64_t)blockIdx.y * kLoraThreads + threadIdx.x;
  if (n >= L.n) return;
  const int32_t id = g.ids[row];
  const int64_t at = row * L.ldb + n, to = row * L.ldy + n;
  float y = L.f32 ? static_cast<const float *>(L.base)[at] : (float)static_cast<const _Float16 *>(L.base)[at];
  if (id >= 0 && id < L.count) {
    const _Float16 *b = reinterpret_cast<const _Float16 *>(L.b) + ((int64_t)id * L.n + n) * L.rank;
    const float *t = L.t + row * L.rank;
    float sum = 0.0f;
    for (int r = 0; r < L.rank; ++r) sum += (float)b[r] * t[r];
    y += sum;
  }
  if (L.f32)
    static_cast<float *>(L.y)[to] = y;
  else
    static_cast<_Float16 *>(L.y)[to] = (_Float16)y;
}

}  // namespace

hipError_t launch_lora(const LoraArgs &a, hipStream_t s) {
  int32_t n = 0;
  for (int i = 0; i < a.count; ++i) n = a.lin[i].n > n ? a.lin[i].n : n;
  hipLaunchKernelGGL(lora_inner_kernel, dim3((unsigned)a.m, (unsigned)a.count), dim3(kLoraThreads), 0, s, a);
  hipLaunchKernelGGL(lora_outer_kernel, dim3((unsigned)a.m, (unsigned)((n + kLoraThreads - 1) / kLoraThreads), (unsigned)a.count),
                     dim3(kLoraThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace wq
