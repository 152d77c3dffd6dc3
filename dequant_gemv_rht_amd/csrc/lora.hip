// Low-rank adapters of many requests beside shared projections (gfx950):
// y = base + scale B (A x), each row with the adapter its id names.
//
// Two launches for all linears of a call, both on the matrix cores:
//   inner  t = scale A x: 16 ranks x 16 rows per v_mfma_f32_16x16x32_f16, K
//          split over workgroups and the four waves of each; a workgroup's
//          waves are added in LDS, workgroups' sums are kept apart
//   outer  y = base + B t: 16 outputs x 16 rows per instruction; t, the sum
//          of the splits, enters as two fp16 parts under a power of two of
//          its row
// Bound by the bytes of the adapters (decode) or of x, base and y (prompts).
// So every adapter is read once for the rows that share it: a workgroup takes
// a group, up to 64 rows of one adapter (16 where a call has no more rows),
// gathered by their ids.  Up to kWholeRows rows one workgroup stands for each
// row: it looks through all ids, and goes on if it is the first of its group.
// Above, a workgroup stands for 64 rows in succession and takes their groups
// in turn.
//
// The matrix instruction's columns are rows of x; a group's last row fills
// the columns it leaves, which are not stored.
#include "wq_internal.h"

namespace wq {
using namespace dev;

namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float4_t __attribute__((ext_vector_type(4)));

constexpr int kLoraThreads = 256;
constexpr int kWaves = kLoraThreads / 64;
constexpr int kBlockRows = 64;

__device__ __forceinline__ half8_t zero8() {
  half8_t z;
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = (_Float16)0.0f;
  return z;
}

__device__ __forceinline__ uint64_t below(int n) { return n >= 64 ? ~0ull : (1ull << n) - 1; }

// Runs f(id, rows in list) for the workgroup's groups; id -1: no adapter.
template <bool WHOLE, int CT, typename F>
__device__ __forceinline__ void for_groups(const LoraArgs &g, int32_t adapters, int32_t *list, uint64_t *masks, F f) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b = blockIdx.x;
  const auto known = [&](int32_t id) { return id >= 0 && id < adapters ? id : -1; };
  if (WHOLE) {
    const int32_t id = known(g.ids[b]);
    const bool same = tid < g.m && known(g.ids[tid < g.m ? tid : 0]) == id;
    const uint64_t ballot = __ballot(same);
    if (lane == 0) masks[wave] = ballot;
    __syncthreads();
    int before = 0, pos = 0, rows = 0;   // rows of the group before b, from b to this thread's, from b on
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const uint64_t at = masks[w], left = below(b - 64 * w < 0 ? 0 : b - 64 * w);
      before += __popcll(at & left);
      rows += __popcll(at & ~left);
      pos += w < wave ? __popcll(at & ~left) : w == wave ? __popcll(at & ~left & below(lane)) : 0;
    }
    if (before % (16 * CT)) return;
    if (rows > 16 * CT) rows = 16 * CT;
    if (same && tid >= b && pos < rows) list[pos] = tid;
    __syncthreads();
    f(id, rows);
  } else {
    const int64_t row = (int64_t)b * kBlockRows + lane;
    const bool live = row < g.m;
    const int32_t mine = live ? known(g.ids[row]) : -1;
    uint64_t left = __ballot(live);
    while (left) {
      const int32_t id = __shfl(mine, __ffsll((unsigned long long)left) - 1);
      const uint64_t same = __ballot(live && mine == id) & left;
      left &= ~same;
      __syncthreads();   // the last group's list is no longer needed
      if (wave == 0 && (same >> lane & 1)) list[__popcll(same & below(lane))] = (int32_t)row;
      __syncthreads();
      f(id, __popcll(same));
    }
  }
}

// One wave's part of A x over 32-wide steps [u0, u1): RT x NC tiles
template <int RT, int NC, int CT>
__device__ __forceinline__ void inner_steps(const _Float16 *const (&ap)[RT], const _Float16 *const (&xp)[CT], int u0, int u1,
                                            float4_t (&acc)[RT][CT]) {
#pragma unroll 4
  for (int u = u0; u < u1; ++u) {
    half8_t a[RT], x[NC];
#pragma unroll
    for (int r = 0; r < RT; ++r) a[r] = *reinterpret_cast<const half8_t *>(ap[r] + 32 * (int64_t)u);
#pragma unroll
    for (int c = 0; c < NC; ++c) x[c] = *reinterpret_cast<const half8_t *>(xp[c] + 32 * (int64_t)u);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[r], x[c], acc[r][c], 0, 0, 0);
  }
}

template <bool WHOLE, int RT, int CT>
__global__ __launch_bounds__(kLoraThreads) void lora_inner_kernel(LoraArgs g) {
  __shared__ int32_t list[kBlockRows];
  __shared__ uint64_t masks[kWaves];
  __shared__ float sums[kWaves][16][RT * 16 + 4];
  const int part = (int)blockIdx.z / g.count;
  const LoraDesc L = g.lin[blockIdx.z - part * g.count];
  const int r0 = part * RT * 16;   // first rank
  if (r0 >= L.rank) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, q = lane >> 4;
  const int units = L.k / 32, slice = (int)blockIdx.y * kWaves + wave, slices = (int)gridDim.y * kWaves;
  const int u0 = (int)((int64_t)units * slice / slices), u1 = (int)((int64_t)units * (slice + 1) / slices);
  for_groups<WHOLE, CT>(g, L.count, list, masks, [&](int32_t id, int rows) {
    if (id < 0) return;
    const _Float16 *ap[RT], *xp[CT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int rank = min(r0 + 16 * r + c, L.rank - 1);   // ranks past the last are not stored
      ap[r] = reinterpret_cast<const _Float16 *>(L.a) + ((int64_t)id * L.rank + rank) * L.k + 8 * q;
    }
#pragma unroll
    for (int t = 0; t < CT; ++t)
      xp[t] = reinterpret_cast<const _Float16 *>(L.x) + list[min(16 * t + c, rows - 1)] * L.ldx + 8 * q;
    float4_t acc[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < CT; ++t) acc[r][t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (CT == 1 || rows <= 16)
      inner_steps<RT, 1, CT>(ap, xp, u0, u1, acc);
    else
      inner_steps<RT, CT, CT>(ap, xp, u0, u1, acc);
    const float scale = L.scales ? L.scales[id] : 1.0f;
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      if (16 * t >= rows) break;
#pragma unroll
      for (int r = 0; r < RT; ++r) *reinterpret_cast<float4_t *>(&sums[wave][c][16 * r + 4 * q]) = acc[r][t];
      __syncthreads();
      const int col = tid >> 4;
      if (16 * t + col < rows) {
        float *out = L.t + ((int64_t)blockIdx.y * g.m + list[16 * t + col]) * L.rank;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const int at = 16 * r + (tid & 15);
          float sum = sums[0][col][at];
#pragma unroll
          for (int w = 1; w < kWaves; ++w) sum += sums[w][col][at];
          if (r0 + at < L.rank) out[r0 + at] = sum * scale;
        }
      }
      __syncthreads();
    }
  });
}

// 8 or 16 neighbours of a row at any alignment
template <typename T, int N>
struct Run {
  T v[N];
};

template <typename T>
__device__ __forceinline__ void add_out(const LoraDesc &L, int32_t row, int n, const float (&add)[16]) {
  const T *base = static_cast<const T *>(L.base) + row * L.ldb + n;
  T *y = static_cast<T *>(L.y) + row * L.ldy + n;
  if (n + 16 <= L.n) {
    Run<T, 16> r;
    __builtin_memcpy(&r, base, sizeof r);
#pragma unroll
    for (int i = 0; i < 16; ++i) r.v[i] = (T)((float)r.v[i] + add[i]);
    __builtin_memcpy(y, &r, sizeof r);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (n + i < L.n) y[i] = (T)((float)base[i] + add[i]);
  }
}

template <typename T>
__device__ __forceinline__ void copy_rows(const LoraDesc &L, const int32_t *list, int rows, int n0, int n1) {
  if (L.y == L.base) return;
  for (int r = 0; r < rows; ++r) {
    const T *base = static_cast<const T *>(L.base) + list[r] * L.ldb;
    T *y = static_cast<T *>(L.y) + list[r] * L.ldy;
    for (int n = n0 + (int)threadIdx.x; n < n1; n += kLoraThreads) y[n] = base[n];
  }
}

// KK: 32-wide steps over the ranks; PACK (ranks up to 16): both parts of t in one step
template <bool WHOLE, int KK, bool PACK, int CT>
__global__ __launch_bounds__(kLoraThreads) void lora_outer_kernel(LoraArgs g) {
  __shared__ int32_t list[kBlockRows];
  __shared__ uint64_t masks[kWaves];
  __shared__ half8_t parts[CT][KK][PACK ? 1 : 2][64];
  __shared__ int32_t powers[CT][16];
  const LoraDesc L = g.lin[blockIdx.z];
  const int n0 = (int)blockIdx.y * g.chunk;
  if (n0 >= L.n) return;
  const int n1 = min(n0 + g.chunk, L.n);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, q = lane >> 4;
  for_groups<WHOLE, CT>(g, L.count, list, masks, [&](int32_t id, int rows) {
    if (id < 0) {
      if (L.f32)
        copy_rows<float>(L, list, rows, n0, n1);
      else
        copy_rows<_Float16>(L, list, rows, n0, n1);
      return;
    }
    // wave w makes the parts of the group's rows 16 w .. 16 w + 15
    if (16 * wave < rows && wave < CT) {
      const int32_t row = list[min(16 * wave + c, rows - 1)];
      float v[KK][8], most = 0.0f;
#pragma unroll
      for (int k = 0; k < KK; ++k) {
        const int rank = PACK ? 8 * (q & 1) : 32 * k + 8 * q;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] = 0.0f;
        if (rank < L.rank)
          for (int s = 0; s < g.splits; ++s) {
            const float4_t *t = reinterpret_cast<const float4_t *>(L.t + ((int64_t)s * g.m + row) * L.rank + rank);
            const float4_t lo = t[0], hi = t[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[k][e] += lo[e];
              v[k][4 + e] += hi[e];
            }
          }
#pragma unroll
        for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(v[k][e]));
      }
      most = fmaxf(most, __shfl_xor(most, 16));
      most = fmaxf(most, __shfl_xor(most, 32));
      // the row's largest into [2^13, 2^14); infinities as they are
      const int power = most > 0.0f && most <= 3.4028234e38f ? 14 - __builtin_amdgcn_frexp_expf(most) : 0;
      if (q == 0) powers[wave][c] = -power;
#pragma unroll
      for (int k = 0; k < KK; ++k) {
        half8_t hi, lo;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = ldexpf(v[k][e], power);
          hi[e] = (_Float16)x;
          const float rest = x - (float)hi[e];
          lo[e] = (_Float16)(rest - rest == 0.0f ? rest : 0.0f);
        }
        if (PACK) {
          parts[wave][k][0][lane] = q < 2 ? hi : lo;
        } else {
          parts[wave][k][0][lane] = hi;
          parts[wave][k][1][lane] = lo;
        }
      }
    }
    __syncthreads();
    for (int n = n0 + 64 * wave; n < n1; n += 64 * kWaves) {
      // instruction j's output row r is output n + 16 (r / 4) + 4 j + r % 4,
      // so that a lane ends up with 16 neighbours
      half8_t b[4][KK];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = min(n + 16 * (c >> 2) + 4 * j + (c & 3), L.n - 1);
        const _Float16 *bp = reinterpret_cast<const _Float16 *>(L.b) + ((int64_t)id * L.n + at) * L.rank;
#pragma unroll
        for (int k = 0; k < KK; ++k) {
          const int rank = PACK ? 8 * (q & 1) : 32 * k + 8 * q;
          b[j][k] = rank < L.rank ? *reinterpret_cast<const half8_t *>(bp + rank) : zero8();
        }
      }
#pragma unroll
      for (int t = 0; t < CT; ++t) {
        if (16 * t >= rows) break;
        float4_t acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < KK; ++k)
#pragma unroll
          for (int p = 0; p < (PACK ? 1 : 2); ++p) {
            const half8_t part = parts[t][k][p][lane];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b[j][k], part, acc[j], 0, 0, 0);
          }
        if (16 * t + c < rows && n + 16 * q < n1) {
          const int power = powers[t][c];
          float add[16];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) add[4 * j + e] = ldexpf(acc[j][e], power);
          if (L.f32)
            add_out<float>(L, list[16 * t + c], n + 16 * q, add);
          else
            add_out<_Float16>(L, list[16 * t + c], n + 16 * q, add);
        }
      }
    }
    if (!WHOLE) __syncthreads();   // the parts are read
  });
}

template <bool WHOLE, int CT>
hipError_t launch(const LoraArgs &a, const LoraPlan &p, hipStream_t s) {
  const dim3 threads(kLoraThreads);
  const auto inner = [&](auto kernel, int tiles) {
    const unsigned parts = (unsigned)((p.rank + 16 * tiles - 1) / (16 * tiles));
    hipLaunchKernelGGL(kernel, dim3((unsigned)p.tiles, (unsigned)p.splits, parts * (unsigned)a.count), threads, 0, s, a);
  };
  if (p.rank <= 16)
    inner(lora_inner_kernel<WHOLE, 1, CT>, 1);
  else if (p.rank <= 32)
    inner(lora_inner_kernel<WHOLE, 2, CT>, 2);
  else
    inner(lora_inner_kernel<WHOLE, 4, CT>, 4);
  const auto outer = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)p.tiles, (unsigned)p.chunks, (unsigned)a.count), threads, 0, s, a);
  };
  if (p.rank <= 16)
    outer(lora_outer_kernel<WHOLE, 1, true, CT>);
  else if (p.rank <= 32)
    outer(lora_outer_kernel<WHOLE, 1, false, CT>);
  else if (p.rank <= 64)
    outer(lora_outer_kernel<WHOLE, 2, false, CT>);
  else
    outer(lora_outer_kernel<WHOLE, 4, false, CT>);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lora(const LoraArgs &a, const LoraPlan &p, hipStream_t s) {
  if (!p.whole) return launch<false, 4>(a, p, s);
  return p.narrow ? launch<true, 1>(a, p, s) : launch<true, 4>(a, p, s);
}

}  // namespace wq
