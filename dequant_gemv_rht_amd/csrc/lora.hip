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
// a group, rows of one adapter, gathered by their ids.  Of few rows, or up to
// kWholeRows with many adapters, one workgroup stands for each row: it looks
// through all ids, and goes on if it is the first of its group (16 rows).
// Otherwise a workgroup stands for 32 (inner) or 64 (outer) rows in succession
// and takes their groups in turn, or every slots-th of them: where there are
// few rows, several workgroups share them in case every row has an adapter of
// its own.  (The host knows how many adapters there are, not the rows' ids.)
//
// Measured: 128 rows with an adapter each, seven projections, rank 32: inner
// 42 us for 218 MB (5.2 TB/s), outer 58 us for 268 MB (4.6); plain reads of
// that size reach 6.4.  64 rows of 28 adapters, two projections, rank 16: 5.6
// and 11.0 us (27 MB), of which starting 900 and 1024 workgroups, 28 of 64 of
// which find a group, is about half.  4001 rows of three requests, three
// projections, rank 64: a call of 59 us (124 MB; with the rows' pieces spread
// over all XCDs, and twice as many of the outputs, 67).  One row: 4.6 and 5.0 us.
//
// What mattered: loads with no branch between them (a branch for each vector,
// or two paths that the compiler joins, keeps them apart or cuts them into
// words: 45 and 75 us for the outer kernel of the 4001 rows), x and A through
// LDS in rows of 512 bytes (straight into the matrix layout, 64 bytes of 16
// rows at a time: 54 us for the 218 MB), 16-byte LDS accesses (the union
// aligned to 16).  Not kept: waves that go their own way over a compact list
// of groups (61 to 75 us), a second set of registers for the next step (three
// instead of five waves a SIMD: 71 to 83 us).
//
// The matrix instruction's columns are rows of x; a group's last row fills
// the columns it leaves, which are not stored.
#include "wq_internal.h"

namespace wq {
using namespace dev;

namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float4_t __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kXcds = 8;
constexpr int kLoraThreads = 64 * kWaves;
static_assert(kWholeRows == kLoraThreads, "a thread looks at one id");

__device__ __forceinline__ half8_t zero8() {
  half8_t z;
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = (_Float16)0.0f;
  return z;
}

__device__ __forceinline__ uint64_t below(int n) { return n >= 64 ? ~0ull : (1ull << n) - 1; }

// Runs f(id, rows in list) for the workgroup's groups, of at most 16 CT rows;
// id -1: no adapter.
template <bool WHOLE, int CT, typename F>
__device__ __forceinline__ void for_groups(const LoraArgs &g, int32_t adapters, int32_t *list, uint64_t *masks, int b, int slot, F f) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
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
    const int64_t row = (int64_t)b * (16 * CT) + lane;
    const bool live = lane < 16 * CT && row < g.m;
    const int32_t mine = live ? known(g.ids[row]) : -1;
    uint64_t left = __ballot(live);
    for (int i = 0; left; ++i) {
      const int32_t id = __shfl(mine, __ffsll((unsigned long long)left) - 1);
      const uint64_t same = __ballot(live && mine == id) & left;
      left &= ~same;
      if (i % g.slots != slot) continue;   // another workgroup's
      __syncthreads();   // the last group's list is no longer needed
      if (wave == 0 && (same >> lane & 1)) list[__popcll(same & below(lane))] = (int32_t)row;
      __syncthreads();
      f(id, __popcll(same));
    }
  }
}

// Which rows, which piece of K or of the outputs, and what else of it a
// workgroup takes.  NEAR: the pieces of some rows follow each other on one
// XCD (workgroups go to the eight in turn), whose L2 then has x or t.
struct Part {
  int tile;
  uint32_t piece;
  int rest;
};

template <bool WHOLE>
__device__ __forceinline__ Part part_of(uint32_t pieces, bool near) {
  if (WHOLE || !near) return {(int)blockIdx.x, blockIdx.y, (int)blockIdx.z};
  return {(int)(blockIdx.z * kXcds + blockIdx.x), blockIdx.y % pieces, (int)(blockIdx.y / pieces)};
}

// The linear that piece `i` of a launch is of, and which of its pieces it is
__device__ __forceinline__ int linear_of(const LoraArgs &g, const uint32_t *to, uint32_t &i) {
  int l = 0;
#pragma unroll
  for (int k = 0; k < kMaxBatch - 1; ++k) l += k + 1 < g.count && i >= to[k];
  l = __builtin_amdgcn_readfirstlane(l);
  i -= l ? to[l - 1] : 0;
  return l;
}

constexpr int kStage = 256;            // channels staged in LDS at once
constexpr int kStageLd = kStage + 8;   // 16 rows of 16 bytes on different banks

// t of RT x CT sixteens of ranks and rows over the workgroup's channels.
// Rows come through LDS, 512 bytes of each at a time: loaded straight into
// the matrix instructions' layout they would be fetched in pieces of 64.  The
// next piece is on its way while this one is multiplied, two 32-wide steps a
// wave; what the waves have is added at the end.
template <bool WHOLE, int RT, int CT>
__global__ __launch_bounds__(kLoraThreads) void lora_inner_kernel(LoraArgs g) {
  constexpr int kRanks = 16 * RT, kRows = 16 * CT, kSumLd = kRanks + 4;
  __shared__ int32_t list[kRows];
  __shared__ uint64_t masks[kWaves];
  __shared__ union alignas(16) {
    _Float16 rows[kRanks + kRows][kStageLd];
    float sums[kWaves][16][kSumLd];
  } lds;
  const Part part = part_of<WHOLE>(g.splits_to[g.count - 1], g.near);
  uint32_t split = part.piece;
  const LoraDesc L = g.lin[linear_of(g, g.splits_to, split)];
  const int slot = part.rest % g.slots, r0 = part.rest / g.slots * kRanks;   // first rank
  const int k0 = (int)split * g.steps * 32, k1 = min(L.k, k0 + g.steps * 32);
  if (r0 >= L.rank) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, q = lane >> 4;
  const int row = tid >> 5, at = 8 * (tid & 31);   // a thread's rows row + 8 i and its 8 channels
  for_groups<WHOLE, CT>(g, L.count, list, masks, part.tile, slot, [&](int32_t id, int rows) {
    if (id < 0) return;
    // ranks and rows past the last repeat it and are not stored; channels
    // past the last are zeros
    half8_t a[2 * RT], x[2 * CT];
    const _Float16 *ap[2 * RT], *xp[2 * CT];
#pragma unroll
    for (int i = 0; i < 2 * RT; ++i)
      ap[i] = reinterpret_cast<const _Float16 *>(L.a) + ((int64_t)id * L.rank + min(r0 + row + 8 * i, L.rank - 1)) * L.k;
#pragma unroll
    for (int i = 0; i < 2 * CT; ++i)
      xp[i] = reinterpret_cast<const _Float16 *>(L.x) + list[min(row + 8 * i, rows - 1)] * L.ldx;
    const auto load = [&](int k) {
      const int from = min(k + at, k1 - 8);
#pragma unroll
      for (int i = 0; i < 2 * RT; ++i) a[i] = *reinterpret_cast<const half8_t *>(ap[i] + from);
#pragma unroll
      for (int i = 0; i < 2 * CT; ++i) x[i] = *reinterpret_cast<const half8_t *>(xp[i] + from);
    };
    const auto clear = [&](int k) {
      const bool in = k + at < k1;
#pragma unroll
      for (int i = 0; i < 2 * RT; ++i) a[i] = in ? a[i] : zero8();
#pragma unroll
      for (int i = 0; i < 2 * CT; ++i) x[i] = in ? x[i] : zero8();
    };
    float4_t acc[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < CT; ++t) acc[r][t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    load(k0);
    for (int k = k0; k < k1; k += kStage) {
      __syncthreads();   // the last piece is multiplied
      if (k + kStage > k1) clear(k);
#pragma unroll
      for (int i = 0; i < 2 * RT; ++i) *reinterpret_cast<half8_t *>(&lds.rows[row + 8 * i][at]) = a[i];
#pragma unroll
      for (int i = 0; i < 2 * CT; ++i) *reinterpret_cast<half8_t *>(&lds.rows[kRanks + row + 8 * i][at]) = x[i];
      __syncthreads();
      if (k + kStage < k1) load(k + kStage);
#pragma unroll
      for (int s = 0; s < kStage / 32 / kWaves; ++s) {
        const int from = 32 * (wave * (kStage / 32 / kWaves) + s) + 8 * q;
        half8_t am[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) am[r] = *reinterpret_cast<const half8_t *>(&lds.rows[16 * r + c][from]);
#pragma unroll
        for (int t = 0; t < CT; ++t) {
          const half8_t xm = *reinterpret_cast<const half8_t *>(&lds.rows[kRanks + 16 * t + c][from]);
#pragma unroll
          for (int r = 0; r < RT; ++r) acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(am[r], xm, acc[r][t], 0, 0, 0);
        }
      }
    }
    const float scale = L.scales ? L.scales[id] : 1.0f;
    float *out = L.t + (int64_t)split * g.m * L.rank + r0;
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      if (16 * t >= rows) break;
      __syncthreads();
#pragma unroll
      for (int r = 0; r < RT; ++r) *reinterpret_cast<float4_t *>(&lds.sums[wave][c][16 * r + 4 * q]) = acc[r][t];
      __syncthreads();
      for (int i = tid; i < 16 * kRanks; i += kLoraThreads) {
        const int col = i / kRanks, rank = i % kRanks;
        if (16 * t + col < rows && r0 + rank < L.rank) {
          float sum = lds.sums[0][col][rank];
#pragma unroll
          for (int w = 1; w < kWaves; ++w) sum += lds.sums[w][col][rank];
          out[(int64_t)list[16 * t + col] * L.rank + rank] = sum * scale;
        }
      }
    }
  });
}

// A lane's 16 outputs of a row in one step of the outer product, 16 bytes
// side by side; vector v's first is 4 V v + V q past the step's.
template <typename T>
struct Run {
  static constexpr int V = 16 / sizeof(T), N = 16 / V;   // of a vector; vectors
  T v[N][V];
};

// FULL: all 64 outputs of the step are there.  The last step of a linear may
// lack some and goes one by one; it has code of its own, a branch for each
// vector would keep the loads apart.
template <bool FULL, typename T>
__device__ __forceinline__ Run<T> load_run(const T *row, int n, int end) {
  constexpr int V = Run<T>::V;
  Run<T> r;
  if constexpr (FULL) {
#pragma unroll
    for (int i = 0; i < Run<T>::N; ++i) __builtin_memcpy(r.v[i], row + n + 4 * V * i, 16);   // at any alignment
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) r.v[i / V][i % V] = row[min(n + 4 * V * (i / V) + i % V, end - 1)];
  }
  return r;
}

template <bool FULL, typename T>
__device__ __forceinline__ void store_run(T *row, int n, int end, const Run<T> &r) {
  constexpr int V = Run<T>::V;
  if constexpr (FULL) {
#pragma unroll
    for (int i = 0; i < Run<T>::N; ++i) __builtin_memcpy(row + n + 4 * V * i, r.v[i], 16);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int at = n + 4 * V * (i / V) + i % V;
      if (at < end) row[at] = r.v[i / V][i % V];
    }
  }
}

// B's part of the 64 outputs from n on: instruction j's output row 4 q + i is
// the output that is element 4 j + i of lane q's run.  Outputs past the last
// repeat it and are not stored; ranks past the last repeat the last eight and
// meet zeros in t.
template <bool FULL, typename T, int KK, bool PACK>
__device__ __forceinline__ void load_b(const LoraDesc &L, int32_t id, int n, half8_t (&b)[4][KK]) {
  constexpr int V = Run<T>::V;
  const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    int at = n + 4 * V * (4 * j / V) + V * (c >> 2) + 4 * j % V + (c & 3);
    if (!FULL) at = min(at, L.n - 1);
    const _Float16 *bp = reinterpret_cast<const _Float16 *>(L.b) + ((int64_t)id * L.n + at) * L.rank;
#pragma unroll
    for (int k = 0; k < KK; ++k) {
      const int rank = PACK ? 8 * (q & 1) : 32 * k + 8 * q;
      b[j][k] = *reinterpret_cast<const half8_t *>(bp + min(rank, L.rank - 8));
    }
  }
}

// t of 16 rows (lane: row c, ranks 8 q ..) as two fp16 parts under a power of
// two of its row: its largest in [2^13, 2^14), infinities as they are.
template <int KK, bool PACK>
__device__ __forceinline__ int load_parts(const LoraArgs &g, const LoraDesc &L, int32_t row,
                                          half8_t (&parts)[KK][PACK ? 1 : 2]) {
  const int q = (threadIdx.x & 63) >> 4, splits = (L.k / 32 + g.steps - 1) / g.steps;
  float v[KK][8], most = 0.0f;
#pragma unroll
  for (int k = 0; k < KK; ++k) {
    const int rank = PACK ? 8 * (q & 1) : 32 * k + 8 * q;
    const bool has = rank < L.rank;
    const float *t = L.t + (int64_t)row * L.rank + (has ? rank : 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[k][e] = 0.0f;
    for (int s0 = 0; s0 < splits; s0 += 4) {   // four splits asked for at once
      float4_t lo[4], hi[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const float4_t *at = reinterpret_cast<const float4_t *>(t + (int64_t)min(s0 + s, splits - 1) * g.m * L.rank);
        lo[s] = at[0];
        hi[s] = at[1];
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const bool adds = has && s0 + s < splits;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[k][e] += adds ? lo[s][e] : 0.0f;
          v[k][4 + e] += adds ? hi[s][e] : 0.0f;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(v[k][e]));
  }
  most = fmaxf(most, __shfl_xor(most, 16));
  most = fmaxf(most, __shfl_xor(most, 32));
  const int power = most > 0.0f && most <= 3.4028234e38f ? 14 - __builtin_amdgcn_frexp_expf(most) : 0;
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
      parts[k][0] = q < 2 ? hi : lo;
    } else {
      parts[k][0] = hi;
      parts[k][1] = lo;
    }
  }
  return -power;
}

template <typename T, int KK, bool PACK>
__device__ __forceinline__ void add_product(Run<T> &out, const half8_t (&b)[4][KK], const half8_t (&parts)[KK][PACK ? 1 : 2],
                                            int power) {
  constexpr int V = Run<T>::V;
  float4_t acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < KK; ++k)
#pragma unroll
    for (int p = 0; p < (PACK ? 1 : 2); ++p)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b[j][k], parts[k][p], acc[j], 0, 0, 0);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      T &o = out.v[4 * j / V][4 * j % V + e];
      o = (T)((float)o + ldexpf(acc[j][e], power));
    }
}

// The outputs [n0, n1) of one group: T base's and y's type.  KK: 32-wide
// steps over the ranks; PACK (ranks up to 16): both parts of t in one.
template <typename T, int KK, bool PACK, int CT>
__device__ __forceinline__ void outer_group(const LoraArgs &g, const LoraDesc &L, const int32_t *list,
                                            half8_t (*shared)[KK][PACK ? 1 : 2][64], int32_t (*powers)[16], int32_t id, int rows,
                                            int n0, int n1) {
  constexpr int V = Run<T>::V;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, q = lane >> 4;
  const int full = n1 < L.n ? n1 : L.n & ~63, end = L.n, own = V * q;   // the lane's first output of a step
  int n = n0 + 64 * wave;
  const T *base[CT];
  T *y[CT];
#pragma unroll
  for (int t = 0; t < CT; ++t) {
    const int32_t row = list[min(16 * t + c, rows - 1)];
    base[t] = static_cast<const T *>(L.base) + row * L.ldb;
    y[t] = static_cast<T *>(L.y) + row * L.ldy;
  }
  if (id < 0) {
    if (L.y == L.base) return;
    for (; n < n1; n += 64 * kWaves)
#pragma unroll
      for (int t = 0; t < CT; ++t) {
        if (16 * t + c >= rows) continue;
        if (n < full)
          store_run<true>(y[t], n + own, end, load_run<true>(base[t], n + own, end));
        else
          store_run<false>(y[t], n + own, end, load_run<false>(base[t], n + own, end));
      }
    return;
  }
  // B and base do not wait for t; tiles past the group's last repeat its last row
  half8_t b[4][KK];
  Run<T> out[CT];
  const auto load = [&](int at) {
    load_b<true, T, KK, PACK>(L, id, at, b);
#pragma unroll
    for (int t = 0; t < CT; ++t) out[t] = load_run<true>(base[t], at + own, end);
  };
  if (n < full) load(n);
  // wave w makes the parts of the group's rows 16 w .. 16 w + 15
  if (wave < CT && 16 * wave < rows) {
    half8_t parts[KK][PACK ? 1 : 2];
    const int power = load_parts<KK, PACK>(g, L, list[min(16 * wave + c, rows - 1)], parts);
    if (q == 0) powers[wave][c] = power;
#pragma unroll
    for (int k = 0; k < KK; ++k)
#pragma unroll
      for (int p = 0; p < (PACK ? 1 : 2); ++p) shared[wave][k][p][lane] = parts[k][p];
  }
  __syncthreads();
  const auto add = [&](int t) {
    half8_t parts[KK][PACK ? 1 : 2];
#pragma unroll
    for (int k = 0; k < KK; ++k)
#pragma unroll
      for (int p = 0; p < (PACK ? 1 : 2); ++p) parts[k][p] = shared[t][k][p][lane];
    add_product<T, KK, PACK>(out[t], b, parts, powers[t][c]);
  };
  while (n < full) {
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      if (16 * t >= rows) break;
      add(t);
      if (16 * t + c < rows) store_run<true>(y[t], n + own, end, out[t]);
    }
    n += 64 * kWaves;
    if (n < full) load(n);
  }
  if (n < n1) {
    load_b<false, T, KK, PACK>(L, id, n, b);
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      if (16 * t >= rows) break;
      out[t] = load_run<false>(base[t], n + own, end);
      add(t);
      if (16 * t + c < rows) store_run<false>(y[t], n + own, end, out[t]);
    }
  }
}

template <bool WHOLE, int KK, bool PACK, int CT>
__global__ __launch_bounds__(kLoraThreads) void lora_outer_kernel(LoraArgs g) {
  __shared__ int32_t list[16 * CT];
  __shared__ uint64_t masks[kWaves];
  __shared__ alignas(16) half8_t parts[CT][KK][PACK ? 1 : 2][64];
  __shared__ int32_t powers[CT][16];
  const Part part = part_of<WHOLE>(g.chunks_to[g.count - 1], g.near);
  uint32_t chunk = part.piece;
  const LoraDesc L = g.lin[linear_of(g, g.chunks_to, chunk)];
  const int n0 = (int)chunk * g.chunk, n1 = min(n0 + g.chunk, L.n);
  for_groups<WHOLE, CT>(g, L.count, list, masks, part.tile, part.rest, [&](int32_t id, int rows) {
    if (L.f32)
      outer_group<float, KK, PACK, CT>(g, L, list, parts, powers, id, rows, n0, n1);
    else
      outer_group<_Float16, KK, PACK, CT>(g, L, list, parts, powers, id, rows, n0, n1);
  });
}

dim3 grid(int64_t tiles, uint32_t pieces, uint32_t rest, bool near) {
  if (near) return dim3(kXcds, pieces * rest, (unsigned)((tiles + kXcds - 1) / kXcds));
  return dim3((unsigned)tiles, pieces, rest);
}

// CI, CO: sixteens of rows of a group in the inner and the outer kernel
template <bool WHOLE, int CI, int CO>
hipError_t launch(const LoraArgs &a, const LoraPlan &p, hipStream_t s) {
  const auto inner = [&](auto kernel, int tiles) {
    const uint32_t parts = (uint32_t)((p.rank + 16 * tiles - 1) / (16 * tiles));
    hipLaunchKernelGGL(kernel, grid(p.inner_tiles, p.splits, parts * (uint32_t)p.slots, a.near), dim3(kLoraThreads), 0,
                       s, a);
  };
  if (p.rank <= 16)
    inner(lora_inner_kernel<WHOLE, 1, CI>, 1);
  else if (p.rank <= 32)
    inner(lora_inner_kernel<WHOLE, 2, CI>, 2);
  else
    inner(lora_inner_kernel<WHOLE, 4, CI>, 4);
  const auto outer = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid(p.outer_tiles, p.chunks, (uint32_t)p.slots, a.near), dim3(kLoraThreads), 0, s, a);
  };
  if (p.rank <= 16)
    outer(lora_outer_kernel<WHOLE, 1, true, CO>);
  else if (p.rank <= 32)
    outer(lora_outer_kernel<WHOLE, 1, false, CO>);
  else if (p.rank <= 64)
    outer(lora_outer_kernel<WHOLE, 2, false, CO>);
  else
    outer(lora_outer_kernel<WHOLE, 4, false, CO>);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lora(const LoraArgs &a, const LoraPlan &p, hipStream_t s) {
  return p.whole ? launch<true, 1, 1>(a, p, s) : launch<false, 2, 4>(a, p, s);
}

}  // namespace wq
