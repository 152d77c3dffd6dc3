// The next token of every row of logits under temperature, top-k, top-p and
// min-p (gfx950).
//
// Logits become keys, whole numbers in the logits' order (-0 as 0, NaN as
// -infinity), and weights w = exp((l - max) / T), computed in fp64 and counted
// in 2^-unit: their sums are exact whole numbers, the same in any order, so
// borders between tokens (1e-6 of the sum apart where a distribution is open)
// fall where 64 bits put them.  What top-k and top-p keep is everything above
// one key and the first few, by index, at it; both keys are found by a search
// over the key's bits, 11, 11 and 10 at a time, with counts (top-k) or sums
// (top-p) of the keys that share the bits found so far.
#include "wq_internal.h"

namespace wq {
using namespace dev;

namespace {

constexpr int kSampleThreads = 1024;
constexpr int kBins = 2048;
constexpr int kTile = 4 * kSampleThreads;          // logits of one turn
constexpr int kTiles = (1 << 20) / kTile;    // most turns
constexpr uint32_t kNoKey = 0x007FFFFFu;     // of -infinity

template <bool F32>
__device__ __forceinline__ float logit(const void *row, int64_t i) {
  if (F32) return static_cast<const float *>(row)[i];
  return (float)static_cast<const _Float16 *>(row)[i];
}

__device__ __forceinline__ uint32_t key_of(float l) {
  if (l != l) return kNoKey;
  const uint32_t b = __builtin_bit_cast(uint32_t, l + 0.0f);
  return b ^ ((int32_t)b < 0 ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ float value_of(uint32_t key) {
  return __builtin_bit_cast(float, key ^ (key & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu));
}

// exp(z) for z <= 0 in fp64: 2^n exp(r), |r| <= ln 2 / 2, the series of exp
// up to r^12 / 12! (its next term is below 2^-57 of the sum)
__device__ __forceinline__ double exp64(double z) {
  if (!(z > -100.0)) return 0.0;   // below any unit
  const double n = rint(z * 1.4426950408889634074);
  const double r = fma(-n, 1.9082149292705877e-10, fma(-n, 0.69314718036912381649, z));
  double p = 1.0 / 479001600.0;
  p = fma(p, r, 1.0 / 39916800.0);
  p = fma(p, r, 1.0 / 3628800.0);
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return ldexp(p, (int)n);
}

struct Scale {
  double max, per;     // the row's largest logit, 1 / T
  uint32_t top;        // its key
  double unit;         // 2^unit
};

__device__ __forceinline__ double weight(uint32_t key, const Scale &s) {
  if (key == s.top) return 1.0;
  if (key <= kNoKey) return 0.0;
  return exp64(((double)value_of(key) - s.max) * s.per);
}

__device__ __forceinline__ uint64_t counted(double w, const Scale &s) { return (uint64_t)rint(w * s.unit); }

template <typename T, typename F>
__device__ __forceinline__ T block_reduce(T v, T *tmp, F f) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = f(v, __shfl_xor(v, d));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
  __syncthreads();
  T r = tmp[0];
  for (int w = 1; w < kSampleThreads / 64; ++w) r = f(r, tmp[w]);
  return r;
}

// the sum of v over the threads before this one
__device__ __forceinline__ uint64_t block_before(uint64_t v, uint64_t *tmp) {
  uint64_t up = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t o = __shfl_up(up, d);
    if ((int)(threadIdx.x & 63) >= d) up += o;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 63) tmp[threadIdx.x >> 6] = up;
  __syncthreads();
  uint64_t before = up - v;
  for (int w = 0; w < (int)(threadIdx.x >> 6); ++w) before += tmp[w];
  return before;
}

struct Shared {
  uint64_t bins[kBins];
  uint64_t sums[kTiles];       // of each turn: w above the key
  uint32_t ties[kTiles];       // of each turn: logits at the key
  uint64_t tmp[kSampleThreads / 64];
  uint32_t digit;
  uint64_t above;
};

// The key at which the sum over falling keys, of counts or of weights, of
// those at or above `floor` first reaches `want` (> 0), and the sum above it.
template <bool F32, bool WEIGHTS>
__device__ uint32_t search(const void *row, int n, const Scale &s, uint32_t floor, uint64_t want, uint64_t &above,
                           Shared &sh) {
  uint32_t prefix = 0;
  above = 0;
  int shift = 32;
  for (int level = 0; level < 3; ++level) {
    const int bits = level == 2 ? 10 : 11, next = shift - bits;
    for (int i = threadIdx.x; i < kBins; i += kSampleThreads) sh.bins[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kSampleThreads) {
      const uint32_t key = key_of(logit<F32>(row, i));
      if (key < floor || (level && key >> shift != prefix >> shift)) continue;
      const uint64_t add = WEIGHTS ? counted(weight(key, s), s) : 1;
      if (add) atomicAdd(reinterpret_cast<unsigned long long *>(&sh.bins[(key >> next) & ((1u << bits) - 1)]), add);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      uint64_t sum = above;
      int d = (1 << bits) - 1;
      for (; d > 0 && sum + sh.bins[d] < want; --d) sum += sh.bins[d];
      sh.digit = d;
      sh.above = sum;
    }
    __syncthreads();
    prefix |= sh.digit << next;
    above = sh.above;
    shift = next;
    __syncthreads();
  }
  return prefix;
}

template <bool F32>
__global__ __launch_bounds__(kSampleThreads) void sample_kernel(SampleArgs a) {
  __shared__ Shared sh;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, n = a.vocab;
  const void *row = F32 ? (const void *)(static_cast<const float *>(a.logits) + r * a.ldl)
                        : (const void *)(static_cast<const uint16_t *>(a.logits) + r * a.ldl);
  const float heat = a.temperature ? a.temperature[r] : 1.0f;
  float u = a.u[r];
  u = u > 0.0f ? (u < 1.0f ? u : 1.0f) : 0.0f;
  const float floor_p = a.min_p ? a.min_p[r] : 0.0f;
  const double at_least = floor_p > 0.0f ? (floor_p < 1.0f ? (double)floor_p : 1.0) : 0.0;
  float top_p = a.top_p ? a.top_p[r] : 1.0f;
  if (!(top_p < 1.0f)) top_p = 1.0f;
  int top_k = a.top_k ? a.top_k[r] : 0;
  if (top_k <= 0 || top_k > n) top_k = n;

  // the largest, and where it is first
  uint64_t best = 0;
  for (int i = tid; i < n; i += kSampleThreads) {
    const uint64_t k = (uint64_t)key_of(logit<F32>(row, i)) << 32 | (uint32_t)~i;
    best = k > best ? k : best;
  }
  best = block_reduce(best, sh.tmp, [](uint64_t x, uint64_t y) { return x > y ? x : y; });
  Scale s;
  s.top = (uint32_t)(best >> 32);
  if (s.top <= kNoKey || !(heat > 0.0f)) {
    if (tid == 0) {
      a.ids[r] = s.top <= kNoKey ? -1 : (int32_t)~(uint32_t)best;
      if (a.logprobs) a.logprobs[r] = s.top <= kNoKey ? -INFINITY : 0.0f;
    }
    return;
  }
  s.max = value_of(s.top);
  s.per = 1.0 / (double)heat;
  s.unit = ldexp(1.0, a.unit);

  // what is kept: keys above `cut`, and the first `ties` at it
  uint32_t cut = 0;
  uint64_t ties = n;
  if (top_k < n) {
    uint64_t above;
    cut = search<F32, false>(row, n, s, 0, top_k, above, sh);
    ties = top_k - above;
  }
  if (top_p < 1.0f) {
    uint64_t sum = 0;
    for (int i = tid; i < n; i += kSampleThreads) {
      const uint32_t key = key_of(logit<F32>(row, i));
      if (key > cut) sum += counted(weight(key, s), s);
    }
    const uint64_t over = block_reduce(sum, sh.tmp, [](uint64_t x, uint64_t y) { return x + y; });
    const uint64_t tie = counted(weight(cut, s), s), all = over + ties * tie;
    // kept are those before which less than p * all lies
    uint64_t want = (uint64_t)ceil((double)(top_p > 0.0f ? top_p : 0.0f) * (double)all);
    if (want == 0) want = 1;
    if (want > over) {   // among top-k's ties
      const uint64_t some = (want - over + tie - 1) / tie;
      ties = some < ties ? some : ties;
    } else {
      uint64_t above;
      cut = search<F32, true>(row, n, s, cut + 1, want, above, sh);
      const uint64_t w = counted(weight(cut, s), s);
      ties = (want - above + w - 1) / w;
    }
  }

  // sums of each turn, in the order of the index
  const double cut_weight = weight(cut, s);
  const uint64_t tie = cut_weight >= at_least ? counted(cut_weight, s) : 0;
  const int turns = (n + kTile - 1) / kTile;
  for (int t = tid; t < turns; t += kSampleThreads) sh.sums[t] = sh.ties[t] = 0;
  __syncthreads();
  for (int t = 0; t < turns; ++t) {
    uint64_t sum = 0;
    uint32_t same = 0;
    for (int i = t * kTile + tid; i < n && i < (t + 1) * kTile; i += kSampleThreads) {
      const uint32_t key = key_of(logit<F32>(row, i));
      same += key == cut;
      if (key > cut) {
        const double w = weight(key, s);
        if (w >= at_least) sum += counted(w, s);
      }
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      sum += __shfl_xor(sum, d);
      same += __shfl_xor(same, d);
    }
    if ((tid & 63) == 0) {
      if (sum) atomicAdd(reinterpret_cast<unsigned long long *>(&sh.sums[t]), sum);
      if (same) atomicAdd(&sh.ties[t], same);
    }
  }
  __syncthreads();
  uint64_t all = 0, seen = 0;
  for (int t = 0; t < turns; ++t) {
    const uint64_t kept = sh.ties[t] < ties - seen ? sh.ties[t] : ties - seen;
    all += sh.sums[t] + kept * tie;
    seen += kept;
  }
  uint64_t target = (uint64_t)floor((double)u * (double)all);
  if (target >= all) target = all - 1;
  uint64_t before = 0;
  seen = 0;
  int t = 0;
  for (;; ++t) {
    const uint64_t kept = sh.ties[t] < ties - seen ? sh.ties[t] : ties - seen;
    const uint64_t here = sh.sums[t] + kept * tie;
    if (before + here > target) break;
    before += here;
    seen += kept;
  }
  // the turn's logits, four in a row to a thread
  const int first = t * kTile + 4 * tid;
  uint32_t key[4];
  uint64_t same = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    key[e] = first + e < n ? key_of(logit<F32>(row, first + e)) : 0;
    same += key[e] == cut && cut;
  }
  uint64_t rank = seen + block_before(same, sh.tmp);
  uint64_t w[4], mine = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    w[e] = 0;
    if (key[e] > cut) {
      const double v = weight(key[e], s);
      if (v >= at_least) w[e] = counted(v, s);
    } else if (key[e] == cut && cut) {
      if (rank < ties) w[e] = tie;
      ++rank;
    }
    mine += w[e];
  }
  uint64_t sum = before + block_before(mine, sh.tmp);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (sum <= target && sum + w[e] > target) {
      a.ids[r] = first + e;
      if (a.logprobs) {
        const double z = key[e] == s.top ? 0.0 : ((double)value_of(key[e]) - s.max) * s.per;
        a.logprobs[r] = (float)(z - log((double)all / s.unit));
      }
    }
    sum += w[e];
  }
}

}  // namespace

hipError_t launch_sample(const SampleArgs &a, hipStream_t s) {
  if (a.f32)
    hipLaunchKernelGGL(sample_kernel<true>, dim3((unsigned)a.rows), dim3(kSampleThreads), 0, s, a);
  else
    hipLaunchKernelGGL(sample_kernel<false>, dim3((unsigned)a.rows), dim3(kSampleThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace wq
