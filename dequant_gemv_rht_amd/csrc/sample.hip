// The next token of every row of logits under temperature, top-k, top-p and
// min-p (gfx950).
//
// A weight w = exp((l - max) / T) is counted in 2^-unit of a power of two near
// the largest, so that sums are whole numbers, exact and the same in any
// order; borders between tokens, 1e-6 of the sum apart and less where a
// distribution is open, fall where 64 bits put them.
//
// Two launches.  The first reads every logit once: a workgroup takes a part
// of a row, kPart logits in registers, and leaves its largest, its sum and,
// for rows with top-k, top-p or min-p, counts and sums in kBins bins of
// equal width (an eighth of a power of two, from its largest down).  Bins of
// all parts line up, so the second launch, a workgroup for each row, finds in
// which bin a cut lies, fetches that bin's logits alone (from the parts that
// have any), finds the cut among them bit by bit, and with it every part's
// sum of what is kept; the part in which the sum passes u times all of it is
// read again, token by token.  Rows for which that does not do (a cut below
// the bins, more logits in its bin than fit in LDS, logits or temperatures
// beyond 2^13 powers of two) are searched in as many passes as it takes.
#include "wq_internal.h"

namespace wq {
using namespace dev;

namespace {

constexpr uint32_t kNoKey = 0x007FFFFFu;     // of -infinity
constexpr int kBins = kSampleBins;
constexpr int kPart = kSamplePart;
constexpr int kPartThreads = 256;
constexpr int kEach = kPart / kPartThreads;  // logits of a thread
constexpr int kMaxParts = (1 << 20) / kPart;
constexpr int kTable = 1024;
constexpr double kFar = 8192.0;              // largest power of two that the bins take

template <bool F32>
__device__ __forceinline__ float logit(const void *row, int64_t i) {
  if (F32) return static_cast<const float *>(row)[i];
  return (float)static_cast<const _Float16 *>(row)[i];
}

// N neighbours from i on, all inside the row, at any alignment
template <bool F32, int N>
__device__ __forceinline__ void logits(const void *row, int64_t i, float (&v)[N]) {
  if (F32) {
    __builtin_memcpy(v, static_cast<const float *>(row) + i, 4 * N);
  } else {
    _Float16 h[N];
    __builtin_memcpy(h, static_cast<const _Float16 *>(row) + i, 2 * N);
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = (float)h[e];
  }
}

// Whole numbers in the logits' order: -0 as 0, NaN as -infinity
__device__ __forceinline__ uint32_t key_of(float l) {
  if (l != l) return kNoKey;
  const uint32_t b = __builtin_bit_cast(uint32_t, l + 0.0f);
  return b ^ ((int32_t)b < 0 ? 0xFFFFFFFFu : 0x80000000u);
}

__device__ __forceinline__ float value_of(uint32_t key) {
  return __builtin_bit_cast(float, key ^ (key & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu));
}

// exp(z) in fp64: 2^n exp(r), |r| <= ln 2 / 2, the series of exp up to
// r^12 / 12! (its next term is below 2^-57 of the sum)
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

// What a row asks for
struct Settings {
  float heat;
  double u, at_least;          // min_p, 0: off
  float top_p;                 // 1: off
  int top_k;                   // vocab: off
  bool greedy, cuts;           // cuts: any of the three
};

__device__ __forceinline__ Settings settings(const SampleArgs &a, int64_t r) {
  Settings s;
  s.heat = a.temperature ? a.temperature[r] : 1.0f;
  s.greedy = !(s.heat > 0.0f);
  const float u = a.u[r];
  s.u = u > 0.0f ? (u < 1.0f ? (double)u : 1.0) : 0.0;
  const float m = a.min_p ? a.min_p[r] : 0.0f;
  s.at_least = m > 0.0f ? (m < 1.0f ? (double)m : 1.0) : 0.0;
  const float p = a.top_p ? a.top_p[r] : 1.0f;
  s.top_p = p < 1.0f ? (p > 0.0f ? p : 0.0f) : 1.0f;
  s.top_k = a.top_k ? a.top_k[r] : 0;
  if (s.top_k <= 0 || s.top_k > a.vocab) s.top_k = a.vocab;
  s.cuts = s.top_k < a.vocab || s.top_p < 1.0f || s.at_least > 0.0;
  return s;
}

// Weights by powers of two: x = l log2(e) / T - power, w = 2^x.  x is split
// at 1024ths: a table of 2^(j / 1024), and 2^g = 1 + e, |g| <= 2^-11, where e
// in fp32 is 2^-35 of w off.
struct Scale {
  double per;                  // log2(e) / T
  double power;                // a whole number
  int unit;
};

struct Split {
  double x;
  int i;                       // 1024 x, rounded
  float g;                     // x - i / 1024
};

__device__ __forceinline__ Split split(float l, const Scale &s) {
  constexpr double kMagic = 6755399441055744.0;   // 1.5 2^52: adding it rounds to whole numbers
  Split p;
  p.x = fmax(fma((double)l, s.per, -s.power), -1000.0);   // NaN and -infinity count as nothing too
  const double q = fma(p.x, 1024.0, kMagic);
  p.i = (int)(uint32_t)__builtin_bit_cast(uint64_t, q);
  p.g = (float)fma(q - kMagic, -1.0 / 1024.0, p.x);
  return p;
}

__device__ __forceinline__ uint64_t counted(const Split &p, const Scale &s, const double *table) {
  const float t = p.g * 0.69314718f, e = t * fmaf(t, fmaf(t, 0.16666667f, 0.5f), 1.0f);
  const double w = table[p.i & (kTable - 1)];
  const double c = ldexp(fma(w, (double)e, w), (p.i >> 10) + s.unit) + 4503599627370496.0;   // 2^52: whole numbers
  return __builtin_bit_cast(uint64_t, c) - 0x4330000000000000ull;
}

// 0: the largest (x from 7 / 8 on); eighths of a power of two
__device__ __forceinline__ int bin_of(const Split &p) { return 8 - (p.i >> 7); }

__device__ __forceinline__ double table_entry(int j) { return exp64((double)j * (0.69314718055994530942 / kTable)); }

template <int THREADS, typename T, typename F>
__device__ __forceinline__ T block_reduce(T v, T *tmp, F f) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = f(v, __shfl_xor(v, d));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
  __syncthreads();
  T r = tmp[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) r = f(r, tmp[w]);
  return r;
}

struct Larger {
  template <typename T>
  __device__ T operator()(T a, T b) const { return a > b ? a : b; }
};
struct Sum {
  template <typename T>
  __device__ T operator()(T a, T b) const { return a + b; }
};

// ---------------------------------------------------------------- parts

template <bool F32>
__global__ __launch_bounds__(kPartThreads) void sample_parts_kernel(SampleArgs a) {
  constexpr int V = F32 ? 4 : 8;   // logits in 16 bytes
  __shared__ double table[kTable];
  __shared__ unsigned long long sums[kBins];
  __shared__ uint32_t counts[kBins];
  __shared__ uint64_t tmp[kPartThreads / 64];
  const int tid = threadIdx.x;
  for (int j = tid; j < kTable; j += kPartThreads) table[j] = table_entry(j);
  const int items = a.rows * a.parts;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int r = item / a.parts, part = item - r * a.parts, from = part * kPart;
    const void *row = F32 ? (const void *)(static_cast<const float *>(a.logits) + r * a.ldl)
                          : (const void *)(static_cast<const uint16_t *>(a.logits) + r * a.ldl);
    float v[kEach];
    if (from + kPart <= a.vocab) {
#pragma unroll
      for (int i = 0; i < kEach / V; ++i) {
        float some[V];
        logits<F32, V>(row, from + (i * kPartThreads + tid) * V, some);
#pragma unroll
        for (int e = 0; e < V; ++e) v[V * i + e] = some[e];
      }
    } else {
      for (int i = 0; i < kEach; ++i) {
        const int at = from + (i / V * kPartThreads + tid) * V + i % V;
        v[i] = at < a.vocab ? logit<F32>(row, at) : -INFINITY;
      }
    }
    const Settings s = settings(a, r);
    if (s.cuts) {
      sums[tid] = 0;
      counts[tid] = 0;
      static_assert(kBins == kPartThreads, "a thread a bin");
    }
    float top = -INFINITY;
    int where = 0, finite = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int at = from + (i / V * kPartThreads + tid) * V + i % V;
      where = v[i] > top ? at : where;
      top = v[i] > top ? v[i] : top;
      finite += v[i] > -INFINITY;
    }
    const uint64_t best =
        block_reduce<kPartThreads>((uint64_t)key_of(top) << 32 | (uint32_t)~where, tmp, Larger());   // and the bins are cleared
    SamplePart head;
    head.best = best;
    head.sum = 0;
    head.power = 0;
    head.finite = 0;
    if (!s.greedy && (uint32_t)(best >> 32) > kNoKey) {
      Scale sc;
      sc.per = 1.4426950408889634074 / (double)s.heat;
      sc.unit = a.unit;
      const double most = (double)value_of((uint32_t)(best >> 32)) * sc.per;
      const bool near = fabs(most) < kFar;
      sc.power = floor(most);
      uint64_t sum = 0;
      if (near) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const Split p = split(v[i], sc);
          const uint64_t w = counted(p, sc, table);
          sum += w;
          const int bin = bin_of(p);
          if (s.cuts && bin < kBins) {
            atomicAdd(&sums[bin], (unsigned long long)w);
            atomicAdd(&counts[bin], 1u);
          }
        }
        head.power = (int32_t)sc.power;
      }
      head.sum = block_reduce<kPartThreads>(sum, tmp, Sum());
      head.finite = (uint32_t)block_reduce<kPartThreads>((uint64_t)finite, tmp, Sum());
      if (!near) head.power = kFarPart;
      if (s.cuts) {
        a.sums[(int64_t)item * kBins + tid] = sums[tid];
        a.counts[(int64_t)item * kBins + tid] = counts[tid];
      }
    }
    if (tid == 0) a.heads[item] = head;
    __syncthreads();
  }
}

// ---------------------------------------------------------------- rows

constexpr int kRowThreads = 1024;
constexpr int kList = 8192;                  // logits of a cut's bin, at most

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

constexpr int kSlowBins = 2048;
constexpr int kTurn = 4 * kRowThreads;       // logits of one turn of the passes
constexpr int kTurns = (1 << 20) / kTurn;

struct Shared {
  double table[kTable];
  uint64_t tmp[kRowThreads / 64];
  unsigned long long bins[kBins];            // the row's
  uint32_t counts[kBins];
  unsigned long long digits[256];            // of a search in the list
  unsigned long long kept[kMaxParts];        // of each part
  SamplePart heads[kMaxParts];
  uint64_t above;
  int32_t found;
  uint32_t list_size;
  union {
    struct {
      uint32_t keys[kList], places[kList];
    } list;
    struct {
      unsigned long long bins[kSlowBins];
      unsigned long long sums[kTurns];       // of each turn: w above the key
      uint32_t ties[kTurns];                 // of each turn: logits at the key
    } slow;
  };
};

// ---- passes over the whole row

struct Far {
  double max, per;     // the row's largest logit, 1 / T
  uint32_t top;        // its key
  double unit;         // 2^unit
};

__device__ __forceinline__ double weight(uint32_t key, const Far &s) {
  if (key == s.top) return 1.0;
  if (key <= kNoKey) return 0.0;
  return exp64(((double)value_of(key) - s.max) * s.per);
}

__device__ __forceinline__ uint64_t counted(double w, const Far &s) { return (uint64_t)rint(w * s.unit); }

// f(key) for every logit of [from, to), from a multiple of 4
template <bool F32, typename F>
__device__ __forceinline__ void each_key(const void *row, int from, int to, F f) {
  int i = from + 4 * (int)threadIdx.x;
  for (; i + 4 <= to; i += kTurn) {
    float v[4];
    logits<F32, 4>(row, i, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) f(key_of(v[e]));
  }
  for (int e = i; e < to && e < i + 4; ++e) f(key_of(logit<F32>(row, e)));
}

// The key at which the sum over falling keys, of counts or of weights, of
// those at or above `floor` first reaches `want` (> 0), and the sum above it:
// 11, 11 and 10 bits at a time.
template <bool F32, bool WEIGHTS>
__device__ uint32_t search_row(const void *row, int n, const Far &s, uint32_t floor, uint64_t want, uint64_t &above, Shared &sh) {
  uint32_t prefix = 0;
  above = 0;
  int shift = 32;
  for (int level = 0; level < 3; ++level) {
    const int bits = level == 2 ? 10 : 11, next = shift - bits;
    for (int i = threadIdx.x; i < kSlowBins; i += kRowThreads) sh.slow.bins[i] = 0;
    __syncthreads();
    each_key<F32>(row, 0, n, [&](uint32_t key) {
      if (key < floor || (level && key >> shift != prefix >> shift)) return;
      const uint64_t add = WEIGHTS ? counted(weight(key, s), s) : 1;
      if (add) atomicAdd(&sh.slow.bins[(key >> next) & ((1u << bits) - 1)], (unsigned long long)add);
    });
    __syncthreads();
    // from the highest down, two bins a thread
    const int d = (1 << bits) - 1 - 2 * (int)threadIdx.x;
    const uint64_t one = d >= 0 ? sh.slow.bins[d] : 0, two = d > 0 ? sh.slow.bins[d - 1] : 0;
    const uint64_t before = above + block_before(one + two, sh.tmp);
    if (d >= 0 && before < want && before + one + two >= want) {
      sh.found = before + one >= want ? d : d - 1;
      sh.above = before + one >= want ? before : before + one;
    }
    __syncthreads();
    prefix |= (uint32_t)sh.found << next;
    above = sh.above;
    shift = next;
    __syncthreads();
  }
  return prefix;
}

template <bool F32>
__device__ void sample_passes(const SampleArgs &a, int64_t r, const void *row, uint32_t top, const Settings &set, Shared &sh) {
  const int tid = threadIdx.x, n = a.vocab;
  Far s;
  s.top = top;
  s.max = value_of(top);
  s.per = 1.0 / (double)set.heat;
  s.unit = ldexp(1.0, a.unit);
  __syncthreads();
  // what is kept: keys above `cut`, and the first `ties` at it
  uint32_t cut = 0;
  uint64_t ties = n;
  if (set.top_k < n) {
    uint64_t above;
    cut = search_row<F32, false>(row, n, s, 0, set.top_k, above, sh);
    ties = set.top_k - above;
  }
  if (set.top_p < 1.0f) {
    uint64_t sum = 0;
    each_key<F32>(row, 0, n, [&](uint32_t key) {
      if (key > cut) sum += counted(weight(key, s), s);
    });
    const uint64_t over = block_reduce<kRowThreads>(sum, sh.tmp, Sum());
    const uint64_t tie = counted(weight(cut, s), s), all = over + ties * tie;
    // kept are those before which less than p * all lies
    uint64_t want = (uint64_t)ceil((double)set.top_p * (double)all);
    if (want == 0) want = 1;
    if (want > over) {   // among top-k's ties
      const uint64_t some = (want - over + tie - 1) / tie;
      ties = some < ties ? some : ties;
    } else {
      uint64_t above;
      cut = search_row<F32, true>(row, n, s, cut + 1, want, above, sh);
      const uint64_t w = counted(weight(cut, s), s);
      ties = (want - above + w - 1) / w;
    }
  }
  // sums of each turn, in the order of the index
  const double cut_weight = weight(cut, s);
  const uint64_t tie = cut_weight >= set.at_least ? counted(cut_weight, s) : 0;
  const int turns = (n + kTurn - 1) / kTurn;
  for (int t = tid; t < turns; t += kRowThreads) sh.slow.sums[t] = sh.slow.ties[t] = 0;
  __syncthreads();
  for (int t = 0; t < turns; ++t) {
    uint64_t sum = 0;
    uint32_t same = 0;
    each_key<F32>(row, t * kTurn, min(n, (t + 1) * kTurn), [&](uint32_t key) {
      same += key == cut;
      if (key > cut) {
        const double w = weight(key, s);
        if (w >= set.at_least) sum += counted(w, s);
      }
    });
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      sum += __shfl_xor(sum, d);
      same += __shfl_xor(same, d);
    }
    if ((tid & 63) == 0) {
      if (sum) atomicAdd(&sh.slow.sums[t], (unsigned long long)sum);
      if (same) atomicAdd(&sh.slow.ties[t], same);
    }
  }
  __syncthreads();
  uint64_t all = 0, seen = 0;
  for (int t = 0; t < turns; ++t) {
    const uint64_t kept = sh.slow.ties[t] < ties - seen ? sh.slow.ties[t] : ties - seen;
    all += sh.slow.sums[t] + kept * tie;
    seen += kept;
  }
  uint64_t target = (uint64_t)floor(set.u * (double)all);
  if (target >= all) target = all - 1;
  uint64_t before = 0;
  seen = 0;
  int t = 0;
  for (;; ++t) {
    const uint64_t kept = sh.slow.ties[t] < ties - seen ? sh.slow.ties[t] : ties - seen;
    const uint64_t here = sh.slow.sums[t] + kept * tie;
    if (before + here > target) break;
    before += here;
    seen += kept;
  }
  // the turn's logits, four in a row to a thread
  const int first = t * kTurn + 4 * tid;
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
      if (v >= set.at_least) w[e] = counted(v, s);
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

// ---- by the parts' bins

// The value at which the sum over falling values, of 1 or of `add`, of the
// list's entries with take(i) first reaches `want` (> 0), and the sum above
// it; if it never does, the lowest.  Eight bits at a time, from the highest
// that differs.
template <typename Take, typename Value, typename Add>
__device__ uint32_t search_list(int size, uint64_t want, uint64_t &above, Shared &sh, Take take, Value value, Add add) {
  const int tid = threadIdx.x;
  uint32_t low = 0xFFFFFFFFu, high = 0;
  for (int i = tid; i < size; i += kRowThreads)
    if (take(i)) {
      const uint32_t v = value(i);
      low = v < low ? v : low;
      high = v > high ? v : high;
    }
  const uint64_t both = block_reduce<kRowThreads>((uint64_t)(~low) , sh.tmp, Larger());
  const uint64_t top = block_reduce<kRowThreads>((uint64_t)high, sh.tmp, Larger());
  low = ~(uint32_t)both;
  high = (uint32_t)top;
  above = 0;
  if (low >= high) return low;
  int shift = 32 - __clz((int)(low ^ high));   // bits from here up are alike
  uint32_t prefix = shift < 32 ? high >> shift << shift : 0;
  while (shift > 0) {
    const int bits = shift < 8 ? shift : 8, next = shift - bits;
    if (tid < 256) sh.digits[tid] = 0;
    if (tid == 0) sh.found = -1;
    __syncthreads();
    for (int i = tid; i < size; i += kRowThreads)
      if (take(i)) {
        const uint32_t v = value(i);
        if (shift == 32 || v >> shift == prefix >> shift)
          atomicAdd(&sh.digits[(v >> next) & ((1u << bits) - 1)], (unsigned long long)add(i));
      }
    __syncthreads();
    const int d = (1 << bits) - 1 - tid;
    const uint64_t here = d >= 0 ? sh.digits[d] : 0;
    const uint64_t before = above + block_before(here, sh.tmp);
    if (d >= 0 && before < want && before + here >= want) {
      sh.found = d;
      sh.above = before;
    }
    __syncthreads();
    if (sh.found < 0) return low;   // (above is that of the last digits)
    prefix |= (uint32_t)sh.found << next;
    above = sh.above;
    shift = next;
    __syncthreads();
  }
  return prefix;
}

// The first of kBins bins in which the sum reaches `want`, and the sum before it; -1: none
template <typename T>
__device__ int find_bin(const T *bins, int end, uint64_t want, uint64_t &above, Shared &sh) {
  const int tid = threadIdx.x;
  if (tid == 0) sh.found = -1;
  const uint64_t here = tid < end ? bins[tid] : 0;
  const uint64_t before = block_before(here, sh.tmp);
  if (tid < end && before < want && before + here >= want) {
    sh.found = tid;
    sh.above = before;
  }
  __syncthreads();
  const int found = sh.found;
  above = sh.above;
  __syncthreads();
  return found;
}

template <bool F32>
__global__ __launch_bounds__(kRowThreads) void sample_rows_kernel(SampleArgs a) {
  extern __shared__ char smem[];
  Shared &sh = *reinterpret_cast<Shared *>(smem);
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, n = a.vocab, parts = a.parts;
  const void *row = F32 ? (const void *)(static_cast<const float *>(a.logits) + r * a.ldl)
                        : (const void *)(static_cast<const uint16_t *>(a.logits) + r * a.ldl);
  const Settings set = settings(a, r);
  const uint64_t *part_sums = a.sums + r * parts * kBins;
  const uint32_t *part_counts = a.counts + r * parts * kBins;

  SamplePart head;
  head.best = 0;
  if (tid < parts) {
    head = a.heads[r * parts + tid];
    sh.heads[tid] = head;
  }
  const uint64_t best = block_reduce<kRowThreads>(head.best, sh.tmp, Larger());
  const uint32_t top = (uint32_t)(best >> 32);
  if (top <= kNoKey || set.greedy) {
    if (tid == 0) {
      a.ids[r] = top <= kNoKey ? -1 : (int32_t)~(uint32_t)best;
      if (a.logprobs) a.logprobs[r] = top <= kNoKey ? -INFINITY : 0.0f;
    }
    return;
  }
  Scale sc;
  sc.per = 1.4426950408889634074 / (double)set.heat;
  sc.unit = a.unit;
  const double most = (double)value_of(top) * sc.per;
  if (!(fabs(most) < kFar)) return sample_passes<F32>(a, r, row, top, set, sh);
  sc.power = floor(most);
  const int power = (int)sc.power;
  for (int j = tid; j < kTable; j += kRowThreads) sh.table[j] = table_entry(j);
  // how far a part's powers are below the row's (64: its weights are nothing)
  const auto behind = [&](int p) {
    const int32_t own = sh.heads[p].power;
    return own == kFarPart || power - own > 63 ? 64 : power - own;
  };
  const auto shifted = [](uint64_t v, int by) { return by < 64 ? v >> by : 0; };
  const auto weight_of = [&](uint32_t key) { return key > kNoKey ? counted(split(value_of(key), sc), sc, sh.table) : 0; };

  // what is kept: keys above `cut`, and of those at it the ones whose index's
  // complement is `last` or more; all of bins before `bin` and, in the list,
  // the logits of that bin
  uint32_t cut = 0, last = 0;
  uint64_t ties = ~0ull;
  int bin = kBins;
  uint64_t all = 0;   // sum of the weights kept
  uint64_t finite = 0;
  for (int p = 0; p < parts; ++p) {
    finite += sh.heads[p].finite;
    all += shifted(sh.heads[p].sum, behind(p));
  }
  int size = 0;       // of the list
  if (set.cuts) {
    if (tid < kBins) {
      sh.bins[tid] = 0;
      sh.counts[tid] = 0;
    }
    __syncthreads();
    for (int i = tid; i < parts * kBins; i += kRowThreads) {
      const int p = i / kBins, by = behind(p), to = i % kBins + 8 * by;
      const uint32_t c = part_counts[i];
      if (by < 64 && to < kBins && c) {
        atomicAdd(&sh.bins[to], (unsigned long long)shifted(part_sums[i], by));
        atomicAdd(&sh.counts[to], c);
      }
    }
    __syncthreads();
    // the logits of a bin into the list, from the parts that have some
    const auto collect = [&](int which) {
      if (which == bin) return true;
      if (sh.counts[which] > (uint32_t)kList) return false;
      __syncthreads();
      if (tid == 0) sh.list_size = 0;
      __syncthreads();
      for (int p = 0; p < parts; ++p) {
        const int by = behind(p), own = which - 8 * by;
        if (by >= 64 || own < 0 || !part_counts[p * kBins + own]) continue;
        Scale ps = sc;
        ps.power = sh.heads[p].power;
        const int from = p * kPart, to = min(n, from + kPart), first = from + 8 * tid;
        float v[8];
        if (first + 8 <= to) {
          logits<F32, 8>(row, first, v);
        } else {
          for (int e = 0; e < 8; ++e) v[e] = first + e < to ? logit<F32>(row, first + e) : -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (bin_of(split(v[e], ps)) == own) {
            const uint32_t at = atomicAdd(&sh.list_size, 1u);
            if (at < (uint32_t)kList) {
              sh.list.keys[at] = key_of(v[e]);
              sh.list.places[at] = (uint32_t)(first + e);
            }
          }
      }
      __syncthreads();
      size = (int)min(sh.list_size, (uint32_t)kList);
      bin = which;
      return true;
    };
    static_assert(kPart == 8 * kRowThreads, "eight logits of a part to a thread");
    // sum of the list's weights above the cut
    const auto list_above = [&]() {
      uint64_t sum = 0;
      for (int i = tid; i < size; i += kRowThreads)
        if (sh.list.keys[i] > cut) sum += weight_of(sh.list.keys[i]);
      return block_reduce<kRowThreads>(sum, sh.tmp, Sum());
    };
    const auto key_at = [&](int i) { return sh.list.keys[i]; };
    uint64_t above, over = 0;   // over: the bins before the list's
    if ((uint64_t)set.top_k < finite) {
      const int at = find_bin(sh.counts, kBins, set.top_k, above, sh);
      if (at < 0 || !collect(at)) return sample_passes<F32>(a, r, row, top, set, sh);
      uint64_t more;
      cut = search_list(size, set.top_k - above, more, sh, [](int) { return true; }, key_at, [](int) { return 1; });
      ties = set.top_k - above - more;
      uint64_t sum = tid < at ? sh.bins[tid] : 0;
      over = block_reduce<kRowThreads>(sum, sh.tmp, Sum());
      all = over + list_above() + ties * weight_of(cut);
    }
    if (set.top_p < 1.0f) {
      uint64_t want = (uint64_t)ceil((double)set.top_p * (double)all);
      if (want == 0) want = 1;
      const int at = find_bin(sh.bins, bin, want, above, sh);
      if (at >= 0) {
        if (!collect(at)) return sample_passes<F32>(a, r, row, top, set, sh);
        uint64_t more;
        cut = search_list(size, want - above, more, sh, [](int) { return true; }, key_at,
                          [&](int i) { return weight_of(sh.list.keys[i]); });
        const uint64_t w = weight_of(cut);
        ties = w ? (want - above - more + w - 1) / w : 1;
        all = above;   // its bins
      } else if (bin < kBins) {   // among top-k's list
        const uint64_t high = over + list_above();
        if (want > high) {
          const uint64_t w = weight_of(cut), some = w ? (want - high + w - 1) / w : 1;
          ties = some < ties ? some : ties;
        } else {
          uint64_t more;
          const uint32_t least = cut;
          cut = search_list(size, want - over, more, sh, [&](int i) { return sh.list.keys[i] > least; }, key_at,
                            [&](int i) { return weight_of(sh.list.keys[i]); });
          const uint64_t w = weight_of(cut);
          ties = w ? (want - over - more + w - 1) / w : 1;
        }
      } else {
        return sample_passes<F32>(a, r, row, top, set, sh);
      }
    }
    if (set.at_least > 0.0) {
      // the lowest key with a weight that is enough: weights rise with keys
      const double max = value_of(top), per = 1.0 / (double)set.heat;
      uint32_t no = kNoKey, yes = top;
      while (yes - no > 1) {
        const uint32_t mid = no + (yes - no) / 2;
        if (exp64(((double)value_of(mid) - max) * per) >= set.at_least)
          yes = mid;
        else
          no = mid;
      }
      if (yes > cut) {
        const int at = bin_of(split(value_of(yes), sc));
        if (at >= kBins || !collect(at)) return sample_passes<F32>(a, r, row, top, set, sh);
        cut = yes;
        ties = ~0ull;
      }
    }
    if (bin < kBins) {
      // of equal ones at the cut the first by index
      uint64_t same = 0;
      for (int i = tid; i < size; i += kRowThreads) same += sh.list.keys[i] == cut;
      same = block_reduce<kRowThreads>(same, sh.tmp, Sum());
      if (ties < same) {
        uint64_t more;
        last = search_list(size, ties, more, sh, [&](int i) { return sh.list.keys[i] == cut; },
                           [&](int i) { return ~sh.list.places[i]; }, [](int) { return 1; });
      }
    }
  }
  // what is kept of each part
  __syncthreads();
  if (tid < kMaxParts) sh.kept[tid] = tid < parts && bin == kBins ? shifted(sh.heads[tid].sum, behind(tid)) : 0;
  __syncthreads();
  if (bin < kBins) {
    for (int i = tid; i < parts * kBins; i += kRowThreads) {
      const int p = i / kBins, by = behind(p);
      if (by < 64 && i % kBins + 8 * by < bin && part_counts[i])
        atomicAdd(&sh.kept[p], (unsigned long long)shifted(part_sums[i], by));
    }
    for (int i = tid; i < size; i += kRowThreads) {
      const uint32_t key = sh.list.keys[i], place = sh.list.places[i];
      if (key > cut || (key == cut && ~place >= last)) atomicAdd(&sh.kept[place / kPart], (unsigned long long)weight_of(key));
    }
    __syncthreads();
  }
  const uint64_t mine = tid < parts ? sh.kept[tid] : 0;
  const uint64_t before = block_before(mine, sh.tmp);
  if (tid == parts - 1) sh.above = before + mine;
  __syncthreads();
  all = sh.above;
  uint64_t target = (uint64_t)floor(set.u * (double)all);
  if (target >= all) target = all - 1;
  __syncthreads();
  if (tid < parts && before <= target && before + mine > target) {
    sh.found = tid;
    sh.above = before;
  }
  __syncthreads();
  const int part = sh.found, from = part * kPart, to = min(n, from + kPart), first = from + 8 * tid;
  const uint64_t start = sh.above;
  float v[8];
  if (first + 8 <= to) {
    logits<F32, 8>(row, first, v);
  } else {
    for (int e = 0; e < 8; ++e) v[e] = first + e < to ? logit<F32>(row, first + e) : -INFINITY;
  }
  uint64_t w[8], sum = 0;
  int final = -1;   // the last that is kept
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t key = key_of(v[e]);
    w[e] = key > cut || (key == cut && ~(uint32_t)(first + e) >= last) ? weight_of(key) : 0;
    sum += w[e];
    if (w[e]) final = first + e;
  }
  uint64_t at = start + block_before(sum, sh.tmp);
  int pick = -1;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (at <= target && at + w[e] > target) pick = first + e;
    at += w[e];
  }
  // (the parts' sums are rounded at another place than the row's weights: a
  // target in the last unit of one is the last token kept)
  const uint64_t chosen = block_reduce<kRowThreads>((uint64_t)(pick >= 0 ? 1u : 0u) << 32 | (uint32_t)(pick >= 0 ? pick : final + 1),
                                                    sh.tmp, Larger());
  const int id = chosen >> 32 ? (int)(uint32_t)chosen : (int)(uint32_t)chosen - 1;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (id == first + e) {
      a.ids[r] = id;
      if (a.logprobs) {
        const double x = fma((double)v[e], sc.per, -sc.power);
        a.logprobs[r] = (float)(x * 0.69314718055994530942 - log(ldexp((double)all, -a.unit)));
      }
    }
}

}  // namespace

hipError_t launch_sample(const SampleArgs &a, hipStream_t s) {
  const int64_t items = (int64_t)a.rows * a.parts;
  const unsigned groups = (unsigned)(items < kSampleGroups ? items : kSampleGroups);
  if (a.f32) {
    hipLaunchKernelGGL(sample_parts_kernel<true>, dim3(groups), dim3(kPartThreads), 0, s, a);
    hipLaunchKernelGGL(sample_rows_kernel<true>, dim3((unsigned)a.rows), dim3(kRowThreads), sizeof(Shared), s, a);
  } else {
    hipLaunchKernelGGL(sample_parts_kernel<false>, dim3(groups), dim3(kPartThreads), 0, s, a);
    hipLaunchKernelGGL(sample_rows_kernel<false>, dim3((unsigned)a.rows), dim3(kRowThreads), sizeof(Shared), s, a);
  }
  return hipGetLastError();
}

}  // namespace wq
