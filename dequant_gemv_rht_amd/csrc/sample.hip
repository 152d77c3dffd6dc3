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
// for rows with top-k, top-p or min-p, running counts and sums over kBins
// bins of equal width (an eighth of a power of two, from its largest down).
// Bins of all parts line up, so the second launch, a workgroup for each row,
// finds in which bin a cut lies, fetches that bin's logits alone (from the
// parts that have any), finds the cut among them, and with it every part's
// sum of what is kept; the part in which the sum passes u times all of it is
// read again, token by token.  Rows for which that does not do (a cut below
// the bins, more logits in its bin than fit in LDS, logits beyond 2^13 powers
// of two) are searched in as many passes as it takes.
//
// The second launch runs once through its code, most of which then comes from
// the L2 line by line: loops there stay rolled, each piece of work has one
// place, and what a wave can find out alone every wave does, without waiting
// for the others.
#include "wq_internal.h"

namespace wq {
using namespace dev;

namespace {

constexpr uint32_t kNoKey = 0x007FFFFFu;     // of -infinity
constexpr int kBins = kSampleBins;
constexpr int kPart = kSamplePart;
constexpr int kPartThreads = 512;
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
  // every array is there (one that the caller left out stands for another), so all are asked for at once
  const float heat = a.temperature[r], u = a.u[r], m = a.min_p[r], p = a.top_p[r];
  const int k = a.top_k[r];
  Settings s;
  s.heat = a.given & kGivenHeat ? heat : 1.0f;
  s.greedy = !(s.heat > 0.0f);
  s.u = u > 0.0f ? (u < 1.0f ? (double)u : 1.0) : 0.0;
  s.at_least = a.given & kGivenMinP && m > 0.0f ? (m < 1.0f ? (double)m : 1.0) : 0.0;
  s.top_p = a.given & kGivenTopP && p < 1.0f ? (p > 0.0f ? p : 0.0f) : 1.0f;
  s.top_k = a.given & kGivenTopK && k > 0 && k < a.vocab ? k : a.vocab;
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
  __shared__ uint32_t tmp_counts[kBins / 64];
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
    if (s.cuts && tid < kBins) {
      sums[tid] = 0;
      counts[tid] = 0;
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
    head.power = kFarPart;   // no bins
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
        // eight at a time: a table entry of one waits behind the sums of none
#pragma unroll
        for (int i = 0; i < kEach; i += 8) {
          Split p[8];
          uint64_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) p[e] = split(v[i + e], sc);
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = counted(p[e], sc, table);
#pragma unroll
          for (int e = 0; e < 8; ++e) sum += w[e];
          if (!s.cuts) continue;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (bin_of(p[e]) < kBins) {
              atomicAdd(&sums[bin_of(p[e])], (unsigned long long)w[e]);
              if (s.top_k < a.vocab) atomicAdd(&counts[bin_of(p[e])], 1u);
            }
        }
        head.power = (int32_t)sc.power;
      }
      head.sum = block_reduce<kPartThreads>(sum, tmp, Sum());
      head.finite = (uint32_t)block_reduce<kPartThreads>((uint64_t)finite, tmp, Sum());
      if (near && s.cuts) {
        // sums up to and with each bin
        uint64_t up = tid < kBins ? sums[tid] : 0;
        uint32_t many = tid < kBins ? counts[tid] : 0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const uint64_t o = __shfl_up(up, d);
          const uint32_t c = __shfl_up(many, d);
          if ((tid & 63) >= d) {
            up += o;
            many += c;
          }
        }
        __syncthreads();
        if ((tid & 63) == 63 && tid < kBins) {
          tmp[tid >> 6] = up;
          tmp_counts[tid >> 6] = many;
        }
        __syncthreads();
        if (tid < kBins) {
          for (int w = 0; w < tid >> 6; ++w) {
            up += tmp[w];
            many += tmp_counts[w];
          }
          a.sums[(int64_t)item * kBins + tid] = up;
          a.counts[(int64_t)item * kBins + tid] = many;
        }
      }
    }
    if (tid == 0) a.heads[item] = head;
    __syncthreads();
  }
}

// ---------------------------------------------------------------- rows

constexpr int kRowThreads = 512;
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
  uint64_t sums[kBins], counts[kBins];       // the row's, up to and with each bin
  unsigned long long digits[256];            // of a search in a long list
  unsigned long long kept[kMaxParts];        // of each part
  uint64_t above;
  int32_t found;
  uint32_t list_size;
  union {
    struct {
      uint64_t weights[kList];
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
    // from the highest down, four bins a thread
    const int d = (1 << bits) - 1 - 4 * (int)threadIdx.x;
    uint64_t here = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) here += d >= e ? sh.slow.bins[d - e] : 0;
    uint64_t before = above + block_before(here, sh.tmp);
    if (before < want && before + here >= want)
      for (int e = 0; e < 4 && d >= e; ++e) {
        const uint64_t one = sh.slow.bins[d - e];
        if (before < want && before + one >= want) {
          sh.found = d - e;
          sh.above = before;
        }
        before += one;
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
__device__ __forceinline__ void sample_passes(const SampleArgs &a, int64_t r, const void *row, uint32_t top, const Settings &set, Shared &sh) {
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

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll 1
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

template <typename T>
__device__ __forceinline__ T wave_max(T v) {
#pragma unroll 1
  for (int d = 32; d; d >>= 1) {
    const T o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}

// the sum of v over the lanes up to this one
__device__ __forceinline__ uint64_t wave_scan(uint64_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll 1
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

__device__ __forceinline__ uint64_t lane_value(uint64_t v, int lane) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
}

// In turn: what top-k leaves, what top-p leaves of that, what min-p leaves of
// that, and which of equal logits at the cut.
enum Stage { kTopK, kTopP, kMinP, kPlace };

template <bool F32>
__global__ __launch_bounds__(kRowThreads) void sample_rows_kernel(SampleArgs a) {
  extern __shared__ char smem[];
  Shared &sh = *reinterpret_cast<Shared *>(smem);
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, n = a.vocab, parts = a.parts;
  const void *row = F32 ? (const void *)(static_cast<const float *>(a.logits) + r * a.ldl)
                        : (const void *)(static_cast<const uint16_t *>(a.logits) + r * a.ldl);
  const uint64_t *part_sums = a.sums + r * parts * kBins;
  const uint32_t *part_counts = a.counts + r * parts * kBins;
  // every wave: parts lane and lane + 64
  static_assert(kMaxParts <= 128, "two parts a lane");
  SamplePart head[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) head[h] = a.heads[r * parts + min(lane + 64 * h, parts - 1)];
  const Settings set = settings(a, r);
  const uint64_t best = wave_max(head[0].best > head[1].best ? head[0].best : head[1].best);
  const uint32_t top = (uint32_t)(best >> 32);
  if (top <= kNoKey || set.greedy) {
    if (tid == 0) {
      a.ids[r] = top <= kNoKey ? -1 : (int32_t)~(uint32_t)best;
      if (a.logprobs) a.logprobs[r] = top <= kNoKey ? -INFINITY : 0.0f;
    }
    return;
  }
#pragma unroll 1
  for (int j = tid; j < kTable; j += kRowThreads) sh.table[j] = table_entry(j);
  Scale sc;
  sc.per = 1.4426950408889634074 / (double)set.heat;
  sc.unit = a.unit;
  const double most = (double)value_of(top) * sc.per;
  sc.power = floor(most);
  // as the first launch counted it: borders of equal weights are exact
  const auto weight_of = [&](float l) { return counted(split(l, sc), sc, sh.table); };
  bool passes = !(fabs(most) < kFar);

  // what is kept: keys above `cut`, and of those at it the ones whose index's
  // complement is `last` or more; all of the bins before `bin` and, in the
  // list, the logits of that bin
  uint32_t cut = 0, last = 0;
  uint64_t ties = ~0ull, all = 0, whole[2];   // sum of the weights kept; of a part's
  int bin = kBins, size = 0, by[2];           // by: how far a part's powers are below the row's (64: too far)
  if (!passes) {
    const int power = (int)sc.power;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = lane + 64 * h < parts && head[h].power != kFarPart && power - head[h].power < 64;
      by[h] = in ? power - head[h].power : 64;
      whole[h] = in ? head[h].sum >> by[h] : 0;
    }
    all = wave_sum(whole[0] + whole[1]);
  }
  if (!passes && set.cuts) {
    const uint32_t finite = wave_sum((lane < parts ? head[0].finite : 0) + (lane + 64 < parts ? head[1].finite : 0));
    const bool counting = (uint32_t)set.top_k < finite;
    // the row's bins: a thread one bin, of every other part
    {
      const int j = tid & (kBins - 1);
      uint64_t sum = 0, many = 0;
#pragma unroll 4
      for (int p = tid / kBins; p < parts; p += kRowThreads / kBins) {
        const int late = __shfl(p < 64 ? by[0] : by[1], p & 63), own = j - 8 * late;   // p is the wave's
        const int64_t i = (int64_t)p * kBins + max(own, 0);
        const uint64_t w = part_sums[i];
        const uint32_t c = part_counts[i];
        sum += late < 64 && own >= 0 ? w >> late : 0;
        many += late < 64 && own >= 0 ? c : 0;
      }
      if (tid >= kBins) {
        sh.sums[j] = sum;
        sh.counts[j] = many;
      }
      __syncthreads();
      if (tid < kBins) {
        sh.sums[j] += sum;
        sh.counts[j] += many;
      }
      static_assert(kRowThreads == 2 * kBins, "two threads a bin");
      __syncthreads();
    }
    uint64_t over = 0;   // top-k: the bins before the list's
#pragma unroll 1
    for (int stage = kTopK; stage <= kPlace; ++stage) {
      int at = -1;            // the bin to look into
      uint64_t want = 0, above = 0;
      uint32_t floor = 0;     // of the keys searched
      if (stage == kTopK) {
        if (!counting) continue;
        want = set.top_k;
      } else if (stage == kTopP) {
        if (!(set.top_p < 1.0f)) continue;
        want = (uint64_t)ceil((double)set.top_p * (double)all);
        if (want == 0) want = 1;
      } else if (stage == kMinP) {
        if (!(set.at_least > 0.0)) continue;
        // the lowest key with a weight that is enough, as weights rise with
        // keys: near where the logarithm puts it, or found by halves
        const double max = value_of(top), per = 1.0 / (double)set.heat;
        const uint32_t guess = key_of((float)(max + (double)set.heat * log(set.at_least)));
        uint32_t no = kNoKey, yes = top;
#pragma unroll 1
        for (int turn = 0; yes - no > 1; ++turn) {
          // 64 keys about the guess, then one
          const bool many = turn == 0 && guess > kNoKey + 64 && guess < 0xFFFFFF00u;
          const uint32_t key = many ? guess - 32 + (uint32_t)lane : no + (yes - no) / 2;
          const uint64_t enough = __ballot(key >= top || exp64(((double)value_of(key) - max) * per) >= set.at_least);
          if (many) {
            if (enough && !(enough & 1)) {
              yes = guess - 32 + (uint32_t)(__ffsll((unsigned long long)enough) - 1);
              no = yes - 1;
            }
          } else if (enough) {
            yes = key;
          } else {
            no = key;
          }
        }
        if (yes <= cut) continue;
        cut = yes;
        ties = ~0ull;
        at = bin_of(split(value_of(yes), sc));
        if (at >= kBins) {
          passes = true;
          break;
        }
      } else {
        if (bin == kBins) continue;
        // of equal ones at the cut the first by index
        uint32_t same = 0;
        for (int i = lane; i < size; i += 64) same += sh.list.keys[i] == cut;
        if (ties >= wave_sum(same)) continue;
        want = ties;
      }
      if (stage <= kTopP) {
        // the first bin with which the sum reaches `want`, and the sum before it
        const uint64_t *bins = stage == kTopK ? sh.counts : sh.sums;
        at = 0;
#pragma unroll 1
        for (int j = 0; j < kBins; j += 64) at += __popcll(__ballot(bins[j + lane] < want));
        above = at ? bins[at - 1] : 0;
        if (at >= bin) {
          if (bin == kBins) {
            passes = true;
            break;
          }
          // among top-k's list
          at = bin;
          uint64_t w = 0;
          for (int i = lane; i < size; i += 64)
            if (sh.list.keys[i] == cut) w = sh.list.weights[i];
          w = wave_max(w);
          const uint64_t high = all - ties * w;
          if (want > high) {
            const uint64_t some = w ? (want - high + w - 1) / w : 1;
            ties = some < ties ? some : ties;
            continue;
          }
          above = over;
          floor = cut;
        }
      }
      if (stage < kPlace && at != bin) {
        // the logits of that bin, from the parts that have some
        __syncthreads();
        if (tid == 0) sh.list_size = 0;
        uint64_t wanted[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int own = at - 8 * by[h];
          const bool in = by[h] < 64 && own >= 0;
          const uint64_t *sums = part_sums + (int64_t)(in ? lane + 64 * h : 0) * kBins + (in ? own : 0);
          const uint64_t up_to = *sums, before = *(in && own ? sums - 1 : sums);
          wanted[h] = __ballot(in && (own ? up_to != before : up_to != 0));
        }
        __syncthreads();
#pragma unroll 1
        while (wanted[0] | wanted[1]) {
          const int h = wanted[0] ? 0 : 1, l = __ffsll((unsigned long long)wanted[h]) - 1, p = l + 64 * h;
          wanted[h] &= wanted[h] - 1;
          const int late = __shfl(h ? by[1] : by[0], l), own = at - 8 * late;
          Scale ps = sc;
          ps.power = sc.power - late;
          const int from = p * kPart, to = min(n, from + kPart);
          uint32_t some = 0;   // of this thread's 16
          if (to - from == kPart) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float eight[8];
              logits<F32, 8>(row, from + (i * kRowThreads + tid) * 8, eight);
#pragma unroll
              for (int e = 0; e < 8; ++e) v[8 * i + e] = eight[e];
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) some |= (uint32_t)(bin_of(split(v[e], ps)) == own) << e;
          } else {
#pragma unroll 1
            for (int e = 0; e < 16; ++e) {
              const int i = from + (e / 8 * kRowThreads + tid) * 8 + e % 8;
              if (i < to) some |= (uint32_t)(bin_of(split(logit<F32>(row, i), ps)) == own) << e;
            }
          }
          static_assert(kPart == 16 * kRowThreads, "16 logits of a part to a thread");
#pragma unroll 1
          for (; some; some &= some - 1) {
            const int e = __ffs((int)some) - 1, i = from + (e / 8 * kRowThreads + tid) * 8 + e % 8;
            const uint32_t to = atomicAdd(&sh.list_size, 1u);
            if (to >= (uint32_t)kList) break;
            const float l = logit<F32>(row, i);
            sh.list.keys[to] = key_of(l);
            sh.list.places[to] = (uint32_t)i;
            sh.list.weights[to] = weight_of(l);
          }
        }
        __syncthreads();
        if (sh.list_size > (uint32_t)kList) {
          passes = true;
          break;
        }
        size = (int)sh.list_size;
        bin = at;
      }
      if (stage == kMinP) continue;
      // The value at which the sum over falling values (keys, or complements
      // of the indices at the cut), of 1 or of weights, of the list reaches
      // `want`, and the sum above it; if it never does, the lowest.
      const auto value = [&](int i) {
        const uint32_t key = sh.list.keys[i];
        return stage == kPlace ? (key == cut ? ~sh.list.places[i] : 0) : key > floor ? key : 0;   // 0: none
      };
      uint32_t found = 0;
      uint64_t more = 0, w = 0, sum = 0;   // w: the weight found; sum: of the weights above it
      want -= above;
      if (size <= 64) {
        // a lane an entry, each against all
        const uint32_t mine = lane < size ? value(lane) : 0;
        const uint64_t weight = lane < size ? sh.list.weights[lane] : 0, add = stage == kTopP ? weight : 1;
        uint64_t higher = 0;
#pragma unroll 1
        for (int j = 0; j < size; ++j) {
          const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)mine, j);
          higher += other > mine ? lane_value(add, j) : 0;
        }
        found = ~wave_max(mine && higher < want ? ~mine : 0);
        const int l = __ffsll((unsigned long long)__ballot(mine == found)) - 1;
        more = lane_value(higher, l);
        w = lane_value(weight, l);
        if (stage == kTopK) sum = wave_sum(mine > found ? weight : 0);
      } else {
        // eight bits at a time, from the highest that differs
        uint32_t low = 0xFFFFFFFFu, high = 0;
        for (int i = lane; i < size; i += 64) {
          const uint32_t v = value(i);
          if (v && v < low) low = v;
          if (v > high) high = v;
        }
        high = wave_max(high);
        low = ~wave_max(~low);
        found = low;
        int shift = low < high ? 32 - __clz((int)(low ^ high)) : 0;   // bits from here up are alike
        if (low < high) found = shift < 32 ? high >> shift << shift : 0;
#pragma unroll 1
        while (shift > 0) {
          const int bits = shift < 8 ? shift : 8, next = shift - bits;
          __syncthreads();
          if (tid < 256) sh.digits[tid] = 0;
          __syncthreads();
          for (int i = tid; i < size; i += kRowThreads) {
            const uint32_t v = value(i);
            if (v && (shift == 32 || v >> shift == found >> shift))
              atomicAdd(&sh.digits[(v >> next) & ((1u << bits) - 1)],
                        (unsigned long long)(stage == kTopP ? sh.list.weights[i] : 1));
          }
          __syncthreads();
          // every wave, from the highest down
          uint64_t so_far = more;
          int d = -1;
#pragma unroll 1
          for (int j = (1 << bits) - 1; j >= 0 && d < 0; j -= 64) {
            const uint64_t here = j >= lane ? sh.digits[j - lane] : 0, up = so_far + wave_scan(here);
            const uint64_t there = __ballot(up >= want);
            if (there) {
              const int l = __ffsll((unsigned long long)there) - 1;
              d = j - l;
              more = lane_value(up - here, l);
            }
            so_far = lane_value(up, 63);
          }
          if (d < 0) {
            found = low;
            break;
          }
          found |= (uint32_t)d << next;
          shift = next;
        }
        for (int i = lane; i < size; i += 64) {
          const uint32_t v = value(i);
          if (v == found) w = sh.list.weights[i];
          if (v > found) sum += sh.list.weights[i];
        }
        w = wave_max(w);
        sum = wave_sum(sum);
      }
      if (stage == kPlace) {
        last = found;
      } else {
        cut = found;
        if (stage == kTopK) {
          ties = want - more;
          over = at ? sh.sums[at - 1] : 0;
          all = over + sum + ties * w;
        } else {
          ties = w ? (want - more + w - 1) / w : 1;
        }
      }
    }
  }
  if (passes) {
    sample_passes<F32>(a, r, row, top, set, sh);
    return;
  }
  // what is kept of each part: a part's sum before the bin, and what the list has
  if (bin < kBins) {
    uint64_t before[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int own = bin - 8 * by[h];
      const bool in = by[h] < 64 && own > 0;
      before[h] = part_sums[(int64_t)(in ? lane + 64 * h : 0) * kBins + (in ? own - 1 : 0)];
      before[h] = in ? before[h] >> by[h] : 0;
    }
    __syncthreads();
    if (tid < 64) {
      sh.kept[lane] = before[0];
      sh.kept[lane + 64] = before[1];
    }
    __syncthreads();
    for (int i = tid; i < size; i += kRowThreads) {
      const uint32_t key = sh.list.keys[i], place = sh.list.places[i];
      if (key > cut || (key == cut && ~place >= last)) atomicAdd(&sh.kept[place / kPart], (unsigned long long)sh.list.weights[i]);
    }
    __syncthreads();
    whole[0] = sh.kept[lane];
    whole[1] = sh.kept[lane + 64];
  }
  // the part in which the sum passes the target
  uint64_t up[2], start = 0;
  up[0] = wave_scan(whole[0]);
  up[1] = parts > 64 ? lane_value(up[0], 63) + wave_scan(whole[1]) : 0;
  all = lane_value(parts > 64 ? up[1] : up[0], 63);
  uint64_t target = (uint64_t)floor(set.u * (double)all);
  if (target >= all) target = all - 1;
  const int h = parts > 64 && lane_value(up[0], 63) <= target ? 1 : 0;
  const int l = __ffsll((unsigned long long)__ballot(up[h] > target)) - 1, part = l + 64 * h;
  start = lane_value(up[h] - whole[h], l);
  __syncthreads();   // (the table, where no list was made)
  // its logits, 16 in a row to a thread
  const int from = part * kPart, to = min(n, from + kPart), first = from + 16 * tid;
  float v[16];
  if (to - from == kPart) {
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
      float eight[8];
      logits<F32, 8>(row, first + i, eight);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i + e] = eight[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = logit<F32>(row, min(first + e, n - 1));
  }
  // their weights' sum
  uint64_t sum = 0;
  int final = -1;   // the last that is kept
  const auto kept = [&](float x, int place) {
    const uint32_t key = key_of(x);
    return place < to && key > kNoKey && (key > cut || (key == cut && ~(uint32_t)place >= last));
  };
#pragma unroll 1
  for (int i = 0; i < 16; i += 4) {
    float four[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) four[e] = i == 0 ? v[e] : i == 4 ? v[4 + e] : i == 8 ? v[8 + e] : v[12 + e];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint64_t w = weight_of(four[e]);
      const bool k = kept(four[e], first + i + e) && w;
      sum += k ? w : 0;
      final = k ? first + i + e : final;
    }
  }
  // the thread in which the sum passes the target; where rounding at other
  // places (of the parts' sums, of the weights) leaves none, the last kept
  uint64_t at = wave_scan(sum);
  __syncthreads();
  if (lane == 63) sh.tmp[tid >> 6] = at;
  if (tid == 0) sh.found = -1;
  __syncthreads();
  at += start - sum;
#pragma unroll 1
  for (int w = 0; w < tid >> 6; ++w) at += sh.tmp[w];
  const bool mine = at <= target && at + sum > target;
  if (mine) sh.found = first;
  __syncthreads();
  const bool none = sh.found < 0;
  if (none) {
    const uint64_t end = wave_max((uint32_t)(final + 1));
    if (lane == 0) sh.tmp[tid >> 6] = end;
    __syncthreads();
    for (int w = 0; w < kRowThreads / 64; ++w) final = max(final, (int)sh.tmp[w] - 1);
    __syncthreads();
  }
  if (none ? tid == 0 : mine) {
    int id = final;
    if (!none)
#pragma unroll 1
      for (int e = 0; e < 16; ++e) {
        const float x = logit<F32>(row, min(first + e, n - 1));
        const uint64_t w = kept(x, first + e) ? weight_of(x) : 0;
        if (w) id = first + e;
        at += w;
        if (at > target) break;
      }
    a.ids[r] = id;
    if (a.logprobs) {
      const double x = fma((double)logit<F32>(row, id), sc.per, -sc.power);
      a.logprobs[r] = (float)(x * 0.69314718055994530942 - log(ldexp((double)all, -a.unit)));
    }
  }
}

}  // namespace

hipError_t launch_sample(const SampleArgs &a, hipStream_t s) {
  const int64_t items = (int64_t)a.rows * a.parts;
  const unsigned groups = (unsigned)(items < kSampleGroups ? items : kSampleGroups);
  static_assert(sizeof(Shared) <= 160 * 1024, "one workgroup's LDS");
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
