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
// read again, token by token.  A cut below the bins lies in one more, of all
// weights that are left (2^-32 to 2^-45 of the largest).  Rows for which that
// does not do (more logits in a cut's bin than fit in LDS, a largest beyond 2^13
// powers of two, temperatures near infinity) take several passes over all.
//
// The first launch is bound by vector instructions, 33 for each 64 logits,
// six of them in fp64 or converting to and from it, and by LDS atomics where
// there are cuts: 66 us for 256 rows of 151936 (156 MB; a plain read 24), of
// which the sums in bins take a third; 7 us for one row.  The second runs
// once through its code, most of which then comes from the L2 line by line
// (92 KB of unrolled code took 49 us for one row where 45 KB take 30): loops
// there stay rolled, each piece of work has one place, and what a wave can
// find out alone every wave does, without waiting for the others.  43 us for
// 64 rows, 54 for 256: the row with the most open top-p, whose cut's bin holds
// thousands of logits in all parts, which one CU reads again.
#include "wq_internal.h"

namespace wq {
using namespace dev;

namespace {

constexpr uint32_t kNoKey = 0x007FFFFFu;     // of -infinity
constexpr int kBins = kSampleBins;
constexpr int kBelow = kBins;                // all weights below the bins, down to a unit's half
constexpr int kNoBin = kBins + 1;
constexpr int kPart = kSamplePart;
constexpr int kPartThreads = 512;
constexpr int kEach = kPart / kPartThreads;  // logits of a thread
constexpr int kMaxParts = (1 << 20) / kPart;
constexpr int kTable = 1024;
constexpr double kFar = 8192.0;              // largest power of two of a row's largest that the bins take
constexpr double kFarOfPart = kFar + 64.0;   // of a part's: one further down has no weight beside a row's within kFar

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
// r^12 / 12! (its next term is below 2^-57 of the sum).  r takes off n ln 2 in
// two parts: ln 2 rounded to fp32, n times which is exact, and what is left.
__device__ __forceinline__ double exp64(double z) {
  if (!(z > -100.0)) return 0.0;   // below any unit
  const double n = rint(z * 1.4426950408889634074);
  const double r = fma(n, 1.904654299957767878e-9, fma(-n, (double)0.69314718055994530942f, z));
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

// Weights by powers of two: x = l log2(e) / T - power, w = 2^x.  One fp64
// multiply-add leaves x in 2^-40s in the low bits of its result, from which
// whole powers, 1024ths (a table of 2^(j / 1024)) and the rest g are cut;
// 2^g = 1 + e, g < 2^-10, where e in fp32 is 2^-34 of w off.
struct Scale {
  double per;                  // log2(e) / T
  double power;                // a whole number
  int unit;
  double shift;                // 1.5 2^12 - power: 2^-40s are its last bit
  float lowest;                // logits below it count as it: x about -1000
};

constexpr uint32_t kShiftHigh = 0x40B80000u;   // the upper half of 1.5 2^12

__device__ __forceinline__ Scale scale(double per, double power, int unit) {
  const double lowest = (power - 1000.0) / per;
  return {per, power, unit, 6144.0 - power, (float)(lowest > -3.4e38 ? lowest : -3.4e38)};
}

// What scale() is for: x of the largest logit, and of -infinity's stand-in, in
// the range of the low bits.
__device__ __forceinline__ bool near(double per, double most, double far) { return fabs(most) < far && per > 1e-30; }

struct Split {
  uint32_t hi, lo;
};

__device__ __forceinline__ Split split(float l, const Scale &s) {
  const uint64_t q = __builtin_bit_cast(uint64_t, fma((double)fmaxf(l, s.lowest), s.per, s.shift));   // (not NaN)
  return {(uint32_t)(q >> 32), (uint32_t)q};
}

__device__ __forceinline__ uint64_t counted(const Split &p, const Scale &s, const double *table) {
  constexpr float kLn2 = 6.3041364e-13f;   // ln 2 / 2^40
  const float g = (float)(p.lo & 0x3FFFFFFFu), e = g * fmaf(g, fmaf(g, kLn2 * kLn2 * kLn2 / 6.0f, kLn2 * kLn2 / 2.0f), kLn2);
  const double w = table[__builtin_amdgcn_alignbit(p.hi, p.lo, 30) & (kTable - 1)];
  const int power = ((int)(p.hi - kShiftHigh) >> 8) + s.unit;
  const double c = ldexp(fma(w, (double)e, w), power) + 4503599627370496.0;   // 2^52: whole numbers
  return __builtin_bit_cast(uint64_t, c) - 0x4330000000000000ull;
}

// Eighths of a power of two, downwards: the largest, x in [0, 1), is in one of
// 1 to 8 (by rounding up to 1 in 0)
__device__ __forceinline__ int bin_of(const Split &p) { return 8 - ((int)(p.hi - kShiftHigh) >> 5); }

__device__ __forceinline__ double table_entry(int j) { return exp64((double)j * (0.69314718055994530942 / kTable)); }

struct Larger {
  template <typename T>
  __device__ T operator()(T a, T b) const { return a > b ? a : b; }
};
struct Sum {
  template <typename T>
  __device__ T operator()(T a, T b) const { return a + b; }
};

// over a wave, in every lane
template <typename T>
__device__ __forceinline__ T wave_sum(T v) { return lane_value(wave_scan(v, (T)0, Sum()), 63); }
template <typename T>
__device__ __forceinline__ T wave_max(T v) { return lane_value(wave_scan(v, (T)0, Larger()), 63); }

// ---------------------------------------------------------------- parts

// the largest of v over a wave, in every lane
__device__ __forceinline__ float wave_max_f32(float v) {
  v = fmaxf(v, dpp<kQuadXor1>(v));
  v = fmaxf(v, dpp<kQuadXor2>(v));
  v = fmaxf(v, dpp<kRowHalfMirror>(v));
  v = fmaxf(v, dpp<kRowMirror>(v));
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}

// The next part's logits and settings are on their way while this one's are
// counted, the bins of one part are summed up by one wave while the others go
// on: two sets of bins, two barriers a part.
template <bool F32>
__global__ __launch_bounds__(kPartThreads) void sample_parts_kernel(SampleArgs a) {
  constexpr int V = F32 ? 4 : 8;   // logits in 16 bytes
  constexpr int kWaves = kPartThreads / 64;
  __shared__ double table[kTable];
  struct Bins {
    alignas(16) unsigned long long sums[kBins];
    alignas(16) uint32_t counts[kBins];
    unsigned long long sum;
    uint32_t nonzero, where;
  };
  __shared__ Bins both[2];
  __shared__ float tops[2][kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int items = a.rows * a.parts;
  const auto fetch = [&](int item, float (&v)[kEach], Settings &s) {
    const int r = item / a.parts, from = (item - r * a.parts) * kPart;
    const void *row = F32 ? (const void *)(static_cast<const float *>(a.logits) + r * a.ldl)
                          : (const void *)(static_cast<const uint16_t *>(a.logits) + r * a.ldl);
    if (from + kPart <= a.vocab) {
#pragma unroll
      for (int i = 0; i < kEach / V; ++i) {
        float some[V];
        logits<F32, V>(row, from + (i * kPartThreads + tid) * V, some);
#pragma unroll
        for (int e = 0; e < V; ++e) v[V * i + e] = some[e];
      }
    } else {   // (a lambda of its own would join the loads of the two)
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int at = from + (i / V * kPartThreads + tid) * V + i % V;
        v[i] = logit<F32>(row, min(at, a.vocab - 1));
        v[i] = at < a.vocab ? v[i] : -INFINITY;
      }
    }
    s = settings(a, r);
  };
  float v[kEach], next[kEach];
  Settings s, next_s;
  if ((int)blockIdx.x < items) fetch(blockIdx.x, v, s);
  for (int j = tid; j < kTable; j += kPartThreads) table[j] = table_entry(j);
  for (int j = tid; j < 2 * kBins; j += kPartThreads) {
    both[j / kBins].sums[j % kBins] = 0;
    both[j / kBins].counts[j % kBins] = 0;
  }
  if (tid < 2) {
    both[tid].sum = 0;
    both[tid].nonzero = 0;
    both[tid].where = 0xFFFFFFFFu;
  }
  int turn = 0;
  for (int item = blockIdx.x; item < items; item += gridDim.x, ++turn) {
    Bins &sh = both[turn & 1];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kEach; ++i) top = fmaxf(top, v[i]);   // (not NaN)
    const float high = wave_max_f32(top);
    if (lane == 0) tops[turn & 1][wave] = high;
    __syncthreads();
    float most = tops[turn & 1][0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) most = fmaxf(most, tops[turn & 1][w]);
    if (top == most) {   // the first of them
#pragma unroll
      for (int i = kEach - 1; i >= 0; --i)
        if (v[i] == most) top = __builtin_bit_cast(float, (i / V * kPartThreads + tid) * V + i % V);
      atomicMin(&sh.where, __builtin_bit_cast(uint32_t, top));
    }
    const double per = 1.4426950408889634074 / (double)s.heat, power = (double)most * per;
    const bool counts_in = !s.greedy && most > -INFINITY && near(per, power, kFarOfPart);
    const Scale sc = scale(per, floor(power), a.unit);
    if (item + (int)gridDim.x < items) fetch(item + gridDim.x, next, next_s);
    if (counts_in) {
      uint64_t sum = 0;
      uint32_t nonzero = 0;   // of the wave
      const bool counts = s.top_k < a.vocab;
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
        if (counts)
#pragma unroll
          for (int e = 0; e < 8; ++e) nonzero += __popcll(__ballot(w[e] != 0));
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (bin_of(p[e]) < kBins) {
            atomicAdd(&sh.sums[bin_of(p[e])], (unsigned long long)w[e]);
            if (counts) atomicAdd(&sh.counts[bin_of(p[e])], 1u);
          }
      }
      sum = wave_sum(sum);
      if (lane == 0) {
        atomicAdd(&sh.sum, (unsigned long long)sum);
        if (counts) atomicAdd(&sh.nonzero, nonzero);
      }
    }
    __syncthreads();
    if (wave == turn % kWaves) {
      if (lane == 0) {
        const int r = item / a.parts;
        SamplePart head;
        head.best = (uint64_t)key_of(most) << 32 | (uint32_t)~((item - r * a.parts) * kPart + sh.where);
        head.sum = sh.sum;
        head.power = counts_in ? (int32_t)sc.power : kFarPart;   // no bins
        head.nonzero = sh.nonzero;
        a.heads[item] = head;
        sh.sum = 0;
        sh.nonzero = 0;
        sh.where = 0xFFFFFFFFu;
      }
      if (counts_in && s.cuts) {
        // sums up to and with each bin, four a lane
        uint64_t up[4];
        uint32_t many[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          up[e] = sh.sums[4 * lane + e] + (e ? up[e - 1] : 0);
          many[e] = sh.counts[4 * lane + e] + (e ? many[e - 1] : 0);
          sh.sums[4 * lane + e] = 0;
          sh.counts[4 * lane + e] = 0;
        }
        static_assert(kBins == 256, "four a lane");
        uint64_t all = wave_scan(up[3], (uint64_t)0, Sum());
        uint32_t all_many = wave_scan(many[3], 0u, Sum());
        all -= up[3];
        all_many -= many[3];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a.sums[(int64_t)item * kBins + 4 * lane + e] = all + up[e];
          a.counts[(int64_t)item * kBins + 4 * lane + e] = all_many + many[e];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) v[i] = next[i];
    s = next_s;
  }
}

// ---------------------------------------------------------------- rows

constexpr int kRowThreads = 1024;
constexpr int kMine = kPart / kRowThreads;   // logits of a part to a thread
static_assert(kMine == 8, "");
constexpr int kList = 8192;                  // logits of a cut's bin, at most

// the sum of v over the threads before this one, and over all
__device__ __forceinline__ uint64_t block_before(uint64_t v, uint64_t *tmp) {
  const uint64_t up = wave_scan(v, (uint64_t)0, Sum());
  __syncthreads();
  if ((threadIdx.x & 63) == 63) tmp[threadIdx.x >> 6] = up;
  __syncthreads();
  uint64_t before = up - v;
#pragma unroll 1
  for (int w = 0; w < (int)(threadIdx.x >> 6); ++w) before += tmp[w];
  return before;
}

__device__ __forceinline__ uint64_t block_sum(uint64_t v, uint64_t *tmp) {
  const uint64_t sum = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = sum;
  __syncthreads();
  uint64_t all = 0;
#pragma unroll 1
  for (int w = 0; w < kRowThreads / 64; ++w) all += tmp[w];
  return all;
}

constexpr int kSlowBins = 2048;
constexpr int kTurn = 4 * kRowThreads;       // logits that a pass takes side by side
constexpr int kTurns = kMaxParts;

struct Shared {
  double table[kTable];
  uint64_t tmp[kRowThreads / 64];
  unsigned long long sums[kBins], counts[kBins];   // the row's, up to and with each bin
  unsigned long long digits[256];            // of a search in a long list
  unsigned long long kept[kMaxParts];        // of each part
  uint64_t above;
  unsigned long long found_weight, found_sum;
  int32_t found;
  uint32_t list_size, low, high;
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

// f(key) for every logit of [from, to)
template <bool F32, typename F>
__device__ __forceinline__ void each_key(const void *row, int from, int to, F f) {
  constexpr int kAtOnce = 4;
  int i = from;
#pragma unroll 1
  for (; i + kAtOnce * kTurn <= to; i += kAtOnce * kTurn) {
    float v[kAtOnce][4];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) logits<F32, 4>(row, i + j * kTurn + 4 * (int)threadIdx.x, v[j]);
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) f(key_of(v[j][e]));
  }
#pragma unroll 1
  for (i += (int)threadIdx.x; i < to; i += kRowThreads) f(key_of(logit<F32>(row, i)));
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
    if (before < want && before + one + two >= want) {
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
    const uint64_t over = block_sum(sum, sh.tmp);
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
  // sums of each part
  const double cut_weight = weight(cut, s);
  const uint64_t tie = cut_weight >= set.at_least ? counted(cut_weight, s) : 0;
  const int turns = (n + kPart - 1) / kPart;
  for (int t = tid; t < turns; t += kRowThreads) sh.slow.sums[t] = sh.slow.ties[t] = 0;
  __syncthreads();
  for (int t = 0; t < turns; ++t) {
    uint64_t sum = 0;
    uint32_t same = 0;
    each_key<F32>(row, t * kPart, min(n, (t + 1) * kPart), [&](uint32_t key) {
      same += key == cut;
      if (key > cut) {
        const double w = weight(key, s);
        if (w >= set.at_least) sum += counted(w, s);
      }
    });
    sum = wave_sum(sum);
    same = wave_sum(same);
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
  // the part's logits, some in a row to a thread
  const int first = t * kPart + kMine * tid;
  uint64_t same = 0;
#pragma unroll 1
  for (int e = 0; e < kMine; ++e) same += first + e < n && cut && key_of(logit<F32>(row, first + e)) == cut;
  const uint64_t rank = seen + block_before(same, sh.tmp);
  const auto weight_at = [&](uint32_t key, uint64_t &place) -> uint64_t {
    if (key > cut) {
      const double v = weight(key, s);
      return v >= set.at_least ? counted(v, s) : 0;
    }
    return key == cut && cut && place++ < ties ? tie : 0;
  };
  uint64_t mine = 0, place = rank;
#pragma unroll 1
  for (int e = 0; e < kMine && first + e < n; ++e) mine += weight_at(key_of(logit<F32>(row, first + e)), place);
  uint64_t sum = before + block_before(mine, sh.tmp);
  if (sum <= target && sum + mine > target) {
    place = rank;
#pragma unroll 1
    for (int e = 0; e < kMine; ++e) {
      const uint32_t key = key_of(logit<F32>(row, first + e));
      sum += weight_at(key, place);
      if (sum > target) {
        a.ids[r] = first + e;
        if (a.logprobs) {
          const double z = key == s.top ? 0.0 : ((double)value_of(key) - s.max) * s.per;
          a.logprobs[r] = (float)(z - log((double)all / s.unit));
        }
        break;
      }
    }
  }
}

// ---- by the parts' bins

// kMine logits of a thread, from `first` on; where fewer are left, those up to
// the row's end: the first of them is at the place returned, and those before
// `first` are another thread's.
template <bool F32>
__device__ __forceinline__ int fetch(const void *row, int first, int n, float (&v)[kMine]) {
  const int place = max(min(first, n - kMine), 0);
  if (n >= kMine) {
    logits<F32, kMine>(row, place, v);
  } else {
#pragma unroll
    for (int e = 0; e < kMine; ++e) v[e] = e < n ? logit<F32>(row, min(e, n - 1)) : NAN;
  }
  return place;
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
  sh.table[tid] = table_entry(tid);
  static_assert(kTable == kRowThreads, "an entry a thread");
  if (tid < kBins) sh.sums[tid] = sh.counts[tid] = 0;
  __syncthreads();
  const double per = 1.4426950408889634074 / (double)set.heat, most = (double)value_of(top) * per;
  const Scale sc = scale(per, floor(most), a.unit);
  // as the first launch counted it: borders of equal weights are exact
  const auto weight_of = [&](float l) { return counted(split(l, sc), sc, sh.table); };
  bool passes = !near(per, most, kFar);

  // what is kept: keys above `cut`, and of those at it the ones whose index's
  // complement is `last` or more; all of the bins before `bin` and, in the
  // list, the logits of that bin
  uint32_t cut = 0, last = 0;
  uint64_t ties = ~0ull, all = 0, whole[2];   // sum of the weights kept; of a part's
  int bin = kNoBin, size = 0, by[2];           // by: how far a part's powers are below the row's (64: too far)
  if (!passes) {
    const int power = (int)sc.power;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = lane + 64 * h < parts && head[h].power != kFarPart && power - head[h].power < 64;
      by[h] = in ? power - head[h].power : 64;
      // Under the row's power weights below half a unit are 0, the sum of
      // thousands is not: it counts, but where top-k is asked for.  There only
      // what is not 0 is sure to be kept, so a part needs a whole unit.
      whole[h] = in && (by[h] <= a.unit || set.top_k >= n) ? head[h].sum >> by[h] : 0;
    }
    all = wave_sum(whole[0] + whole[1]);
  }
  if (!passes && set.cuts) {
    // top-k matters if it leaves out a logit whose weight is not 0: parts so far
    // below the row's that theirs are have none, the others at most their own
    uint32_t nonzero = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) nonzero += by[h] < a.unit + 2 ? head[h].nonzero : 0;
    const bool counting = (uint32_t)set.top_k < wave_sum(nonzero);
    // the row's bins: a thread one bin of some parts
    {
      const int j = tid & (kBins - 1);
      uint64_t sum = 0, many = 0;
#pragma unroll 5
      for (int p = tid / kBins; p < parts; p += kRowThreads / kBins) {
        const int late = __shfl(p < 64 ? by[0] : by[1], p & 63), own = j - 8 * late;   // p is the wave's
        const int64_t i = (int64_t)p * kBins + max(own, 0);
        const uint64_t w = part_sums[i];
        const uint32_t c = part_counts[i];
        sum += late < 64 && own >= 0 ? w >> late : 0;
        many += late < 64 && own >= 0 ? c : 0;
      }
      atomicAdd(&sh.sums[j], (unsigned long long)sum);
      atomicAdd(&sh.counts[j], (unsigned long long)many);
      static_assert(kRowThreads % kBins == 0, "threads of a bin");
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
        at = min(bin_of(split(value_of(yes), sc)), kBelow);
      } else {
        if (bin == kNoBin) continue;
        // of equal ones at the cut the first by index
        __syncthreads();
        if (tid == 0) sh.list_size = 0;   // (size has it)
        __syncthreads();
        uint32_t same = 0;
        for (int i = tid; i < size; i += kRowThreads) same += sh.list.keys[i] == cut;
        same = wave_sum(same);
        if (lane == 0 && same) atomicAdd(&sh.list_size, same);
        __syncthreads();
        if (ties >= sh.list_size) continue;
        want = ties;
      }
      if (stage <= kTopP) {
        // the first bin with which the sum reaches `want`, and the sum before it
        const unsigned long long *bins = stage == kTopK ? sh.counts : sh.sums;
        at = 0;
#pragma unroll 1
        for (int j = 0; j < kBins; j += 64) at += __popcll(__ballot(bins[j + lane] < want));
        above = at ? bins[at - 1] : 0;
        if (at >= bin) {
          // among top-k's list
          at = bin;
          const uint64_t w = weight_of(value_of(cut)), high = all - ties * w;
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
          const bool in = at == kBelow ? by[h] < a.unit + 2 : by[h] < 64 && own >= 0;
          const uint64_t *sums = part_sums + (int64_t)(in ? lane + 64 * h : 0) * kBins;
          const uint64_t binned = sums[min(max(own, 0), kBins - 1)], before = sums[max(own - 1, 0)];
          const uint64_t up_to = at == kBelow ? head[h].sum : binned;
          wanted[h] = __ballot(in && (own > 0 ? up_to != before : up_to != 0));
        }
        __syncthreads();
        // The bin's logits are those from `from_value` up to `to_value`, whose
        // keys are the lowest of the bin and of the next higher: near where
        // the logarithm puts them (64 keys at once), or by halves.
        float from_value = 0.0f, to_value = 0.0f;
#pragma unroll 1
        for (int edge = 0; edge < 2; ++edge) {
          const int lowest = edge ? at - 1 : at == kBelow ? 8 * (a.unit + 2) : at;   // the bin that starts there
          const uint32_t guess = key_of((float)(((double)(8 - lowest) * 0.125 + sc.power) / sc.per));
          uint32_t no = kNoKey, yes = top + 1;
#pragma unroll 1
          for (int turn = 0; yes - no > 1; ++turn) {
            const bool many = turn == 0 && guess > kNoKey + 64 && guess <= top;
            const uint32_t key = many ? guess - 32 + (uint32_t)lane : no + (yes - no) / 2;
            const uint64_t there = __ballot(key > top || bin_of(split(value_of(key), sc)) <= lowest);
            if (many) {
              if (there && !(there & 1)) {
                yes = guess - 32 + (uint32_t)(__ffsll((unsigned long long)there) - 1);
                no = yes - 1;
              }
            } else if (there) {
              yes = key;
            } else {
              no = key;
            }
          }
          from_value = edge ? from_value : value_of(yes);
          to_value = yes > top ? INFINITY : value_of(yes);   // above the largest: nothing is that high
        }
#pragma unroll 1
        while (wanted[0] | wanted[1]) {
          // four parts asked for at once
          int which[4];
          float four[4][kMine];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool low = wanted[0] != 0;
            const uint64_t left = low ? wanted[0] : wanted[1];
            which[j] = left ? __ffsll((unsigned long long)left) - 1 + (low ? 0 : 64) : -1;
            wanted[0] &= wanted[0] - (low ? 1 : 0);
            wanted[1] &= wanted[1] - (low || !left ? 0 : 1);
            fetch<F32>(row, max(which[j], 0) * kPart + kMine * tid, n, four[j]);
          }
#pragma unroll 1
          for (int j = 0; j < 4; ++j) {
            const int p = j < 2 ? (j ? which[1] : which[0]) : j == 2 ? which[2] : which[3];
            if (p < 0) break;
            const int first = p * kPart + kMine * tid, from = max(min(first, n - kMine), 0);
            float v[kMine];
#pragma unroll
            for (int e = 0; e < kMine; ++e) v[e] = j < 2 ? (j ? four[1][e] : four[0][e]) : j == 2 ? four[2][e] : four[3][e];
            if ((p + 1) * kPart > n) {
#pragma unroll
              for (int e = 0; e < kMine; ++e) v[e] = from + e >= first ? v[e] : NAN;   // another thread's
            }
            uint32_t some = 0;
#pragma unroll
            for (int e = 0; e < kMine; ++e) some |= v[e] >= from_value && v[e] < to_value ? 1u << e : 0;
            // one of each lane at a time (rarely more than a few)
#pragma unroll 1
            for (uint64_t lanes; (lanes = __ballot(some)) != 0; some &= some - 1) {
              uint32_t to = 0;
              if (lane == 0) to = atomicAdd(&sh.list_size, (uint32_t)__popcll(lanes));
              const uint32_t i = (uint32_t)__builtin_amdgcn_readfirstlane((int)to) +
                                 __builtin_amdgcn_mbcnt_hi((uint32_t)(lanes >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)lanes, 0));
              if (some && i < (uint32_t)kList) sh.list.places[i] = (uint32_t)(from + __ffs((int)some) - 1);
            }
          }
        }
        __syncthreads();
        if (sh.list_size > (uint32_t)kList) {
          passes = true;
          break;
        }
        size = (int)sh.list_size;
        bin = at;
#pragma unroll 1
        for (int i = tid; i < size; i += kRowThreads) {
          const float l = logit<F32>(row, (int64_t)sh.list.places[i]);
          sh.list.keys[i] = key_of(l);
          sh.list.weights[i] = weight_of(l);
        }
        __syncthreads();
      }
      if (stage == kMinP) continue;
      if (stage < kPlace && at == kBelow && (size == 0 || (stage == kTopK && want - above >= (uint64_t)size))) {
        over = sh.sums[kBins - 1];   // (all that has a weight)
        continue;
      }
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
        __syncthreads();
        if (tid == 0) {
          sh.low = 0xFFFFFFFFu;
          sh.high = 0;
          sh.found_weight = sh.found_sum = 0;
        }
        __syncthreads();
        uint32_t low = 0xFFFFFFFFu, high = 0;
        for (int i = tid; i < size; i += kRowThreads) {
          const uint32_t v = value(i);
          if (v && v < low) low = v;
          if (v > high) high = v;
        }
        high = wave_max(high);
        low = ~wave_max(~low);
        if (lane == 0) {
          atomicMax(&sh.high, high);
          atomicMin(&sh.low, low);
        }
        __syncthreads();
        high = sh.high;
        low = sh.low;
        found = low;
        int shift = low < high ? 32 - __clz((int)(low ^ high)) : 0;   // bits from here up are alike
        if (low < high) found = shift < 32 ? high >> shift << shift : 0;
#pragma unroll 1
        while (shift > 0) {
          const int bits = shift < 8 ? shift : 8, next = shift - bits, end = (1 << bits) - 1;
          if (tid < 256) sh.digits[tid] = 0;
          __syncthreads();
          for (int i = tid; i < size; i += kRowThreads) {
            const uint32_t v = value(i);
            if (v && (shift == 32 || v >> shift == found >> shift))
              atomicAdd(&sh.digits[end - ((v >> next) & end)],   // from the highest on
                        (unsigned long long)(stage == kTopP ? sh.list.weights[i] : 1));
          }
          __syncthreads();
          // every wave: four digits a lane
          uint64_t up[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) up[e] = sh.digits[4 * lane + e] + (e ? up[e - 1] : 0);
          const uint64_t before = more + wave_scan(up[3], (uint64_t)0, Sum()) - up[3];
          const uint64_t there = __ballot(before + up[3] >= want);
          __syncthreads();
          if (!there) {
            found = low;
            break;
          }
          const int l = __ffsll((unsigned long long)there) - 1;
          int e = 0;
          uint64_t higher = before;
#pragma unroll
          for (int f = 0; f < 3; ++f)
            if (before + up[f] < want) {
              e = f + 1;
              higher = before + up[f];
            }
          more = lane_value(higher, l);
          found |= (uint32_t)(end - (4 * l + __builtin_amdgcn_readlane(e, l))) << next;
          shift = next;
        }
        for (int i = tid; i < size; i += kRowThreads) {
          const uint32_t v = value(i);
          if (v == found) sh.found_weight = sh.list.weights[i];
          if (v > found) sum += sh.list.weights[i];
        }
        sum = wave_sum(sum);
        if (lane == 0 && sum) atomicAdd(&sh.found_sum, (unsigned long long)sum);
        __syncthreads();
        w = sh.found_weight;
        sum = sh.found_sum;
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
  if (bin < kNoBin) {
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
  uint64_t up[2], start;
  up[0] = wave_scan(whole[0], (uint64_t)0, Sum());
  up[1] = parts > 64 ? lane_value(up[0], 63) + wave_scan(whole[1], (uint64_t)0, Sum()) : 0;
  all = lane_value(parts > 64 ? up[1] : up[0], 63);
  uint64_t target = (uint64_t)floor(set.u * (double)all);
  const bool end = target >= all;   // u = 1: the last one kept
  if (end) target = all - 1;
  const int h = parts > 64 && lane_value(up[0], 63) <= target ? 1 : 0;
  const int l = __ffsll((unsigned long long)__ballot(up[h] > target)) - 1, part = l + 64 * h;
  start = lane_value(up[h] - whole[h], l);
  // In a row that is open to the end the part's logits are weighed as the first
  // launch did, under the part's own power, which adds up to the sum that the
  // part was chosen by: under the row's power each of them may be 0.  With a
  // cut what it was chosen by are bins of 2^-32 and more and the list's weights
  // under the row's power, with top-k alone a part's largest is a unit or more.
  const int below = bin < kNoBin || set.top_k < n ? 0 : (int)lane_value((uint32_t)(h ? by[1] : by[0]), l);
  Scale own = sc;
  own.power -= below;
  own.shift += below;
  target = end ? ~0ull : (target - start) << below;
  __syncthreads();   // (the table, where no list was made)
  // its logits, some in a row to a thread
  const int first = part * kPart + kMine * tid, to = min(n, (part + 1) * kPart);
  float v[kMine];
  const int from = fetch<F32>(row, first, n, v);
  const auto taken = [&](float x, int place) {
    const uint32_t key = key_of(x);
    return key > kNoKey && (key > cut || (key == cut && ~(uint32_t)place >= last));
  };
  // their weights' sum
  uint64_t sum = 0;
  int final = -1;   // the last that is kept
#pragma unroll 1
  for (int i = 0; i < kMine; i += 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = i ? v[4 + e] : v[e];
      const uint64_t w = counted(split(x, own), own, sh.table);
      const bool k = from + i + e >= first && from + i + e < to && taken(x, from + i + e) && w;
      sum += k ? w : 0;
      final = k ? from + i + e : final;
    }
  }
  // the wave and the thread in which the sum passes the target; where
  // rounding at other places (of the parts' sums, of the weights under the
  // row's power) leaves none, or u is 1, the last kept
  uint64_t at = wave_scan(sum, (uint64_t)0, Sum());
  __syncthreads();
  if (lane == 63) sh.tmp[tid >> 6] = at;
  if (tid == 0) sh.found = -1;
  __syncthreads();
  at -= sum;
#pragma unroll 1
  for (int w = 0; w < tid >> 6; ++w) at += sh.tmp[w];
  const uint64_t owner = __ballot(at <= target && at + sum > target);
  if (owner && lane == 0) sh.found = 0;
  __syncthreads();
  const bool none = sh.found < 0;
  int id = -1;
  if (none) {
    const uint64_t last_here = wave_max((uint32_t)(final + 1));
    if (lane == 0) sh.tmp[tid >> 6] = last_here;
    __syncthreads();
    for (int w = 0; w < kRowThreads / 64; ++w) id = max(id, (int)sh.tmp[w] - 1);
    if (id < 0) id = (int)~(uint32_t)best;   // no place outside the row, whatever the sums
    if (tid) return;
  } else {
    if (!owner) return;
    // the thread's logits, one to a lane
    const int o = __ffsll((unsigned long long)owner) - 1, place = __builtin_amdgcn_readlane(first, o) + lane;
    const float x = logit<F32>(row, min(place, n - 1));
    const uint64_t w = lane < kMine && place < to && taken(x, place) ? counted(split(x, own), own, sh.table) : 0;
    const uint64_t up = lane_value(at, o) + wave_scan(w, (uint64_t)0, Sum());
    const uint64_t passed = __ballot(up > target);
    id = __builtin_amdgcn_readlane(place, __ffsll((unsigned long long)passed) - 1);
    if (lane) return;
  }
  a.ids[r] = id;
  if (a.logprobs) {
    const float l = logit<F32>(row, id);
    const double x = fma((double)l, sc.per, -sc.power);
    // more than half of the sum: from the others', whose digits the logarithm
    // of the chance would lose
    const uint64_t w = weight_of(l);
    const bool most = w >= all / 2;
    const double ln = log1p(most ? -(double)(w < all ? all - w : 0) / (double)all : ldexp((double)all, -a.unit) - 1.0);
    a.logprobs[r] = (float)(most ? ln : x * 0.69314718055994530942 - ln);
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
