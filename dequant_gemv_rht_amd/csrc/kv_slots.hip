// Pages, slots and positions of a serving step's tokens (gfx950): two prefix
// sums over the sequences (rows, then pages), then one look-up for each row.
//
// Nothing to compute and little to move (12 bytes a row): the time is the
// launch and three round trips to memory.  So it is one launch without
// anything between workgroups: a workgroup takes kRows rows, adds up the
// sequences before them for itself (1024 sequences a turn, 8 KB from the
// caches), keeps a record for each sequence that has rows among its own, and
// a maximum over the rows spreads the records.  A new page's entry of the
// table is written by the row that opens the page, and no workgroup reads an
// entry that another writes: pages from the free list are looked up there.
#include "wq_internal.h"

namespace wq {

namespace {

constexpr int kSlotThreads = 256;
constexpr int kItems = 4;                    // sequences, and rows, of a thread
constexpr int kRows = kSlotThreads * kItems;

// exclusive sums of v over the workgroup's threads, and the total
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *sums, int64_t &total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t up = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_up(up, d);
    if (lane >= d) up += o;
  }
  __syncthreads();   // the last use of sums is over
  if (lane == 63) sums[wave] = up;
  __syncthreads();
  int64_t before = up - v;
  total = 0;
#pragma unroll
  for (int w = 0; w < kSlotThreads / 64; ++w) {
    if (w < wave) before += sums[w];
    total += sums[w];
  }
  return before;
}

struct Record {
  int32_t seq;       // -1: not served
  int32_t shift;     // position - row
  int32_t held;      // pages the sequence holds already
  int32_t place;     // of its first new page in the free list
};

__global__ __launch_bounds__(kSlotThreads) void kv_slots_kernel(SlotsArgs a) {
  __shared__ int64_t sums[kSlotThreads / 64];
  __shared__ Record rec[kRows];
  __shared__ int32_t mark[kRows], tops[kSlotThreads / 64];
  const int tid = threadIdx.x;
  const int64_t row0 = (int64_t)blockIdx.x * kRows, row1 = row0 + kRows < a.tokens ? row0 + kRows : a.tokens;
  const int32_t used = *a.used, mask = (1 << a.page_shift) - 1;
  const int64_t room = used >= 0 && used <= a.free_count ? a.free_count - used : 0;
  for (int i = tid; i < kRows; i += kSlotThreads) mark[i] = -1;

  int64_t rows = 0, need_sum = 0, taken = 0;   // before the turn; pages given out
  const int turns = (a.seqs + kRows - 1) / kRows;
  // turn t's sequences are written by workgroup t % gridDim, used_out by the
  // last turn's; a workgroup stops after its last such turn once the rows are
  // past its own
  const int grid = (int)gridDim.x, group = (int)blockIdx.x;
  const int until = group < turns ? group + (turns - 1 - group) / grid * grid : -1;
  for (int t = 0; t < turns; ++t) {
    if (rows >= row1 && t > until) break;
    const bool writes = t % grid == group;
    int32_t len[kItems], add[kItems];
    int64_t mine = 0;
#pragma unroll
    for (int e = 0; e < kItems; ++e) {
      const int64_t s = (int64_t)t * kRows + tid * kItems + e;
      len[e] = s < a.seqs ? a.lens[s] : 0;
      add[e] = s < a.seqs ? a.new_tokens[s] : 0;
      if (add[e] < 0) add[e] = 0;
      mine += add[e];
    }
    int64_t total;
    int64_t begin = rows + block_scan(mine, sums, total);
    rows += total;
    int32_t need[kItems], held[kItems];
    bool fits[kItems];
    int64_t at = begin, pages = 0;
#pragma unroll
    for (int e = 0; e < kItems; ++e) {
      const int64_t l = len[e] > 0 ? len[e] : 0, to = l + add[e];
      at += add[e];
      held[e] = (int32_t)((l + mask) >> a.page_shift);
      fits[e] = at <= a.tokens && to <= ((int64_t)a.table_pages << a.page_shift);
      need[e] = fits[e] ? (int32_t)((to + mask) >> a.page_shift) - held[e] : 0;
      pages += need[e];
    }
    int64_t place = need_sum + block_scan(pages, sums, total);
    need_sum += total;
#pragma unroll
    for (int e = 0; e < kItems; ++e) {
      const int64_t s = (int64_t)t * kRows + tid * kItems + e;
      const bool served = fits[e] && (need[e] == 0 || place + need[e] <= room);
      if (s < a.seqs) {
        if (served && need[e]) taken = place + need[e];
        if (writes) {
          a.lens_out[s] = served ? (len[e] > 0 ? len[e] : 0) + add[e] : len[e];
          a.last[s] = served && add[e] ? (int32_t)(begin + add[e] - 1) : -1;
        }
        // its first row here, if it has one
        const int64_t first = begin > row0 ? begin : row0;
        if (add[e] && first < row1 && begin + add[e] > row0) {
          const int i = (int)(first - row0);
          mark[i] = i;
          rec[i] = {served ? (int32_t)s : -1, (int32_t)((len[e] > 0 ? len[e] : 0) - begin), held[e],
                    served ? (int32_t)(used + place) : 0};
        }
      }
      begin += add[e];
      place += need[e];
    }
  }
  // what the last served sequence took: places only grow
  if ((turns ? turns - 1 : 0) % grid == group) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = __shfl_xor(taken, d);
      taken = o > taken ? o : taken;
    }
    __syncthreads();
    if ((tid & 63) == 0) sums[tid >> 6] = taken;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kSlotThreads / 64; ++w) taken = sums[w] > taken ? sums[w] : taken;
      *a.used_out = (int32_t)(used + taken);
    }
  }
  __syncthreads();
  // each row's record: the last mark up to it
  int32_t r[kItems], top = -1;
#pragma unroll
  for (int e = 0; e < kItems; ++e) {
    const int32_t m = mark[tid * kItems + e];
    top = m > top ? m : top;
    r[e] = top;
  }
  int32_t up = top;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t o = __shfl_up(up, d);
    if ((tid & 63) >= d && o > up) up = o;
  }
  if ((tid & 63) == 63) tops[tid >> 6] = up;
  int32_t before = __shfl_up(up, 1);
  if ((tid & 63) == 0) before = -1;
  __syncthreads();
  for (int w = 0; w < tid >> 6; ++w) before = tops[w] > before ? tops[w] : before;
#pragma unroll
  for (int e = 0; e < kItems; ++e) {
    const int64_t row = row0 + tid * kItems + e;
    if (row >= row1) break;
    const int32_t i = r[e] > before ? r[e] : before;
    int32_t slot = -1, pos = -1, seq = -1;
    if (i >= 0 && row < rows && rec[i].seq >= 0) {
      const Record c = rec[i];
      seq = c.seq;
      pos = (int32_t)(row + c.shift);
      const int32_t index = pos >> a.page_shift;
      int32_t *entry = a.table + seq * a.ld_table + index;
      int32_t page;
      if (index < c.held) {
        page = *entry;
      } else {
        page = a.free_pages[c.place + (index - c.held)];
        if ((pos & mask) == 0) *entry = page;
      }
      if (page >= 0 && page < a.pages) slot = (page << a.page_shift) + (pos & mask);
    }
    a.slots[row] = slot;
    a.positions[row] = pos;
    a.seq_of[row] = seq;
  }
}

}  // namespace

hipError_t launch_kv_slots(const SlotsArgs &a, hipStream_t s) {
  const int64_t groups = a.tokens ? ((int64_t)a.tokens + kRows - 1) / kRows : 1;
  hipLaunchKernelGGL(kv_slots_kernel, dim3((unsigned)groups), dim3(kSlotThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace wq
