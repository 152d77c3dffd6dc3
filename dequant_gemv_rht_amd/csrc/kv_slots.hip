// Pages, slots and positions of a serving step's tokens (gfx950): two prefix
// sums over the sequences (rows, then pages), then one look-up for each row.
//
// Nothing to compute and little to move (12 bytes a row): the time is the
// launch and three round trips to memory, 4.6 us for 64 sequences of one new
// token and 5.9 for 1024 sequences with 44000 rows in a kernel trace (an empty
// kernel takes 2.2).  So it is one launch without anything between workgroups:
// a workgroup takes kRows rows, adds up the sequences before them for itself
// (1024 sequences a turn, 8 KB from the caches), keeps a record for each
// sequence that has rows among its own, and a maximum over the rows spreads
// the records.  Sums in 32 bits that stop past the step's rows, by DPP moves: in
// 64 bits and by shuffles the first of these took 5.6 us.  A new page's entry
// of the table is written by the row that opens the page, and no workgroup
// reads an entry that another writes: pages from the free list are looked up
// there.
#include "wq_internal.h"

namespace wq {
using namespace dev;

namespace {

constexpr int kSlotThreads = 256;
constexpr int kItems = 4;                    // sequences, and rows, of a thread
constexpr int kRows = kSlotThreads * kItems;

constexpr int kWaves = kSlotThreads / 64;

// Sums that stop at `most` (so that they stay in 32 bits), over the threads
// before this one and over all, on top of `so_far`.  Every call has a `sums`
// of its own until the next barrier but one.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t most, uint32_t *sums, uint32_t &so_far) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const auto add = [&](uint32_t a, uint32_t b) { return min(a + b, most); };
  const uint32_t up = wave_scan(v, 0u, add);
  if (lane == 63) sums[wave] = up;
  __syncthreads();
  uint32_t before = so_far, all = so_far;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const uint32_t s = sums[w];
    if (w < wave) before = add(before, s);
    all = add(all, s);
  }
  so_far = all;
  return add(before, lane_before(up, 0));
}

struct Record {
  int32_t seq;       // -1: not served
  int32_t shift;     // position - row
  int32_t held;      // pages the sequence holds already
  int32_t place;     // of its first new page in the free list
};

__global__ __launch_bounds__(kSlotThreads) void kv_slots_kernel(SlotsArgs a) {
  __shared__ uint32_t sums[4][kWaves];
  __shared__ Record rec[kRows];
  __shared__ alignas(16) int32_t mark[kRows];
  __shared__ int32_t tops[kWaves];
  const int tid = threadIdx.x;
  const uint32_t row0 = blockIdx.x * kRows, row1 = min(row0 + kRows, (uint32_t)a.tokens);
  const int32_t used = *a.used, mask = (1 << a.page_shift) - 1;
  const uint32_t room = used >= 0 && used <= a.free_count ? a.free_count - used : 0;
#pragma unroll
  for (int e = 0; e < kItems; ++e) mark[tid * kItems + e] = -1;

  // before the turn: rows, up to one more than the step has, and pages (each
  // page counted has a row, or there would be no room for it)
  uint32_t rows = 0, asked = 0, taken = 0;
  const uint32_t most = (uint32_t)a.tokens + 1;
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
    uint32_t mine = 0;
#pragma unroll
    for (int e = 0; e < kItems; ++e) {
      const int s = t * kRows + tid * kItems + e;
      len[e] = s < a.seqs ? a.lens[s] : 0;
      add[e] = s < a.seqs ? a.new_tokens[s] : 0;
    }
#pragma unroll
    for (int e = 0; e < kItems; ++e) {
      if (add[e] < 0) add[e] = 0;
      mine = min(mine + (uint32_t)add[e], most);
    }
    uint32_t begin = block_scan(mine, most, sums[2 * (t & 1)], rows);
    int32_t need[kItems], held[kItems];
    bool fits[kItems];
    uint32_t at = begin, pages = 0;
#pragma unroll
    for (int e = 0; e < kItems; ++e) {
      const int64_t l = len[e] > 0 ? len[e] : 0, to = l + add[e];
      at = min(at + (uint32_t)add[e], most);
      held[e] = (int32_t)((l + mask) >> a.page_shift);
      fits[e] = at < most && to <= ((int64_t)a.table_pages << a.page_shift);
      need[e] = fits[e] ? (int32_t)((to + mask) >> a.page_shift) - held[e] : 0;
      pages += need[e];
    }
    uint32_t place = block_scan(pages, 0x7FFFFFFFu, sums[2 * (t & 1) + 1], asked);
#pragma unroll
    for (int e = 0; e < kItems; ++e) {
      const int s = t * kRows + tid * kItems + e;
      const bool served = fits[e] && (need[e] == 0 || place + need[e] <= room);
      if (s < a.seqs) {
        if (served && need[e]) taken = place + need[e];
        if (writes) {
          a.lens_out[s] = served ? (len[e] > 0 ? len[e] : 0) + add[e] : len[e];
          a.last[s] = served && add[e] ? (int32_t)(begin + add[e] - 1) : -1;
        }
        // its first row here, if it has one
        const uint32_t first = max(begin, row0);
        if (add[e] && first < row1 && min(begin + (uint32_t)add[e], most) > row0) {
          const int i = (int)(first - row0);
          mark[i] = i;
          rec[i] = {served ? s : -1, (int32_t)((uint32_t)(len[e] > 0 ? len[e] : 0) - begin), held[e],
                    served ? (int32_t)((uint32_t)used + place) : 0};
        }
      }
      begin = min(begin + (uint32_t)add[e], most);
      place += need[e];
    }
  }
  // what the last served sequence took: places only grow
  if ((turns ? turns - 1 : 0) % grid == group) {
    const uint32_t top = wave_scan(taken, 0u, [](uint32_t x, uint32_t y) { return max(x, y); });
    __syncthreads();
    if ((tid & 63) == 63) sums[0][tid >> 6] = top;
    __syncthreads();
    if (tid == 0) {
      taken = sums[0][0];
      for (int w = 1; w < kWaves; ++w) taken = max(taken, sums[0][w]);
      *a.used_out = (int32_t)((uint32_t)used + taken);
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
  const auto later = [](uint32_t x, uint32_t y) { return (uint32_t)max((int32_t)x, (int32_t)y); };
  const uint32_t up = wave_scan((uint32_t)top, 0xFFFFFFFFu, later);
  if ((tid & 63) == 63) tops[tid >> 6] = (int32_t)up;
  int32_t before = (int32_t)lane_before(up, 0xFFFFFFFFu);
  __syncthreads();
  for (int w = 0; w < tid >> 6; ++w) before = max(before, tops[w]);
#pragma unroll
  for (int e = 0; e < kItems; ++e) {
    const uint32_t row = row0 + tid * kItems + e;
    if (row >= row1) break;
    const int32_t i = r[e] > before ? r[e] : before;
    int32_t slot = -1, pos = -1, seq = -1;
    if (i >= 0 && row < rows && rec[i].seq >= 0) {
      const Record c = rec[i];
      seq = c.seq;
      pos = (int32_t)(row + (uint32_t)c.shift);
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
