// Host-only exercise of the argument checks and plans of the slots, adapters
// and sampling calls, built with AddressSanitizer and
// UndefinedBehaviorSanitizer around serve_api.cpp and serve_plan.cpp.  Every
// call is a size query, does nothing, or has a defect that the host must
// refuse before any HIP call, so no GPU is needed.  Exit status 0: every
// answer was as expected; the sanitizers abort the run on the first error.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../dequant_gemv_rht_amd/csrc/wq_internal.h"

namespace {

int failures = 0;
long checked = 0;

void expect(bool ok, const char *what, long long a, long long b) {
  ++checked;
  if (!ok) {
    std::fprintf(stderr, "FAIL %s (%lld, %lld): %s\n", what, a, b, wq_last_error());
    ++failures;
  }
}

template <typename T>
T *at(uintptr_t a) {
  return reinterpret_cast<T *>(a);   // never dereferenced
}

}  // namespace

int main() {
  const int64_t counts[] = {0, 1, 63, 1000, (int64_t)1 << 20, (int64_t)1 << 31, INT64_MAX, -1, INT64_MIN};
  const int32_t sizes[] = {16, 64, 1 << 30, 0, 24, INT_MIN, INT_MAX};
  const uintptr_t places[] = {0, 1 << 20, (1 << 20) + 2, UINTPTR_MAX - 3, (uintptr_t)1 << 63};

  // slots: used_out on used, so that nothing gets past the checks
  for (int32_t page : sizes)
    for (int64_t pages : counts)
      for (int64_t seqs : counts)
        for (int64_t tokens : counts)
          for (int64_t n : counts)
            for (uintptr_t p : places) {
              const int32_t *in = at<int32_t>(p);
              int32_t *out = at<int32_t>(p);
              expect(wq_kv_slots(page, pages, out, n, tokens, in, in, seqs, in, n, in, tokens, out, out, out, out, out, out,
                                 nullptr) < 0, "slots", seqs, tokens);
            }

  // adapters
  for (int32_t count : {1, 8, 0, 9, INT_MIN, INT_MAX})
    for (int32_t rank : {8, 128, 16, 0, 12, INT_MIN, INT_MAX})
      for (int64_t n : counts)
        for (int64_t m : counts)
          for (int64_t ld : counts)
            for (uintptr_t p : {places[1], places[2], places[3]}) {
              wq_adapters w[8];
              const uint16_t *x[8];
              const void *base[8];
              void *y[8];
              int64_t l[8];
              wq_dtype t[8];
              for (int i = 0; i < 8; ++i) {
                w[i] = {n, n < 0 || n > ((int64_t)1 << 55) ? n : n * 128, rank, rank, at<uint16_t>(p), at<uint16_t>(p), at<float>(p)};
                x[i] = at<uint16_t>(p);
                base[i] = at<void>(p);
                y[i] = at<void>(p);
                l[i] = ld;
                t[i] = WQ_F32;
              }
              const size_t need = wq_lora_workspace(count, w, m);
              (void)need;
              // x and y at one place: refused at the latest there, or nothing to do
              const wq_status st = wq_lora(count, w, x, l, m, at<int32_t>(p), base, l, y, l, t, at<void>(p), SIZE_MAX, nullptr);
              expect(m == 0 ? st <= 0 : st < 0, "lora", n, m);
            }

  // sampling: ids on u
  for (int64_t rows : counts)
    for (int64_t vocab : counts)
      for (int64_t ld : counts)
        for (uintptr_t p : places) {
          (void)wq_sample_workspace(rows, vocab);
          const wq_status st = wq_sample(at<void>(p), WQ_F16, rows, vocab, ld, at<float>(p), at<float>(p), at<int32_t>(p),
                                         at<float>(p), nullptr, at<int32_t>(p), at<float>(p), at<void>(p), SIZE_MAX, nullptr);
          expect(rows == 0 ? st <= 0 : st < 0, "sample", rows, vocab);
        }
  size_t last = 0;
  for (int64_t rows = 0; rows < 3000; rows += 1 + rows / 3) {
    const size_t s = wq_sample_workspace(rows, 151936);
    expect(s != (size_t)-1 && s >= last, "sample workspace", rows, 0);
    last = s;
  }

  // plans: whole of K and of the outputs is dealt out, the launch and the workspace hold it
  for (int64_t k = 128; k < 20000; k += 128 * (1 + k / 700))
    for (int64_t n = 1; n < 30000; n += 1 + n / 2)
      for (int32_t count = 1; count <= 8; count += 3) {
        wq_adapters w[8];
        for (int i = 0; i < count; ++i) w[i] = {n + 100 * i, k, 4, 8 * (i + 1), nullptr, nullptr, nullptr};
        size_t before = 0;
        for (int64_t m = 1; m < 1 << 20; m += 1 + m / 4) {
          const wq::LoraPlan p = wq::lora_plan(count, w, m);
          const size_t ws = wq::lora_workspace(w[0], m);
          expect(p.steps > 0 && p.steps % 4 == 0 && p.chunk > 0 && p.chunk % 256 == 0, "whole 128s", k, m);
          uint32_t splits = 0, chunks = 0;
          for (int i = 0; i < count; ++i) {
            const int64_t of_k = p.splits_to[i] - splits, of_n = p.chunks_to[i] - chunks;
            expect(of_k * p.steps * 32 >= k && (of_k - 1) * p.steps * 32 < k, "K", k, m);
            expect(of_n * p.chunk >= w[i].n && (of_n - 1) * p.chunk < w[i].n, "outputs", n, m);
            expect((size_t)of_k * m * w[i].rank * sizeof(float) <= wq::lora_workspace(w[i], m), "workspace", of_k, m);
            splits = p.splits_to[i];
            chunks = p.chunks_to[i];
          }
          expect(splits == p.splits && chunks == p.chunks && ws >= before, "sums", p.splits, m);
          expect(p.rank == 8 * count, "rank", p.rank, count);
          expect(p.inner_tiles * p.splits * p.slots * 2 <= wq::kMaxGroups256 && p.splits <= 65535 && p.chunks <= 65535 &&
                     p.outer_tiles * p.chunks * p.slots <= wq::kMaxGroups256 && p.slots >= 1 && (p.slots == 1 || !p.whole),
                 "launch", p.inner_tiles, p.chunks);
          expect(!p.near || (!p.whole && p.inner_tiles <= 8 * 65535 && p.splits * p.slots * 2 <= 65535 &&
                             p.chunks * p.slots <= 65535),
                 "launch by XCD", p.inner_tiles, p.chunks);
          before = ws;
        }
      }
  std::printf("checked %ld answers\n", checked);
  return failures ? 1 : 0;
}
