// Host-only exercise of the argument checks and workspace planning of the
// key-value cache, attention and rotary calls, built with AddressSanitizer
// and UndefinedBehaviorSanitizer around kv_api.cpp.  Every call is a size
// query, does nothing, or has a defect that the host must refuse before any
// HIP call, so no GPU is needed.  Exit status 0: every answer was as
// expected; the sanitizers abort the run on the first error they find.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "wq.h"

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

void *const P16 = reinterpret_cast<void *>(uintptr_t(1) << 20);   // never dereferenced
void *const P2 = reinterpret_cast<void *>((uintptr_t(1) << 20) + 2);

wq_kv_cache cache(int bits, int d, int heads, int page, int64_t pages, bool rotated) {
  wq_kv_cache c;
  std::memset(&c, 0, sizeof c);
  c.bits = bits;
  c.head_dim = d;
  c.kv_heads = heads;
  c.page_size = page;
  c.pages = pages;
  c.k = c.v = P16;
  c.k_params = c.v_params = static_cast<uint16_t *>(P16);
  if (rotated) {
    c.rht_signs = static_cast<uint32_t *>(P16);
    c.rht_block = 128;
  }
  return c;
}

}  // namespace

int main() {
  const int bits_list[] = {4, 8, 16, 3, 0, INT_MIN, INT_MAX};
  const int dims[] = {64, 128, 256, 0, 96, INT_MIN, INT_MAX};
  const int heads_list[] = {1, 8, 1000, 1 << 24, INT_MAX, 0, INT_MIN};
  const int pages_of[] = {16, 1024, 1 << 30, 0, 24, INT_MIN, INT_MAX};
  const int64_t counts[] = {1, 1000, (int64_t)1 << 31, INT64_MAX, 0, -1, INT64_MIN};
  const uint16_t *x = static_cast<const uint16_t *>(P16);
  uint16_t *y = static_cast<uint16_t *>(P16);
  const int32_t *odd = static_cast<const int32_t *>(P2);   // misaligned: refused at the last check

  for (int bits : bits_list)
    for (int d : dims)
      for (int heads : heads_list)
        for (int page : pages_of)
          for (int64_t n : counts)
            for (int rot = 0; rot < 2; ++rot) {
              const wq_kv_cache c = cache(bits, d, heads, page, n, rot != 0);
              for (int64_t m : counts) {
                const int64_t ld = INT64_MAX / 8 * 8;
                if (m == 0) continue;
                expect(wq_kv_write(&c, x, ld, x, ld, odd, m, nullptr) < 0, "write", heads, m);
                expect(wq_kv_read(&c, odd, m, y, ld, y, ld, nullptr) < 0, "read", heads, m);
                (void)wq_attn_decode_workspace(&c, m, heads, n, m);
                (void)wq_attn_decode_workspace(&c, n, INT_MAX, m, 0);
                expect(wq_attn_decode(&c, x, ld, heads, m, odd, ld, odd, n, 0, 1.0f, y, ld, P16, SIZE_MAX, nullptr) < 0,
                       "attend", heads, m);
              }
              expect(wq_attn_decode(nullptr, x, 8, 1, 1, odd, 8, odd, 1, 0, 1.0f, y, 8, P16, 0, nullptr) == WQ_E_ARG,
                     "null cache", 0, 0);
            }

  // the workspace never shrinks as the batch or the bound of the lengths grows
  const wq_kv_cache good = cache(8, 128, 8, 64, 1 << 20, true);
  for (int window = 0; window < 3000; window += 999)
    for (int group = 1; group < 40; group += 6)
      for (int64_t seqs = 1; seqs < 300; seqs += 1 + seqs / 3) {
        size_t last = 0;
        for (int64_t len = 0; len < 200000; len += 1 + len / 5) {
          const size_t w = wq_attn_decode_workspace(&good, seqs, 8 * group, len, window);
          expect(w != (size_t)-1 && w >= last, "workspace in max_len", seqs, len);
          expect(wq_attn_decode_workspace(&good, seqs + 1, 8 * group, len, window) >= w, "workspace in seqs", seqs, len);
          last = w;
        }
      }

  const int64_t lds[] = {0, 8, 128, 1 << 20, INT64_MAX / 8 * 8, -8, INT64_MIN};
  const uint8_t axis[128] = {0};
  for (int count : {0, 1, 8, 9, INT_MIN, INT_MAX})
    for (int heads : heads_list)
      for (int64_t ld : lds)
        for (int64_t tokens : counts)
          for (int d : dims)
            for (int rot : {16, 64, 256, 0, 8, INT_MIN, INT_MAX})
              for (int axes : {1, 4, 5, 0, INT_MIN}) {
                const uint16_t *xs[8];
                uint16_t *ys[8];
                int64_t l[8];
                int32_t h[8];
                for (int i = 0; i < 8; ++i) {
                  xs[i] = x;
                  ys[i] = y;
                  l[i] = ld;
                  h[i] = heads;
                }
                const wq_status st =
                    wq_rope(count, xs, l, ys, l, h, tokens, d, rot, static_cast<const float *>(P16),
                            static_cast<const float *>(P16), 10, odd, INT64_MAX / 16, axes, axis, 0, nullptr);
                expect(tokens == 0 ? st <= 0 : st < 0, "rope", heads, tokens);
              }
  std::printf("checked %ld answers\n", checked);
  return failures ? 1 : 0;
}
