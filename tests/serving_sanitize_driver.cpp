// Host-side driver for the sanitizer build of the serving calls: size queries over
// sizes at and past the limits, and calls that each return before any launch (a
// null pointer is refused at the latest).  No GPU is needed or used.
#include <cstdint>
#include <cstdio>
#include <limits>

#include "gptq.h"

static int g_fail = 0;

#define REFUSED(call)                                                     \
  do {                                                                    \
    const gptq_status st = (call);                                        \
    if (st != GPTQ_ERR_INVALID_ARG && st != GPTQ_ERR_WORKSPACE) {         \
      std::fprintf(stderr, "FAILED line %d: %d\n", __LINE__, (int)st);    \
      ++g_fail;                                                           \
    }                                                                     \
  } while (0)

int main() {
  void* f = reinterpret_cast<void*>(uintptr_t{1} << 20);  // never dereferenced
  float* ff = static_cast<float*>(f);
  int32_t* fi = static_cast<int32_t*>(f);
  int64_t* fs = static_cast<int64_t*>(f);
  int8_t* fc = static_cast<int8_t*>(f);
  const int64_t big = std::numeric_limits<int64_t>::max(), least = std::numeric_limits<int64_t>::min();
  const int32_t big32 = std::numeric_limits<int32_t>::max();
  const int64_t sizes[] = {least, -1, 1, 16, 4096, 1 << 20, int64_t{1} << 30, (int64_t{1} << 30) + 1, int64_t{1} << 60, big};
  const int32_t counts[] = {std::numeric_limits<int32_t>::min(), -1, 0, 1, 16, 255, 256, 65536, 1 << 20, big32};
  size_t all = 0;
  for (int64_t pages : {least, int64_t{0}, int64_t{4096}, int64_t{1} << 31, big})
    for (int32_t page : counts)
      for (int32_t kv : counts)
        for (int32_t hd : {-16, 16, 80, 256, 272})
          for (int32_t bits : {2, 4, 8}) {
            const gptq_cache c{pages, page, kv, hd, bits, f, f, ff, ff};
            for (int64_t t : sizes) {
              for (int32_t heads : {1, kv, big32})
                for (int32_t seq : {-1, 0, 1, 1 << 20, big32})
                  for (int64_t table : {int64_t{1}, int64_t{1} << 22, int64_t{1} << 60, big})
                    all += gptq_attention_workspace_size(&c, t, heads, seq, table);
              REFUSED(gptq_cache_write(&c, nullptr, f, GPTQ_BF16, t, big - 7, big - 7, fs, nullptr));
              REFUSED(gptq_cache_read(&c, nullptr, t, f, f, GPTQ_BF16, nullptr));
              REFUSED(gptq_cache_attention(&c, nullptr, GPTQ_BF16, t, int64_t{1} << 40, kv, fi, 4, fi, fi, 1, 0.1f, f,
                                           int64_t{1} << 40, f, 1, nullptr));
            }
          }
  for (int64_t m : sizes)
    for (int64_t a : sizes)
      for (int64_t b : sizes)
        for (int t : {0, 1, 2, 3}) {
          all += gptq_integer_workspace_size(m, t, a, b);
          REFUSED(gptq_integer_matmul(nullptr, t, nullptr, nullptr, m, a, big, fc, ff, nullptr, b, f, GPTQ_F32, f, 1, nullptr));
          REFUSED(gptq_quantize_tokens(nullptr, t, m, a, b, nullptr, nullptr, nullptr, nullptr));
          REFUSED(gptq_integer_weight(nullptr, nullptr, 8, a, b, nullptr, nullptr, nullptr));
        }
  std::printf("%s (%zu)\n", g_fail ? "failures" : "all checks passed", all);
  return g_fail != 0;
}
