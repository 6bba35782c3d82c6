// Host check of a streamed row's chunks (ls_chunks.h): each fits its place in shared memory, and
// together they are the row, up to the largest rows that the token statistics take.
#include <cstdio>

#include "ls_chunks.h"

constexpr int kGroup = 64, kPer = 384;

int main() {
  // groups: of 1 to a few chunks, and of 2^30 values of 2 and 4 bytes, an odd one more or less
  const int32_t most[] = {1 << 25, 1 << 26};
  for (int c = 0; c < 2000 + 6; ++c) {
    const int32_t n = c < 2000 ? c + 1 : most[(c - 2000) / 3] + (c - 2000) % 3 - 1;
    const int32_t chunks = (n + kPer - 1) / kPer;
    int64_t sum = 0;
    for (int32_t k = 0; k < chunks; ++k) {
      const uint32_t b = ls_chunk_bytes<kGroup, kPer>(n, k);
      if (b == 0 || b > kGroup * kPer || b % 16 != 0) {
        std::printf("FAIL chunk %d of %d groups: %u bytes\n", k, n, b);
        return 1;
      }
      sum += b;
    }
    if (sum != (int64_t)n * kGroup) {
      std::printf("FAIL %d groups: %lld bytes\n", n, (long long)sum);
      return 1;
    }
  }
  std::printf("chunks ok\n");
  return 0;
}
