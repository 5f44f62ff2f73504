// The layout of attention's tiles in LDS (csrc/attn_internal.h), on the host: every chunk has a place
// of its own within the tile, the copies' places add up, and the reads of 16 rows and the transposing
// reads fall on all 64 banks.
#include <cstdio>
#include <set>

#include "../mixed_precision_int8_amd/csrc/attn_internal.h"

using namespace llmint8;

static int bad = 0;
#define CHECK(x)                                          \
  do {                                                    \
    if (!(x)) std::printf("%s:%d: %s (DP %d)\n", __FILE__, __LINE__, #x, DP), ++bad; \
  } while (0)

template <int DP>
static int place(int row, int chunk) {
  using T = AttnTile<DP>;
  return T::at(row) + (chunk ^ T::swizzle(row)) * 16;
}

template <int DP>
static void check() {
  using T = AttnTile<DP>;
  std::set<int> all;
  for (int r = 0; r < 64; ++r)
    for (int c = 0; c < T::kChunks; ++c) {
      const int p = place<DP>(r, c);
      CHECK(p >= 0 && p % 16 == 0 && p + 16 <= T::kBytes);
      CHECK((c ^ T::swizzle(r)) < T::kChunks);
      all.insert(p);
    }
  CHECK((int)all.size() == 64 * T::kChunks);
  // a wavefront's copies: 1 KB of whole rows each, one after the other in LDS
  for (int W : {4, 8}) {
    const int rows = 1024 / T::kPitch, issues = 64 / rows / W;
    for (int w = 0; w < W; ++w)
      for (int i = 0; i < issues; ++i) {
        const int first = (i * W + w) * rows;
        CHECK(T::at(first) == T::at(w * rows) + T::at(i * W * rows));
        for (int r = 0; r < rows; ++r) {
          CHECK(T::at(first + r) == T::at(first) + r * T::kPitch);
          CHECK(T::swizzle(first + r) == T::swizzle(w * rows + r));
        }
      }
  }
  // 16 rows at one chunk (256 bytes of 64 banks)
  for (int r0 = 0; r0 < 64; r0 += 16)
    for (int c = 0; c < DP / 8; ++c) {
      std::set<int> banks;
      for (int r = 0; r < 16; ++r) banks.insert(place<DP>(r0 + r, c) % 256);
      CHECK((int)banks.size() == 16);
    }
  // four rows of four chunks
  for (int r0 = 0; r0 < 64; r0 += 4)
    for (int c0 = 0; c0 < DP / 8; c0 += 4) {
      std::set<int> banks;
      for (int r = 0; r < 4; ++r)
        for (int c = 0; c < 4; ++c) banks.insert(place<DP>(r0 + r, c0 + c) % 256);
      CHECK((int)banks.size() == 16);
    }
}

int main() {
  check<64>();
  check<96>();
  check<128>();
  check<256>();
  if (!bad) std::printf("tiles ok\n");
  return bad != 0;
}
