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
  // a wavefront's copies: 64 chunks each, one after the other in LDS, by an address that adds up
  for (int W : {4, 8}) {
    if (T::kMiddle && W == 8) continue;  // three halves of a copy to a wavefront
    const int copies = 64 * T::kChunks / 64;
    CHECK(copies % W == 0);
    for (int n = 0; n < copies; ++n) {
      const int w = n % W;
      CHECK(T::copy_at(n) == T::copy_at(w) + T::copy_at(n - w));
      for (int lane = 0; lane < 64; ++lane) {
        const int at = n * 64 + lane, row = at / T::kChunks, slot = at % T::kChunks;
        CHECK(T::copy_at(n) + lane * 16 == T::at(row) + slot * 16);
        CHECK(T::kMiddle || T::swizzle(row) == T::swizzle(row % (W * 1024 / T::kPitch)));  // one offset for all
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
