// Host sweep of the index arithmetic that the key/value cache's kernels share with
// it (mixed_precision_int8_amd/csrc/kv_internal.h). Built and run by
// tests/test_kvcache_index.py; the argument names the check.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>

#include "../mixed_precision_int8_amd/csrc/kv_internal.h"

using namespace llmint8;

static int failures = 0;
#define EXPECT(c, ...)                          \
  do {                                          \
    if (!(c) && ++failures < 10) {              \
      std::fprintf(stderr, "failed: %s: ", #c); \
      std::fprintf(stderr, __VA_ARGS__);        \
      std::fprintf(stderr, "\n");               \
    }                                           \
  } while (0)

static std::mt19937 rng(7);
static int draw(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); }

// Random batches of rising cu, some with rows past the last sequence's: every row
// with a position is worked on by one item of the launch, no other row by any, both
// as pages of tokens (append, gather) and as tiles of rows (attention).
static void items() {
  for (int round = 0; round < 4000; ++round) {
    const int page_shift = draw(4, 7), B = draw(1, 9), per = draw(1, 9), shift = draw(4, 8);
    std::vector<int> cu{0}, len;
    for (int b = 0; b < B; ++b) {
      const int kind = draw(0, 3), n = kind == 0 ? 0 : kind == 1 ? 1 : draw(1, kind == 2 ? 20 : 300);
      cu.push_back(cu.back() + n);
      len.push_back(draw(0, 9) == 0 ? draw(0, n) : n + draw(0, 300));  // now and then rows without a position
    }
    const int T = cu[B] + (draw(0, 1) ? 0 : draw(1, 300));
    for (int tiles = 0; tiles < 2; ++tiles) {
      const int p = tiles ? per : 1, s = tiles ? shift : page_shift;
      std::vector<int> seen((size_t)T * p, 0);
      const int launched = (int)(((int64_t)T * p) >> s) + B;
      for (int item = 0; item < launched; ++item) {
        int b = -1;  // the last sequence whose items begin no later, as kv_find counts it
        while (b + 1 < B && kv_items(b + 1, cu[b + 1], cu[b + 2] - cu[b + 1], p, s).first <= item) ++b;
        if (b < 0) continue;
        const int n = cu[b + 1] - cu[b], pos0 = len[b] - n;
        const KvItems own = kv_items(b, cu[b], n, p, s);
        const int index = kv_item_index(own, item);
        if (index < 0) continue;
        if (tiles) {
          for (int r = index << s; r < std::min((index + 1) << s, n * p); ++r) ++seen[(size_t)cu[b] * p + r];
          continue;
        }
        const KvEntries e = kv_item_entries(pos0, index, own.count, s);
        for (int i = e.first; i < e.first + e.count; ++i)
          for (int at = std::max(pos0, i << s); at < std::min(len[b], (i + 1) << s); ++at) ++seen[cu[b] + at - pos0];
      }
      for (int b = 0; b <= B; ++b)
        for (int r = cu[b]; r < (b < B ? cu[b + 1] : T); ++r)
          for (int k = 0; k < p; ++k) {
            const bool live = b < B && (tiles || len[b] - (cu[b + 1] - cu[b]) + r - cu[b] >= 0);
            EXPECT(seen[(size_t)r * p + k] == (live ? 1 : 0), "%d times: row %d of %d (%d in the batch), page or tile 2^%d, per %d",
                   seen[(size_t)r * p + k], r, T, cu[B], s, p);
          }
    }
  }
}

// Lengths past the table, up to the largest: a row keeps its position, tokens that
// the table has no entry for are on entries past it, and nothing is out of range.
static void positions() {
  for (int round = 0; round < 200000; ++round) {
    const int page_shift = draw(4, 7), width = draw(1, 40), T = draw(1, 500), P = 1 << page_shift;
    const int64_t room = (int64_t)width << page_shift;
    const int hostile[] = {-5, 0, T, T + 9, INT32_MAX, INT32_MIN};
    const int kind = draw(0, 9);
    const int cu0 = kind == 0 ? hostile[draw(0, 5)] : draw(0, T), cu1 = kind < 2 ? hostile[draw(0, 5)] : draw(cu0 < 0 || cu0 > T ? 0 : cu0, T);
    const int length = draw(0, 3) ? draw(0, (int)room + 300) : draw(0, 1) ? draw(INT32_MAX - 300, INT32_MAX) : draw(-9, 9);
    const KvSeq q = kv_seq_of(3, cu0, cu1, length, T, room);
    EXPECT(q.row0 >= 0 && q.n >= 0 && q.row0 + q.n <= T, "cu %d %d of %d", cu0, cu1, T);
    EXPECT(q.len == std::max<int64_t>(0, std::min<int64_t>(length, room)), "len %d, room %ld", length, (long)room);
    const KvItems own = kv_items(3, q.row0, q.n, 1, page_shift);
    std::vector<int> seen(q.n, 0);
    for (int item = own.first; item < own.first + own.count; ++item) {
      const KvEntries e = kv_item_entries(q.pos0, kv_item_index(own, item), own.count, page_shift);
      for (int entry = e.first; entry < e.first + e.count; ++entry) {
        const KvOnPage on = kv_on_page(q, entry, page_shift);
        if (on.t0 >= on.t1) continue;
        EXPECT(on.t0 >= on.base && on.t1 - 1 - on.base < P && on.base == entry * (int64_t)P, "entry %d", entry);
        for (int64_t at = on.t0; at < on.t1; ++at) {
          const int64_t row = at - q.pos0;
          EXPECT(row >= 0 && row < q.n, "position %ld of %d", (long)at, length);
          if (row < 0 || row >= q.n) continue;
          ++seen[row];
          // row i is token len - n + i, on entry (len - n + i) / P
          EXPECT(at == std::max(length, 0) - (int64_t)q.n + row && at / P == entry, "position %ld of %d", (long)at, length);
        }
      }
    }
    for (int i = 0; i < q.n; ++i) {
      const bool live = std::max(length, 0) - (int64_t)q.n + i >= 0;
      EXPECT(seen[i] == (live ? 1 : 0), "row %d of %d, length %d", i, q.n, length);
    }
  }
}

// Any two numbers that a row's note may hold: what is read of the workspace for it
// is within the parts' rows.
static void notes() {
  const int runs[] = {16, 32, 128, 256}, sizes[] = {1, 2, 3, 64, 1536, 1 << 22};
  for (int run : runs)
    for (int max_parts : sizes)
      for (int round = 0; round < 200000; ++round) {
        const int kind = draw(0, 2);
        const int where = kind == 0 ? (int)rng() : kind == 1 ? draw(-3, 600) : (max_parts + draw(-2, 2)) << kKvNoteShift | draw(0, 255);
        const int parts = draw(0, 1) ? (int)rng() : draw(-2, max_parts + 2);
        const KvNote n = kv_note(where, parts, run, max_parts);
        EXPECT(n.parts >= 0 && n.slot >= 0 && n.place >= 0, "note %d %d", where, parts);
        const int64_t last = ((int64_t)n.slot + n.parts - 1) * run + n.place;
        EXPECT(n.parts == 0 || last < (int64_t)max_parts * run, "note %d %d of %d parts of %d rows", where, parts, max_parts, run);
        const int64_t first = where >> kKvNoteShift, row = where & 255;
        if (where >= 0 && row < run && parts >= 1 && first + parts <= max_parts)
          EXPECT(n.slot == first && n.place == row && n.parts == parts, "note %d %d", where, parts);
      }
}

int main(int, char** argv) {
  const char* what = argv[1];
  if (!std::strcmp(what, "items")) items();
  else if (!std::strcmp(what, "notes")) notes();
  else if (!std::strcmp(what, "positions")) positions();
  else return 2;
  if (!failures) std::printf("%s ok\n", what);
  return failures ? 1 : 0;
}
