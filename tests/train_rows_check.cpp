// How rows are dealt to launches (csrc/train_internal.h), on the host: every row is in one launch, no launch
// has too many work items, and a launch's arguments are those of its first row.
#include <cstdio>

#include "../mixed_precision_int8_amd/csrc/train_internal.h"

using namespace llmint8;

static int bad = 0;
#define CHECK(x)                                                        \
  do {                                                                  \
    if (!(x)) std::printf("%s:%d: %s\n", __FILE__, __LINE__, #x), ++bad; \
  } while (0)

static void check(int64_t rows, int64_t items, int threads, int64_t max_items) {
  int64_t next = 0;
  int launches = 0;
  const hipError_t e = launch_rows(
      rows, items, threads,
      [&](int64_t at, int64_t n) {
        CHECK(at == next && n > 0);
        CHECK((n * items + threads - 1) / threads * threads < max_items);
        next = at + n;
        ++launches;
        return hipSuccess;
      },
      max_items);
  CHECK(e == hipSuccess && next == rows);
  CHECK(launches <= 2 * ((rows * items + max_items - 1) / max_items) + 1);
}

int main() {
  for (int threads : {256, 1024})
    for (int64_t items : {1, 3, 64, 1000, 1024})
      for (int64_t rows : {0, 1, 2, 7, 100, 4095, 4096, 5000}) check(rows, items, threads, 8192);
  check((int64_t(1) << 31) - 1, 64, 256, kMaxWorkItems);
  check((int64_t(1) << 31) - 1, 1024, 1024, kMaxWorkItems);
  check(int64_t(1) << 29, int64_t(1) << 30, 256, kMaxWorkItems);
  int calls = 0;
  CHECK(launch_rows(100, 64, 256, [&](int64_t, int64_t) { return ++calls, hipErrorUnknown; }, 1024) == hipErrorUnknown && calls == 1);

  static char x[100], y[100], dy[100];
  static float stats[100];
  NormArgs a{};
  a.x = x, a.y = y, a.stats = stats, a.rows = 9, a.x_row = 5, a.y_row = 7, a.dy_row = 3;
  NormArgs b = norm_rows_of(a, 4, 5, 2);
  CHECK(b.x == x + 40 && b.y == y + 56 && b.stats == stats + 8 && b.rows == 5 && !b.dy);
  a.dy = dy, a.stats = nullptr;
  b = norm_rows_of(a, 2, 3, 4);
  CHECK(b.x == x + 40 && b.y == y + 56 && b.dy == dy + 24 && !b.stats && b.rows == 3);

  static uint16_t p[1000];
  static int32_t pos[100];
  RopeArgs r{};
  r.x[0] = {p, 10, 2}, r.y[0] = {p + 500, 20, 2}, r.heads[0] = 2, r.pos = pos, r.axes = 3, r.rows = 9;
  RopeArgs s = rope_rows_of(r, 4, 5);
  CHECK(s.x[0].p == p + 40 && s.y[0].p == p + 580 && s.pos == pos + 12 && s.rows == 5 && !s.x[1].p);
  r.x[1] = {p, 30, 2}, r.y[1] = {p, 30, 2}, r.heads[1] = 1;
  s = rope_rows_of(r, 1, 1);
  CHECK(s.x[1].p == p + 30 && s.y[1].p == p + 30 && s.rows == 1);
  std::printf(bad ? "%d bad\n" : "rows ok\n", bad);
  return bad != 0;
}
