// Four<B> gives a row's elements four at a time, wherever the array starts and ends, and loads nothing outside the
// array: by words the rows that cut() lets pass, by elements any.
#include <stdio.h>
#include <string.h>

#include "four_of_row.h"

static long outside, loads, whole;
static const char *g_first, *g_end;

struct Load {
  template <typename T>
  T operator()(const T* p) const {
    const char* c = reinterpret_cast<const char*>(p);
    ++loads;
    if (c < g_first || c + sizeof(T) > g_end || (uintptr_t)p % sizeof(T)) ++outside;
    T v;
    memcpy(&v, c, sizeof(T));   // room on both sides
    return v;
  }
};

// rows of n elements of B bytes, the array `shift` bytes past a 16-byte boundary; the kernel's order of calls
template <int B>
static int check(int rows, int n, int shift) {
  alignas(16) static char room[4096];
  memset(room, 0xee, sizeof room);
  char* a = room + 64 + shift;
  for (int i = 0; i < rows * n; ++i) {
    const uint16_t v = (uint16_t)(i * 2654435761u >> 16 | 1);
    memcpy(a + i * B, &v, B);
  }
  g_first = a, g_end = a + rows * n * B;
  int bad = 0;
  for (int r = 0; r < rows; ++r)
    for (int from = 0; from < n; from += 4)   // a part of the row, as blocks that share it take
      for (int step = 1; step <= 2; ++step) {
        const char* row = a + (r * n + from) * B;
        auto walk = [&](auto f) {
          f.fetch(0, Load());
          for (int b = 0; b * 4 < n - from; b += step) {
            const auto v = f.value(b, Load());
            f.fetch(b + step, Load());
            for (int j = 0; j < 4 && b * 4 + j < n - from; ++j)
              bad += memcmp(reinterpret_cast<const char*>(&v) + j * B, row + (b * 4 + j) * B, B) != 0;
          }
        };
        const moe::Four<B> f(row, n - from);
        if (!f.cut(g_first, g_end)) ++whole, walk(f);
        else if (!moe::ends_cut(g_first, rows * n, B)) ++bad;
        walk(moe::Four<B, true>(row, n - from));
      }
  return bad;
}
template <int B>
static int check_all() {
  int bad = 0;
  for (int rows = 1; rows <= 5; ++rows)
    for (int n = 1; n <= 21; ++n)
      for (int shift = 0; shift < 16; shift += B) bad += check<B>(rows, n, shift);
  return bad;
}
int main() {
  const int bad = check_all<1>() + check_all<2>();
  moe::Four<1> none(nullptr, 0);
  const long before = loads;
  none.fetch(0, Load());
  none.fetch(3, Load());
  if (none.cut(nullptr, nullptr)) ++outside;
  printf("%d wrong elements, %ld loads outside the array, %ld loads of none\n", bad, outside, loads - before);
  return bad || outside || loads != before || loads < 1000 || whole < 1000;
}
