// Two blocks of w4_tile_kernel never share an SM, whatever its registers: each takes more than half of its shared memory.
#include <stdio.h>

#include "w4_tile.h"

constexpr size_t kSm = 228 * 1024, kReserved = 1024, kMost = 232448;   // of an SM, of it for the system in each block, of a block

template <int NT>
static int check() {
  int bad = 0;
  for (int E = 1; E <= moe::kMaxExperts; ++E) {
    const size_t n = moe::tile_smem<NT>(E);
    if (2 * (n + kReserved) <= kSm || n + 1024 > kMost) {   // the block's static arrays take less than 1 KB more
      if (!bad) printf("width %d, %d experts: %zu bytes\n", NT, E, n);
      ++bad;
    }
    if (n > moe::tile_smem<NT>(moe::kMaxExperts)) printf("more than with all experts\n"), ++bad;
  }
  return bad;
}
int main() { return check<32>() + check<64>() + check<128>() ? 1 : 0; }
