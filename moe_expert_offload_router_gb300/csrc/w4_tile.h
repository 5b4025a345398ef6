// Sizes of w4_tile_kernel's blocks (4-bit products of many rows), without device code: a host program can check them.
#pragma once

#include <stddef.h>

namespace moe {

constexpr int kMaxExperts = 2048;
constexpr int kTileStages = 8, kCodeBytes = 128 * 64;
constexpr int kAStages = 4, kACols = 256;   // A: four steps in the last 256 columns of tensor memory

template <int NT>
struct TileCfg {
  static constexpr int kStage = kCodeBytes + NT / 2 * 256;
  static constexpr int kBufs = kACols / NT;   // accumulators
  static constexpr int kRing = kTileStages * kStage;
  // warps: TMA, MMA, two that only fill a group of four, 8 of codes, and 4 of sums for every kCols columns: 32, since 64
  // a thread do not stay in its registers
  static constexpr int kCols = NT == 128 ? 32 : NT / 2, kParts = NT / kCols;
  static constexpr int kThreads = (12 + 4 * kParts) * 32;
  static constexpr int kExchange = kParts * 16 * 64 * 4;
};
// A block takes all of an SM's tensor memory, together with its pair's, and may do so before the launch ahead has
// ended: two of them on an SM (of this launch and the next one, or of two streams) could each hold half of what
// the other waits for.  So each takes more than half of an SM's 228 KB, of which 1 KB a block is the system's, whatever
// its ring needs (105 KB at a width of 32); the projection's kernels, which allocate tensor memory for
// clusters too, take more than that.
constexpr size_t kAloneBytes = 116 * 1024;
static_assert(2 * (kAloneBytes + 1024) > 228 * 1024, "two blocks must not fit an SM");
template <int NT>
inline size_t tile_smem(int E) {
  const size_t n = (size_t)TileCfg<NT>::kRing + TileCfg<NT>::kExchange + 1024 + (size_t)(E + 1) * 8;
  return n > kAloneBytes ? n : kAloneBytes;
}

}  // namespace moe
