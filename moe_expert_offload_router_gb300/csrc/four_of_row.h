// Four neighbouring elements at a time of a row's scales or zero points.  Compiled for the host too, where a test
// watches its loads.
#pragma once

#include <stdint.h>

#include <type_traits>

#if defined(__CUDACC__)
#define MOE_DEVICE __device__ __forceinline__
#else
#define MOE_DEVICE inline
#endif

namespace moe {

// Four neighbouring elements of B bytes of a row's array, fetched a batch ahead: a lane's row is
// its own cache line, and a load of every element by itself takes the L1's time 32 times.
// Rows start anywhere: the two aligned words that hold the four are loaded (one where they
// are aligned themselves) and shifted.
//
// The outermost words can pass the array's ends (cut(): in its first and last rows, where it is not aligned
// itself).  Such a row is taken one element at a time where they are used, CUT, by a copy of the caller's
// loop: a test at each load or use cost the loop without it 3 to 20 % (4001 x 4096 x 4096 in groups of 64:
// 239 us at the loads, 267 at the uses, 221 without).
template <int B, bool CUT = false>
struct Four {
  using W = typename std::conditional<B == 2, uint64_t, uint32_t>::type;
  using T = typename std::conditional<B == 2, uint16_t, uint8_t>::type;
  static constexpr uintptr_t kLow = 4 * B - 1;
  const char *row, *end;
  W lo = 0, hi = 0;
  MOE_DEVICE Four(const void* p, int n) : row((const char*)p), end((const char*)p + (long long)n * B) {}
  // whether words around the row pass the ends of its array
  MOE_DEVICE bool cut(const void* array, const void* array_end) const {
    return ((uintptr_t)row & ~kLow) < (uintptr_t)array || (((uintptr_t)end + kLow) & ~kLow) > (uintptr_t)array_end;
  }
  template <typename L>
  MOE_DEVICE void fetch(int batch, L load) {   // elements 4 batch to 4 batch + 3, those that there are
    if (CUT) return;
    const char* at = row + (long long)batch * (4 * B);
    const W* w = reinterpret_cast<const W*>((uintptr_t)at & ~kLow);
    if (at < end) lo = load(w);
    if ((const char*)w != at && (const char*)(w + 1) < end) hi = load(w + 1);
  }
  template <typename L>
  MOE_DEVICE W value(int batch, L load) const {
    const char* at = row + (long long)batch * (4 * B);
    if (CUT) {
      W v = 0;
      for (int i = 0; i < 4; ++i)
        if (at + i * B < end) v |= (W)load(reinterpret_cast<const T*>(at) + i) << (8 * B * i);
      return v;
    }
    const int sh = (int)((uintptr_t)at & kLow) * 8;
    return sh ? lo >> sh | hi << (32 * B - sh) : lo;
  }
};

// Whether an array of n elements of B bytes has rows, however they divide it, that its ends cut.
inline bool ends_cut(const void* array, long long n, int B) {
  return (uintptr_t)array % (4 * B) != 0 || n % 4 != 0;
}

}  // namespace moe
