// How the key steps of all sequences are shared out among the teams of the 4-bit attention (attend_q4.cu):
// plain integer arithmetic, the same on the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define FA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define FA_HOST_DEVICE inline
#endif

namespace fa {

// The shares of equal length: team i of N takes units [T i / N, T (i + 1) / N) of the T units of all
// sequences, key heads and row blocks in order, however long each sequence is.  N is all teams, or less
// where a share would fall under kQ4MinUnits.  Of whole row blocks: those that begin in that stretch.
constexpr int kQ4MinUnits = 1;
struct Q4Share {
  long long total;                                            // T
  int n;                                                      // N
  uint32_t each, rest;                                        // T / N (< 2^31: no team has more), T % N
  FA_HOST_DEVICE void set(long long t, int most) {
    total = t;
    const long long by_units = t / kQ4MinUnits;
    n = by_units < 1 ? 1 : by_units < most ? static_cast<int>(by_units) : most;
    // (a 64-bit division is some hundred instructions, and this one stands before the first load of keys)
    each = t < (1LL << 32) ? static_cast<uint32_t>(t) / static_cast<uint32_t>(n) : static_cast<uint32_t>(t / n);
    rest = static_cast<uint32_t>(t - static_cast<long long>(each) * n);
  }
  // T i / N
  FA_HOST_DEVICE long long begin(int i) const {
    return static_cast<long long>(each) * i + rest * static_cast<uint32_t>(i) / static_cast<uint32_t>(n);
  }
  // The team that has unit u.  (Both sides have to fit for the 32-bit division: of 2^32 units and more the
  // first ones have a small x.)
  FA_HOST_DEVICE int owner(long long u) const {
    const long long x = (u + 1) * n - 1;
    const bool small = x < (1LL << 32) && total < (1LL << 32);
    return small ? static_cast<int>(static_cast<uint32_t>(x) / static_cast<uint32_t>(total)) : static_cast<int>(x / total);
  }
};

}  // namespace fa
