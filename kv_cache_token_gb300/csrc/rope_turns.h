// The rotation's frequencies as fractions of a turn per position (host).
// No CUDA types, so that they can be tested without a GPU.
#pragma once
#include <cmath>
#include <cstdint>

namespace kve {

constexpr int kRopePairs = 64;      // rotated pairs of a head at most

// Fractions of a turn per position of the r/2 pairs: base^(-2i/r) / 2 pi,
// mod 1, in units of 2^-64.  base^(-2i/r) is the product of the factors of
// i's bits, so the host takes at most 6 powers, not 64.
inline void turn_fractions(double base, int r, uint64_t* f) {
  constexpr double kTau = 6.283185307179586476925286766559;
  double p[kRopePairs];
  p[0] = 1.0;
  for (int i = 1; i < r / 2; ++i) {
    const int low = i & -i;
    p[i] = i == low ? std::pow(base, -2.0 * low / r) : p[i - low] * p[low];
  }
  for (int i = 0; i < r / 2; ++i) {
    double t = p[i] / kTau;
    t -= std::floor(t);
    f[i] = t >= 1.0 ? 0ull : static_cast<unsigned long long>(t * 18446744073709551616.0);
  }
}

// The same, kept from call to call: a model asks for one base, or for a few
// that its layers take in turn.  Each host thread has tables of its own, so
// calls from several threads need no lock.  Valid until the thread's next call.
inline const uint64_t* turn_table(double base, int r) {
  struct Table {
    double base;
    int r;
    uint64_t f[kRopePairs];
  };
  constexpr int kTables = 4;
  static thread_local Table tables[kTables];      // r 0: none (rotating nothing reads no table)
  static thread_local int oldest = 0;
  for (const Table& t : tables)
    if (t.r == r && t.base == base) return t.f;
  Table& t = tables[oldest];
  oldest = (oldest + 1) % kTables;
  t.base = base;
  t.r = r;
  turn_fractions(base, r, t.f);
  return t.f;
}

}  // namespace kve
