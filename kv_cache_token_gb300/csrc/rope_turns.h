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
//
// In long double (64 bits on x86, 113 on Arm; doubles left 2^-24 turn at
// position 2^31).  With 64 bits the powers are off by an ulp, 2^-63, each, the
// products, the exponent and the division by 2^-64: at most 20 * 2^-64 of
// 1 / 2 pi for bases from 1, and 2^-64 for the fraction's end, under 2^-61 turn
// a position; 2^-30 at position 2^31.  Below base 1 the frequencies, and their
// error with them, grow to 1 / base times that.
inline void turn_fractions(double base, int r, uint64_t* f) {
  constexpr long double kTau = 6.283185307179586476925286766559005768L;
  long double p[kRopePairs];
  p[0] = 1.0L;
  for (int i = 1; i < r / 2; ++i) {
    const int low = i & -i;
    p[i] = i == low ? std::pow(static_cast<long double>(base), -2.0L * low / r) : p[i - low] * p[low];
  }
  for (int i = 0; i < r / 2; ++i) {
    long double t = p[i] / kTau;
    t -= std::floor(t);
    f[i] = t >= 1.0L ? 0ull : static_cast<unsigned long long>(t * 18446744073709551616.0L);
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
