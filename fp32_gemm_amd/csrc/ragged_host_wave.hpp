// ragged_host_wave.hpp -- a wave of 64 lanes for ragged_order.hpp on the host.
#pragma once

#include "ragged_order.hpp"

namespace fp32gemm {

struct HostWave {
  static constexpr int N = 64;
  template <class T>
  struct Lanes {
    T v[N] = {};
    template <class F>
    static Lanes each(F f) {
      Lanes r;
      for (int i = 0; i < N; ++i) r.v[i] = f(i);
      return r;
    }
  };
  using Int = Lanes<int>;
  using Flag = Lanes<bool>;
  struct Spans { Int lo, hi; };

  Spans spans(const Groups& g, int e0) const {
    Spans s;
    for (int i = 0; i < N; ++i) {
      const RowSpan r = e0 + i < g.groups ? g.span(e0 + i) : RowSpan{0, 0};
      s.lo.v[i] = r.lo;
      s.hi.v[i] = r.hi;
    }
    return s;
  }
  static Int sum_below(const Int& a) {
    unsigned sum = 0;  // wraps, as the device's sums do
    return Int::each([&](int i) { return static_cast<int>(sum += static_cast<unsigned>(a.v[i])); });
  }
  static int at(const Int& a, int l) { return a.v[l & (N - 1)]; }
  static unsigned long long where(const Flag& f) {
    unsigned long long m = 0;
    for (int i = 0; i < N; ++i) m |= static_cast<unsigned long long>(f.v[i]) << i;
    return m;
  }
  static Int rank(unsigned long long m) {
    return Int::each([&](int i) { return __builtin_popcountll(m & ((1ull << i) - 1)); });
  }
  static Flag in(unsigned long long m) {
    return Flag::each([&](int i) { return (m >> i & 1) != 0; });
  }
  static Int lanes() { return Int::each([](int i) { return i; }); }

  friend Int operator+(const Int& a, int b) {
    return Int::each([&](int i) { return static_cast<int>(static_cast<unsigned>(a.v[i]) + static_cast<unsigned>(b)); });
  }
  friend Int operator-(const Int& a, const Int& b) { return Int::each([&](int i) { return a.v[i] - b.v[i]; }); }
  friend Int operator/(const Int& a, int b) { return Int::each([&](int i) { return a.v[i] / b; }); }
  friend Int operator%(const Int& a, int b) { return Int::each([&](int i) { return a.v[i] % b; }); }
  friend Int& operator+=(Int& a, const Flag& b) {
    for (int i = 0; i < N; ++i) a.v[i] += b.v[i];
    return a;
  }
  friend Flag operator>(const Int& a, int b) { return Flag::each([&](int i) { return a.v[i] > b; }); }
  friend Flag operator<(const Int& a, int b) { return Flag::each([&](int i) { return a.v[i] < b; }); }
  friend Flag operator==(const Int& a, int b) { return Flag::each([&](int i) { return a.v[i] == b; }); }
  friend Flag operator&(const Flag& a, const Flag& b) { return Flag::each([&](int i) { return a.v[i] && b.v[i]; }); }
  friend Flag operator|(const Flag& a, const Flag& b) { return Flag::each([&](int i) { return a.v[i] || b.v[i]; }); }
};

}  // namespace fp32gemm
