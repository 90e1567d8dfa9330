// Frequencies of the rotary tables (host).
//
// An error in a pair's turns a position counts by the position, up to 2^31: those of double, 2^-55 turns
// and more, would leave 2^-24 of a turn.  Here numbers are unevaluated sums of two doubles (Dekker), right
// to some 2^-100, at the cost of a few multiplications; long double is as good, but on Arm a power of it
// takes longer than the tables.
#pragma once

#include <cmath>

namespace sba {

struct TwoDoubles {
  double hi, lo;
};
inline TwoDoubles exact_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
inline TwoDoubles exact_product(double a, double b) {
  const double p = a * b;
  return {p, std::fma(a, b, -p)};
}
inline TwoDoubles operator*(TwoDoubles a, TwoDoubles b) {
  const TwoDoubles p = exact_product(a.hi, b.hi);
  return exact_sum(p.hi, p.lo + (a.hi * b.lo + a.lo * b.hi));
}
inline TwoDoubles operator+(TwoDoubles a, double b) {
  const TwoDoubles s = exact_sum(a.hi, b);
  return exact_sum(s.hi, s.lo + a.lo);
}
inline TwoDoubles operator/(TwoDoubles a, TwoDoubles b) {
  const double q = a.hi / b.hi;
  const TwoDoubles p = b * TwoDoubles{q, 0.0};
  return exact_sum(q, ((a.hi - p.hi) + (a.lo - p.lo)) / b.hi);
}

// turns[i], i < rot / 2: turns a position of a pair, in steps of 2^-64, each right to less than a step.
inline void rotary_turns(int rot, double base, double factor, int original_length, double slow, double fast,
                         unsigned long long* turns) {
  const int n = rot / 2;
  // r = base^(-1 / n): one Newton step from the power in double.  base r^n is taken as (base h) h with
  // h = r^(n / 2), n even, so that no base overflows or underflows it.
  const double first = std::pow(base, -1.0 / n);
  TwoDoubles h{1.0, 0.0}, square{first, 0.0};
  for (int k = n / 2; k > 0; k >>= 1) {
    if (k & 1) h = h * square;
    square = square * square;
  }
  const TwoDoubles t = TwoDoubles{base, 0.0} * h * h;  // within 2^-44 of 1
  const TwoDoubles off = (t + -1.0) / TwoDoubles{-1.0 * n, 0.0};
  const double e = (t + -1.0).hi;
  // 1 / t - 1 over n, to the second order: ((1 + e)^(-1 / n) - 1
  const TwoDoubles r = TwoDoubles{first, 0.0} * ((off + 0.5 * (1.0 + n) / n / n * e * e) + 1.0);
  TwoDoubles f{0.15915494309189535, -9.839338337591243e-18};  // 1 / (2 pi)
  const TwoDoubles range = exact_sum(fast, -slow);
  for (int i = 0; i < n; ++i, f = f * r) {
    TwoDoubles keep{0.0, 0.0};
    if (original_length > 0) {
      keep = (f * TwoDoubles{static_cast<double>(original_length), 0.0} + -slow) / range;
      if (!(keep.hi > 0.0)) keep = {0.0, 0.0};
      if (keep.hi >= 1.0) keep = {1.0, 0.0};
    }
    // f (keep + (1 - keep) / factor)
    const TwoDoubles share = keep * (TwoDoubles{factor, 0.0} + -1.0) + 1.0;
    const TwoDoubles g = f * share / TwoDoubles{factor, 0.0};
    // the high part is a whole number of steps, or has none of them but its fraction
    const double hi = std::ldexp(g.hi, 64), lo = std::ldexp(g.lo, 64), whole = std::floor(hi);
    turns[i] = static_cast<unsigned long long>(whole) + static_cast<unsigned long long>(
        static_cast<long long>(std::floor((hi - whole) + lo + 0.5)));
  }
}

}  // namespace sba
