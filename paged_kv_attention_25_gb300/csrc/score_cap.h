// The short way of capped scores, computed on the host for a call.
#pragma once
#include <cfloat>
#include <cmath>

namespace pkv {

// cap_out tanh(base x) for |x| < small as x (q0 + q1 x^2 + q2 x^4 + q3 x^6): tanh(y) / y interpolated at Chebyshev nodes of
// y^2 in [0, 1/4], off by 6e-7 of it.  small = 0, and no score counts as small, where a coefficient, which grows as a power
// of base (up to the seventh) times cap_out, is no normal number of fp32: caps of 30 to 50 have the short way for a
// base from 2^-18 to 2^18.
struct CapPoly {
  float small, q[4];
};
inline CapPoly cap_poly(float base, float cap_out) {
  const double c[4] = {0.9999994510270872, -0.3332628423141671, 0.13189939425594752, -0.04439273843261177};
  CapPoly p{0.5f / base, {}};
  double f = static_cast<double>(base) * cap_out;
  for (int i = 0; i < 4; ++i, f *= static_cast<double>(base) * base) {
    const double q = c[i] * f;
    if (!(std::fabs(q) >= FLT_MIN && std::fabs(q) <= FLT_MAX)) return CapPoly{};
    p.q[i] = static_cast<float>(q);
  }
  return p;
}

}  // namespace pkv
