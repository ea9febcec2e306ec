// The row that an acceptance draws from.  Nothing here is the GPU's own, so
// that a host build can run it on loads that it watches.
#pragma once

#include <math.h>
#include <stdint.h>

namespace gdn {

// The target's row, less what was tried there.
template <typename IO>
struct AcceptRow {
  const void *p, *q;      // the target's and the draft's row
  int m;                  // rejected children
  const double* scale;    // 1 / Z in front of each rejection
  const int* tried;       // their tokens (certain drafts)

  // The draft's row takes part: with nothing rejected it does not, and behind
  // a node without children there need be none.
  __device__ inline bool two() const { return q != nullptr && m > 0; }
  __device__ inline double less(float pv, float qv, int x) const {
    double w = pv > 0.f ? pv : 0.f;  // (a NaN counts nothing)
    for (int j = 0; j < m; ++j) {
      const double by = q != nullptr ? static_cast<double>(qv) : x == tried[j] ? 1.0 : 0.0;
      w = fmax(fma(w, scale[j], -by), 0.0);
    }
    return w;
  }
  // The values of tokens x on, zeros from hi on; all loads in front of their
  // use, so that one wait is for all of a row's.
  template <int N>
  __device__ inline void take(int x, int hi, double (&w)[N]) const {
    float pv[N], qv[N];
    for (int e = 0; e < N; ++e) pv[e] = x + e < hi ? IO::load(p, x + e) : 0.f;
    for (int e = 0; e < N; ++e) qv[e] = 0.f;
    if (two())
      for (int e = 0; e < N; ++e) qv[e] = x + e < hi ? IO::load(q, x + e) : 0.f;
    for (int e = 0; e < N; ++e) w[e] = x + e < hi ? less(pv[e], qv[e], x + e) : 0.0;
  }
};

}  // namespace gdn
