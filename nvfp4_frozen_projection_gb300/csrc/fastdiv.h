// Division by an invariant integer, prepared on the host.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pact {

// n / d for n < 2^31 by a multiply-high and a shift (Granlund and Montgomery's
// division by invariant integers): p = 31 + ceil(log2 d), m = ceil(2^p / d).
struct FastDiv {
  uint32_t d, m, s;
  __host__ static FastDiv make(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    const uint64_t p2 = 1ull << (31 + l);
    FastDiv f;
    f.d = d;
    f.m = (uint32_t)((p2 + d - 1) / d);
    f.s = l - 1;  // (n * m) >> (31 + l) == umulhi(n, m) >> (l - 1) for l >= 1
    return f;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return d == 1 ? n : (__umulhi(n, m) >> s);
  }
};

}  // namespace pact
