#pragma once

#include <cuda_runtime.h>

namespace gdn {

// Quotients by a divisor that the host knows, for dividends below 2^31: with l = ceil(log2 d)
// and m = floor(2^32 (2^l - d) / d) + 1, n / d = (mulhi(m, n) + n) >> l.
struct FastDiv {
  unsigned d, m, l;
  FastDiv() = default;
  explicit FastDiv(unsigned div) : d(div), l(0) {
    while ((1ull << l) < d) ++l;
    m = (unsigned)(((1ull << 32) * ((1ull << l) - d)) / d + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int div(int n) const { return (int)((__umulhi(m, (unsigned)n) + (unsigned)n) >> l); }
#endif
};

}  // namespace gdn
