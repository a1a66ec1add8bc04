// Index arithmetic of the paged cache that host and device share.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define GDN_HD __host__ __device__ __forceinline__
#else
#define GDN_HD inline
#endif

namespace gdn {

// Column of the page table that holds `token`, exact for every token that starts a unit of 16 below
// 2^30 (the longest slot) and every page of 16 m tokens, m in 1..64.  With n = token / 16 < 2^26 and
// inv = ceil(2^32 / m) = (2^32 + e) / m, 0 <= e < m, the product's high word is
// floor(n / m + n e / (m 2^32)), and n e < 2^26 * 64 = 2^32 keeps the second term below 1 / m.
GDN_HD uint32_t page_units_inv(int32_t page_size) {  // 0 for pages of one unit, which need no quotient
  const uint32_t m = uint32_t(page_size) / 16;
  return uint32_t(((1ull << 32) + m - 1) / m);
}
GDN_HD int32_t page_column(int32_t token, uint32_t inv) {
  const uint32_t n = uint32_t(token) / 16;
  return int32_t(inv ? uint32_t((uint64_t(n) * inv) >> 32) : n);
}

}  // namespace gdn
