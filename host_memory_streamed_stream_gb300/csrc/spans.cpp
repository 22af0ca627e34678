// Spans and positions of packed documents: host arrays in, host arrays out, like the token ids they
// go with. And the check that an entry's outputs do not lie over its inputs.
#include <algorithm>
#include <cstdint>

#include "kernels.h"

namespace mt {

bool columns_overlap(const bf16* a, int64_t lda, int64_t cols_a, const bf16* b, int64_t ldb, int64_t cols_b,
                     int64_t rows) {
  using Wide = __int128;  // any stride times any number of rows
  const Wide pa = reinterpret_cast<uintptr_t>(a) / sizeof(bf16), pb = reinterpret_cast<uintptr_t>(b) / sizeof(bf16);
  if (pa + Wide(rows - 1) * lda + cols_a <= pb || pb + Wide(rows - 1) * ldb + cols_b <= pa) return false;
  if (lda != ldb) return true;
  const Wide d = ((pb - pa) % lda + lda) % lda;  // b's first column in rows that start at a
  return d < cols_a || d + cols_b > lda;
}

bool doc_spans(const int32_t* bounds, int n_docs, const int32_t* prefix, int B, int s, int32_t* lo, int32_t* hi,
               int32_t* positions) {
  if (!bounds || !lo || !hi || n_docs < 0 || B <= 0 || s <= 0) return false;
  const int64_t T = static_cast<int64_t>(B) * s;
  if (T > INT32_MAX || bounds[0] < 0 || bounds[n_docs] > T) return false;
  for (int d = 0; d < n_docs; ++d)
    if (bounds[d + 1] < bounds[d] || (prefix && prefix[d] < 0)) return false;
  std::fill(lo, lo + T, 0);
  std::fill(hi, hi + T, 0);
  if (positions) std::fill(positions, positions + T, 0);
  for (int d = 0; d < n_docs; ++d) {
    for (int64_t t = bounds[d]; t < bounds[d + 1];) {  // the document's part in each sequence
      const int64_t base = t / s * s, end = std::min<int64_t>(bounds[d + 1], base + s);
      const int64_t keep = prefix ? std::min<int64_t>(end, t + prefix[d]) : t;
      for (int64_t i = t; i < end; ++i) {
        lo[i] = static_cast<int32_t>(t - base);
        hi[i] = static_cast<int32_t>(std::max(i + 1, keep) - base);
        if (positions) positions[i] = static_cast<int32_t>(i - t);
      }
      t = end;
    }
  }
  return true;
}

}  // namespace mt
