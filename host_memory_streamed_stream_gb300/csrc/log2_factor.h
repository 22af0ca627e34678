// c = a log2 e as two floats, for powers 2^(c z). Computed on the host, once a call.
#pragma once
#include <cmath>
#include <cstdint>
#include <cstring>

namespace mt {

constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = 1.4426950408889634 - static_cast<double>(kLog2e);

// One float is off by up to 2^-25, which moves a row's logp by that times the label's distance from the mean, always
// the same way (1e-7 a token, which a sequence of 1000 tokens adds up); hi + lo is good to 2^-34: hi has 12 bits, so
// that what lo adds to c z is not below its last place, where it would always be lost. hi is strictly below the rounded
// product, so that lo > 0 also where that was rounded up to a number of 12 bits: a logit of -inf times lo has to stay
// -inf.
struct Factor {
  float one, hi, lo;
};
inline Factor factor(float scale) {
  const float one = scale * kLog2e;
  uint32_t bits;
  std::memcpy(&bits, &one, sizeof(bits));
  bits = (bits - 1) & 0xfffff000u;
  float hi;
  std::memcpy(&hi, &bits, sizeof(hi));
  return {one, hi, std::fmaf(scale, kLog2e, -hi) + scale * kLog2eLow};
}

}  // namespace mt
