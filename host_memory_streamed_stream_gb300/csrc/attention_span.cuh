// What the forward and backward of attention over spans share: the span of keys each query row
// sees, its summary over a tile of rows, and the score's cap and distance bias.
//
// Query i sees the keys lo_i <= j < hi_i. Causal, document, prefix and two-sided masks are all of
// this form, a tile's key range follows from its rows' smallest lo and largest hi, and a score's
// visibility is two comparisons, so no mask is ever read or stored per pair.
#pragma once
#include <atomic>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace mt {
namespace span {

constexpr float kLog2e = 1.4426950408889634f;

struct Spans {
  const int32_t* lo;  // [B*s] or null: 0
  const int32_t* hi;  // [B*s] or null: i + 1
};

// The span of row i of sequence b as given (a row past the end has none). Loaded ahead of its use and
// clamped where it is used: an operation on the loaded values would wait for them.
__device__ __forceinline__ int2 fetch_span(const Spans& sp, int b, int i, int s) {
  if (i >= s) return make_int2(0, 0);
  const int64_t at = static_cast<int64_t>(b) * s + i;
  return make_int2(sp.lo ? __ldg(sp.lo + at) : 0, sp.hi ? __ldg(sp.hi + at) : i + 1);
}
// Clamped to the sequence; an empty one is (0, 0).
__device__ __forceinline__ int2 clamp_span(int2 r, int s) {
  const int lo = max(r.x, 0), hi = min(r.y, s);
  return lo < hi ? make_int2(lo, hi) : make_int2(0, 0);
}
__device__ __forceinline__ int2 load_span(const Spans& sp, int b, int i, int s) {
  return clamp_span(fetch_span(sp, b, i, s), s);
}

// Summary of a tile of rows: the keys some row sees lie in [min_lo, max_hi); every row sees the
// keys [max_lo, min_hi) (an empty row makes that range empty).
struct Hull {
  int min_lo, max_hi, max_lo, min_hi;
};
// What one row adds to it; a row past the end of the sequence (live = false) adds nothing.
__device__ __forceinline__ Hull row_hull(int2 r, bool live) {
  if (!live) return {INT_MAX, 0, 0, INT_MAX};
  if (r.x >= r.y) return {INT_MAX, 0, INT_MAX, 0};
  return {r.x, r.y, r.x, r.y};
}
__device__ __forceinline__ Hull warp_hull(Hull h) {
  return {__reduce_min_sync(0xffffffffu, h.min_lo), __reduce_max_sync(0xffffffffu, h.max_hi),
          __reduce_max_sync(0xffffffffu, h.max_lo), __reduce_min_sync(0xffffffffu, h.min_hi)};
}
__device__ __forceinline__ Hull join(const Hull& a, const Hull& b) {
  return {min(a.min_lo, b.min_lo), max(a.max_hi, b.max_hi), max(a.max_lo, b.max_lo), min(a.min_hi, b.min_hi)};
}
// Whether all rows see all keys [k0, k1).
__device__ __forceinline__ bool sees_all(const Hull& h, int k0, int k1) { return h.max_lo <= k0 && k1 <= h.min_hi; }

// Bits [0, n) of a word, n clamped to 0..32.
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
// Bits of [lo, hi) relative to base.
__device__ __forceinline__ uint32_t span_bits(int2 r, int base) { return bits_below(r.y - base) & ~bits_below(r.x - base); }

// 32x32 bit transpose over the warp: bit c of lane r becomes bit r of lane c (five exchanges of
// halves of shrinking blocks).
__device__ __forceinline__ uint32_t warp_transpose(uint32_t x, int lane) {
  uint32_t m = 0x0000ffffu;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) {
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, j);
    x = (lane & j) ? ((x & ~m) | ((y & ~m) >> j)) : ((x & m) | ((y & m) << j));
    m ^= m << (j >> 1);
  }
  return x;
}

__device__ __forceinline__ float ex2(float x) {  // hardware 2^x (ex2.approx, flush to zero)
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {  // hardware 1/x (1/inf = 0)
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {  // three-input max (sm_100+)
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Scores in log2 units from the raw products x = q.k: scale log2(e) x, or, capped, c log2(e) times
// the tanh of scale x / c.
struct ScoreArgs {
  float scale_log2;  // scale log2(e)
  float scale;
  float cap_x;       // scale / c
  float cap_log2;    // c log2(e)
};
inline ScoreArgs score_args(const AttnSpanArgs& g) {
  return {g.scale * kLog2e, g.scale, g.cap > 0.f ? g.scale / g.cap : 0.f, g.cap * kLog2e};
}

// v = tanh(v cap_x) for a warp's N values a lane. While every |v cap_x| of the warp is at most 1
// (scores up to the cap itself) by a polynomial: tanh(t) = t p(t^2), p fitted to tanh(sqrt y)/sqrt y on
// [0, 1] with the smallest relative error for its degree, 5e-8; with fp32 arithmetic the result is
// within 1.6e-7 of its size. It runs two values at a time on the FMA units, which are idle here. Else
// tanh(t) = 1 - 2 / (1 + e^(2t)) for all of them, right at both ends (e^(2t) = 0 or inf) and within
// 2^-22 (absolute): its exponential and reciprocal share one slow unit with the softmax's exponential
// and made the capped kernels 1.4 (backward) to 2 times (forward) slower than the plain ones.
template <int N>
__device__ __forceinline__ void cap_tanh(float (&v)[N], const ScoreArgs& a) {
  const float2 k = make_float2(a.cap_x, a.cap_x);
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 t = __fmul2_rn(make_float2(v[i], v[i + 1]), k);
    const float2 y = __fmul2_rn(t, t);
    far = fmax3(far, y.x, y.y);
    v[i] = t.x;
    v[i + 1] = t.y;
  }
  if (__any_sync(0xffffffffu, far > 1.f)) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = fmaf(-2.f, rcp(1.f + ex2(v[i] * (2.f * kLog2e))), 1.f);
    return;
  }
  constexpr float kC[7] = {0.9999999403953552f,   -0.33332839608192444f,  0.13325203955173492f, -0.05345702916383743f,
                           0.020289979875087738f, -0.006203379016369581f, 0.0010410225950181484f};
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 t = make_float2(v[i], v[i + 1]);
    const float2 y = __fmul2_rn(t, t);
    float2 p = make_float2(kC[6], kC[6]);
#pragma unroll
    for (int d = 5; d >= 0; --d) p = __ffma2_rn(p, y, make_float2(kC[d], kC[d]));
    p = __fmul2_rn(p, t);
    v[i] = p.x;
    v[i + 1] = p.y;
  }
}

// Store 32 rows of NC 16-byte chunks, lane l holding row l: transposed within groups of NC lanes
// (log2 NC exchanges) so that a store instruction writes 32 / NC rows' whole runs of NC chunks.
// base: row 0, chunk 0; rows past `rows` are left out.
template <int NC>
__device__ __forceinline__ void store_rows(bf16* base, int64_t ld, int rows, uint4 (&c)[NC], int lane) {
#pragma unroll
  for (int b = 1; b < NC; b <<= 1) {
    const bool up = (lane & b) != 0;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      if (k & b) continue;
      uint4& lo = c[k];
      uint4& hi = c[k | b];
      const uint4 give = make_uint4(up ? lo.x : hi.x, up ? lo.y : hi.y, up ? lo.z : hi.z, up ? lo.w : hi.w);
      const uint4 got = make_uint4(__shfl_xor_sync(0xffffffffu, give.x, b), __shfl_xor_sync(0xffffffffu, give.y, b),
                                   __shfl_xor_sync(0xffffffffu, give.z, b), __shfl_xor_sync(0xffffffffu, give.w, b));
      lo = up ? got : lo;
      hi = up ? hi : got;
    }
  }
  const int first = lane / NC * NC;
#pragma unroll
  for (int k = 0; k < NC; ++k)
    if (first + k < rows) *reinterpret_cast<uint4*>(base + (first + k) * ld + (lane % NC) * 8) = c[k];
}

// Zero the 128 bytes of one 64-column slice of an operand row in shared memory. The 128-byte
// swizzle moves 16-byte chunks within a row only, so it does not matter here.
__device__ __forceinline__ void zero_slice_row(uint8_t* slice, int row) {
  uint4* p = reinterpret_cast<uint4*>(slice + row * 128);
#pragma unroll
  for (int i = 0; i < 8; ++i) p[i] = make_uint4(0u, 0u, 0u, 0u);
}

// Allow a kernel its dynamic shared memory, once for each device (a bit of `ready`).
template <class K>
cudaError_t allow_smem(K* kernel, int bytes, std::atomic<uint64_t>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && (ready.load() >> dev & 1))) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) ready.fetch_or(uint64_t{1} << dev);
  return e;
}

// One of the eight kernels of a direction: f(head_dim, capped, biased) as compile-time constants.
template <class F>
cudaError_t dispatch(const AttnSpanArgs& g, F&& f) {
  auto pick = [&](auto hd) {
    auto capped = [&](auto cap) {
      return g.slopes ? f(hd, cap, std::true_type{}) : f(hd, cap, std::false_type{});
    };
    return g.cap > 0.f ? capped(std::true_type{}) : capped(std::false_type{});
  };
  return g.hd == 64 ? pick(std::integral_constant<int, 64>{}) : pick(std::integral_constant<int, 128>{});
}

}  // namespace span
}  // namespace mt
