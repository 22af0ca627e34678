// Log-probabilities of given tokens and the losses on them: the clipped policy loss with a KL term, forward and
// backward in one pass over the logits, and the preference loss over pairs of sequences.
//
//   lse_t = log sum_v exp(a z_tv),  logp_t = a z_t,label - lse_t,  dlogits_tv = a dlogp_t ([v = label] - p_tv)
//
// Sums of exponentials run in fp32 as powers of two, 2^(c z - m) with c = a log2 e, against a whole number m that is
// raised where a term would pass 1: rescaling is exact. What an approximation loses always in one direction adds up
// over the tokens of a sequence, so that c is held as two floats (log2_factor.h), and the average error of the power is
// put back. Rows of 1001 to 152064 columns whose lse is near 0, so that its own rounding is nothing: off by 5e-8 in the
// root mean square, 2.6e-7 at most, below 9e-9 in the mean (1.9e-7 without the two); storing a logp of 8 to 16 as fp32
// adds 2.8e-7. The label's logit, m and the logarithm meet in pairs of floats: a ratio of policies is exp of a small
// difference of numbers of size 10, of which one float would lose 2^-21.
//
// Bound by HBM. Log-probabilities: 6000 rows of 32000 fp32 114 us, 6.7 TB/s, 3000 of 152064 bf16 135 us, 6.8 TB/s
// (where the exponential unit is 70 % busy). Policy loss, whose second look at a row reads the L2: 198 us, 5.8 TB/s,
// and 341 us, 5.3 TB/s; rows of 3000 to 10000 columns 1.4 to 1.6 times their bytes' time (8192 x 5268 fp32 56 us of
// 39), as a small block waits for its loads and at its barrier between two looks. Gradient alone: 4048 rows of 152064
// bf16, a quarter of them masked, 313 us, 6.9 TB/s with what the L2 still holds. What did not help the policy loss: a
// ring of shared memory that holds the row, filled by cp.async (1.8 times as long), bulk prefetches of the next row
// into the L2 (1.3), persistent blocks (1.05).
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "follow.cuh"
#include "kernels.h"
#include "log2_factor.h"
#include "mt_kernels.h"
#include "rows.cuh"

namespace mt {

namespace {

constexpr float kMinScale = 0x1p-64f;
constexpr float kLn2 = 0.6931471805599453f, kLn2Low = 0.6931471805599453 - static_cast<double>(kLn2);

__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The mean relative error of pow2 over any stretch of [-20, 0], measured against 64 bits: -4.9e-8 to -5.1e-8. (Above 0
// it is 3.4e-8: exponents are kept at or below 0.)
constexpr float kPow2Error = -5.0e-8f;

// Sum of 2^(c z - m), m a whole number; -inf: nothing but -inf so far, sum 0. +inf: beyond the range of c z.
struct MaxSum {
  float m, s;
};
// 2^(a - b) for whole a <= b.
__device__ __forceinline__ float down(float a, float b) {
  return a == b ? 1.f : __int_as_float((static_cast<int>(fmaxf(a - b, -127.f)) + 127) << 23);
}
constexpr float kRoom = 1.f;  // that a raised m leaves: few rows raise it again
template <int N>
__device__ __forceinline__ void add_terms(MaxSum& r, const float* z, const Factor& c) {
  float top = z[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, z[i]);
  top *= c.one;
  if (top > r.m) {
    const float m = ceilf(top) + kRoom;
    r.s *= down(r.m, m);
    r.m = m;
  }
  const float m = r.m == -INFINITY ? 0.f : r.m;
  if constexpr (N == 1) {
    r.s += pow2(fmaf(z[0], c.lo, fmaf(z[0], c.hi, -m)));
  } else {
    const float2 hi = make_float2(c.hi, c.hi), lo = make_float2(c.lo, c.lo), low = make_float2(-m, -m);
    // their own sum first: bf16 logits have few values, whose roundings against a long sum are the same each time
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 q = make_float2(z[i], z[i + 1]), x = __ffma2_rn(q, lo, __ffma2_rn(q, hi, low));
      sum = __fadd2_rn(sum, make_float2(pow2(x.x), pow2(x.y)));
    }
    r.s += sum.x + sum.y;
  }
}
// Beyond this m (logits of 45000 at scale 1) c z is no longer good to 2^-20, and finally out of range: such rows are
// summed again with the largest logit z0 subtracted before the product, as are rows of nothing but -inf.
constexpr float kFarthest = 65536.f;
__device__ __forceinline__ bool too_far(const MaxSum& r) { return !(fabsf(r.m) <= kFarthest); }
// The sum over a warp's lanes, the same in all of them.
__device__ __forceinline__ MaxSum merge_warp(MaxSum r) {
  const int i = __float_as_int(r.m), ordered = __reduce_max_sync(0xffffffffu, i ^ (i >> 31 & 0x7fffffff));
  const float m = __int_as_float(ordered ^ (ordered >> 31 & 0x7fffffff));
  r.s *= down(r.m, m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r.s += __shfl_xor_sync(0xffffffffu, r.s, o);
  return {m, r.s};
}

// A number held as two floats, the second what the first has lost: a few instructions of 4 cycles where 64-bit
// arithmetic takes 40 cycles each, in the one thread that a whole row waits for.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair add(const Pair& a, const Pair& b) {
  const float s = a.hi + b.hi, x = s - a.hi;
  return {s, (a.hi - (s - x)) + (b.hi - x) + (a.lo + b.lo)};
}
__device__ __forceinline__ Pair add_warp(Pair a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = add(a, {__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)});
  return a;
}
__device__ __forceinline__ Pair product(const Pair& a, float b) {
  const float p = a.hi * b;
  return {p, fmaf(a.hi, b, -p) + a.lo * b};
}
__device__ __forceinline__ Pair negative(const Pair& a) { return {-a.hi, -a.lo}; }
// With an infinity or NaN among the parts the second float may be NaN where the sum is not.
__device__ __forceinline__ float value(const Pair& a) { return isfinite(a.hi) ? a.hi + a.lo : a.hi; }
// The logarithm, to 2^-24 of its fraction rather than of its size.
__device__ __forceinline__ Pair log_pair(float s) {
  int e;
  float f = frexpf(s, &e);
  if (f < 0.70710678f) f *= 2.f, e -= 1;
  if (!(s > 0.f && s < INFINITY)) return {logf(s), 0.f};
  return add(product({kLn2, kLn2Low}, static_cast<float>(e)), {logf(f), 0.f});
}

struct TokenRows {
  const void* logits;
  int64_t ld;
  const int32_t* labels;
  int T, V;
  float scale;
  Factor c;     // of scale
  float per_c;  // 1 / c
  float* logp;
  float* lse;  // token_logprobs
  // policy loss
  const float *old_logp, *adv, *ref, *weights;
  float clip_low, clip_high, kl;
  bf16* dlogits;
  int64_t ldd;
  float* row_loss;
  int* err;
};

// A row's numbers besides its logits, loaded ahead of where they are used (and converted there: the thread goes on).
template <class Z>
struct RowInputs {
  Z z_label;
  float old_logp, adv, ref, weight;
  __device__ __forceinline__ float label() const { return to_f32(z_label); }
};
template <class Z, bool POLICY>
__device__ __forceinline__ RowInputs<Z> row_inputs(const TokenRows& g, int64_t t, int label) {
  RowInputs<Z> r{};
  r.z_label = static_cast<const Z*>(g.logits)[t * g.ld + label];
  if constexpr (POLICY) {
    r.old_logp = g.old_logp[t];
    r.adv = g.adv[t];
    r.ref = g.kl != 0.f ? g.ref[t] : 0.f;
    r.weight = g.weights ? g.weights[t] : 1.f / static_cast<float>(g.T);
  }
  return r;
}
// What the second look at a row needs: dlogits_v = kp 2^(c (z_v - z0) - m) + k [v = label].
struct RowGrad {
  float z0, m, k, kp;
};
// Of sums of 2^(c (z - z0) - m). The second look has c in one float, whose error times z would scale all of p (6e-4 at
// logits of 40000): it subtracts about m / c from z first, and then what is left of m.
__device__ __forceinline__ RowGrad row_grad(const TokenRows& g, float z0, float m, float k, float kp) {
  const float near = m * g.per_c;  // 0 where z0 is not
  return {z0 + near, fmaf(-g.c.lo, near, fmaf(-g.c.hi, near, m)), k, kp};
}
// The row's log-probability, and for the policy loss its loss and d loss / d logp, from the sum r of
// 2^(c (z - z0) - m). `write`: of several callers, one.
template <bool POLICY, class Z>
__device__ __forceinline__ RowGrad finish_row(const TokenRows& g, int64_t t, const RowInputs<Z>& in, float z0,
                                              const MaxSum& r, bool write) {
  Pair log_sum = add(product({kLn2, kLn2Low}, r.m), log_pair(r.s));
  // A power of two is mostly a sum of exact terms. (Other sums of them, as of three equal logits of 0, are off by
  // 5e-8.)
  if ((__float_as_uint(r.s) & 0x7fffffu) != 0) log_sum = add(log_sum, {-kPow2Error, 0.f});
  Pair logp = add(product(add({in.label(), 0.f}, {-z0, 0.f}), g.scale), negative(log_sum));
  if (logp.hi > 0.f) logp = {0.f, 0.f};  // by rounding, where the label has all of the probability
  if (write) g.logp[t] = value(logp);
  if constexpr (!POLICY) {
    if (write) g.lse[t] = value(add(product({z0, 0.f}, g.scale), log_sum));
    return {};
  } else {
    float ratio = expf(value(add(logp, {-in.old_logp, 0.f})));
    if (ratio == INFINITY) ratio = FLT_MAX;  // times an advantage of 0 it is 0
    const float lo = 1.f - g.clip_low, hi = 1.f + g.clip_high;
    // comparisons rather than fminf, which would drop a NaN
    const float cut = ratio < lo ? lo : ratio > hi ? hi : ratio;
    const bool held = ratio * in.adv > cut * in.adv;
    float loss = held ? -cut * in.adv : -ratio * in.adv;
    float d = held ? 0.f : -ratio * in.adv;
    if (g.kl != 0.f) {
      const float far = value(add({in.ref, 0.f}, negative(logp)));
      const float em1 = expm1f(far);
      loss += g.kl * (em1 < INFINITY ? em1 - far : em1);  // infinite, also where far itself is; NaN stays
      d -= g.kl * em1;
    }
    if (in.weight == 0.f && loss == loss) loss = d = 0.f;  // where exp has passed fp32's range too
    if (write) g.row_loss[t] = in.weight * loss;
    const float k = in.weight * d * g.scale;
    return row_grad(g, z0, r.m, k, -k / r.s);
  }
}

// ------------------------------------------------------------------ rows
// In chunks of 16 bytes; neighbouring threads take neighbouring chunks.
template <class Z>
constexpr int kChunk = 16 / static_cast<int>(sizeof(Z));  // columns of a chunk

template <class Z>
__device__ __forceinline__ void unpack_chunk(const uint4& u, float* v) {
  if constexpr (sizeof(Z) == 2) {
    unpack8(u, v);
  } else {
    v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
  }
}
// A chunk's gradient, which nothing here reads again.
template <class Z>
__device__ __forceinline__ void write_chunk(bf16* d, float* v, const RowGrad& q, const Factor& c, int to_label) {
  constexpr int N = kChunk<Z>;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 x = __ffma2_rn(__fadd2_rn(make_float2(v[i], v[i + 1]), make_float2(-q.z0, -q.z0)),
                                make_float2(c.one, c.one), make_float2(-q.m, -q.m));
    const float2 p = __fmul2_rn(make_float2(pow2(x.x), pow2(x.y)), make_float2(q.kp, q.kp));
    v[i] = p.x, v[i + 1] = p.y;
  }
  if (static_cast<unsigned>(to_label) < N) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += i == to_label ? q.k : 0.f;
  }
  if constexpr (N == 8) __stcs(reinterpret_cast<uint4*>(d), pack8(v));
  else __stcs(reinterpret_cast<uint2*>(d), make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])));
}
template <class Z>
__device__ __forceinline__ bf16 one_grad(Z z, const RowGrad& q, const Factor& c, bool hot) {
  return __float2bfloat16_rn(q.kp * pow2(fmaf(to_f32(z) - q.z0, c.one, -q.m)) + (hot ? q.k : 0.f));
}
// Zeros in the columns [0, n) of a row, by `threads` threads.
__device__ __forceinline__ void zero_row(bf16* d, int n, int at, int threads) {
  for (int i = at * 8; i < (n & ~7); i += threads * 8) *reinterpret_cast<uint4*>(d + i) = make_uint4(0, 0, 0, 0);
  for (int i = (n & ~7) + at; i < n; i += threads) d[i] = __float2bfloat16_rn(0.f);
}
template <bool POLICY>
__device__ __forceinline__ void masked_row(const TokenRows& g, int64_t t, int label) {
  if (label >= g.V) record_bad_token(g.err);
  g.logp[t] = 0.f;
  if (POLICY) g.row_loss[t] = 0.f;
  else g.lse[t] = 0.f;
}

// Short rows, up to 32 x kWarpChunks chunks: a warp a row, in registers.
constexpr int kWarpChunks = 8;
template <class Z, bool POLICY>
__global__ void __launch_bounds__(128) token_warp_kernel(const TokenRows g) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  constexpr int N = kChunk<Z>;
  wait_for_previous();
  let_next_start();
  if (t >= g.T) return;
  const Z* z = static_cast<const Z*>(g.logits) + t * g.ld;
  bf16* d = POLICY ? g.dlogits + t * g.ldd : nullptr;
  const int label = g.labels[t];
  if (label < 0 || label >= g.V) {
    if (lane == 0) masked_row<POLICY>(g, t, label);
    if (POLICY) zero_row(d, g.V, lane, 32);
    return;
  }
  RowInputs<Z> in{};
  if (lane == 0) in = row_inputs<Z, POLICY>(g, t, label);
  uint4 raw[kWarpChunks];
#pragma unroll
  for (int j = 0; j < kWarpChunks; ++j) {
    const int col = (j * 32 + lane) * N;
    if (col + N <= g.V) raw[j] = *reinterpret_cast<const uint4*>(z + col);
  }
  const Factor c = g.c;
  MaxSum r{-INFINITY, 0.f};
  float v[N];
#pragma unroll
  for (int j = 0; j < kWarpChunks; ++j) {
    const int col = (j * 32 + lane) * N;
    if (col + N <= g.V) {
      unpack_chunk<Z>(raw[j], v);
      add_terms<N>(r, v, c);
    } else {
      for (int i = col; i < g.V; ++i) {
        v[0] = to_f32(z[i]);
        add_terms<1>(r, v, c);
      }
    }
  }
  r = merge_warp(r);
  float z0 = 0.f;
  if (too_far(r)) {
    z0 = -INFINITY;
    for (int i = lane; i < g.V; i += 32) z0 = fmaxf(z0, to_f32(z[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z0 = fmaxf(z0, __shfl_xor_sync(0xffffffffu, z0, o));
    r = {0.f, 0.f};
    for (int i = lane; i < g.V; i += 32) r.s += pow2((to_f32(z[i]) - z0) * c.one);
    r = merge_warp(r);
  }
  RowGrad q{};
  if (lane == 0) q = finish_row<POLICY>(g, t, in, z0, r, true);
  if constexpr (POLICY) {
    q = row_grad(g, z0, r.m, __shfl_sync(0xffffffffu, q.k, 0), __shfl_sync(0xffffffffu, q.kp, 0));
#pragma unroll
    for (int j = 0; j < kWarpChunks; ++j) {
      const int col = (j * 32 + lane) * N;
      if (col + N <= g.V) {
        unpack_chunk<Z>(raw[j], v);
        write_chunk<Z>(d + col, v, q, c, label - col);
      } else {
        for (int i = col; i < g.V; ++i) d[i] = one_grad(z[i], q, c, i == label);
      }
    }
  }
}

// Longer rows: a block a row, or, for very wide and for few rows, a cluster of blocks that split it by columns, with
// two loads of a thread in flight (policy loss at 32000 fp32: one 1.18 times as long, four at half the threads 1.3).
// The policy loss reads the row a second time, from the L2, for its gradient.
// *p of block `rank` of the cluster = v.
__device__ __forceinline__ void cluster_store(MaxSum* p, unsigned rank, const MaxSum& v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.m), "f"(v.s) : "memory");
}

template <class Z, bool POLICY, int NT>
__global__ void __launch_bounds__(NT, 2048 / NT) token_rows_kernel(const TokenRows g, int share) {
  constexpr int N = kChunk<Z>, WARPS = NT / 32;
  __shared__ MaxSum part[2][WARPS], others[2][8];
  __shared__ RowGrad shared;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned rank = cluster_rank(), blocks = cluster_blocks();
  const int64_t t = blockIdx.x / blocks;
  const int c0 = static_cast<int>(rank) * share, cols = min(share, g.V - c0), whole = cols / N * N;
  wait_for_previous();
  let_next_start();
  const int label = g.labels[t];
  if (label < 0 || label >= g.V) {  // the same for all blocks of the cluster
    if (rank == 0 && threadIdx.x == 0) masked_row<POLICY>(g, t, label);
    if (POLICY) zero_row(g.dlogits + t * g.ldd + c0, cols, threadIdx.x, NT);
    return;
  }
  if (blocks > 1) cluster_arrive();
  const Z* z = static_cast<const Z*>(g.logits) + t * g.ld + c0;
  RowInputs<Z> in{};
  if (threadIdx.x == 0) in = row_inputs<Z, POLICY>(g, t, label);
  const Factor c = g.c;
  MaxSum r{-INFINITY, 0.f};
  int i = threadIdx.x * N;
  for (; i + NT * N < whole; i += 2 * NT * N) {
    const uint4 x = *reinterpret_cast<const uint4*>(z + i), y = *reinterpret_cast<const uint4*>(z + i + NT * N);
    float v[2 * N];
    unpack_chunk<Z>(x, v);
    unpack_chunk<Z>(y, v + N);
    add_terms<2 * N>(r, v, c);
  }
  if (i < whole) {
    float v[N];
    unpack_chunk<Z>(*reinterpret_cast<const uint4*>(z + i), v);
    add_terms<N>(r, v, c);
  }
  if (whole + static_cast<int>(threadIdx.x) < cols) {
    const float v = to_f32(z[whole + threadIdx.x]);
    add_terms<1>(r, &v, c);
  }
  int turn = 0;
  bool started = false;  // all blocks of the cluster
  auto meet = [&](MaxSum v) {  // over the blocks of the row, in every thread
    v = merge_warp(v);
    if (lane == 0) part[turn][warp] = v;
    __syncthreads();
    v = merge_warp(lane < WARPS ? part[turn][lane] : MaxSum{-INFINITY, 0.f});
    if (blocks > 1) {
      if (!started) cluster_wait();
      started = true;
      if (warp == 0 && lane < static_cast<int>(blocks)) cluster_store(&others[turn][rank], lane, v);
      cluster_sync();
      v = merge_warp(lane < static_cast<int>(blocks) ? others[turn][lane] : MaxSum{-INFINITY, 0.f});
    }
    turn ^= 1;
    return v;
  };
  r = meet(r);
  float z0 = 0.f;
  if (too_far(r)) {
    r = {-INFINITY, 0.f};
    for (i = threadIdx.x; i < cols; i += NT) r.m = fmaxf(r.m, to_f32(z[i]));
    z0 = meet(r).m;
    r = {0.f, 0.f};
    for (i = threadIdx.x; i < cols; i += NT) r.s += pow2((to_f32(z[i]) - z0) * c.one);
    r = meet(r);
  }
  if (threadIdx.x == 0) shared = finish_row<POLICY>(g, t, in, z0, r, rank == 0);
  if constexpr (POLICY) {
    __syncthreads();
    const RowGrad q = shared;
    bf16* d = g.dlogits + t * g.ldd + c0;
    const int at = label - c0;
    i = threadIdx.x * N;
    for (; i + NT * N < whole; i += 2 * NT * N) {
      const uint4 x = __ldcs(reinterpret_cast<const uint4*>(z + i));
      const uint4 y = __ldcs(reinterpret_cast<const uint4*>(z + i + NT * N));
      float v[N];
      unpack_chunk<Z>(x, v);
      write_chunk<Z>(d + i, v, q, c, at - i);
      unpack_chunk<Z>(y, v);
      write_chunk<Z>(d + i + NT * N, v, q, c, at - i - NT * N);
    }
    if (i < whole) {
      float v[N];
      unpack_chunk<Z>(__ldcs(reinterpret_cast<const uint4*>(z + i)), v);
      write_chunk<Z>(d + i, v, q, c, at - i);
    }
    i = whole + threadIdx.x;
    if (i < cols) d[i] = one_grad(z[i], q, c, i == at);
  }
}

// dlogits of given dlogp and lse: a pass over the logits, from the last row to the first, since the L2 still holds some
// of the last rows that token_logprobs read.
constexpr int kGradChunks = 4, kGradThreads = 256;  // chunks of a thread
// Up to here p takes on lse's rounding, 2^-14 of it at most. Beyond, lse no longer has the sum's logarithm (or is out
// of fp32's range), and one block takes the whole row, which it sums again with the largest logit subtracted (all rows
// of 2048 x 32000 bf16 far: 138 us for 44).
constexpr float kFarLse = 1024.f;

// A far row, in place or not: all of it is read before any of it is written.
template <class Z>
__device__ __noinline__ void far_row_grad(const Z* z, bf16* d, int V, float scale, float k, int label) {
  __shared__ float red[2][kGradThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float c = scale * kLog2e;
  float top = -INFINITY, sum = 0.f;
#pragma unroll 8
  for (int i = threadIdx.x; i < V; i += kGradThreads) top = fmaxf(top, to_f32(z[i]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) red[0][warp] = top;
  __syncthreads();
  for (int w = 0; w < kGradThreads / 32; ++w) top = fmaxf(top, red[0][w]);
#pragma unroll 8
  for (int i = threadIdx.x; i < V; i += kGradThreads) sum += pow2((to_f32(z[i]) - top) * c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) red[1][warp] = sum;
  __syncthreads();
  sum = 0.f;
  for (int w = 0; w < kGradThreads / 32; ++w) sum += red[1][w];
  const float kp = -k / sum;
#pragma unroll 4
  for (int i = threadIdx.x; i < V; i += kGradThreads)
    d[i] = __float2bfloat16_rn(kp * pow2((to_f32(z[i]) - top) * c) + (i == label ? k : 0.f));
}
template <class Z>
__global__ void __launch_bounds__(kGradThreads) token_grad_kernel(const TokenRows g, const float* dlogp) {
  constexpr int N = kChunk<Z>, STEP = kGradThreads * N;
  const int64_t t = gridDim.y - 1 - blockIdx.y;
  const Z* z = static_cast<const Z*>(g.logits) + t * g.ld;
  bf16* d = g.dlogits + t * g.ldd;
  wait_for_previous();
  let_next_start();
  const int label = g.labels[t], whole = g.V / N * N, first = blockIdx.x * STEP * kGradChunks + threadIdx.x * N;
  const float lse = g.lse[t];
  const bool masked = label < 0 || label >= g.V, far = !(fabsf(lse) <= kFarLse);
  if (masked | far) {  // one test, so that lse is not loaded behind the label's
    if (masked) {
      const int c0 = blockIdx.x * STEP * kGradChunks;
      zero_row(d + c0, min(STEP * kGradChunks, g.V - c0), threadIdx.x, kGradThreads);
    } else if (blockIdx.x == 0) {
      far_row_grad(z, d, g.V, g.scale, dlogp[t] * g.scale, label);
    }
    return;
  }
  uint4 raw[kGradChunks];
#pragma unroll
  for (int j = 0; j < kGradChunks; ++j)
    if (first + j * STEP < whole) raw[j] = __ldcs(reinterpret_cast<const uint4*>(z + first + j * STEP));
  const float k = dlogp[t] * g.scale;
  const RowGrad q{lse / g.scale, 0.f, k, -k};
  const Factor c = g.c;
#pragma unroll
  for (int j = 0; j < kGradChunks; ++j) {
    const int i = first + j * STEP;
    if (i < whole) {
      float v[N];
      unpack_chunk<Z>(raw[j], v);
      write_chunk<Z>(d + i, v, q, c, label - i);
    } else {
      for (int n = i; n < min(i + N, g.V); ++n) d[n] = one_grad(z[n], q, c, n == label);
    }
  }
}

// out = sum of v[0..n) times f in a fixed order.
__global__ void __launch_bounds__(1024) sum_kernel(const float* v, int n, float f, float* out) {
  __shared__ Pair red[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_for_previous();
  let_next_start();
  Pair s{0.f, 0.f};
  for (int i = threadIdx.x; i < n; i += 8 * blockDim.x) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = i + j * static_cast<int>(blockDim.x) < n ? v[i + j * blockDim.x] : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = add(s, {x[j], 0.f});
  }
  s = add_warp(s);
  if (lane == 0) red[warp] = s;
  __syncthreads();
  if (warp == 0) {
    s = add_warp(red[lane]);
    if (lane == 0) *out = value(s) * f;
  }
}

__device__ Pair block_total(Pair v, Pair* red) {
  v = add_warp(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = {0.f, 0.f};
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) v = add(v, red[i]);
  return v;
}

struct Preference {
  const float *logp, *ref;
  const int32_t *labels, *bounds;
  int pairs, T, kind;
  float beta, margin, smoothing;
  bool average;
  float *pair_loss, *rewards, *dlogp;
};

// A row's part of its sequence's score, added to v where the row is trained. Scores are held in pairs of floats: two
// sums of thousands, of which a float's step is 2^-11, differ by little.
__device__ __forceinline__ Pair add_score(const Preference& g, Pair v, int i, bool on) {
  const float a = g.logp[i], b = g.ref ? g.ref[i] : 0.f;
  v = add(v, {on ? a : 0.f, 0.f});
  return g.ref ? add(v, {on ? -b : 0.f, 0.f}) : v;
}
// A pair's loss from its two scores, and the derivative by their difference times beta (h).
__device__ __forceinline__ float pair_loss(const Preference& g, const Pair& s0, const Pair& s1, float& d) {
  const float h = g.beta * value(add(s0, negative(s1))) - g.margin;
  float loss;
  if (g.kind == MTK_PREF_SIGMOID) {
    const float e = expf(-fabsf(h)), l = log1pf(e);  // softplus(-|h|)
    // an infinite h times a smoothing of 0 is nothing
    loss = l + (h <= 0.f ? (g.smoothing - 1.f) * h : g.smoothing > 0.f || h != h ? g.smoothing * h : 0.f);
    d = g.smoothing - (h > 0.f ? e : 1.f) / (1.f + e);
  } else if (g.kind == MTK_PREF_HINGE) {
    loss = h >= 1.f ? 0.f : 1.f - h;
    d = h < 1.f ? -1.f : h >= 1.f ? 0.f : h;  // NaN stays
  } else {
    const float u = (h - 0.5f) / g.beta;
    loss = u * u;
    d = 2.f * u / g.beta;
  }
  return loss;
}
// The row at which sequence j begins, or the one before it ends.
__device__ __forceinline__ int bound_of(const Preference& g, int j) { return min(max(g.bounds[j], 0), g.T); }

// Few rows of few sequences: one block does all of it, several warps a sequence. Against a block a pair and another
// launch for the mean, with a reference and labels: 322 rows of 4 sequences 2.7 and 4.7 us, 4096 of 2 3.9 and 7.6, of 8
// 3.9 and 4.6, of 32 3.6 and 4.5. With warps that took more sequences in turn, 64 took 5.3 and 4.5, 2048 69 and 13.
constexpr int kFewRows = 4096, kFewPairs = 16;
__global__ void __launch_bounds__(1024) preference_few_kernel(const Preference g, float* loss) {
  __shared__ Pair score[2 * kFewPairs];
  __shared__ float share[2 * kFewPairs];
  __shared__ float4 part[32];  // a warp's sum and count
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = 2 * g.pairs;
  const int team = 32 / n, j = warp / team, mate = warp % team;  // a team of warps for each sequence
  wait_for_previous();
  let_next_start();
  int lo = 0, hi = 0;
  if (j < n) lo = bound_of(g, j), hi = bound_of(g, j + 1);
  Pair v{0.f, 0.f};
  float count = 0.f;
#pragma unroll 8
  for (int i = lo + mate * 32 + lane; i < hi; i += team * 32) {
    const bool on = !g.labels || g.labels[i] >= 0;
    v = add_score(g, v, i, on);
    count += on ? 1.f : 0.f;
  }
  v = add_warp(v);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) count += __shfl_xor_sync(0xffffffffu, count, o);
  if (lane == 0) part[warp] = make_float4(v.hi, v.lo, count, 0.f);
  __syncthreads();
  if (lane == 0 && mate == 0 && j < n) {
    for (int k = warp + 1; k < warp + team; ++k) v = add(v, {part[k].x, part[k].y}), count += part[k].z;
    share[j] = g.average ? 1.f / fmaxf(count, 1.f) : 1.f;
    score[j] = product(v, share[j]);
    g.rewards[j] = g.beta * value(score[j]);
  }
  __syncthreads();
  if (warp == 0) {
    Pair sum{0.f, 0.f};
    if (lane < g.pairs) {
      float d;
      const float l = pair_loss(g, score[2 * lane], score[2 * lane + 1], d);
      g.pair_loss[lane] = l;
      sum = {l, 0.f};
      const float k = g.beta * d / static_cast<float>(g.pairs);
      share[2 * lane] *= k;
      share[2 * lane + 1] *= -k;
    }
    sum = add_warp(sum);
    if (lane == 0) *loss = value(sum) / static_cast<float>(g.pairs);
  }
  __syncthreads();
  const float k = j < n ? share[j] : 0.f;
#pragma unroll 4
  for (int i = lo + mate * 32 + lane; i < hi; i += team * 32) g.dlogp[i] = g.labels && g.labels[i] < 0 ? 0.f : k;
  const int first = bound_of(g, 0), last = max(first, bound_of(g, n));
  for (int i = threadIdx.x; i < first; i += 1024) g.dlogp[i] = 0.f;
  for (int i = last + threadIdx.x; i < g.T; i += 1024) g.dlogp[i] = 0.f;
}

// One block a pair: the sums of its two sequences, its loss, and its rows' dlogp. The last block zeroes the rows
// of no sequence.
__global__ void __launch_bounds__(512) preference_kernel(const Preference g) {
  __shared__ Pair red[16];
  wait_for_previous();
  let_next_start();
  const int p = blockIdx.x;
  if (p == g.pairs) {
    const int first = bound_of(g, 0), last = max(first, bound_of(g, 2 * g.pairs));
    for (int i = threadIdx.x; i < first; i += blockDim.x) g.dlogp[i] = 0.f;
    for (int i = last + threadIdx.x; i < g.T; i += blockDim.x) g.dlogp[i] = 0.f;
    return;
  }
  Pair s[2];
  float share[2];
  int lo[2], hi[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    lo[j] = bound_of(g, 2 * p + j);
    hi[j] = bound_of(g, 2 * p + j + 1);
    Pair v{0.f, 0.f};
    float n = 0.f;
    for (int i = lo[j] + threadIdx.x; i < hi[j]; i += blockDim.x) {
      if (g.labels && g.labels[i] < 0) continue;
      v = add_score(g, v, i, true);
      n += 1.f;
    }
    v = block_total(v, red);
    if (g.average) n = value(block_total({n, 0.f}, red));
    share[j] = g.average ? 1.f / fmaxf(n, 1.f) : 1.f;
    s[j] = product(v, share[j]);
  }
  float d;
  const float loss = pair_loss(g, s[0], s[1], d);
  if (threadIdx.x == 0) {
    g.pair_loss[p] = loss;
    g.rewards[2 * p] = g.beta * value(s[0]);
    g.rewards[2 * p + 1] = g.beta * value(s[1]);
  }
  const float k = g.beta * d / static_cast<float>(g.pairs);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float kj = (j ? -k : k) * share[j];
    for (int i = lo[j] + threadIdx.x; i < hi[j]; i += blockDim.x)
      g.dlogp[i] = g.labels && g.labels[i] < 0 ? 0.f : kj;
  }
}

void set_scale(TokenRows& g, float scale) {
  g.scale = scale;
  g.c = factor(scale);
  g.per_c = 1.f / g.c.one;
}
bool rows_args_ok(const TokenRows& g, int type) {
  return row_type_ok(type) && g.T > 0 && g.T <= kMaxRows && g.V > 0 && g.V <= kMaxVocab &&
         rows_ok(g.logits, g.ld, g.V) && vec_ok(g.labels, 4) && g.scale >= kMinScale && g.scale <= 1.f / kMinScale &&
         (!g.err || vec_ok(g.err, 4));
}
// The gradient's rows: apart from the logits', or the bf16 logits themselves.
bool grad_ok(const TokenRows& g, int type) {
  if (!rows_ok(g.dlogits, g.ldd, g.V)) return false;
  if (type == kRowBf16 && g.dlogits == g.logits) return g.ldd == g.ld;
  return !spans_overlap(g.logits, g.ld, row_type_bytes(type), g.dlogits, g.ldd, 2, g.T, g.V);
}
// Blocks of a row. The policy loss: as many as keep the rows that are being worked on, two on an SM, within what the L2
// holds of them (3000 rows of 152064 bf16, 304 KB: one block 344 us, two 338, four 428; 6000 of 128 KB: one 198, two
// 220). Few rows: as many as have 2048 columns each to do, up to two on an SM.
constexpr int kShareBytes = 160 << 10;
int row_blocks(int T, int V, int esz, bool policy) {
  int n = 1;
  while (policy && n < 8 && static_cast<int64_t>(V) * esz > static_cast<int64_t>(n) * kShareBytes) n *= 2;
  while (n < 8 && static_cast<int64_t>(T) * n <= kSms && V / (2 * n) >= 2048) n *= 2;
  return n;
}

template <class Z, bool POLICY, int NT>
cudaError_t launch_blocks(const TokenRows& g, int blocks, cudaStream_t s) {
  const int share = ((g.V + blocks - 1) / blocks + 7) / 8 * 8;
  return launch_cluster_following(token_rows_kernel<Z, POLICY, NT>, dim3(static_cast<unsigned>(g.T) * blocks), NT,
                                  blocks, 0, s, g, share);
}
template <class Z, bool POLICY>
cudaError_t launch_rows(const TokenRows& g, cudaStream_t s) {
  if (g.V <= 32 * kWarpChunks * kChunk<Z>)
    return launch_following(token_warp_kernel<Z, POLICY>, dim3((g.T + 3) / 4), 128, 0, s, g);
  const int blocks = row_blocks(g.T, g.V, sizeof(Z), POLICY);
  const int bytes = g.V / blocks * static_cast<int>(sizeof(Z));
  // About eight chunks a thread, so that the starts of many rows overlap (4127 rows of 10.5 KB: 256 threads 40 us with
  // the call, 128 35), and, without a second look, sixteen and more (128 KB rows: 1024 threads 127 us, 512 118).
  if (bytes <= 16 << 10) return launch_blocks<Z, POLICY, 128>(g, blocks, s);
  if (bytes <= 32 << 10) return launch_blocks<Z, POLICY, 256>(g, blocks, s);
  if constexpr (POLICY)
    if (bytes > 64 << 10) return launch_blocks<Z, POLICY, 1024>(g, blocks, s);
  return launch_blocks<Z, POLICY, 512>(g, blocks, s);
}

}  // namespace

cudaError_t token_logprobs(const void* logits, int type, int64_t ld, const int32_t* labels, float* logp, float* lse,
                           int T, int V, float scale, int* err, cudaStream_t s) {
  TokenRows g{};
  g.logits = logits, g.ld = ld, g.labels = labels, g.T = T, g.V = V, g.logp = logp, g.lse = lse;
  set_scale(g, scale);
  g.err = err;
  if (!rows_args_ok(g, type) || !vec_ok(logp, 4) || !vec_ok(lse, 4)) return cudaErrorInvalidValue;
  return type == kRowF32 ? launch_rows<float, false>(g, s) : launch_rows<bf16, false>(g, s);
}

cudaError_t token_logprobs_bwd(const void* logits, int type, int64_t ld, const int32_t* labels, const float* lse,
                               const float* dlogp, bf16* dlogits, int64_t ldd, int T, int V, float scale,
                               cudaStream_t s) {
  TokenRows g{};
  g.logits = logits, g.ld = ld, g.labels = labels, g.T = T, g.V = V;
  set_scale(g, scale);
  g.lse = const_cast<float*>(lse), g.dlogits = dlogits, g.ldd = ldd;
  if (!rows_args_ok(g, type) || !vec_ok(lse, 4) || !vec_ok(dlogp, 4) || !grad_ok(g, type)) return cudaErrorInvalidValue;
  auto* k = type == kRowF32 ? token_grad_kernel<float> : token_grad_kernel<bf16>;
  const int columns = kGradThreads * kGradChunks * (16 / row_type_bytes(type));
  for (int end = T; end > 0; end -= 65535) {
    TokenRows a = g;
    const int n = std::min(end, 65535), t = end - n;
    a.logits = static_cast<const char*>(logits) + t * ld * row_type_bytes(type);
    a.dlogits = dlogits + t * ldd;
    a.labels += t;
    a.lse += t;
    const cudaError_t e = launch_following(k, dim3((V + columns - 1) / columns, n), kGradThreads, 0, s, a,
                                           dlogp + t);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t policy_loss(const void* logits, int type, int64_t ld, const int32_t* labels, const float* old_logp,
                        const float* adv, const float* ref, const float* weights, float clip_low, float clip_high,
                        float kl, float scale, bf16* dlogits, int64_t ldd, float* logp, float* row_loss, float* loss,
                        int T, int V, int* err, cudaStream_t s) {
  TokenRows g{};
  g.logits = logits, g.ld = ld, g.labels = labels, g.T = T, g.V = V, g.logp = logp, g.err = err;
  g.old_logp = old_logp, g.adv = adv, g.ref = ref, g.weights = weights;
  g.clip_low = clip_low, g.clip_high = clip_high, g.kl = kl;
  g.dlogits = dlogits, g.ldd = ldd, g.row_loss = row_loss;
  set_scale(g, scale);
  if (!rows_args_ok(g, type) || !vec_ok(old_logp, 4) || !vec_ok(adv, 4) || !vec_ok(logp, 4) || !vec_ok(row_loss, 4) ||
      !vec_ok(loss, 4) || (weights && !vec_ok(weights, 4)) || (ref && !vec_ok(ref, 4)) || !grad_ok(g, type))
    return cudaErrorInvalidValue;
  if (!(clip_low >= 0.f && clip_low <= 1.f) || !(clip_high >= 0.f) || !std::isfinite(clip_high) || !(kl >= 0.f) ||
      !std::isfinite(kl) || (kl > 0.f && !ref))
    return cudaErrorInvalidValue;
  const cudaError_t e = type == kRowF32 ? launch_rows<float, true>(g, s) : launch_rows<bf16, true>(g, s);
  if (e != cudaSuccess) return e;
  return launch_following(sum_kernel, dim3(1), 1024, 0, s, row_loss, T, 1.f, loss);
}

cudaError_t preference_loss(const float* logp, const float* ref, const int32_t* labels, const int32_t* bounds,
                            int pairs, int T, int kind, float beta, float margin, float smoothing, bool average,
                            float* pair_loss, float* loss, float* rewards, float* dlogp, cudaStream_t s) {
  if (pairs <= 0 || pairs > kPreferenceMaxPairs || T <= 0 || T > kMaxRows || kind < MTK_PREF_SIGMOID ||
      kind > MTK_PREF_SQUARE || !(beta > 0.f) || !std::isfinite(beta) || !std::isfinite(margin) ||
      !(smoothing >= 0.f && smoothing <= 0.5f))
    return cudaErrorInvalidValue;
  if (!vec_ok(logp, 4) || (ref && !vec_ok(ref, 4)) || (labels && !vec_ok(labels, 4)) || !vec_ok(bounds, 4) ||
      !vec_ok(pair_loss, 4) || !vec_ok(loss, 4) || !vec_ok(rewards, 4) || !vec_ok(dlogp, 4))
    return cudaErrorInvalidValue;
  const Preference g{logp, ref, labels, bounds, pairs, T, kind, beta, margin, smoothing, average, pair_loss, rewards,
                     dlogp};
  if (T <= kFewRows && pairs <= kFewPairs)
    return launch_following(preference_few_kernel, dim3(1), 1024, 0, s, g, loss);
  const cudaError_t e = launch_following(preference_kernel, dim3(pairs + 1), 512, 0, s, g);
  if (e != cudaSuccess) return e;
  return launch_following(sum_kernel, dim3(1), 1024, 0, s, pair_loss, pairs, 1.f / static_cast<float>(pairs), loss);
}

}  // namespace mt
