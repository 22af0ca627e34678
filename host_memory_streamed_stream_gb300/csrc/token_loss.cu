// Log-probabilities of given tokens and the losses on them: the clipped policy loss with a KL term, forward and
// backward in one pass over the logits, and the preference loss over pairs of sequences.
//
//   lse_t = log sum_v exp(a z_tv),  logp_t = a z_t,label - lse_t,  dlogits_tv = a dlogp_t ([v = label] - p_tv)
//
// Sums of exponentials run in fp32 against a running maximum, as powers of two (c = a log2 e). The maximum is
// subtracted before the product with c, which keeps masks of the type's lowest value in range. The label's
// logit, the maximum and the logarithm meet in 64 bits: a ratio of policies is exp of a small difference of
// numbers of size 10, of which fp32 would lose 2^-21.
#include <cmath>

#include "follow.cuh"
#include "kernels.h"
#include "mt_kernels.h"
#include "rows.cuh"

namespace mt {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr double kLn2 = 0.6931471805599453;

__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Running maximum and sum of 2^(c (z - max)). max = -inf: nothing but -inf so far, sum 0.
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ MaxSum merge(const MaxSum& a, const MaxSum& b, float c) {
  const float m = fmaxf(a.m, b.m);
  const float mm = m == -INFINITY ? 0.f : m;
  return {m, a.s * pow2((a.m - mm) * c) + b.s * pow2((b.m - mm) * c)};
}
template <int N>
__device__ __forceinline__ void add_terms(MaxSum& r, const float* z, float c) {
  float top = z[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, z[i]);
  if (top > r.m) {
    r.s *= pow2((r.m - top) * c);
    r.m = top;
  }
  const float m = r.m == -INFINITY ? 0.f : r.m;
#pragma unroll
  for (int i = 0; i < N; ++i) r.s += pow2((z[i] - m) * c);
}

// log2 of a sum of exponentials, to 2^-24 of its fraction rather than of its size.
__device__ __forceinline__ double log2_split(float s) {
  int e;
  const float f = frexpf(s, &e);
  return static_cast<double>(e) + static_cast<double>(log2f(f));
}

struct TokenRows {
  const void* logits;
  int64_t ld;
  const int32_t* labels;
  int T, V;
  float scale;
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

// What one row's label gives: its log-probability, and for the policy loss the row's loss and d loss / d logp.
template <bool POLICY>
__device__ __forceinline__ float finish_row(const TokenRows& g, int t, float z_label, const MaxSum& r) {
  const float c = g.scale * kLog2e;
  const double log2_sum = log2_split(r.s);
  const double logp = ((static_cast<double>(z_label) - r.m) * c - log2_sum) * kLn2;
  g.logp[t] = static_cast<float>(logp);
  if constexpr (!POLICY) {
    g.lse[t] = static_cast<float>((static_cast<double>(r.m) * c + log2_sum) * kLn2);
    return 0.f;
  } else {
    const float w = g.weights ? g.weights[t] : 1.f / static_cast<float>(g.T);
    const float adv = g.adv[t];
    const float ratio = expf(static_cast<float>(logp - static_cast<double>(g.old_logp[t])));
    const float lo = 1.f - g.clip_low, hi = 1.f + g.clip_high;
    // comparisons rather than fminf, which would drop a NaN
    const float cut = ratio < lo ? lo : ratio > hi ? hi : ratio;
    const bool held = ratio * adv > cut * adv;
    float loss = held ? -cut * adv : -ratio * adv;
    float d = held ? 0.f : -ratio * adv;
    if (g.kl != 0.f) {
      const float far = static_cast<float>(static_cast<double>(g.ref[t]) - logp);
      const float em1 = expm1f(far);
      loss += g.kl * (em1 - far);
      d -= g.kl * em1;
    }
    g.row_loss[t] = w * loss;
    return w * d;
  }
}

// One block a row: maximum and sum over the row, then, for the policy loss, the row once more (from the L2)
// for its gradient.
template <class Z, bool POLICY>
__global__ void __launch_bounds__(512) token_rows_kernel(const TokenRows g) {
  __shared__ MaxSum part[16];
  __shared__ float shared_k, shared_m, shared_inv;
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const Z* z = static_cast<const Z*>(g.logits) + t * g.ld;
  bf16* d = POLICY ? g.dlogits + t * g.ldd : nullptr;
  const int label = g.labels[t], whole = g.V & ~7;
  if (label < 0 || label >= g.V) {  // nothing of the row is read
    if (threadIdx.x == 0) {
      if (label >= g.V) record_bad_token(g.err);
      g.logp[t] = 0.f;
      if (POLICY) g.row_loss[t] = 0.f;
      else g.lse[t] = 0.f;
    }
    if constexpr (POLICY) {
      for (int i = threadIdx.x * 8; i < whole; i += blockDim.x * 8)
        *reinterpret_cast<uint4*>(d + i) = make_uint4(0, 0, 0, 0);
      for (int i = whole + threadIdx.x; i < g.V; i += blockDim.x) d[i] = __float2bfloat16_rn(0.f);
    }
    return;
  }
  const float c = g.scale * kLog2e;
  MaxSum r{-INFINITY, 0.f};
  float v[8];
  for (int i = threadIdx.x * 8; i < whole; i += blockDim.x * 8) {
    unpack8(load8(z + i), v);
    add_terms<8>(r, v, c);
  }
  for (int i = whole + threadIdx.x; i < g.V; i += blockDim.x) {
    v[0] = to_f32(z[i]);
    add_terms<1>(r, v, c);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    r = merge(r, {__shfl_xor_sync(0xffffffffu, r.m, o), __shfl_xor_sync(0xffffffffu, r.s, o)}, c);
  if (lane == 0) part[warp] = r;
  __syncthreads();
  if (warp == 0) {
    r = lane < warps ? part[lane] : MaxSum{-INFINITY, 0.f};
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
      r = merge(r, {__shfl_xor_sync(0xffffffffu, r.m, o), __shfl_xor_sync(0xffffffffu, r.s, o)}, c);
    if (lane == 0) {
      shared_k = finish_row<POLICY>(g, t, to_f32(z[label]), r) * g.scale;
      shared_m = r.m == -INFINITY ? 0.f : r.m;
      shared_inv = 1.f / r.s;
    }
  }
  if constexpr (POLICY) {
    __syncthreads();
    const float k = shared_k, m = shared_m, kp = -k * shared_inv;
    for (int i = threadIdx.x * 8; i < whole; i += blockDim.x * 8) {
      unpack8(load8(z + i), v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = kp * pow2((v[j] - m) * c) + (i + j == label ? k : 0.f);
      store8(d + i, v);
    }
    for (int i = whole + threadIdx.x; i < g.V; i += blockDim.x)
      d[i] = __float2bfloat16_rn(kp * pow2((to_f32(z[i]) - m) * c) + (i == label ? k : 0.f));
  }
}

// dlogits of given dlogp and lse: a pass over the logits.
template <class Z>
__global__ void __launch_bounds__(256) token_grad_kernel(const TokenRows g, const float* dlogp) {
  const int t = blockIdx.y;
  const Z* z = static_cast<const Z*>(g.logits) + t * g.ld;
  bf16* d = g.dlogits + t * g.ldd;
  const int label = g.labels[t], whole = g.V & ~7;
  const bool on = label >= 0 && label < g.V;
  const float k = on ? dlogp[t] * g.scale : 0.f;
  const float lse = on ? g.lse[t] : 0.f;
  const int stride = gridDim.x * blockDim.x, first = blockIdx.x * blockDim.x + threadIdx.x;
  for (int i = first * 8; i < whole; i += stride * 8) {
    float v[8] = {};
    if (on) {
      unpack8(load8(z + i), v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = -k * pow2(fmaf(v[j], g.scale, -lse) * kLog2e) + (i + j == label ? k : 0.f);
    }
    store8(d + i, v);
  }
  for (int i = whole + first; i < g.V; i += stride)
    d[i] = __float2bfloat16_rn(on ? -k * pow2(fmaf(to_f32(z[i]), g.scale, -lse) * kLog2e) + (i == label ? k : 0.f) : 0.f);
}

// out = sum of v[0..n) times f, in 64 bits and a fixed order.
__global__ void __launch_bounds__(1024) sum_kernel(const float* v, int n, double f, float* out) {
  __shared__ double red[32];
  wait_for_previous();
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) s += static_cast<double>(v[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) s += red[i];
    *out = static_cast<float>(s * f);
  }
}

__device__ float block_total(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) v += red[i];
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

// One block a pair: the sums of its two sequences, its loss, and its rows' dlogp. The last block zeroes the rows
// of no sequence.
__global__ void __launch_bounds__(512) preference_kernel(const Preference g) {
  __shared__ float red[16];
  wait_for_previous();
  let_next_start();
  auto bound = [&](int j) { return min(max(g.bounds[j], 0), g.T); };
  const int p = blockIdx.x;
  if (p == g.pairs) {
    const int first = bound(0), last = max(first, bound(2 * g.pairs));
    for (int i = threadIdx.x; i < first; i += blockDim.x) g.dlogp[i] = 0.f;
    for (int i = last + threadIdx.x; i < g.T; i += blockDim.x) g.dlogp[i] = 0.f;
    return;
  }
  float s[2], share[2];
  int lo[2], hi[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    lo[j] = bound(2 * p + j);
    hi[j] = bound(2 * p + j + 1);
    float v = 0.f, n = 0.f;
    for (int i = lo[j] + threadIdx.x; i < hi[j]; i += blockDim.x) {
      if (g.labels && g.labels[i] < 0) continue;
      v += g.ref ? g.logp[i] - g.ref[i] : g.logp[i];
      n += 1.f;
    }
    v = block_total(v, red);
    n = g.average ? block_total(n, red) : 1.f;
    share[j] = 1.f / fmaxf(n, 1.f);
    s[j] = v * share[j];
  }
  const float h = g.beta * (s[0] - s[1]) - g.margin;
  float loss, d;
  if (g.kind == MTK_PREF_SIGMOID) {
    const float e = expf(-fabsf(h)), l = log1pf(e);  // softplus(-|h|)
    loss = l + (h > 0.f ? g.smoothing * h : (g.smoothing - 1.f) * h);
    d = g.smoothing - (h > 0.f ? e : 1.f) / (1.f + e);
  } else if (g.kind == MTK_PREF_HINGE) {
    loss = 1.f - h > 0.f ? 1.f - h : 0.f * h;
    d = h < 1.f ? -1.f : 0.f * h;
  } else {
    const float u = (h - 0.5f) / g.beta;
    loss = u * u;
    d = 2.f * u / g.beta;
  }
  if (threadIdx.x == 0) {
    g.pair_loss[p] = loss;
    g.rewards[2 * p] = g.beta * s[0];
    g.rewards[2 * p + 1] = g.beta * s[1];
  }
  const float k = g.beta * d / static_cast<float>(g.pairs);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float kj = (j ? -k : k) * share[j];
    for (int i = lo[j] + threadIdx.x; i < hi[j]; i += blockDim.x)
      g.dlogp[i] = g.labels && g.labels[i] < 0 ? 0.f : kj;
  }
}

bool rows_args_ok(const TokenRows& g, int type) {
  return row_type_ok(type) && g.T > 0 && g.V > 0 && rows_ok(g.logits, g.ld, g.V) && vec_ok(g.labels, 4) &&
         std::isfinite(g.scale) && g.scale > 0.f && (!g.err || vec_ok(g.err, 4));
}
// The gradient's rows: apart from the logits', or the bf16 logits themselves.
bool grad_ok(const TokenRows& g, int type) {
  if (!rows_ok(g.dlogits, g.ldd, g.V)) return false;
  if (type == kRowBf16 && g.dlogits == g.logits) return g.ldd == g.ld;
  return !spans_overlap(g.logits, g.ld, row_type_bytes(type), g.dlogits, g.ldd, 2, g.T, g.V);
}
unsigned row_threads(int V) { return V <= 1024 ? 128 : V <= 8192 ? 256 : 512; }

}  // namespace

cudaError_t token_logprobs(const void* logits, int type, int64_t ld, const int32_t* labels, float* logp, float* lse,
                           int T, int V, float scale, int* err, cudaStream_t s) {
  TokenRows g{};
  g.logits = logits, g.ld = ld, g.labels = labels, g.T = T, g.V = V, g.scale = scale, g.logp = logp, g.lse = lse;
  g.err = err;
  if (!rows_args_ok(g, type) || !vec_ok(logp, 4) || !vec_ok(lse, 4)) return cudaErrorInvalidValue;
  auto* k = type == kRowF32 ? token_rows_kernel<float, false> : token_rows_kernel<bf16, false>;
  k<<<T, row_threads(V), 0, s>>>(g);
  return cudaGetLastError();
}

cudaError_t token_logprobs_bwd(const void* logits, int type, int64_t ld, const int32_t* labels, const float* lse,
                               const float* dlogp, bf16* dlogits, int64_t ldd, int T, int V, float scale,
                               cudaStream_t s) {
  TokenRows g{};
  g.logits = logits, g.ld = ld, g.labels = labels, g.T = T, g.V = V, g.scale = scale;
  g.lse = const_cast<float*>(lse), g.dlogits = dlogits, g.ldd = ldd;
  if (!rows_args_ok(g, type) || !vec_ok(lse, 4) || !vec_ok(dlogp, 4) || !grad_ok(g, type)) return cudaErrorInvalidValue;
  auto* k = type == kRowF32 ? token_grad_kernel<float> : token_grad_kernel<bf16>;
  for (int t = 0; t < T; t += 65535) {
    TokenRows a = g;
    const int n = T - t < 65535 ? T - t : 65535;
    a.logits = static_cast<const char*>(logits) + t * ld * row_type_bytes(type);
    a.dlogits = dlogits + t * ldd;
    a.labels += t;
    a.lse += t;
    k<<<dim3((V + 4095) / 4096, n), 256, 0, s>>>(a, dlogp + t);
  }
  return cudaGetLastError();
}

cudaError_t policy_loss(const void* logits, int type, int64_t ld, const int32_t* labels, const float* old_logp,
                        const float* adv, const float* ref, const float* weights, float clip_low, float clip_high,
                        float kl, float scale, bf16* dlogits, int64_t ldd, float* logp, float* row_loss, float* loss,
                        int T, int V, int* err, cudaStream_t s) {
  const TokenRows g{logits, ld, labels, T, V, scale, logp, nullptr, old_logp, adv, ref, weights, clip_low, clip_high,
                    kl, dlogits, ldd, row_loss, err};
  if (!rows_args_ok(g, type) || !vec_ok(old_logp, 4) || !vec_ok(adv, 4) || !vec_ok(logp, 4) || !vec_ok(row_loss, 4) ||
      !vec_ok(loss, 4) || (weights && !vec_ok(weights, 4)) || (ref && !vec_ok(ref, 4)) || !grad_ok(g, type))
    return cudaErrorInvalidValue;
  if (!(clip_low >= 0.f && clip_low <= 1.f) || !(clip_high >= 0.f) || !std::isfinite(clip_high) || !(kl >= 0.f) ||
      !std::isfinite(kl) || (kl > 0.f && !ref))
    return cudaErrorInvalidValue;
  auto* k = type == kRowF32 ? token_rows_kernel<float, true> : token_rows_kernel<bf16, true>;
  k<<<T, row_threads(V), 0, s>>>(g);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_following(sum_kernel, dim3(1), 1024, 0, s, row_loss, T, 1.0, loss);
}

cudaError_t preference_loss(const float* logp, const float* ref, const int32_t* labels, const int32_t* bounds,
                            int pairs, int T, int kind, float beta, float margin, float smoothing, bool average,
                            float* pair_loss, float* loss, float* rewards, float* dlogp, cudaStream_t s) {
  if (pairs <= 0 || pairs > kPreferenceMaxPairs || T <= 0 || kind < MTK_PREF_SIGMOID || kind > MTK_PREF_SQUARE ||
      !(beta > 0.f) || !std::isfinite(beta) || !std::isfinite(margin) || !(smoothing >= 0.f && smoothing <= 0.5f))
    return cudaErrorInvalidValue;
  if (!vec_ok(logp, 4) || (ref && !vec_ok(ref, 4)) || (labels && !vec_ok(labels, 4)) || !vec_ok(bounds, 4) ||
      !vec_ok(pair_loss, 4) || !vec_ok(loss, 4) || !vec_ok(rewards, 4) || !vec_ok(dlogp, 4))
    return cudaErrorInvalidValue;
  const Preference g{logp, ref, labels, bounds, pairs, T, kind, beta, margin, smoothing, average, pair_loss, rewards,
                     dlogp};
  const cudaError_t e = launch_following(preference_kernel, dim3(pairs + 1), 512, 0, s, g);
  if (e != cudaSuccess) return e;
  return launch_following(sum_kernel, dim3(1), 1024, 0, s, pair_loss, pairs, 1.0 / pairs, loss);
}

}  // namespace mt
