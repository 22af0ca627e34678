// Layer norm, forward and backward, on rows of fp32 or bf16.
//
//   mean = sum x / h,  rstd = 1 / sqrt(sum (x - mean)^2 / h + eps),  n = (x - mean) rstd,  y = n gamma + beta
//   u = dy gamma,  dx = dres + rstd (u - sum u / h - n sum(u n) / h),  dgamma = sum_t dy n,  dbeta = sum_t dy
//
// Bound by HBM: a row stays in the registers of its threads, so that every element is read once and the sum of
// squares is taken of centred values.
#include <algorithm>
#include <cmath>

#include "follow.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace mt {

namespace {

constexpr int kUnits = 2;        // units of eight columns a thread holds of a row
constexpr int kNormThreads = 256;  // at least so many threads a block, in groups of whole warps that share a row

struct NormShape {
  int group, groups;  // threads a row, rows a block at a time
};
NormShape norm_shape(int h) {
  const int units = h / 8;
  const int group = ((units + kUnits - 1) / kUnits + 31) / 32 * 32;
  return {group, std::max(1, kNormThreads / group)};
}

// Sums over the threads of a row: N values at a time through shuffles and, where the row has several warps, shared
// memory. `red`: N floats a warp of the block. Every thread adds the warps' sums in the same order.
template <int N>
__device__ __forceinline__ void row_sum(float* v, float* red, int group, int id) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (group == 32) return;
  const int warps = group >> 5, first = id * warps;
  auto sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(group) : "memory"); };
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[(threadIdx.x >> 5) * N + i] = v[i];
  sync();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int w = first; w < first + warps; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += red[w * N + i];
  sync();
}

struct LnFwd {
  const void* x;
  int64_t ldx;
  const bf16 *gamma, *beta;
  bf16* y;
  int64_t ldy;
  float *mean, *rstd;
  int T, h, group;
  float eps;
};

template <class X>
__global__ void __launch_bounds__(1024) ln_fwd_kernel(const LnFwd g) {
  __shared__ float red[32];
  const int id = threadIdx.x / g.group, at = threadIdx.x - id * g.group;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / g.group) + id;
  if (t >= g.T) return;  // a whole group
  const X* x = static_cast<const X*>(g.x) + t * g.ldx;
  float v[kUnits][8], s = 0.f;
  Raw8<X> raw[kUnits];
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int c = (at + k * g.group) * 8;
    if (c < g.h) raw[k] = load8(x + c);
  }
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int c = (at + k * g.group) * 8;
    if (c >= g.h) break;
    unpack8(raw[k], v[k]);
#pragma unroll
    for (int j = 0; j < 8; ++j) s += v[k][j];
  }
  const float inv_h = 1.f / static_cast<float>(g.h);
  row_sum<1>(&s, red, g.group, id);
  const float mean = s * inv_h;
  s = 0.f;
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    if ((at + k * g.group) * 8 >= g.h) break;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[k][j] -= mean;
      s += v[k][j] * v[k][j];
    }
  }
  row_sum<1>(&s, red, g.group, id);
  const float r = rsqrtf(s * inv_h + g.eps);
  if (at == 0) {
    g.mean[t] = mean;
    g.rstd[t] = r;
  }
  bf16* y = g.y + t * g.ldy;
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int c = (at + k * g.group) * 8;
    if (c >= g.h) break;
    float a[8], b[8] = {};
    unpack8(load8(g.gamma + c), a);
    if (g.beta) unpack8(load8(g.beta + c), b);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[k][j] = v[k][j] * r * a[j] + b[j];
    store8(y + c, v[k]);
  }
}

struct LnBwd {
  const void* dy;
  int64_t lddy;
  const void* x;
  int64_t ldx;
  const bf16* gamma;
  const float *mean, *rstd;
  const void* dres;
  int64_t lddres;
  void* dx;
  bf16* dx_bf16;
  float* partial;  // [blocks][2][h]
  int T, h, group;
};

// Each block takes the rows blockIdx + k gridDim (by groups), and adds dy n and dy of its rows in registers.
template <class X, class D>
__global__ void __launch_bounds__(1024) ln_bwd_kernel(const LnBwd g) {
  extern __shared__ float sums[];  // [groups - 1][2][h]
  __shared__ float red[64];
  const int groups = blockDim.x / g.group, id = threadIdx.x / g.group, at = threadIdx.x - id * g.group;
  float dg[kUnits][8] = {}, db[kUnits][8] = {};
  const float inv_h = 1.f / static_cast<float>(g.h);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * groups + id; t < g.T;
       t += static_cast<int64_t>(gridDim.x) * groups) {
    const X* x = static_cast<const X*>(g.x) + t * g.ldx;
    const D* dy = static_cast<const D*>(g.dy) + t * g.lddy;
    const float r = g.rstd[t], mean = g.mean[t];
    float n[kUnits][8], u[kUnits][8], s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int c = (at + k * g.group) * 8;
      if (c >= g.h) break;
      float a[8];
      unpack8(load8(x + c), n[k]);
      unpack8(load8(dy + c), u[k]);
      unpack8(load8(g.gamma + c), a);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[k][j] = (n[k][j] - mean) * r;
        dg[k][j] += u[k][j] * n[k][j];
        db[k][j] += u[k][j];
        u[k][j] *= a[j];
        s[0] += u[k][j];
        s[1] += u[k][j] * n[k][j];
      }
    }
    row_sum<2>(s, red, g.group, id);
    const float a0 = s[0] * inv_h, a1 = s[1] * inv_h;
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int c = (at + k * g.group) * 8;
      if (c >= g.h) break;
#pragma unroll
      for (int j = 0; j < 8; ++j) u[k][j] = r * (u[k][j] - a0 - n[k][j] * a1);
      if (g.dres) {
        float d[8];
        unpack8(load8(static_cast<const X*>(g.dres) + t * g.lddres + c), d);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[k][j] += d[j];
      }
      store8(static_cast<X*>(g.dx) + t * g.h + c, u[k]);
      if (g.dx_bf16) store8(g.dx_bf16 + t * g.h + c, u[k]);
    }
  }
  float* out = g.partial + static_cast<int64_t>(blockIdx.x) * 2 * g.h;
  if (id > 0) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int c = (at + k * g.group) * 8;
      if (c >= g.h) break;
      store8(sums + (2 * (id - 1)) * g.h + c, dg[k]);
      store8(sums + (2 * (id - 1) + 1) * g.h + c, db[k]);
    }
  }
  __syncthreads();
  if (id == 0) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int c = (at + k * g.group) * 8;
      if (c >= g.h) break;
      for (int o = 0; o < groups - 1; ++o)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dg[k][j] += sums[2 * o * g.h + c + j];
          db[k][j] += sums[(2 * o + 1) * g.h + c + j];
        }
      store8(out + c, dg[k]);
      store8(out + g.h + c, db[k]);
    }
  }
}

// dgamma and dbeta: the blocks' sums added in a fixed order, 32 columns a block.
__global__ void __launch_bounds__(512) ln_gain_kernel(const float* partial, int parts, int h, bf16* dgamma,
                                                      bf16* dbeta) {
  __shared__ float acc[16][33];
  wait_for_previous();
  const int c = threadIdx.x & 31, w = threadIdx.x >> 5, j = blockIdx.x * 32 + c;
  float s = 0.f;
  if (j < 2 * h)
    for (int p = w; p < parts; p += 16) s += partial[static_cast<int64_t>(p) * 2 * h + j];
  acc[w][c] = s;
  __syncthreads();
  if (w == 0 && j < 2 * h) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += acc[k][c];
    bf16* out = j < h ? dgamma + j : dbeta ? dbeta + j - h : nullptr;
    if (out) *out = __float2bfloat16_rn(s);
  }
}

bool ln_shape_ok(int T, int h) { return T > 0 && h > 0 && h % 8 == 0 && h <= kLayerNormMaxWidth; }

}  // namespace

cudaError_t layernorm_fwd(const void* x, int type, int64_t ldx, const bf16* gamma, const bf16* beta, bf16* y,
                          int64_t ldy, float* mean, float* rstd, int T, int h, float eps, cudaStream_t s) {
  if (!row_type_ok(type) || !ln_shape_ok(T, h) || !rows_ok(x, ldx, h) || !rows_ok(y, ldy, h) || !vec_ok(gamma, 16) ||
      (beta && !vec_ok(beta, 16)) || !vec_ok(mean, 4) || !vec_ok(rstd, 4) || !(eps >= 0.f) || std::isinf(eps) ||
      spans_overlap(x, ldx, row_type_bytes(type), y, ldy, 2, T, h))
    return cudaErrorInvalidValue;
  const NormShape n = norm_shape(h);
  const LnFwd g{x, ldx, gamma, beta, y, ldy, mean, rstd, T, h, n.group, eps};
  auto* k = type == kRowF32 ? ln_fwd_kernel<float> : ln_fwd_kernel<bf16>;
  k<<<(T + n.groups - 1) / n.groups, n.group * n.groups, 0, s>>>(g);
  return cudaGetLastError();
}

int layernorm_bwd_parts(int T, int h) {
  if (!ln_shape_ok(T, h)) return 0;
  const NormShape n = norm_shape(h);
  return std::min((T + n.groups - 1) / n.groups, 2 * kSms);
}

cudaError_t layernorm_bwd(const void* dy, int dy_type, int64_t lddy, const void* x, int type, int64_t ldx,
                          const bf16* gamma, const float* mean, const float* rstd, const void* dres, int64_t lddres,
                          void* dx, bf16* dx_bf16, float* partial, bf16* dgamma, bf16* dbeta, int T, int h,
                          cudaStream_t s) {
  if (!row_type_ok(type) || !row_type_ok(dy_type) || !ln_shape_ok(T, h) || !rows_ok(dy, lddy, h) ||
      !rows_ok(x, ldx, h) || (dres && !rows_ok(dres, lddres, h)) || !vec_ok(dx, 16) ||
      (dx_bf16 && (!vec_ok(dx_bf16, 16) || type != kRowF32)) || !vec_ok(gamma, 16) || !vec_ok(mean, 4) ||
      !vec_ok(rstd, 4) || !vec_ok(partial, 16) || !vec_ok(dgamma, 2) || (dbeta && !vec_ok(dbeta, 2)))
    return cudaErrorInvalidValue;
  const int esz = row_type_bytes(type);
  const void* outs[2] = {dx, dx_bf16};
  for (int i = 0; i < 2; ++i) {
    const int e = i ? 2 : esz;
    if (!outs[i]) continue;
    const bool same = dres == outs[i] && lddres == h && i == 0;  // added to in place
    if (spans_overlap(outs[i], h, e, x, ldx, esz, T, h) ||
        spans_overlap(outs[i], h, e, dy, lddy, row_type_bytes(dy_type), T, h) ||
        (dres && !same && spans_overlap(outs[i], h, e, dres, lddres, esz, T, h)))
      return cudaErrorInvalidValue;
  }
  if (dx_bf16 && spans_overlap(dx, h, esz, dx_bf16, h, 2, T, h)) return cudaErrorInvalidValue;
  const NormShape n = norm_shape(h);
  const LnBwd g{dy, lddy, x, ldx, gamma, mean, rstd, dres, lddres, dx, dx_bf16, partial, T, h, n.group};
  const int parts = layernorm_bwd_parts(T, h);
  const size_t smem = static_cast<size_t>(n.groups - 1) * 2 * h * 4;  // below 28 KB: more groups only for narrow rows
  auto* k = type == kRowF32 ? (dy_type == kRowF32 ? ln_bwd_kernel<float, float> : ln_bwd_kernel<float, bf16>)
                            : (dy_type == kRowF32 ? ln_bwd_kernel<bf16, float> : ln_bwd_kernel<bf16, bf16>);
  k<<<parts, n.group * n.groups, smem, s>>>(g);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_following(ln_gain_kernel, dim3((2 * h + 31) / 32), 512, 0, s, partial, parts, h, dgamma, dbeta);
}

}  // namespace mt
