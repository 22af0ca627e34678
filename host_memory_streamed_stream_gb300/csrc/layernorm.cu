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

constexpr int kNormCols = 16;      // columns a thread holds of a row
constexpr int kNormThreads = 256;  // at least so many threads a block, in groups of whole warps that share a row

struct NormShape {
  int group, groups;  // threads a row, rows a block at a time
};
NormShape norm_shape(int cols) {
  const int group = ((cols + kNormCols - 1) / kNormCols + 31) / 32 * 32;
  return {group, std::max(1, kNormThreads / group)};
}

// A copy of W neighbouring columns, 8 or 16 bytes, into shared memory.
template <class T, int W>
__device__ __forceinline__ void copy_cols(void* dst, const T* src) {
  if constexpr (W * sizeof(T) == 16) cp_async_chunk(dst, src);
  else cp_async_half(dst, src);
}

// Sums over the threads of a row, N values at a time: shuffles and, where the row has several warps, shared memory
// (two copies in turn, so that one barrier a sum is enough). Every thread adds the warps' sums in the same order.
template <int N>
struct RowSum {
  float red[2][32][N];
};
template <int N>
__device__ __forceinline__ void row_sum(float* v, RowSum<N>& s, int& turn, int group, int id) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (group == 32) return;
  const int warps = group >> 5, first = id * warps;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) s.red[turn][threadIdx.x >> 5][i] = v[i];
  asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(group) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int w = first; w < first + warps; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += s.red[turn][w][i];
  turn ^= 1;
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

// A group a row, with its columns in registers. MAX threads a block at most; the smaller kind leaves room for six blocks
// on an SM, whose rows overlap.
template <class X, int MAX>
__global__ void __launch_bounds__(MAX, MAX == kNormThreads ? 6 : 1) ln_fwd_kernel(const LnFwd g) {
  constexpr int W = 16 / sizeof(X), K = kNormCols / W;
  __shared__ RowSum<1> sums;
  const int id = threadIdx.x / g.group, at = threadIdx.x - id * g.group;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / g.group) + id;
  if (t >= g.T) return;  // a whole group
  const X* x = static_cast<const X*>(g.x) + t * g.ldx;
  const float inv_h = 1.f / static_cast<float>(g.h);
  int turn = 0;
  uint4 raw[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (at + k * g.group) * W;
    if (c < g.h) raw[k] = *reinterpret_cast<const uint4*>(x + c);
  }
  float v[K][W], s = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if ((at + k * g.group) * W >= g.h) break;
    read_cols<X, W>(reinterpret_cast<const X*>(&raw[k]), v[k]);
#pragma unroll
    for (int j = 0; j < W; ++j) s += v[k][j];
  }
  row_sum<1>(&s, sums, turn, g.group, id);
  const float mean = s * inv_h;
  s = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if ((at + k * g.group) * W >= g.h) break;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      v[k][j] -= mean;
      s += v[k][j] * v[k][j];
    }
  }
  row_sum<1>(&s, sums, turn, g.group, id);
  const float r = rsqrtf(s * inv_h + g.eps);
  if (at == 0) {
    g.mean[t] = mean;
    g.rstd[t] = r;
  }
  bf16* y = g.y + t * g.ldy;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (at + k * g.group) * W;
    if (c >= g.h) break;
    float a[W], b[W] = {};
    read_cols<bf16, W>(g.gamma + c, a);
    if (g.beta) read_cols<bf16, W>(g.beta + c, b);
#pragma unroll
    for (int j = 0; j < W; ++j) v[k][j] = v[k][j] * r * a[j] + b[j];
    write_cols<bf16, W>(y + c, v[k]);
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
  int T, h, group, stages, stage_bytes, share;
};

// Persistent blocks whose groups take rows in turn; each thread copies its columns of the rows ahead into its own part
// of a ring in shared memory, so that the loads go on through a row's sums. dy n and dy add up in registers. Rows wider than 512 threads hold are shared by two blocks of a cluster (CL = 2), by columns.
template <class X, class D, int CL>
__global__ void __launch_bounds__(512) ln_bwd_kernel(const LnBwd g) {
  constexpr int W = sizeof(X) == 4 || sizeof(D) == 4 ? 4 : 8, K = kNormCols / W;
  constexpr int BX = W * sizeof(X), BD = W * sizeof(D);
  extern __shared__ __align__(16) char bwd_ring[];  // [stages][dy, x, dres][K][threads]; at the end [groups - 1][2][h]
  __shared__ RowSum<2> sums;
  __shared__ float2 halves[2][2];
  const unsigned rank = CL > 1 ? cluster_rank() : 0;
  const int groups = blockDim.x / g.group, id = threadIdx.x / g.group, at = threadIdx.x - id * g.group;
  const int c0 = static_cast<int>(rank) * g.share, cols = CL > 1 ? min(g.share, g.h - c0) : g.h;
  const int64_t step = static_cast<int64_t>(gridDim.x / CL) * groups;
  const float inv_h = 1.f / static_cast<float>(g.h);
  const X* x = static_cast<const X*>(g.x) + c0;
  const D* dy = static_cast<const D*>(g.dy) + c0;
  const X* res = g.dres ? static_cast<const X*>(g.dres) + c0 : nullptr;
  int turn = 0, stage = 0, half_turn = 0;
  int64_t t = static_cast<int64_t>(blockIdx.x / CL) * groups + id, ahead = t;
  auto slot = [&](int st, int bytes_before, int bytes, int k) {
    return bwd_ring + st * g.stage_bytes + (bytes_before * K) * blockDim.x + (k * blockDim.x + threadIdx.x) * bytes;
  };
  auto load = [&](int st) {
    if (ahead < g.T) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (at + k * g.group) * W;
        if (c < cols) {
          copy_cols<D, W>(slot(st, 0, BD, k), dy + ahead * g.lddy + c);
          copy_cols<X, W>(slot(st, BD, BX, k), x + ahead * g.ldx + c);
          if (res) copy_cols<X, W>(slot(st, BD + BX, BX, k), res + ahead * g.lddres + c);
        }
      }
      ahead += step;
    }
    cp_async_end_group();
  };
  for (int i = 0; i < g.stages; ++i) load(i);
  uint32_t gain[K][W / 2];
  float dg[K][W] = {}, db[K][W] = {};
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (at + k * g.group) * W;
    if (c >= cols) break;
#pragma unroll
    for (int j = 0; j < W / 2; ++j) gain[k][j] = reinterpret_cast<const uint32_t*>(g.gamma + c0 + c)[j];
  }
  float r = 0.f, mean = 0.f;
  if (t < g.T) r = g.rstd[t], mean = g.mean[t];
  for (; t < g.T; t += step) {
    cp_async_wait_groups(g.stages - 1);
    float n[K][W], u[K][W], d[K][W], s[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if ((at + k * g.group) * W >= cols) break;
      read_cols<D, W>(reinterpret_cast<const D*>(slot(stage, 0, BD, k)), u[k]);
      read_cols<X, W>(reinterpret_cast<const X*>(slot(stage, BD, BX, k)), n[k]);
      if (res) read_cols<X, W>(reinterpret_cast<const X*>(slot(stage, BD + BX, BX, k)), d[k]);
    }
    load(stage);
    stage = stage + 1 == g.stages ? 0 : stage + 1;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if ((at + k * g.group) * W >= cols) break;
      float gk[W];
#pragma unroll
      for (int j = 0; j < W / 2; ++j) unpack2(gain[k][j], gk + 2 * j);
#pragma unroll
      for (int j = 0; j < W; ++j) {
        n[k][j] = (n[k][j] - mean) * r;
        dg[k][j] += u[k][j] * n[k][j];
        db[k][j] += u[k][j];
        u[k][j] *= gk[j];
        s[0] += u[k][j];
        s[1] += u[k][j] * n[k][j];
      }
    }
    const float rt = r;
    if (t + step < g.T) r = g.rstd[t + step], mean = g.mean[t + step];
    row_sum<2>(s, sums, turn, g.group, id);
    if constexpr (CL > 1) {
      if (threadIdx.x < CL) {
        uint32_t a;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(&halves[half_turn][rank])), "r"(threadIdx.x));
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(s[0]), "f"(s[1]) : "memory");
      }
      cluster_sync();
      s[0] = halves[half_turn][0].x + halves[half_turn][1].x;
      s[1] = halves[half_turn][0].y + halves[half_turn][1].y;
      half_turn ^= 1;
    }
    const float a0 = s[0] * inv_h, a1 = s[1] * inv_h;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (at + k * g.group) * W;
      if (c >= cols) break;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        u[k][j] = rt * (u[k][j] - a0 - n[k][j] * a1);
        if (res) u[k][j] += d[k][j];
      }
      write_cols<X, W>(static_cast<X*>(g.dx) + t * g.h + c0 + c, u[k]);
      if (g.dx_bf16) write_cols<bf16, W>(g.dx_bf16 + t * g.h + c0 + c, u[k]);
    }
  }
  if constexpr (CL > 1) cluster_sync();  // no block ends while the other may write its half here
  float* out = g.partial + static_cast<int64_t>(blockIdx.x / CL) * 2 * g.h + c0;
  if (groups > 1) {
    cp_async_wait_groups(0);
    __syncthreads();  // the ring is free
    float* other = reinterpret_cast<float*>(bwd_ring);
    if (id > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (at + k * g.group) * W;
        if (c >= cols) break;
#pragma unroll
        for (int j = 0; j < W; ++j) {
          other[2 * (id - 1) * g.h + c + j] = dg[k][j];
          other[(2 * id - 1) * g.h + c + j] = db[k][j];
        }
      }
    }
    __syncthreads();
    if (id > 0) return;
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (at + k * g.group) * W;
    if (c >= cols) break;
    if (groups > 1) {
      const float* other = reinterpret_cast<const float*>(bwd_ring);
      for (int o = 0; o < groups - 1; ++o)
#pragma unroll
        for (int j = 0; j < W; ++j) {
          dg[k][j] += other[2 * o * g.h + c + j];
          db[k][j] += other[(2 * o + 1) * g.h + c + j];
        }
    }
#pragma unroll
    for (int j = 0; j < W; j += 4) {
      *reinterpret_cast<float4*>(out + c + j) = make_float4(dg[k][j], dg[k][j + 1], dg[k][j + 2], dg[k][j + 3]);
      *reinterpret_cast<float4*>(out + g.h + c + j) = make_float4(db[k][j], db[k][j + 1], db[k][j + 2], db[k][j + 3]);
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

constexpr int kNormRing = 192 << 10;  // bytes of the rings on an SM

struct BwdShape {
  int group, groups, cluster, blocks, share;  // blocks on an SM; columns of a block of the cluster
};
BwdShape bwd_shape(int h) {
  const int cluster = h > 512 * kNormCols ? 2 : 1;
  const int share = cluster > 1 ? (h / 2 + 7) / 8 * 8 : h;
  const NormShape n = norm_shape(share);
  return {n.group, n.groups, cluster, n.group * n.groups > kNormThreads ? 1 : 2, share};
}
template <class X, class D>
cudaError_t launch_bwd(const LnBwd& g, const BwdShape& n, int parts, int threads, int smem, cudaStream_t s) {
  auto* k = n.cluster > 1 ? ln_bwd_kernel<X, D, 2> : ln_bwd_kernel<X, D, 1>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {static_cast<unsigned>(n.cluster), 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(parts * n.cluster);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = n.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k, g);
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
  const int threads = n.group * n.groups;
  const LnFwd g{x, ldx, gamma, beta, y, ldy, mean, rstd, T, h, n.group, eps};
  auto* k = threads <= kNormThreads ? (type == kRowF32 ? ln_fwd_kernel<float, kNormThreads> : ln_fwd_kernel<bf16, kNormThreads>)
                                    : (type == kRowF32 ? ln_fwd_kernel<float, 1024> : ln_fwd_kernel<bf16, 1024>);
  k<<<(T + n.groups - 1) / n.groups, threads, 0, s>>>(g);
  return cudaGetLastError();
}

int layernorm_bwd_parts(int T, int h) {
  if (!ln_shape_ok(T, h)) return 0;
  const BwdShape n = bwd_shape(h);
  return std::min((T + n.groups - 1) / n.groups, kSms * n.blocks / n.cluster);
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
  const BwdShape n = bwd_shape(h);
  const int threads = n.group * n.groups, parts = layernorm_bwd_parts(T, h);
  const int row = threads * kNormCols * (row_type_bytes(dy_type) + esz * (dres ? 2 : 1));
  const int stages = std::max(1, std::min(4, kNormRing / n.blocks / row));
  // at the end the ring holds the sums of all groups but one
  const int smem = std::max(stages * row, (n.groups - 1) * 2 * h * 4);
  const LnBwd g{dy, lddy, x, ldx, gamma, mean, rstd, dres, lddres, dx, dx_bf16, partial, T, h, n.group, stages, row,
                n.share};
  cudaError_t e;
  if (type == kRowF32)
    e = dy_type == kRowF32 ? launch_bwd<float, float>(g, n, parts, threads, smem, s)
                           : launch_bwd<float, bf16>(g, n, parts, threads, smem, s);
  else
    e = dy_type == kRowF32 ? launch_bwd<bf16, float>(g, n, parts, threads, smem, s)
                           : launch_bwd<bf16, bf16>(g, n, parts, threads, smem, s);
  if (e != cudaSuccess) return e;
  return launch_following(ln_gain_kernel, dim3((2 * h + 31) / 32), 512, 0, s, partial, parts, h, dgamma, dbeta);
}

}  // namespace mt
