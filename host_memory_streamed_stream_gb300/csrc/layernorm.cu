// Layer norm, forward and backward, on rows of fp32 or bf16.
//
//   mean = sum x / h,  rstd = 1 / sqrt(sum (x - mean)^2 / h + eps),  n = (x - mean) rstd,  y = n gamma + beta
//   u = dy gamma,  dx = dres + rstd (u - sum u / h - n sum(u n) / h),  dgamma = sum_t dy n,  dbeta = sum_t dy
//
// Bound by HBM: a row stays in the registers of its threads, so that every element is read once and the sum of squares
// is taken of centred values. Measured at 8192 x 4096: forward of fp32 rows 35.2 us, 5.7 TB/s (a cast of the same bytes
// takes 32), of bf16 ones 27 (20 for the bytes: four warps a scheduler, as 128 registers allow, fill half of its issue
// slots between the latencies of a row's steps); backward of fp32 rows with the residual's gradient 97.2 us, 6.2 TB/s
// with the gains' sums, of bf16 ones 50, 5.4 TB/s, bound by its instructions. At 8000 x 5120: forward 44 and 34 us,
// backward 138 (one block of 320 threads an SM; 110 for the bytes) and 66. One row of 5120: 3 us on the device.
#include <algorithm>
#include <cmath>

#include "follow.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace mt {

namespace {

// Threads hold 32 columns of a row each in the forward (16: 43.5 us instead of 35) and 16 in the backward (8: 141
// instead of 98), whose gains' sums take as many registers again; an SM holds 512 of them, with 128 registers each.
// Rows share a block in groups of whole warps. Arithmetic is in packed pairs: with scalar instructions these kernels
// are bound by issuing them (forward 43.5 us, of bf16 rows 35).
constexpr int kFwdCols = 32, kBwdCols = 16;
constexpr int kFwdThreads = 128, kBwdThreads = 256;  // of a block, at least
constexpr int kSmThreads = 512;
constexpr int kNormRing = 192 << 10;  // bytes of the rings on an SM

struct NormShape {
  int group, groups, blocks;  // threads a row, rows a block at a time, blocks on an SM
};
NormShape norm_shape(int cols, int each, int least) {
  NormShape n;
  n.group = ((cols + each - 1) / each + 31) / 32 * 32;
  n.groups = std::max(1, least / n.group);
  n.blocks = std::max(1, kSmThreads / (n.group * n.groups));
  return n;
}
// Rows that a block's ring holds.
int ring_stages(const NormShape& n, int row_bytes) {
  return std::max(1, std::min(4, kNormRing / n.blocks / row_bytes));
}

// A copy of W neighbouring columns, 8 or 16 bytes, into shared memory.
template <class T, int W>
__device__ __forceinline__ void copy_cols(void* dst, const T* src) {
  if constexpr (W * sizeof(T) == 16) cp_async_chunk(dst, src);
  else cp_async_half(dst, src);
}
// W columns as pairs.
template <class T, int W>
__device__ __forceinline__ void read_pairs(const T* p, float2* v) {
  float a[W];
  read_cols<T, W>(p, a);
#pragma unroll
  for (int j = 0; j < W / 2; ++j) v[j] = make_float2(a[2 * j], a[2 * j + 1]);
}
template <class T, int W>
__device__ __forceinline__ void write_pairs(T* p, const float2* v) {
  float a[W];
#pragma unroll
  for (int j = 0; j < W / 2; ++j) a[2 * j] = v[j].x, a[2 * j + 1] = v[j].y;
  write_cols<T, W>(p, a);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 unpacked(uint32_t p) {
  return make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u));
}

template <int N>
__device__ __forceinline__ void lane_sums(float* v, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}
// The threads of a group meet; `id` of its block.
__device__ __forceinline__ void group_sync(int id, int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(group) : "memory");
}
__device__ __forceinline__ int lanes_for(int warps) {
  return warps > 16 ? 32 : warps > 8 ? 16 : warps > 4 ? 8 : warps > 2 ? 4 : warps;
}

struct LnFwd {
  const void* x;
  int64_t ldx;
  const bf16 *gamma, *beta;
  bf16* y;
  int64_t ldy;
  float *mean, *rstd;
  int T, h, group, stages;
  float eps;
};

// Persistent blocks whose groups take rows in turn; each thread copies its columns of the rows ahead into its own part
// of a ring in shared memory, so that the loads go on through a row's sums. Mean and squares meet at one barrier: each
// warp sums the squares about its own mean, and what that leaves out is the warps' means about the row's.
template <class X>
__global__ void __launch_bounds__(kSmThreads) ln_fwd_kernel(const LnFwd g) {
  constexpr int W = 16 / sizeof(X), K = kFwdCols / W;
  extern __shared__ uint4 ring[];  // [stages][K][threads]
  __shared__ float4 meet[2][32];   // a warp's columns, mean and squares; two in turn
  const int id = threadIdx.x / g.group, at = threadIdx.x - id * g.group, groups = blockDim.x / g.group;
  const int lane = threadIdx.x & 31, warps = g.group >> 5, lanes = lanes_for(warps);
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t t = static_cast<int64_t>(blockIdx.x) * groups + id, ahead = t;
  wait_for_previous();
  let_next_start();
  auto slot = [&](int st, int k) { return ring + (st * K + k) * blockDim.x + threadIdx.x; };
  auto load = [&](int st) {
    if (ahead < g.T) {
      const X* x = static_cast<const X*>(g.x) + ahead * g.ldx;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (at + k * g.group) * W;
        if (c < g.h) cp_async_chunk(slot(st, k), x + c);
      }
      ahead += step;
    }
    cp_async_end_group();
  };
  for (int i = 0; i < g.stages; ++i) load(i);
  float2 gain[K][W / 2], bias[K][W / 2] = {};
  int mine = 0;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (at + k * g.group) * W;
    if (c >= g.h) break;
    mine += W;
    read_pairs<bf16, W>(g.gamma + c, gain[k]);
    if (g.beta) read_pairs<bf16, W>(g.beta + c, bias[k]);
  }
  const float count = static_cast<float>(__reduce_add_sync(0xffffffffu, mine));
  const float inv_count = count > 0.f ? 1.f / count : 0.f, inv_h = 1.f / static_cast<float>(g.h);
  int turn = 0, stage = 0;
  for (; t < g.T; t += step) {
    cp_async_wait_groups(g.stages - 1);
    float2 v[K][W / 2], part[2] = {};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k * W >= mine) break;
      read_pairs<X, W>(reinterpret_cast<const X*>(slot(stage, k)), v[k]);
#pragma unroll
      for (int j = 0; j < W / 2; ++j) part[j & 1] = __fadd2_rn(part[j & 1], v[k][j]);
    }
    load(stage);
    stage = stage + 1 == g.stages ? 0 : stage + 1;
    float mean = (part[0].x + part[0].y) + (part[1].x + part[1].y);
    lane_sums<1>(&mean, 32);
    mean *= inv_count;
    part[0] = part[1] = both(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k * W >= mine) break;
#pragma unroll
      for (int j = 0; j < W / 2; ++j) {
        const float2 d = __fadd2_rn(v[k][j], both(-mean));
        part[j & 1] = __ffma2_rn(d, d, part[j & 1]);
      }
    }
    float squares = (part[0].x + part[0].y) + (part[1].x + part[1].y);
    lane_sums<1>(&squares, 32);
    if (warps > 1) {
      if (lane == 0) meet[turn][threadIdx.x >> 5] = make_float4(count, mean, squares, 0.f);
      group_sync(id, g.group);
      const int w = lane & (lanes - 1);
      const float4 q = w < warps ? meet[turn][id * warps + w] : make_float4(0.f, 0.f, 0.f, 0.f);
      mean = q.x * q.y;
      lane_sums<1>(&mean, lanes);
      mean *= inv_h;
      squares = q.z + q.x * (q.y - mean) * (q.y - mean);
      lane_sums<1>(&squares, lanes);
      turn ^= 1;
    }
    const float r = rsqrtf(squares * inv_h + g.eps);
    if (at == 0) {
      g.mean[t] = mean;
      g.rstd[t] = r;
    }
    bf16* y = g.y + t * g.ldy;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k * W >= mine) break;
#pragma unroll
      for (int j = 0; j < W / 2; ++j) {
        const float2 n = __fmul2_rn(__fadd2_rn(v[k][j], both(-mean)), both(r));
        v[k][j] = __ffma2_rn(n, gain[k][j], bias[k][j]);
      }
      write_pairs<bf16, W>(y + (at + k * g.group) * W, v[k]);
    }
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

// The same with dy, x and dres of a row in the ring; dy n and dy add up in registers over a block's rows. dres is read
// after the sums, when registers are free again (before them: 101.8 us, and 69.6 for bf16 rows). Rows wider than 512
// threads hold are shared by two blocks of a cluster (CL = 2), by columns. FULL: a row has
// a multiple of 512 columns, so that no thread tests its own; for bf16 x and dy, bound by instructions (8192 x 4096:
// 55.9 us with the tests, 49.4 without; of fp32 97.1 and 100.8).
template <class X, class D, int CL, bool FULL>
__global__ void __launch_bounds__(kSmThreads) ln_bwd_kernel(const LnBwd g) {
  constexpr int W = sizeof(X) == 4 || sizeof(D) == 4 ? 4 : 8, K = kBwdCols / W;
  constexpr int BX = W * sizeof(X), BD = W * sizeof(D);
  extern __shared__ __align__(16) char bwd_ring[];  // [stages][dy, x, dres][K][threads]; at the end [groups - 1][2][h]
  __shared__ float2 meet[2][32], halves[2][2];
  const unsigned rank = CL > 1 ? cluster_rank() : 0;
  const int groups = blockDim.x / g.group, id = threadIdx.x / g.group, at = threadIdx.x - id * g.group;
  const int lane = threadIdx.x & 31, warps = g.group >> 5, lanes = lanes_for(warps);
  const int c0 = static_cast<int>(rank) * g.share, cols = CL > 1 ? min(g.share, g.h - c0) : g.h;
  const int64_t step = static_cast<int64_t>(gridDim.x / CL) * groups;
  const float inv_h = 1.f / static_cast<float>(g.h);
  const X* x = static_cast<const X*>(g.x) + c0;
  const D* dy = static_cast<const D*>(g.dy) + c0;
  const X* res = g.dres ? static_cast<const X*>(g.dres) + c0 : nullptr;
  int turn = 0, stage = 0, half_turn = 0;
  int64_t t = static_cast<int64_t>(blockIdx.x / CL) * groups + id, ahead = t;
  if constexpr (CL > 1) cluster_arrive();
  wait_for_previous();
  let_next_start();
  auto slot = [&](int st, int bytes_before, int bytes, int k) {
    return bwd_ring + st * g.stage_bytes + (bytes_before * K) * blockDim.x + (k * blockDim.x + threadIdx.x) * bytes;
  };
  auto load = [&](int st) {  // dy and x of the row ahead, whose slots are read first
    if (ahead >= g.T) return;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (at + k * g.group) * W;
      if (FULL || c < cols) {
        copy_cols<D, W>(slot(st, 0, BD, k), dy + ahead * g.lddy + c);
        copy_cols<X, W>(slot(st, BD, BX, k), x + ahead * g.ldx + c);
      }
    }
  };
  auto load_rest = [&](int st) {
    if (ahead < g.T) {
      if (res) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int c = (at + k * g.group) * W;
          if (FULL || c < cols) copy_cols<X, W>(slot(st, BD + BX, BX, k), res + ahead * g.lddres + c);
        }
      }
      ahead += step;
    }
    cp_async_end_group();
  };
  for (int i = 0; i < g.stages; ++i) {
    load(i);
    load_rest(i);
  }
  uint32_t gain[K][W / 2];
  float2 dg[K][W / 2] = {}, db[K][W / 2] = {};
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (at + k * g.group) * W;
    if (!FULL && c >= cols) break;
#pragma unroll
    for (int j = 0; j < W / 2; ++j) gain[k][j] = reinterpret_cast<const uint32_t*>(g.gamma + c0 + c)[j];
  }
  float r = 0.f, mean = 0.f;
  if (t < g.T) r = g.rstd[t], mean = g.mean[t];
  if constexpr (CL > 1) cluster_wait();  // both have started
  for (; t < g.T; t += step) {
    cp_async_wait_groups(g.stages - 1);
    float2 n[K][W / 2], u[K][W / 2], sum[2] = {};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!FULL && (at + k * g.group) * W >= cols) break;
      read_pairs<D, W>(reinterpret_cast<const D*>(slot(stage, 0, BD, k)), u[k]);
      read_pairs<X, W>(reinterpret_cast<const X*>(slot(stage, BD, BX, k)), n[k]);
    }
    load(stage);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!FULL && (at + k * g.group) * W >= cols) break;
#pragma unroll
      for (int j = 0; j < W / 2; ++j) {
        n[k][j] = __fmul2_rn(__fadd2_rn(n[k][j], both(-mean)), both(r));
        dg[k][j] = __ffma2_rn(u[k][j], n[k][j], dg[k][j]);
        db[k][j] = __fadd2_rn(db[k][j], u[k][j]);
        u[k][j] = __fmul2_rn(u[k][j], unpacked(gain[k][j]));
        sum[0] = __fadd2_rn(sum[0], u[k][j]);
        sum[1] = __ffma2_rn(u[k][j], n[k][j], sum[1]);
      }
    }
    float s[2] = {sum[0].x + sum[0].y, sum[1].x + sum[1].y};
    const float rt = r;
    if (t + step < g.T) r = g.rstd[t + step], mean = g.mean[t + step];
    lane_sums<2>(s, 32);
    if (warps > 1) {
      if (lane == 0) meet[turn][threadIdx.x >> 5] = make_float2(s[0], s[1]);
      group_sync(id, g.group);
      const int w = lane & (lanes - 1);
      const float2 q = w < warps ? meet[turn][id * warps + w] : make_float2(0.f, 0.f);
      s[0] = q.x, s[1] = q.y;
      lane_sums<2>(s, lanes);
      turn ^= 1;
    }
    if constexpr (CL > 1) {
      if (threadIdx.x < CL) {
        uint32_t a;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(a)
                     : "r"(smem_addr(&halves[half_turn][rank])), "r"(threadIdx.x));
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(s[0]), "f"(s[1]) : "memory");
      }
      cluster_sync();
      s[0] = halves[half_turn][0].x + halves[half_turn][1].x;
      s[1] = halves[half_turn][0].y + halves[half_turn][1].y;
      half_turn ^= 1;
    }
    const float2 a0 = both(-s[0] * inv_h), a1 = both(-s[1] * inv_h);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (at + k * g.group) * W;
      if (!FULL && c >= cols) break;
      float2 d[W / 2];
      if (res) read_pairs<X, W>(reinterpret_cast<const X*>(slot(stage, BD + BX, BX, k)), d);
#pragma unroll
      for (int j = 0; j < W / 2; ++j) {
        u[k][j] = __ffma2_rn(n[k][j], a1, __fadd2_rn(u[k][j], a0));
        u[k][j] = res ? __ffma2_rn(u[k][j], both(rt), d[j]) : __fmul2_rn(u[k][j], both(rt));
      }
      write_pairs<X, W>(static_cast<X*>(g.dx) + t * g.h + c0 + c, u[k]);
      if (g.dx_bf16) write_pairs<bf16, W>(g.dx_bf16 + t * g.h + c0 + c, u[k]);
    }
    load_rest(stage);
    stage = stage + 1 == g.stages ? 0 : stage + 1;
  }
  if constexpr (CL > 1) cluster_sync();  // no block ends while the other may write its half here
  float* out = g.partial + static_cast<int64_t>(blockIdx.x / CL) * 2 * g.h + c0;
  float2* other = reinterpret_cast<float2*>(bwd_ring);  // [groups - 1][2][h / 2]
  if (groups > 1) {
    cp_async_wait_groups(0);
    __syncthreads();  // the ring is free
    if (id > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (at + k * g.group) * W;
        if (!FULL && c >= cols) break;
#pragma unroll
        for (int j = 0; j < W / 2; ++j) {
          other[(id - 1) * g.h + c / 2 + j] = dg[k][j];
          other[(id - 1) * g.h + (g.h + c) / 2 + j] = db[k][j];
        }
      }
    }
    __syncthreads();
    if (id > 0) return;
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (at + k * g.group) * W;
    if (!FULL && c >= cols) break;
    for (int o = 0; o < groups - 1; ++o)
#pragma unroll
      for (int j = 0; j < W / 2; ++j) {
        dg[k][j] = __fadd2_rn(dg[k][j], other[o * g.h + c / 2 + j]);
        db[k][j] = __fadd2_rn(db[k][j], other[o * g.h + (g.h + c) / 2 + j]);
      }
#pragma unroll
    for (int j = 0; j < W / 2; j += 2) {
      *reinterpret_cast<float4*>(out + c + 2 * j) = make_float4(dg[k][j].x, dg[k][j].y, dg[k][j + 1].x, dg[k][j + 1].y);
      *reinterpret_cast<float4*>(out + g.h + c + 2 * j) =
          make_float4(db[k][j].x, db[k][j].y, db[k][j + 1].x, db[k][j + 1].y);
    }
  }
}

// dgamma and dbeta: the blocks' sums added in a fixed order, 32 columns a block, each warp a part of the sums (304 x 2
// x 4096 cold: 8 us, with 128 columns a block 11).
constexpr int kGainWarps = 16;
__global__ void __launch_bounds__(32 * kGainWarps) ln_gain_kernel(const float* partial, int parts, int h, bf16* dgamma,
                                                                  bf16* dbeta) {
  __shared__ float acc[kGainWarps][33];
  wait_for_previous();
  let_next_start();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, j = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (j < 2 * h) {
#pragma unroll 10
    for (int p = w; p < parts; p += kGainWarps) s += partial[static_cast<int64_t>(p) * 2 * h + j];
  }
  acc[w][lane] = s;
  __syncthreads();
  if (w == 0 && j < 2 * h) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < kGainWarps; ++k) s += acc[k][lane];
    bf16* out = j < h ? dgamma + j : dbeta ? dbeta + j - h : nullptr;
    if (out) *out = __float2bfloat16_rn(s);
  }
}

template <class X>
cudaError_t launch_fwd(LnFwd g, cudaStream_t s) {
  const NormShape n = norm_shape(g.h, kFwdCols, kFwdThreads);
  const int threads = n.group * n.groups, row = threads * kFwdCols * static_cast<int>(sizeof(X));
  g.group = n.group;
  g.stages = ring_stages(n, row);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(ln_fwd_kernel<X>, kNormRing, done);
  if (e != cudaSuccess) return e;
  return launch_following(ln_fwd_kernel<X>, dim3(std::min((g.T + n.groups - 1) / n.groups, kSms * n.blocks)), threads,
                          g.stages * row, s, g);
}

struct BwdShape {
  NormShape n;
  int cluster, share;  // blocks of a row, and columns of each
};
BwdShape bwd_shape(int h) {
  const int cluster = h > kSmThreads * kBwdCols ? 2 : 1;
  const int share = cluster > 1 ? (h / 2 + 7) / 8 * 8 : h;
  return {norm_shape(share, kBwdCols, kBwdThreads), cluster, share};
}
template <class X, class D>
cudaError_t launch_bwd(LnBwd g, const BwdShape& b, int parts, cudaStream_t s) {
  const int threads = b.n.group * b.n.groups;
  const int row = threads * kBwdCols * static_cast<int>(sizeof(D) + sizeof(X) * (g.dres ? 2 : 1));
  g.stages = ring_stages(b.n, row);
  g.stage_bytes = row;
  // at the end the ring holds the sums of all groups but one
  const int smem = std::max(g.stages * row, (b.n.groups - 1) * 2 * g.h * 4);
  auto* k = b.cluster > 1 ? ln_bwd_kernel<X, D, 2, false> : ln_bwd_kernel<X, D, 1, false>;
  int which = b.cluster > 1;
  if constexpr (sizeof(X) == 2 && sizeof(D) == 2)
    if (b.cluster == 1 && g.h == b.n.group * kBwdCols) k = ln_bwd_kernel<X, D, 1, true>, which = 2;
  static std::atomic<uint64_t> done[3];
  const cudaError_t e = allow_shared(k, kNormRing, done[which]);
  if (e != cudaSuccess) return e;
  return launch_cluster_following(k, dim3(parts * b.cluster), threads, b.cluster, smem, s, g);
}

bool ln_shape_ok(int T, int h) { return T > 0 && T <= kMaxRows && h > 0 && h % 8 == 0 && h <= kLayerNormMaxWidth; }

}  // namespace

cudaError_t layernorm_fwd(const void* x, int type, int64_t ldx, const bf16* gamma, const bf16* beta, bf16* y,
                          int64_t ldy, float* mean, float* rstd, int T, int h, float eps, cudaStream_t s) {
  if (!row_type_ok(type) || !ln_shape_ok(T, h) || !rows_ok(x, ldx, h) || !rows_ok(y, ldy, h) || !vec_ok(gamma, 16) ||
      (beta && !vec_ok(beta, 16)) || !vec_ok(mean, 4) || !vec_ok(rstd, 4) || !(eps >= 0.f) || std::isinf(eps) ||
      spans_overlap(x, ldx, row_type_bytes(type), y, ldy, 2, T, h))
    return cudaErrorInvalidValue;
  return type == kRowF32 ? launch_fwd<float>({x, ldx, gamma, beta, y, ldy, mean, rstd, T, h, 0, 0, eps}, s)
                         : launch_fwd<bf16>({x, ldx, gamma, beta, y, ldy, mean, rstd, T, h, 0, 0, eps}, s);
}

int layernorm_bwd_parts(int T, int h) {
  if (!ln_shape_ok(T, h)) return 0;
  const BwdShape b = bwd_shape(h);
  return std::min((T + b.n.groups - 1) / b.n.groups, kSms * b.n.blocks / b.cluster);
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
  const BwdShape b = bwd_shape(h);
  const int parts = layernorm_bwd_parts(T, h);
  const LnBwd g{dy, lddy, x, ldx, gamma, mean, rstd, dres, lddres, dx, dx_bf16, partial, T, h, b.n.group, 0, 0,
                b.share};
  cudaError_t e;
  if (type == kRowF32)
    e = dy_type == kRowF32 ? launch_bwd<float, float>(g, b, parts, s)
                           : launch_bwd<float, bf16>(g, b, parts, s);
  else
    e = dy_type == kRowF32 ? launch_bwd<bf16, float>(g, b, parts, s)
                           : launch_bwd<bf16, bf16>(g, b, parts, s);
  if (e != cudaSuccess) return e;
  return launch_following(ln_gain_kernel, dim3((2 * h + 31) / 32), 32 * kGainWarps, 0, s, partial, parts, h, dgamma,
                          dbeta);
}

}  // namespace mt
