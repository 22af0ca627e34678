// Embedding lookup with a scale, and the gradient of the table by sorted tokens.
//
//   x_t = scale E[tok_t],   dE[v] = scale sum over t with tok_t = v of dx_t   (negative ids: padding, no gradient)
//
// Gradient: one cluster sorts the (token, row) pairs stably while the other blocks write zeros to the rows of the table
// that no token uses; then the sorted rows are summed by chunks of equal length, however long a token's run is: a run
// inside a chunk goes straight to the table, one that crosses a border leaves fp32 sums that a last
// kernel adds in order. No floating-point atomics: the result does not change from run to run.
#include <algorithm>
#include <cmath>

#include "follow.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace mt {

namespace {

// ------------------------------------------------------------------ lookup
// A thread takes eight columns of a token; consecutive threads consecutive columns.
template <class X>
__global__ void __launch_bounds__(256) lookup_kernel(const int32_t* tok, const bf16* E, X* x, int T, int h, int V,
                                                     float scale, int* err) {
  const int units = h / 8;
  const int64_t total = static_cast<int64_t>(T) * units, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += step) {
    const int64_t t = i / units;
    const int c = static_cast<int>(i - t * units) * 8;
    const int v = tok[t];
    float a[8] = {};
    if (v >= 0 && v < V) {
      unpack8(load8(E + static_cast<int64_t>(v) * h + c), a);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] *= scale;
    } else if (v >= V && c == 0) {
      record_bad_token(err);
    }
    store8(x + t * h + c, a);
  }
}

// ------------------------------------------------------------------ sort
constexpr int kSortBlocks = 8;     // one cluster, the largest that is portable
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortBits = 9;       // of a digit at most: 16 x 512 counters a block
constexpr int kSortBins = 1 << kSortBits;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// *p of block `rank` of this cluster.
__device__ __forceinline__ int cluster_load(const int* p, int rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

struct SortArgs {
  const int32_t* tok;
  int2 *a, *b;  // pairs (token or V, row): the passes go from one to the other
  int T, V, passes, bits;
  bf16* dE;
  int64_t h;
  bool zero;
  int* err;
};

// Least significant digit first. Each warp of the cluster owns T / 128 consecutive pairs and counts their digits;
// the place of a digit's first pair of a warp is the sum of what comes before it in (digit, block, warp) order, which
// keeps equal digits in order.
__device__ void sort_pairs(const SortArgs& g, int (*count)[kSortBins], int* total, int* base, int* warp_sum) {
  const int rank = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bins = 1 << g.bits;
  const int each = (g.T + kSortBlocks * kSortWarps - 1) / (kSortBlocks * kSortWarps);
  const int64_t first = static_cast<int64_t>(rank * kSortWarps + warp) * each;
  const int lo = static_cast<int>(first < g.T ? first : g.T), hi = min(g.T, lo + each);
  for (int pass = 0; pass < g.passes; ++pass) {
    const int2* src = pass & 1 ? g.a : g.b;
    int2* dst = pass & 1 ? g.b : g.a;
    const int shift = pass * g.bits;
    auto pair = [&](int i) {
      if (pass > 0) return __ldcg(src + i);
      int v = g.tok[i];
      if (v >= g.V) record_bad_token(g.err);
      return make_int2(v < 0 || v >= g.V ? g.V : v, i);
    };
    for (int i = threadIdx.x; i < kSortWarps * kSortBins; i += kSortThreads) count[0][i] = 0;
    __syncthreads();
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      const unsigned active = __ballot_sync(0xffffffffu, i < hi);
      if (i < hi) {
        const int d = pair(i).x >> shift & (bins - 1);
        const unsigned same = __match_any_sync(active, d);
        if (lane == __ffs(same) - 1) count[warp][d] += __popc(same);
      }
      __syncwarp();
    }
    __syncthreads();
    // per digit: exclusive sums over the block's warps, and the block's total
    for (int d = threadIdx.x; d < bins; d += kSortThreads) {
      int s = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = count[w][d];
        count[w][d] = s;
        s += c;
      }
      total[d] = s;
    }
    cluster_sync();
    // what comes before this block's pairs of a digit: those of smaller digits, and of lower blocks
    const int d = threadIdx.x;  // bins <= kSortThreads
    int below = 0, all = 0;
    if (d < bins)
#pragma unroll
      for (int r = 0; r < kSortBlocks; ++r) {
        const int c = cluster_load(total + d, r);
        below += r < rank ? c : 0;
        all += c;
      }
    int s = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += v;
    }
    if (lane == 31) warp_sum[warp] = s;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    if (d < bins) base[d] = before + s - all + below;
    __syncthreads();
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      const unsigned active = __ballot_sync(0xffffffffu, i < hi);
      if (i < hi) {
        const int2 p = pair(i);
        const int k = p.x >> shift & (bins - 1);
        const unsigned same = __match_any_sync(active, k);
        const int at = base[k] + count[warp][k] + __popc(same & ((1u << lane) - 1));
        dst[at] = p;
        __syncwarp(active);
        if (lane == __ffs(same) - 1) count[warp][k] += __popc(same);
      }
      __syncwarp();
    }
    cluster_sync();  // pairs written, totals read
  }
}

__global__ void __cluster_dims__(kSortBlocks, 1, 1) __launch_bounds__(kSortThreads) sort_kernel(const SortArgs g) {
  __shared__ int count[kSortWarps][kSortBins];
  __shared__ int total[kSortBins], base[kSortBins], warp_sum[kSortWarps];
  wait_for_previous();
  let_next_start();
  if (blockIdx.x < kSortBlocks) {
    sort_pairs(g, count, total, base, warp_sum);
    return;
  }
  // the other clusters: zeros in the rows of this block's share of the table that no token uses
  const int blocks = gridDim.x - kSortBlocks, b = blockIdx.x - kSortBlocks;
  const int v0 = static_cast<int>(static_cast<int64_t>(g.V) * b / blocks);
  const int v1 = static_cast<int>(static_cast<int64_t>(g.V) * (b + 1) / blocks);
  unsigned* used = reinterpret_cast<unsigned*>(count);  // a bit for each row: 2^18 of them
  const int units = static_cast<int>(g.h / 8);
  for (int r0 = v0; r0 < v1; r0 += 32 * kSortWarps * kSortBins) {
    const int r1 = min(v1, r0 + 32 * kSortWarps * kSortBins);
    __syncthreads();
    for (int i = threadIdx.x; i < (r1 - r0 + 31) / 32; i += kSortThreads) used[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < g.T; i += kSortThreads) {
      const int v = g.tok[i];
      if (v >= r0 && v < r1) atomicOr(used + (v - r0) / 32, 1u << ((v - r0) & 31));
    }
    __syncthreads();
    for (int r = r0 + (threadIdx.x >> 5); r < r1; r += kSortWarps) {
      if (used[(r - r0) / 32] >> ((r - r0) & 31) & 1) continue;
      uint4* row = reinterpret_cast<uint4*>(g.dE + r * g.h);
      for (int i = threadIdx.x & 31; i < units; i += 32) row[i] = make_uint4(0, 0, 0, 0);
    }
  }
}

// ------------------------------------------------------------------ sums of runs
constexpr int kSumThreads = 128;  // of eight columns each: 1024 columns a block

struct SumArgs {
  const int2* pairs;
  const void* dx;
  bf16* dE;
  float* partial;  // [chunks][2][h]: a run from the chunk before (0), one that goes on into the next (1)
  int T, V, h, chunk;
  float scale;
  bool add;
};
__device__ __forceinline__ void write_row(const SumArgs& g, int v, int c, const float* acc) {
  bf16* p = g.dE + static_cast<int64_t>(v) * g.h + c;
  float out[8], old[8] = {};
  if (g.add) unpack8(load8(p), old);
#pragma unroll
  for (int j = 0; j < 8; ++j) out[j] = fmaf(acc[j], g.scale, old[j]);
  store8(p, out);
}

template <class X>
__global__ void __launch_bounds__(kSumThreads) run_sum_kernel(const SumArgs g) {
  wait_for_previous();
  let_next_start();
  const int c = (blockIdx.y * kSumThreads + threadIdx.x) * 8;
  if (c >= g.h) return;
  const int p0 = blockIdx.x * g.chunk, p1 = min(g.T, p0 + g.chunk);
  const X* dx = static_cast<const X*>(g.dx);
  float acc[8] = {}, a[8];
  int cur = __ldcg(&g.pairs[p0].x);
  if (cur == g.V) return;
  bool from_before = p0 > 0 && __ldcg(&g.pairs[p0 - 1].x) == cur;
  for (int p = p0; p < p1; ++p) {
    const int2 q = __ldcg(g.pairs + p);
    if (q.x != cur) {
      if (from_before) store8(g.partial + static_cast<int64_t>(blockIdx.x) * 2 * g.h + c, acc);
      else write_row(g, cur, c, acc);
      from_before = false;
      cur = q.x;
      if (cur == g.V) return;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    }
    unpack8(load8(dx + static_cast<int64_t>(q.y) * g.h + c), a);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += a[j];
  }
  const bool goes_on = p1 < g.T && __ldcg(&g.pairs[p1].x) == cur;
  if (from_before) store8(g.partial + static_cast<int64_t>(blockIdx.x) * 2 * g.h + c, acc);
  else if (goes_on) store8(g.partial + (static_cast<int64_t>(blockIdx.x) * 2 + 1) * g.h + c, acc);
  else write_row(g, cur, c, acc);
}

// The runs that cross a border: one block for each chunk in which such a run begins.
__global__ void __launch_bounds__(kSumThreads) run_join_kernel(const SumArgs g) {
  wait_for_previous();
  const int c = (blockIdx.y * kSumThreads + threadIdx.x) * 8;
  if (c >= g.h) return;
  const int p0 = blockIdx.x * g.chunk;
  int64_t end = static_cast<int64_t>(p0) + g.chunk;
  if (end >= g.T) return;
  const int cur = __ldcg(&g.pairs[end - 1].x);
  if (cur == g.V || __ldcg(&g.pairs[end].x) != cur) return;           // no run goes on
  if (p0 > 0 && __ldcg(&g.pairs[p0 - 1].x) == cur) return;            // it began in an earlier chunk
  const float* part = g.partial + (static_cast<int64_t>(blockIdx.x) * 2 + 1) * g.h + c;
  float acc[8], a[8];
  unpack8(load8(part), acc);
  for (int k = blockIdx.x + 1; end < g.T && __ldcg(&g.pairs[end].x) == cur; ++k, end += g.chunk) {
    unpack8(load8(g.partial + static_cast<int64_t>(k) * 2 * g.h + c), a);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += a[j];
  }
  write_row(g, cur, c, acc);
}

bool embed_shape_ok(int T, int V, int h) {
  return T > 0 && T <= kEmbedMaxTokens && V > 0 && V <= kEmbedMaxVocab && h > 0 && h % 8 == 0 && h <= kEmbedMaxWidth;
}
uint64_t table_bytes(int V, int h) { return static_cast<uint64_t>(V) * h * sizeof(bf16); }
// Sorted rows a block sums.
int sum_chunk(int T) { return T <= 4096 ? 16 : T <= 32768 ? 32 : 128; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

cudaError_t embed_lookup(const int32_t* tok, const bf16* E, void* x, int type, int T, int h, int V, float scale,
                         int* err, cudaStream_t s) {
  if (!row_type_ok(type) || !embed_shape_ok(T, V, h) || !vec_ok(tok, 4) || !vec_ok(E, 16) || !vec_ok(x, 16) ||
      (err && !vec_ok(err, 4)) || !std::isfinite(scale) ||
      ranges_overlap(E, table_bytes(V, h), x, static_cast<uint64_t>(T) * h * row_type_bytes(type)))
    return cudaErrorInvalidValue;
  const int64_t blocks = (static_cast<int64_t>(T) * (h / 8) + 255) / 256;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(blocks, kSms * 16));
  if (type == kRowF32)
    lookup_kernel<float><<<grid, 256, 0, s>>>(tok, E, static_cast<float*>(x), T, h, V, scale, err);
  else
    lookup_kernel<bf16><<<grid, 256, 0, s>>>(tok, E, static_cast<bf16*>(x), T, h, V, scale, err);
  return cudaGetLastError();
}

uint64_t embed_lookup_bwd_scratch(int T, int h) {
  const int chunk = sum_chunk(T);
  const size_t chunks = (T + chunk - 1) / chunk;
  return 2 * round256(static_cast<size_t>(T) * sizeof(int2)) + chunks * 2 * h * sizeof(float);
}

cudaError_t embed_lookup_bwd(const int32_t* tok, const void* dx, int type, bf16* dE, void* scratch, int T, int h,
                             int V, float scale, bool add, int* err, cudaStream_t s) {
  if (!row_type_ok(type) || !embed_shape_ok(T, V, h) || !vec_ok(tok, 4) || !vec_ok(dx, 16) || !vec_ok(dE, 16) ||
      !vec_ok(scratch, 16) || (err && !vec_ok(err, 4)) || !std::isfinite(scale))
    return cudaErrorInvalidValue;
  const uint64_t table = table_bytes(V, h), rows = static_cast<uint64_t>(T) * h * row_type_bytes(type);
  if (ranges_overlap(dE, table, dx, rows) || ranges_overlap(dE, table, scratch, embed_lookup_bwd_scratch(T, h)) ||
      ranges_overlap(dx, rows, scratch, embed_lookup_bwd_scratch(T, h)))
    return cudaErrorInvalidValue;
  int bits = 1;
  while ((V >> bits) > 0) ++bits;  // of the keys 0 .. V
  const int passes = (bits + kSortBits - 1) / kSortBits;
  char* at = static_cast<char*>(scratch);
  int2* a = reinterpret_cast<int2*>(at);
  int2* b = reinterpret_cast<int2*>(at + round256(static_cast<size_t>(T) * sizeof(int2)));
  float* partial = reinterpret_cast<float*>(at + 2 * round256(static_cast<size_t>(T) * sizeof(int2)));
  const SortArgs g{tok, a, b, T, V, passes, (bits + passes - 1) / passes, dE, h, !add, err};
  const unsigned blocks = add ? kSortBlocks : kSortBlocks + 2 * kSms / kSortBlocks * kSortBlocks;
  cudaError_t e = launch_following(sort_kernel, dim3(blocks), kSortThreads, 0, s, g);
  if (e != cudaSuccess) return e;
  const int chunk = sum_chunk(T);
  const SumArgs r{passes & 1 ? a : b, dx, dE, partial, T, V, h, chunk, scale, add};
  const dim3 grid((T + chunk - 1) / chunk, (h / 8 + kSumThreads - 1) / kSumThreads);
  e = launch_following(type == kRowF32 ? run_sum_kernel<float> : run_sum_kernel<bf16>, grid, kSumThreads, 0, s, r);
  if (e != cudaSuccess) return e;
  return launch_following(run_join_kernel, grid, kSumThreads, 0, s, r);
}

}  // namespace mt
