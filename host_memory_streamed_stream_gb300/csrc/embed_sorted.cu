// Embedding lookup with a scale, and the gradient of the table by sorted tokens.
//
//   x_t = scale E[tok_t],   dE[v] = scale sum over t with tok_t = v of dx_t   (negative ids: padding, no gradient)
//
// Gradient: the (token, row) pairs are sorted stably, and the sorted rows are summed by chunks of equal length, however
// long a token's run is: a run inside a chunk goes straight to the table, one that crosses a border leaves fp32 sums
// that a last kernel adds in order. Rows of no token get zeros, up to 32768 tokens beside the sort, which is then one
// cluster's, else beside the sums. No floating-point atomics: the result does not change from run to run.
//
// Bound by HBM, with a sort of 13 us (8192 tokens) and joins of 6 us that it cannot hide all of. Measured: 8192 tokens
// x 4096 fp32, 32000 rows 71 us (zeros and sort 42, sums 24, joins 6), 5.4 TB/s; 131072 x 4096 bf16 227 us (sort 25,
// sums 190, joins 12), 5.9 TB/s. Added to a gradient that is there: 60 us, of which the bytes take 28 (nothing hides
// the sort), and 8192 x 256 19 us of 2. Lookup of 4096 x 5120 to fp32: 18 us on the device, 20.8 in a row of calls, 5.2
// TB/s. Zeroing most rows beside the sums for few tokens too, which would hide the sort, measured 90 us.
#include <algorithm>
#include <cmath>
#include <utility>

#include "follow.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace mt {

namespace {

// ------------------------------------------------------------------ lookup
constexpr int kLookupBlocks = 64;  // on an SM, of which 8 at a time: a block's start costs as much as a short row
// W columns a thread at a time, 16 bytes of x: blockDim.x threads a row, blockDim.y rows a block. (45359 x 640 fp32: 64
// threads a row 21.6 us, 160, of one load each, 26.2.)
template <class X>
__global__ void __launch_bounds__(256) lookup_kernel(const int32_t* tok, const bf16* E, X* x, int T, int h, int V,
                                                     float scale, int* err) {
  constexpr int W = 16 / sizeof(X);
  wait_for_previous();
  let_next_start();
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; t < T;
       t += static_cast<int64_t>(gridDim.x) * blockDim.y) {
    const int v = tok[t];
    const bool on = v >= 0 && v < V;
    if (v >= V && threadIdx.x == 0) record_bad_token(err);
    const bf16* row = E + static_cast<int64_t>(on ? v : 0) * h;
#pragma unroll 4
    for (int c = threadIdx.x * W; c < h; c += blockDim.x * W) {
      float a[W] = {};
      if (on) {
        read_cols<bf16, W>(row + c, a);
#pragma unroll
        for (int j = 0; j < W; ++j) a[j] *= scale;
      }
      write_cols<X, W>(x + t * h + c, a);
    }
  }
}

// ------------------------------------------------------------------ sort
constexpr int kSortBlocks = 8;     // one cluster, the largest that is portable
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortBits = 9;       // of a digit at most
constexpr int kSortBins = 1 << kSortBits;
constexpr int kSortAhead = 8;      // loads a thread has in flight
constexpr int kSortSmem = kSortWarps * kSortBins * 4;  // counters
// Up to here one cluster sorts, and zeros are written beside it; beyond, 128 blocks sort in two launches a pass and
// zeros are written beside the sums. Both ways, 32000 rows of 4096 fp32: 8192 tokens 72 and 119 us, 16384 103 and 137,
// 32768 150 and 155, 49152 208 and 189, 131072 428 and 380; 256 columns: 32768 33 and 36, 65536 50 and 38. Added to a
// gradient, without zeros, they meet earlier: 16384 of 4096 99 and 96, of 256 24 and 26, 32768 33 and 29.
constexpr int kClusterTokens = 32768;
constexpr int kGapBlocks = 240;  // that write zeros in the launch of the sums (131072 x 4096: 120 244 us, 240 234)

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
  int* number;  // of a pair among the equal digits of its block
  int* counts;  // [blocks][bins] of a pass, where the blocks are not a cluster
  int T, V, passes, bits;
  bf16* dE;
  int64_t h;
  int* err;
};

// Least significant digit first. The blocks own consecutive pairs, and so do a block's warps: each counts the digits
// of its pairs and numbers equal ones; the place of a digit's first pair of a warp is the sum of what comes before
// it in (digit, block, warp) order, which keeps equal digits in order.
struct PassView {
  const SortArgs& g;
  const int2* src;
  int2* dst;
  int shift, bins, lo, hi;  // this warp's pairs
  bool first;
  __device__ PassView(const SortArgs& a, int pass, int block, int blocks)
      : g(a), src(pass & 1 ? a.a : a.b), dst(pass & 1 ? a.b : a.a), shift(pass * a.bits), bins(1 << a.bits),
        first(pass == 0) {
    const int each = (a.T + blocks * kSortWarps - 1) / (blocks * kSortWarps);
    const int64_t begin = static_cast<int64_t>(block * kSortWarps + (threadIdx.x >> 5)) * each;
    lo = static_cast<int>(begin < a.T ? begin : a.T);
    hi = min(a.T, lo + each);
  }
  __device__ __forceinline__ int key(int i) const {
    if (!first) return __ldcg(&src[i].x);
    const int v = g.tok[i];
    if (v >= g.V) record_bad_token(g.err);
    return v < 0 || v >= g.V ? g.V : v;
  }
  __device__ __forceinline__ int digit(int k) const { return k >> shift & (bins - 1); }
};
// count[warp][digit] = pairs of this digit in the block's warps before; total[digit] of the block; numbers of the pairs
// within their warp.
__device__ void count_digits(const PassView& p, int* count, int* total) {
  const int lane = threadIdx.x & 31;
  int* mine = count + (threadIdx.x >> 5) * p.bins;
  for (int i = threadIdx.x; i < kSortWarps * p.bins; i += kSortThreads) count[i] = 0;
  __syncthreads();
  for (int i0 = p.lo; i0 < p.hi; i0 += 32 * kSortAhead) {
    int k[kSortAhead];
#pragma unroll
    for (int j = 0; j < kSortAhead; ++j) {
      const int i = i0 + 32 * j + lane;
      k[j] = i < p.hi ? p.key(i) : 0;
    }
#pragma unroll
    for (int j = 0; j < kSortAhead; ++j) {
      const int i = i0 + 32 * j + lane;
      const unsigned active = __ballot_sync(0xffffffffu, i < p.hi);
      if (i < p.hi) {
        const int d = p.digit(k[j]);
        const unsigned same = __match_any_sync(active, d);
        const int n = mine[d], below = __popc(same & ((1u << lane) - 1));
        p.g.number[i] = n + below;
        __syncwarp(active);
        if (below == 0) mine[d] = n + __popc(same);
      }
      __syncwarp();
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < p.bins; d += kSortThreads) {
    int s = 0;
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = count[w * p.bins + d];
      count[w * p.bins + d] = s;
      s += c;
    }
    total[d] = s;
  }
}
// Where the block's pairs of each digit begin, from digit threadIdx.x's pairs in all blocks and in those before it.
__device__ void digit_bases(const PassView& p, int all, int below, int* base, int* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = threadIdx.x;  // bins <= kSortThreads
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
  if (d < p.bins) base[d] = before + s - all + below;
  __syncthreads();
}
__device__ void place_pairs(const PassView& p, const int* count, const int* base) {
  const int lane = threadIdx.x & 31;
  const int* mine = count ? count + (threadIdx.x >> 5) * p.bins : nullptr;
  for (int i0 = p.lo; i0 < p.hi; i0 += 32 * kSortAhead) {
    int2 q[kSortAhead];
    int n[kSortAhead];
#pragma unroll
    for (int j = 0; j < kSortAhead; ++j) {
      const int i = i0 + 32 * j + lane;
      if (i >= p.hi) continue;
      if (p.first) q[j] = make_int2(p.key(i), i);
      else q[j] = __ldcg(p.src + i);
      n[j] = __ldcg(p.g.number + i);
    }
#pragma unroll
    for (int j = 0; j < kSortAhead; ++j) {
      if (i0 + 32 * j + lane >= p.hi) continue;
      const int d = p.digit(q[j].x);
      p.dst[base[d] + (mine ? mine[d] : 0) + n[j]] = q[j];
    }
  }
}

// Up to kClusterTokens one cluster does all passes, and its blocks read each other's totals.
__device__ void sort_pairs(const SortArgs& g, int* count, int* total, int* base, int* warp_sum) {
  const int rank = blockIdx.x, d = threadIdx.x;
  for (int pass = 0; pass < g.passes; ++pass) {
    const PassView p(g, pass, rank, kSortBlocks);
    count_digits(p, count, total);
    cluster_sync();
    int below = 0, all = 0;
    if (d < p.bins) {
#pragma unroll
      for (int r = 0; r < kSortBlocks; ++r) {
        const int c = cluster_load(total + d, r);
        below += r < rank ? c : 0;
        all += c;
      }
    }
    digit_bases(p, all, below, base, warp_sum);
    place_pairs(p, count, base);
    cluster_sync();  // pairs written, totals read
  }
}

// More tokens: a launch that counts and one that places for each pass, over up to kManyBlocks blocks.
constexpr int kManyBlocks = 128;
__global__ void __launch_bounds__(kSortThreads) digit_count_kernel(const SortArgs g, int pass) {
  extern __shared__ __align__(128) char sort_smem[];
  wait_for_previous();
  let_next_start();
  const PassView p(g, pass, blockIdx.x, gridDim.x);
  int* count = reinterpret_cast<int*>(sort_smem);
  count_digits(p, count, g.counts + blockIdx.x * p.bins);
  __syncthreads();
  // numbers within the block, which the next launch needs alone
  const int* mine = count + (threadIdx.x >> 5) * p.bins;
  for (int i = p.lo + (threadIdx.x & 31); i < p.hi; i += 32) g.number[i] += mine[p.digit(p.key(i))];
}
__global__ void __launch_bounds__(kSortThreads) digit_place_kernel(const SortArgs g, int pass) {
  __shared__ int base[kSortBins], warp_sum[kSortWarps];
  wait_for_previous();
  let_next_start();
  const PassView p(g, pass, blockIdx.x, gridDim.x);
  // the blocks' counts of digit d, in as many shares as there are threads for
  __shared__ int sums[2][kSortThreads];
  const int d = threadIdx.x & (p.bins - 1), rank = blockIdx.x, shares = kSortThreads >> g.bits;
  int below = 0, all = 0;
#pragma unroll 16
  for (int r = threadIdx.x >> g.bits; r < static_cast<int>(gridDim.x); r += shares) {
    const int c = __ldcg(g.counts + r * p.bins + d);
    below += r < rank ? c : 0;
    all += c;
  }
  sums[0][threadIdx.x] = below;
  sums[1][threadIdx.x] = all;
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < p.bins)
    for (int i = 1; i < shares; ++i) {
      below += sums[0][threadIdx.x + i * p.bins];
      all += sums[1][threadIdx.x + i * p.bins];
    }
  else
    below = all = 0;
  digit_bases(p, all, below, base, warp_sum);
  place_pairs(p, nullptr, base);
}

__global__ void __cluster_dims__(kSortBlocks, 1, 1) __launch_bounds__(kSortThreads) sort_kernel(const SortArgs g) {
  extern __shared__ __align__(128) char sort_smem[];
  __shared__ int total[kSortBins], base[kSortBins], warp_sum[kSortWarps];
  wait_for_previous();
  let_next_start();
  sort_pairs(g, reinterpret_cast<int*>(sort_smem), total, base, warp_sum);
}

// Zeros in the rows of the table that no token uses, beside the sort: this kernel starts once the sort's blocks have
// seen the kernel before them end, needs nothing of theirs, and ends after them. Many short blocks, which go where
// there is room: 4096 tokens, 152064 rows of 5120 243 us with 2432 blocks; with one an SM (bulk copies or not) 247 to
// 277, by the GPU, with blocks that share SMs 365; as blocks of the sort's launch, placed in clusters, up to 439.
constexpr int kZeroThreads = 256;
constexpr int kZeroRows = 8192;  // a bit each
__global__ void __launch_bounds__(kZeroThreads) zero_kernel(const SortArgs g) {
  __shared__ unsigned used[kZeroRows / 32];
  let_next_start();
  const int v0 = static_cast<int>(static_cast<int64_t>(g.V) * blockIdx.x / gridDim.x);
  const int v1 = static_cast<int>(static_cast<int64_t>(g.V) * (blockIdx.x + 1) / gridDim.x);
  const int units = static_cast<int>(g.h) / 8;
  for (int r0 = v0; r0 < v1; r0 += kZeroRows) {
    const int r1 = min(v1, r0 + kZeroRows);
    __syncthreads();
    for (int i = threadIdx.x; i < (r1 - r0 + 31) / 32; i += kZeroThreads) used[i] = 0;
    __syncthreads();
    for (int i0 = threadIdx.x; i0 < g.T; i0 += kZeroThreads * kSortAhead) {
      int v[kSortAhead];
#pragma unroll
      for (int j = 0; j < kSortAhead; ++j) {
        const int i = i0 + j * kZeroThreads;
        v[j] = i < g.T ? __ldcg(g.tok + i) : -1;
      }
#pragma unroll
      for (int j = 0; j < kSortAhead; ++j)
        if (v[j] >= r0 && v[j] < r1) atomicOr(used + (v[j] - r0) / 32, 1u << ((v[j] - r0) & 31));
    }
    __syncthreads();
    for (int r = r0 + (threadIdx.x >> 5); r < r1; r += kZeroThreads / 32) {
      if (used[(r - r0) / 32] >> ((r - r0) & 31) & 1) continue;
      uint4* row = reinterpret_cast<uint4*>(g.dE + r * g.h);
      for (int i = threadIdx.x & 31; i < units; i += 32) row[i] = make_uint4(0, 0, 0, 0);
    }
  }
  wait_for_previous();
}
// About 96 KB of the table each, but no more blocks than read the tokens for 20 million in all.
int zero_blocks(int T, int V, int h) {
  const int64_t most = std::min<int64_t>(2432, 20000000 / T);
  const int64_t blocks = (static_cast<int64_t>(V) * h * 2 + 98303) / 98304;
  return static_cast<int>(std::min(most, blocks));
}

// ------------------------------------------------------------------ sums of runs
constexpr int kSumThreads = 256;  // of 16 bytes of a row each
constexpr int kSumAhead = 8;      // rows a thread has in flight
constexpr int kSumChunk = 256;    // sorted rows a block sums, at most

struct SumArgs {
  const int2* pairs;
  const void* dx;
  bf16* dE;
  float* partial;  // [chunks][2][h]: a run from the chunk before (0), one that goes on into the next (1)
  int T, V, h, chunk, chunks;
  float scale;
  bool add;
};
// Zeros in the rows of no token, with the tokens sorted: part `b` of `parts` of the table, a thread a row, which looks
// its token up among the pairs.
constexpr int kGapZeros = 4096;  // bytes
__device__ void zero_gaps(const SumArgs& g, uint4* zeros, int b, int parts) {
  const int v0 = static_cast<int>(static_cast<int64_t>(g.V) * b / parts);
  const int v1 = static_cast<int>(static_cast<int64_t>(g.V) * (b + 1) / parts);
  for (int i = threadIdx.x; i < kGapZeros / 16; i += blockDim.x) zeros[i] = make_uint4(0, 0, 0, 0);
  fence_async_shared();
  __syncthreads();
  const int row_bytes = g.h * 2;
  for (int r = v0 + threadIdx.x; r < v1; r += blockDim.x) {
    int lo = 0, hi = g.T;  // the first pair of a token from r on
    while (lo < hi) {
      const int mid = lo + (hi - lo) / 2;
      if (__ldcg(&g.pairs[mid].x) < r) lo = mid + 1;
      else hi = mid;
    }
    if (lo < g.T && __ldcg(&g.pairs[lo].x) == r) continue;
    char* row = reinterpret_cast<char*>(g.dE + static_cast<int64_t>(r) * g.h);
    for (int i = 0; i < row_bytes; i += kGapZeros) bulk_store(row + i, zeros, min(kGapZeros, row_bytes - i));
  }
  bulk_store_end_group();
  bulk_store_wait_read();
}
template <int W>
__device__ __forceinline__ void write_row(const SumArgs& g, int v, int c, const float* acc) {
  bf16* p = g.dE + static_cast<int64_t>(v) * g.h + c;
  float out[W], old[W] = {};
  if (g.add) read_cols<bf16, W>(p, old);
#pragma unroll
  for (int j = 0; j < W; ++j) out[j] = fmaf(acc[j], g.scale, old[j]);
  write_cols<bf16, W>(p, out);
}
template <int W>
__device__ __forceinline__ void write_partial(const SumArgs& g, int chunk, int which, int c, const float* acc) {
  float* p = g.partial + (static_cast<int64_t>(chunk) * 2 + which) * g.h + c;
#pragma unroll
  for (int j = 0; j < W; j += 4)
    *reinterpret_cast<float4*>(p + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
}

template <class X>
__global__ void __launch_bounds__(kSumThreads) run_sum_kernel(const SumArgs g) {
  constexpr int W = 16 / sizeof(X);
  __shared__ __align__(128) uint4 zeros[kGapZeros / 16];
  __shared__ int2 pairs[kSumChunk];
  __shared__ int ends[2];  // the tokens before and behind the chunk
  wait_for_previous();
  let_next_start();
  if (static_cast<int>(blockIdx.x) >= g.chunks) {
    zero_gaps(g, zeros, (blockIdx.x - g.chunks) * gridDim.y + blockIdx.y, (gridDim.x - g.chunks) * gridDim.y);
    return;
  }
  const int p0 = blockIdx.x * g.chunk, n = min(g.T - p0, g.chunk);
  for (int i = threadIdx.x; i < n; i += blockDim.x) pairs[i] = __ldcg(g.pairs + p0 + i);
  if (threadIdx.x == 0) ends[0] = p0 > 0 ? __ldcg(&g.pairs[p0 - 1].x) : -1;
  if (threadIdx.x == 0) ends[1] = p0 + n < g.T ? __ldcg(&g.pairs[p0 + n].x) : -1;
  __syncthreads();
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * W;
  if (c >= g.h) return;
  const X* dx = static_cast<const X*>(g.dx) + c;
  float acc[W] = {};
  int cur = pairs[0].x;
  bool from_before = ends[0] == cur;
  for (int i0 = 0; i0 < n; i0 += kSumAhead) {
    uint4 raw[kSumAhead];
#pragma unroll
    for (int j = 0; j < kSumAhead; ++j)
      if (i0 + j < n && pairs[i0 + j].x != g.V)
        raw[j] = *reinterpret_cast<const uint4*>(dx + static_cast<int64_t>(pairs[i0 + j].y) * g.h);
#pragma unroll
    for (int j = 0; j < kSumAhead; ++j) {
      if (i0 + j >= n) break;
      const int v = pairs[i0 + j].x;
      if (v != cur) {
        if (from_before) write_partial<W>(g, blockIdx.x, 0, c, acc);
        else write_row<W>(g, cur, c, acc);
        from_before = false;
        cur = v;
#pragma unroll
        for (int k = 0; k < W; ++k) acc[k] = 0.f;
      }
      if (cur == g.V) return;  // padding, at the end
      float a[W];
      read_cols<X, W>(reinterpret_cast<const X*>(&raw[j]), a);
#pragma unroll
      for (int k = 0; k < W; ++k) acc[k] += a[k];
    }
  }
  if (from_before) write_partial<W>(g, blockIdx.x, 0, c, acc);
  else if (ends[1] == cur) write_partial<W>(g, blockIdx.x, 1, c, acc);
  else write_row<W>(g, cur, c, acc);
}

// The runs that cross a border: one block for each chunk in which such a run begins. blockDim.x threads of 4 columns,
// and blockDim.y shares of the chunks that the run goes on into, which meet in shared memory in order.
constexpr int kJoinThreads = 512;
__global__ void __launch_bounds__(kJoinThreads) run_join_kernel(const SumArgs g) {
  __shared__ float4 meet[kJoinThreads];
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * 4, tid = threadIdx.y * blockDim.x + threadIdx.x;
  const int threads = blockDim.x * blockDim.y, p0 = blockIdx.x * g.chunk;
  wait_for_previous();
  const int64_t end = static_cast<int64_t>(p0) + g.chunk;
  if (end >= g.T) return;
  const int before = p0 > 0 ? __ldcg(&g.pairs[p0 - 1].x) : -1;
  const int cur = __ldcg(&g.pairs[end - 1].x), next = __ldcg(&g.pairs[end].x);
  if (cur == g.V || next != cur || before == cur) return;  // no run goes on, or it began in an earlier chunk
  // the chunks that it goes on into
  const int first = blockIdx.x + 1;
  int last = first;
  for (int k0 = first;; k0 += threads) {
    const int k = k0 + tid;
    const int n = __syncthreads_count(k < g.chunks && __ldcg(&g.pairs[static_cast<int64_t>(k) * g.chunk].x) == cur);
    last = k0 + n;
    if (n < threads) break;
  }
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const int share = (last - first + blockDim.y - 1) / blockDim.y;
  const int lo = first + threadIdx.y * share, hi = min(last, lo + share);
  if (c < g.h) {
    const float* part = g.partial + static_cast<int64_t>(lo) * 2 * g.h + c;
#pragma unroll 8
    for (int k = lo; k < hi; ++k, part += 2 * g.h) {
      const float4 a = *reinterpret_cast<const float4*>(part);
      acc.x += a.x, acc.y += a.y, acc.z += a.z, acc.w += a.w;
    }
  }
  meet[tid] = acc;
  __syncthreads();
  if (threadIdx.y > 0 || c >= g.h) return;
  const float4 q = *reinterpret_cast<const float4*>(g.partial + (static_cast<int64_t>(blockIdx.x) * 2 + 1) * g.h + c);
  float sum[4] = {q.x, q.y, q.z, q.w};
  for (int y = 0; y < static_cast<int>(blockDim.y); ++y) {
    const float4 a = meet[y * blockDim.x + threadIdx.x];
    sum[0] += a.x, sum[1] += a.y, sum[2] += a.z, sum[3] += a.w;
  }
  write_row<4>(g, cur, c, sum);
}

bool embed_shape_ok(int T, int V, int h) {
  return T > 0 && T <= kEmbedMaxTokens && V > 0 && V <= kEmbedMaxVocab && h > 0 && h % 8 == 0 && h <= kEmbedMaxWidth;
}
uint64_t table_bytes(int V, int h) { return static_cast<uint64_t>(V) * h * sizeof(bf16); }
// Sorted rows a block sums: as many as leave the SMs 65536 threads (of eight columns each), which leaves fewer sums at
// borders. (8192 x 4096 fp32: 32 73.1 us, here 64 71.7; 131072 x 4096 bf16: 128 234 us, here 256 227, 512 228, and 108,
// which would make whole waves, 250; 77765 x 672 bf16: 256 70 us, here 64 43.)
int sum_chunk(int T, int h) {
  const int64_t most = static_cast<int64_t>(T) * (h / 8) / 65536;
  int chunk = 16;
  while (chunk < kSumChunk && 2 * chunk <= most) chunk *= 2;
  return chunk;
}
// Threads that go over `units` in the fewest turns of at most `most`, and then as evenly as whole warps can.
int threads_of(int units, int most) {
  const int turns = (units + most - 1) / most;
  return ((units + turns - 1) / turns + 31) / 32 * 32;
}
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

cudaError_t embed_lookup(const int32_t* tok, const bf16* E, void* x, int type, int T, int h, int V, float scale,
                         int* err, cudaStream_t s) {
  if (!row_type_ok(type) || !embed_shape_ok(T, V, h) || !vec_ok(tok, 4) || !vec_ok(E, 16) || !vec_ok(x, 16) ||
      (err && !vec_ok(err, 4)) || !std::isfinite(scale) ||
      ranges_overlap(E, table_bytes(V, h), x, static_cast<uint64_t>(T) * h * row_type_bytes(type)))
    return cudaErrorInvalidValue;
  const int threads = std::min(256, (h * row_type_bytes(type) / 16 + 127) / 128 * 32);  // four loads each, or more
  const dim3 block(threads, 256 / threads);
  const dim3 grid(std::min<unsigned>((T + block.y - 1) / block.y, kSms * kLookupBlocks));
  if (type == kRowF32)
    return launch_following(lookup_kernel<float>, grid, block, 0, s, tok, E, static_cast<float*>(x), T, h, V, scale,
                            err);
  return launch_following(lookup_kernel<bf16>, grid, block, 0, s, tok, E, static_cast<bf16*>(x), T, h, V, scale, err);
}

uint64_t embed_lookup_bwd_scratch(int T, int h) {
  const int chunk = sum_chunk(T, h);
  const size_t n = T, chunks = (n + chunk - 1) / chunk;
  return 2 * round256(n * sizeof(int2)) + round256(n * sizeof(int)) +
         (T > kClusterTokens ? kManyBlocks * kSortBins * sizeof(int) : 0) + chunks * 2 * h * sizeof(float);
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
  auto take = [&at](size_t bytes) { return std::exchange(at, at + round256(bytes)); };
  int2* a = reinterpret_cast<int2*>(take(static_cast<size_t>(T) * sizeof(int2)));
  int2* b = reinterpret_cast<int2*>(take(static_cast<size_t>(T) * sizeof(int2)));
  int* number = reinterpret_cast<int*>(take(static_cast<size_t>(T) * sizeof(int)));
  const bool many = T > kClusterTokens;
  int* counts = reinterpret_cast<int*>(take(many ? kManyBlocks * kSortBins * sizeof(int) : 0));
  const SortArgs g{tok, a, b, number, counts, T, V, passes, (bits + passes - 1) / passes, dE, h, err};
  cudaError_t e;
  if (many) {
    for (int pass = 0; pass < passes; ++pass) {
      const int smem = kSortWarps * (1 << g.bits) * 4;
      e = launch_following(digit_count_kernel, dim3(kManyBlocks), kSortThreads, smem, s, g, pass);
      if (e == cudaSuccess) e = launch_following(digit_place_kernel, dim3(kManyBlocks), kSortThreads, 0, s, g, pass);
      if (e != cudaSuccess) return e;
    }
  } else {
    e = launch_following(sort_kernel, dim3(kSortBlocks), kSortThreads, kSortSmem, s, g);
    if (e == cudaSuccess && !add) e = launch_following(zero_kernel, dim3(zero_blocks(T, V, h)), kZeroThreads, 0, s, g);
    if (e != cudaSuccess) return e;
  }
  const int chunk = sum_chunk(T, h), chunks = (T + chunk - 1) / chunk;
  const SumArgs r{passes & 1 ? a : b, dx, dE, reinterpret_cast<float*>(at), T, V, h, chunk, chunks, scale, add};
  auto grid = [&](int units, unsigned& threads) {
    threads = threads_of(units, kSumThreads);
    return dim3(chunks, (units + threads - 1) / threads);
  };
  unsigned threads;
  dim3 blocks_xy = grid(h * row_type_bytes(type) / 16, threads);
  if (many && !add) blocks_xy.x += (kGapBlocks + blocks_xy.y - 1) / blocks_xy.y;
  e = launch_following(type == kRowF32 ? run_sum_kernel<float> : run_sum_kernel<bf16>, blocks_xy, threads, 0, s, r);
  if (e != cudaSuccess || chunks == 1) return e;
  blocks_xy = grid(h / 4, threads);
  return launch_following(run_join_kernel, blocks_xy, dim3(threads, kJoinThreads / threads), 0, s, r);
}

}  // namespace mt
