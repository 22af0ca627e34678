// Attention over spans, backward, on the tcgen05 tensor cores. Deterministic, no atomics.
//
// The tiles are worked on as in the causal backward (attention_bwd_tc.cu): lsd pairs
// (-lse2, -delta) per query row; dK/dV per (128-key tile, kv head, sequence) over the 128-query
// tiles of its group's heads,
//     S^T = K Q^T, dP^T = V dO^T, P^T = 2^(z - lse2), dS^T = P^T (dP^T - delta) z',
//     dV += P^T dO, dK += dS^T Q;
// dQ per (128-query tile, head, sequence) over 128-key tiles, dQ += dS K; 128 x 128 tiles, two
// 128-column score slots in TMEM, P and dS written back over the scores as bf16 pairs and read from
// TMEM, each in two halves of 64 columns. What differs:
//  * z is the capped and biased score and z' the cap's derivative 1 - tanh^2;
//  * the delta kernel also writes each query tile's hull; dQ walks the key tiles of its hull, dK/dV
//    the query tiles from the first to the last whose hull meets its keys, and a tile that meets
//    nothing writes zeros;
//  * documents make these walks short (six tiles on average at a mean of 700 tokens, one for the
//    shortest), and what a block spends around them (its start, the first loads and scores, the
//    last products, the stores) cost more than the walks. The kernels are therefore persistent, one
//    block per SM that takes items (a tile with its walk) from a counter, heaviest ranks first, and
//    the roles run ahead across items: the next item's operands are loaded and its first scores
//    computed while the last item's gradients are stored;
//  * a tile that some row does not see whole is masked by words of 32 bits: a query row's span is a
//    run of bits over its key columns; in dK/dV, where a thread holds a key row, 32 lanes make the
//    runs of 32 query columns and transpose them through the warp;
//  * operand rows that must not count (padding rows, keys outside the hull) are zeroed in shared
//    memory before the products that sum over them, as 0 x NaN is NaN: padding may hold anything.
//
// Measured (head size 128): two 4096-token sequences of 32 heads, packed documents of 700 tokens on
// average, 343 to 349 us (delta 27, dQ 123, dK/dV 188), 7 products over 1.35 times the visible scores; 4096
// tokens, 40/8 heads, capped, 635 us (18, 239, 378; the longest walk is 1.15 times the mean load of an SM). The
// delta kernel is bound by HBM; the others keep the tensor cores 51 % (dQ) and 46 % (dK/dV) busy and wait for
// one another's halves in turn. A tile of dK/dV moves 192 KB of operands, 64 KB of TMA writes and 845
// wavefronts of ordinary accesses (most of them the pairs' broadcasts) through shared memory; smaller
// products that start earlier (S^T by halves) move more and end later: 349 us.
#include <algorithm>
#include <cstdint>

#include "attention_span.cuh"
#include "follow.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "tile_order.cuh"
#include "tma.h"

namespace mt {

namespace {

using namespace span;

// Warps of a block with EW elementwise warps (8 or 16): 0 takes items and loads one ring, 1 issues
// MMAs, 2 .. EW+1 elementwise (EW/4 on each TMEM lane quadrant), the last two load.
template <int EW>
struct Roles {
  static constexpr int kElem = EW * 32;      // elementwise threads
  static constexpr int kCols = 256 / EW;     // score columns an elementwise warp takes per half tile
  static constexpr int kRingWarp = EW + 2;   // loads the other ring
  static constexpr int kItemWarp = EW + 3;   // loads an item's own operands, stores its gradients
  static constexpr int kThreads = EW * 32 + 128;
  static constexpr int kItemReaders = EW + 3;  // lane 0 of every warp but the one that takes items
};
constexpr int kPartItems = 512;       // items that few key tiles' walks are cut into
constexpr int kSlice128 = 128 * 128;  // bytes of a [128 rows][64 bf16] swizzle-atom-wide slice

__host__ __device__ __forceinline__ int pad128(int s) { return (s + 127) & ~127; }

// Pack the 16 values v[o .. o + 15] into 8 bf16 pairs and store them to 8 TMEM columns of this
// thread's lane (the A-operand layout: element k of a row in column k/2, even k in the low half).
template <int N>
__device__ __forceinline__ void store_pairs16(uint32_t taddr, const float (&v)[N], int o) {
  uint32_t w[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) w[c] = pack_bf16(v[o + 2 * c], v[o + 2 * c + 1]);
  tmem_st_8cols(taddr, w);
}

// N (16 or 32) columns of S and of dP of one row behind a single wait.
template <int N>
__device__ __forceinline__ void tmem_ld_pair(uint32_t ta, uint32_t tb, float (&a)[N], float (&b)[N]) {
  uint32_t ra[N], rb[N];
  if constexpr (N == 32) {
    tmem_ld_32cols(ta, ra);
    tmem_ld_32cols(tb, rb);
  } else {
    tmem_ld_16cols(ta, ra);
    tmem_ld_16cols(tb, rb);
  }
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    a[i] = __uint_as_float(ra[i]);
    b[i] = __uint_as_float(rb[i]);
  }
}

// An item's gradients leave through shared memory: each thread converts its share of a row (W columns
// from col0) of the accumulator and writes it to the ring stage that the item's last tile was read
// from, in the swizzled layout of a TMA store, which the warp that loads the items' own operands
// issues. (Each lane storing its own row to global memory touches 32 lines an instruction: 7500 cycles for the two 128 x 128
// gradients of a key tile, two tiles' work. Rows transposed through the warp first: 4700.)
template <int W>
__device__ __forceinline__ void stage_cols(uint32_t taddr, int col0, float scale, uint8_t* tile, int row) {
  constexpr int N = W < 32 ? 16 : 32;
#pragma unroll
  for (int c = 0; c < W; c += N) {
    uint32_t r[N];
    const int col = col0 + c;
    if constexpr (N == 32) tmem_ld_32cols(taddr + col, r);
    else tmem_ld_16cols(taddr + col, r);
    tmem_ld_wait();
    uint8_t* line = tile + (col >> 6) * kSlice128 + row * 128;
#pragma unroll
    for (int v = 0; v < N / 8; ++v) {
      uint4 u;
      u.x = pack_bf16(__uint_as_float(r[8 * v + 0]) * scale, __uint_as_float(r[8 * v + 1]) * scale);
      u.y = pack_bf16(__uint_as_float(r[8 * v + 2]) * scale, __uint_as_float(r[8 * v + 3]) * scale);
      u.z = pack_bf16(__uint_as_float(r[8 * v + 4]) * scale, __uint_as_float(r[8 * v + 5]) * scale);
      u.w = pack_bf16(__uint_as_float(r[8 * v + 6]) * scale, __uint_as_float(r[8 * v + 7]) * scale);
      *reinterpret_cast<uint4*>(line + ((((col & 63) >> 3) + v) ^ (row & 7)) * 16) = u;
    }
  }
}

// W columns (from col0) of one row of an fp32 accumulator to the item's partial sums, laid out [group of
// 4 columns][128 rows][4]: a warp's 32 rows are 512 contiguous bytes an instruction.
template <int W>
__device__ __forceinline__ void partial_cols(uint32_t taddr, int col0, float* dst, int row) {
  constexpr int N = W < 32 ? 16 : 32;
#pragma unroll
  for (int c = 0; c < W; c += N) {
    uint32_t r[N];
    if constexpr (N == 32) tmem_ld_32cols(taddr + col0 + c, r);
    else tmem_ld_16cols(taddr + col0 + c, r);
    tmem_ld_wait();
#pragma unroll
    for (int v = 0; v < N / 4; ++v)
      reinterpret_cast<float4*>(dst)[((col0 + c) / 4 + v) * 128 + row] =
          make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]), __uint_as_float(r[4 * v + 2]),
                      __uint_as_float(r[4 * v + 3]));
  }
}

// Zeros to `rows` rows of HD columns (an item without a walk): the elementwise threads, 16 bytes each.
template <int HD>
__device__ __forceinline__ void zero_rows(bf16* dst, int64_t ld, int rows, int elem, int threads) {
  for (int i = elem; i < rows * (HD / 8); i += threads)
    *reinterpret_cast<uint4*>(dst + i / (HD / 8) * ld + i % (HD / 8) * 8) = make_uint4(0u, 0u, 0u, 0u);
}

// ------------------------------------------------------------------ items
// The items a block works on, handed from the warp that takes them to the others through two slots.
struct Item {
  int lin;    // index in the heaviest-first order, -1: no more
  int first;  // first tile of the walk
  int count;  // its tiles (per query head of the group in dK/dV)
  int begin;  // dK/dV: first step of the item's part of the walk over the group's heads
  int steps;  // and its steps
  Hull hull;  // dQ: of the query tile
};
struct ItemRing {
  uint64_t* full;   // [2]
  uint64_t* empty;  // [2]
  Item* slot;       // [2]
  int* err;
};
constexpr int kTakeAhead = 2;     // the next item is taken with the last this many loads of an item

// Barriers used in turn (turn_bar), as their waits are not needed for the very next phase; of the others, every
// waiter is.
// acc_empty, by items: the accumulators' release is waited for by the MMA warp and by the warp that stores
// the item's gradients, which has by then loaded what the next item needs. An item of one or two tiles
// can end before it looks; item n + 2 needs operands that it loads after its wait for item n.
constexpr int kAccTurns = 2;
// dQ's second half of dS, by tiles: the MMA warp has issued the next tile's scores when it waits for it, which
// is all that the elementwise warps need to finish that tile too; the scores of tile g + 2 come after.
constexpr int kLastHalfTurns = 2;

// Publish item number n (one thread).
__device__ __forceinline__ bool put_item(const ItemRing& r, int n, const Item& it) {
  if (!mbar_wait(&r.empty[n & 1], ((n >> 1) & 1) ^ 1u, r.err, kErrTimeoutAttn)) return false;
  r.slot[n & 1] = it;
  mbar_arrive(&r.full[n & 1]);
  return true;
}
// The same value in every lane, as a warp reduction's result: what the compiler can see to be uniform
// stays in uniform registers. The MMA warp's descriptors follow from the items' tile counts, and
// computed per lane they have to be moved for every MMA it issues.
__device__ __forceinline__ int uniform(int v) { return __reduce_max_sync(0xffffffffu, v); }

// Item number n, for a whole warp; false if there is none.
__device__ __forceinline__ bool get_item_warp(const ItemRing& r, int n, Item& it) {
  if (!mbar_wait_warp(&r.full[n & 1], (n >> 1) & 1, r.err, kErrTimeoutAttn)) return false;
  const Item s = r.slot[n & 1];
  it.lin = uniform(s.lin);
  it.first = uniform(s.first);
  it.count = uniform(s.count);
  it.begin = uniform(s.begin);
  it.steps = uniform(s.steps);
  it.hull = {uniform(s.hull.min_lo), uniform(s.hull.max_hi), uniform(s.hull.max_lo), uniform(s.hull.min_hi)};
  if ((threadIdx.x & 31) == 0) mbar_arrive(&r.empty[n & 1]);
  return it.lin >= 0;
}
// The same for a single thread.
__device__ __forceinline__ bool get_item(const ItemRing& r, int n, Item& it) {
  if (!mbar_wait(&r.full[n & 1], (n >> 1) & 1, r.err, kErrTimeoutAttn)) return false;
  it = r.slot[n & 1];
  mbar_arrive(&r.empty[n & 1]);
  return it.lin >= 0;
}

// ------------------------------------------------------------------ delta and hulls
// One block per 128 query rows of a (sequence, head): HD/8 lanes per row (16-byte loads). A row
// whose span is empty (or past the end, or without a finite score) gets (-inf, -0): every
// probability of it is 0. The blocks of head 0 also reduce their rows' spans to the tile's hull.
// Block 0 clears the counters the next two kernels take their items from.
template <int HD>
__global__ void __launch_bounds__(256)
    span_delta_kernel(const bf16* __restrict__ o, int64_t ldo, const bf16* __restrict__ dout, int64_t lddo,
                      const float* __restrict__ lse, Spans spans, float2* __restrict__ lsd, Hull* __restrict__ hulls,
                      int* __restrict__ taken, int s, int nh, int n_t) {
  constexpr int kLanes = HD / 8;  // lanes per row
  let_next_start();  // (dQ and dK/dV do not: the next one's blocks among theirs cost 17 us of 362 at 7B)
  if (blockIdx.x == 0 && threadIdx.x < 2) taken[threadIdx.x] = 0;  // items taken by dQ and by dK/dV
  __shared__ Hull parts[4];
  const int tile = blockIdx.x % n_t;
  const int bh = blockIdx.x / n_t;  // b * nh + head
  const int b = bh / nh, head = bh % nh;
  const int sp = pad128(s);
  const int sub = threadIdx.x % kLanes;
#pragma unroll 4
  for (int r = threadIdx.x / kLanes; r < 128; r += 256 / kLanes) {
    const int i = tile * 128 + r;
    float acc = 0.f;
    bool live = false;
    float l2 = 0.f;
    if (i < s) {
      const int64_t t = static_cast<int64_t>(b) * s + i;
      const uint4 x = reinterpret_cast<const uint4*>(o + t * ldo + static_cast<int64_t>(head) * HD)[sub];
      const uint4 d = reinterpret_cast<const uint4*>(dout + t * lddo + static_cast<int64_t>(head) * HD)[sub];
      const int2 seen = load_span(spans, b, i, s);
      l2 = lse[static_cast<int64_t>(bh) * s + i];
      live = seen.x < seen.y && l2 != -INFINITY;
      const uint32_t xv[4] = {x.x, x.y, x.z, x.w}, dv[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        acc += __uint_as_float(xv[k] << 16) * __uint_as_float(dv[k] << 16) +
               __uint_as_float(xv[k] & 0xffff0000u) * __uint_as_float(dv[k] & 0xffff0000u);
    }
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (sub == 0)
      lsd[static_cast<int64_t>(bh) * sp + i] = live ? make_float2(-l2, -acc) : make_float2(-INFINITY, -0.f);
  }
  if (head != 0) return;
  if (threadIdx.x < 128) {
    const int i = tile * 128 + threadIdx.x;
    const Hull h = warp_hull(row_hull(i < s ? load_span(spans, b, i, s) : make_int2(0, 0), i < s));
    if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = h;
  }
  __syncthreads();
  if (threadIdx.x == 0)
    hulls[static_cast<int64_t>(b) * n_t + tile] = join(join(parts[0], parts[1]), join(parts[2], parts[3]));
}

struct BwdArgs {
  Spans spans;
  const float* slopes;
  const float2* lsd;
  const Hull* hulls;   // [B][tiles] of the query tiles
  int2* q_ranges;      // [B][tiles] first and last query tile that meets a key tile (last -1: none)
  int* taken;          // [2] items taken: dQ, dK/dV
  int parts;           // parts of a key tile's walk
  float* partial;      // with more than one, their sums: [B][nkv][parts][tiles][2][HD/4][128][4]
  bf16 *dq, *dk, *dv;
  int64_t lddq, lddk, lddv;
  int B, s, nh, nkv;
  ScoreArgs score;
  int* err;
};

// Query tiles of a key tile's walk (per query head of the group), and where part `k` of `parts` of `steps`
// steps begins.
__device__ __forceinline__ int walk_tiles(int2 range) { return range.y < 0 ? 0 : range.y - range.x + 1; }
__device__ __forceinline__ int part_begin(int steps, int k, int parts) {
  // steps <= kSpanMaxWalk / 128, k <= parts <= kPartItems
  return static_cast<uint32_t>(steps * k) / static_cast<uint32_t>(parts);
}

// P and dS of one pair of columns: scores (capped: their tanh) and dP in, P and dS out. nl = -lse2,
// nd = -delta of the columns' (or the row's) queries; dist = |i - j| where there is a bias.
template <bool CAP, bool BIAS>
__device__ __forceinline__ void p_and_ds(float2& sv, float2& dv, float2 nl, float2 nd, float2 dist, float slope2,
                                         const ScoreArgs& a) {
  const float to_log2 = CAP ? a.cap_log2 : a.scale_log2;
  if constexpr (BIAS) nl = __ffma2_rn(make_float2(-slope2, -slope2), dist, nl);
  const float2 e = __ffma2_rn(sv, make_float2(to_log2, to_log2), nl);
  const float2 p = make_float2(ex2(e.x), ex2(e.y));
  float2 d = __fmul2_rn(p, __fadd2_rn(dv, nd));
  if constexpr (CAP) d = __fmul2_rn(d, __ffma2_rn(make_float2(-sv.x, -sv.y), sv, make_float2(1.f, 1.f)));
  sv = p;
  dv = d;
}

// ------------------------------------------------------------------ dK, dV (KV-outer)
template <int HD>
struct SmemKV {
  static constexpr int NSL = HD / 64;
  static constexpr int QS = 3, DS = 2;                  // Q ring and dO ring depths
  static constexpr int TILE = NSL * kSlice128;          // one 128-row tile: NSL x [128][64]
  static constexpr int K = 0;
  static constexpr int V = K + TILE;
  static constexpr int Q = V + TILE;                    // QS tiles
  static constexpr int DO = Q + QS * TILE;              // DS x (tile, then 128 (-lse2, -delta) pairs)
  static constexpr int DSTAGE = TILE + 1024;
  static constexpr int BAR = DO + DS * DSTAGE;
  static constexpr int BYTES = BAR + 320;               // the dynamic window is 1024-aligned (checked)
  static_assert(BYTES <= 232448, "dK/dV shared memory above the 227 KB per-CTA limit");
};

template <int HD, bool CAP, bool BIAS, int EW, bool PARTIAL>
__global__ void __launch_bounds__(Roles<EW>::kThreads, 1)
    attn_span_dkdv_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do,
                          const __grid_constant__ CUtensorMap map_dk, const __grid_constant__ CUtensorMap map_dv,
                          const __grid_constant__ BwdArgs a) {
  using L = SmemKV<HD>;
  using R = Roles<EW>;
  // A tile's halves: with 32 columns a warp the unrolled loop misses the instruction cache (7B packed
  // documents 362 us, rolled 345); with 16 it fits (14B capped 632 us, rolled 645)
  constexpr int kUnroll = CAP ? 2 : 1;
  constexpr int kCols = R::kCols;
  constexpr int QS = L::QS, DS = L::DS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  int* err = a.err;
  if (smem_addr(sm) & 1023) {  // the swizzled layouts need a 1024-byte aligned base
    if (threadIdx.x == 0) record_give_up(err, kErrTimeoutAttn);
    return;
  }
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint64_t* kv_full = bar + 0;
  uint64_t* kv_empty = bar + 1;          // every MMA that reads the item's K and V has completed
  uint64_t* q_full = bar + 2;            // [QS]
  uint64_t* q_empty = bar + 5;           // [QS]
  uint64_t* d_full = bar + 8;            // [DS]
  uint64_t* d_empty = bar + 10;          // [DS]
  uint64_t* sdp_full = bar + 12;         // [2]: the tile's S^T and that half of its dP^T are complete
  uint64_t* dp_free = bar + 14;          // every warp holds its dP^T columns in registers
  uint64_t* p_half = bar + 15;           // [2]: every warp has written P^T/dS^T of that half
  uint64_t* acc_full = bar + 17;         // the item's accumulating MMAs have completed
  uint64_t* acc_empty = bar + 18;        // [kAccTurns]: every warp has read its part of dK and dV and staged it
  const ItemRing ring{bar + 20, bar + 22, reinterpret_cast<Item*>(bar + 25), err};
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + 24);
  uint64_t* drained = bar + 34;          // the MMA warp's last products have completed
  static_assert(25 * 8 + 2 * sizeof(Item) <= 34 * 8, "item slots past their shared memory");

  const int s = a.s, nh = a.nh, nkv = a.nkv;
  const int group = nh / nkv;
  const int parts = PARTIAL ? a.parts : 1;  // items that share the walk of a key tile
  const int n_t = (s + 127) / 128, n_hb = nkv * parts * a.B;
  const int sp = pad128(s);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // item -> key tile (the first key tile is seen by the most queries under a causal mask), part of its
  // walk, key head, sequence
  struct Where {
    int kt, part, kvh, b;
  };
  auto where = [&](int lin) -> Where {
    const TileSlot slot = heavy_first_slot(lin, n_t, n_hb);
    const int hb = slot.hb / parts;
    return {slot.rank, slot.hb % parts, hb % nkv, hb / nkv};
  };

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    mbar_init(kv_empty, 1);
    for (int i = 0; i < QS; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < DS; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], 1);
    }
    mbar_init(&sdp_full[0], 1);
    mbar_init(&sdp_full[1], 1);
    mbar_init(dp_free, EW);
    mbar_init(&p_half[0], EW);
    mbar_init(&p_half[1], EW);
    mbar_init(acc_full, 1);
    mbar_init(drained, 1);
    for (int i = 0; i < kAccTurns; ++i) mbar_init(&acc_empty[i], EW);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ring.full[i], 1);
      mbar_init(&ring.empty[i], R::kItemReaders);
    }
    fence_mbar_init();
    tma_prefetch_map(&map_q);
    tma_prefetch_map(&map_k);
    tma_prefetch_map(&map_v);
    tma_prefetch_map(&map_do);
  }
  if (warp == 1) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  wait_for_previous();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  const uint32_t tdV = tbase + 256, tdK = tbase + 256 + HD;
  // g numbers the block's tiles across its items, n its items with a walk
  auto s_slot = [&](int g) { return tbase + (g & 1) * 128; };        // S^T, then P^T | dS^T pairs
  auto d_slot = [&](int g) { return tbase + ((g & 1) ^ 1) * 128; };  // dP^T

  if (warp == 0) {
    // takes the items and loads the Q ring. The next item is taken with the last loads of this one, a
    // few tiles before its end: taken with the item itself, the items no longer go to the blocks that
    // are done first (14B heads, 256 unequal items: 385 -> 470 us); taken any later, the next item's
    // first loads come late
    if (lane == 0) {
      const int items = n_t * n_hb;
      auto take = [&](int lin) -> Item {
        Item it{-1, 0, 0, 0, 0, {0, 0, 0, 0}};
        if (lin < items) {
          const Where w = where(lin);
          const int2 r = a.q_ranges[static_cast<int64_t>(w.b) * n_t + w.kt];
          it.lin = lin;
          it.first = r.x;
          it.count = walk_tiles(r);
          it.begin = part_begin(group * it.count, w.part, parts);
          it.steps = part_begin(group * it.count, w.part + 1, parts) - it.begin;
        }
        return it;
      };
      Item cur = take(blockIdx.x);
      bool ok = put_item(ring, 0, cur);
      int g = 0;
      for (int m = 1; ok && cur.lin >= 0; ++m) {
        const Where w = where(cur.lin);
        const int total = cur.steps, early = max(total - kTakeAhead, 0);
        Item next;
        auto hand_on = [&] {
          next = take(gridDim.x + atomicAdd(a.taken + 1, 1));
          return put_item(ring, m, next);
        };
        if (total == 0 && !(ok = hand_on())) break;
        for (int i = 0; i < total; ++i, ++g) {
          if (i == early && !(ok = hand_on())) break;
          const int st = g % QS;
          if (!(ok = mbar_wait(&q_empty[st], ((g / QS) & 1) ^ 1u, err, kErrTimeoutAttn))) break;
          mbar_arrive_expect_tx(&q_full[st], L::TILE);
          const int x = (PARTIAL ? cur.begin : 0) + i;
          tma_load_4d(sm + L::Q + st * L::TILE, &map_q, &q_full[st], 0, (cur.first + x % cur.count) * 128,
                      (w.kvh * group + x / cur.count) * (HD / 64), w.b);
        }
        cur = next;
      }
      ring_drain<QS>(q_full, g);
    }
  } else if (warp == R::kRingWarp) {
    // the dO ring with the (-lse2, -delta) pairs
    if (lane == 0) {
      Item it;
      bool ok = true;
      int g = 0;
      for (int m = 0; ok && get_item(ring, m, it); ++m) {
        const Where w = where(it.lin);
        const int begin = PARTIAL ? it.begin : 0;
        for (int i = begin; i < begin + it.steps; ++i, ++g) {
          const int st = g % DS;
          const int hq = w.kvh * group + i / it.count, q0 = (it.first + i % it.count) * 128;
          if (!(ok = mbar_wait(&d_empty[st], ((g / DS) & 1) ^ 1u, err, kErrTimeoutAttn))) break;
          mbar_arrive_expect_tx(&d_full[st], L::TILE + 1024);
          uint8_t* base = sm + L::DO + st * L::DSTAGE;
          tma_load_4d(base, &map_do, &d_full[st], 0, q0, hq * (HD / 64), w.b);
          bulk_load_1d(base + L::TILE, a.lsd + (static_cast<int64_t>(w.b) * nh + hq) * sp + q0, 1024, &d_full[st]);
        }
      }
      ring_drain<DS>(d_full, g);
    }
  } else if (warp == R::kItemWarp) {
    // K and V, once per item; and the gradients of the item before, from the stages of its last tile,
    // which are released when they have been read
    if (lane == 0) {
      Item it;
      Where out{0, 0, 0, 0};
      bool ok = true;
      auto store = [&](int n, int g) -> bool {  // item n, which ended with tile g
        if (!mbar_wait(turn_bar<kAccTurns>(acc_empty, n), turn_parity<kAccTurns>(n), err, kErrTimeoutAttn))
          return false;
        if constexpr (!PARTIAL) {
          tma_store_4d(&map_dk, sm + L::Q + (g % QS) * L::TILE, 0, out.kt * 128, out.kvh * (HD / 64), out.b);
          tma_store_4d(&map_dv, sm + L::DO + (g % DS) * L::DSTAGE, 0, out.kt * 128, out.kvh * (HD / 64), out.b);
          bulk_commit();
          bulk_wait_read();
        }
        mbar_arrive(&q_empty[g % QS]);
        mbar_arrive(&d_empty[g % DS]);
        return true;
      };
      int n = 0, g = 0, stored = 0;
      for (int m = 0; ok && get_item(ring, m, it); ++m) {
        const Where w = where(it.lin);
        const int last = g - 1;
        if (it.steps > 0) {
          if (!(ok = mbar_wait(kv_empty, (n & 1) ^ 1u, err, kErrTimeoutAttn))) break;
          mbar_arrive_expect_tx(kv_full, 2 * L::TILE);
          tma_load_4d(sm + L::K, &map_k, kv_full, 0, w.kt * 128, w.kvh * (HD / 64), w.b);
          tma_load_4d(sm + L::V, &map_v, kv_full, 0, w.kt * 128, w.kvh * (HD / 64), w.b);
        }
        if (stored < n) ok = store(stored++, last);
        if (it.steps > 0) {
          out = w;
          g += it.steps;
          ++n;
        }
      }
      if (ok && stored < n) store(stored, g - 1);
      if (n > 0) mbar_drain(kv_full, (n - 1) & 1);
      bulk_wait();
    }
  } else if (warp == 1) {
    // the whole warp runs the issuing loop; elect.sync picks the lane that issues each MMA
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t idesc_dh = idesc_bf16_f32(128, 64, false, false);
    constexpr uint32_t idesc_acc = idesc_bf16_f32(128, HD, false, true);
    const uint64_t kd = smem_desc_sw128(smem_addr(sm + L::K), 16, 1024);
    const uint64_t vd = smem_desc_sw128(smem_addr(sm + L::V), 16, 1024);
    // S^T = K Q^T of tile g into its TMEM slot, once its Q tile is in
    auto s_scores = [&](int g) -> bool {
      if (!mbar_wait_warp(&q_full[g % QS], (g / QS) & 1, err, kErrTimeoutAttn)) return false;
      tc_fence_after();
      const uint64_t bd = smem_desc_sw128(smem_addr(sm + L::Q + (g % QS) * L::TILE), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        const uint32_t off = (kk >> 2) * kSlice128 + (kk & 3) * 32;
        umma_bf16_warp(s_slot(g), desc_advance(kd, off), desc_advance(bd, off), idesc_s, kk > 0 ? 1u : 0u);
      }
      return true;
    };
    // half h of dP^T = V dO^T of tile g into columns [64 h, 64 h + 64) of its TMEM slot
    auto dp_half = [&](int g, int h) -> bool {
      if (!mbar_wait_warp(&d_full[g % DS], (g / DS) & 1, err, kErrTimeoutAttn)) return false;
      tc_fence_after();
      const uint64_t bd = smem_desc_sw128(smem_addr(sm + L::DO + (g % DS) * L::DSTAGE), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        const uint32_t off = (kk >> 2) * kSlice128 + (kk & 3) * 32;
        umma_bf16_warp(d_slot(g) + h * 64, desc_advance(vd, off), desc_advance(bd, off + h * 8192), idesc_dh,
                       kk > 0 ? 1u : 0u);
      }
      return true;
    };
    Item it;
    bool ok = true;
    for (int m = 0, n = 0, g = 0; ok && get_item_warp(ring, m, it); ++m) {
      const int total = it.steps;
      if (total == 0) continue;
      // the item's first scores: both TMEM slots are free of what the last item left in them once
      // its products, issued before, have run and every warp holds its dP^T columns
      if (!(ok = mbar_wait_warp(kv_full, n & 1, err, kErrTimeoutAttn))) break;
      if (g > 0 && !(ok = mbar_wait_warp(dp_free, (g - 1) & 1, err, kErrTimeoutAttn))) break;
      if (!(ok = s_scores(g) && dp_half(g, 0))) break;
      umma_commit_warp(&sdp_full[0]);
      if (!(ok = dp_half(g, 1))) break;
      umma_commit_warp(&sdp_full[1]);
      if (total == 1) umma_commit_warp(kv_empty);
      for (int i = 0; i < total && ok; ++i, ++g) {
        // B operands of the accumulating MMAs: dO and Q tiles read MN-major (16 queries per step)
        const uint64_t qd = smem_desc_sw128(smem_addr(sm + L::Q + (g % QS) * L::TILE), kSlice128, 1024);
        const uint64_t dd = smem_desc_sw128(smem_addr(sm + L::DO + (g % DS) * L::DSTAGE), kSlice128, 1024);
        const uint32_t ts = s_slot(g);
        for (int h = 0; h < 2 && ok; ++h) {
          if (h == 1 && i + 1 < total) {
            // the next tile's first dP^T half over this tile's first P^T/dS^T pairs, after the MMAs
            // reading them; then the next S^T into the dP^T slot, free once every warp holds its columns
            if (!(ok = dp_half(g + 1, 0))) break;
            if (!(ok = mbar_wait_warp(dp_free, g & 1, err, kErrTimeoutAttn))) break;
            tc_fence_after();
            if (!(ok = s_scores(g + 1))) break;
            umma_commit_warp(&sdp_full[0]);
          }
          if (!(ok = mbar_wait_warp(&p_half[h], g & 1, err, kErrTimeoutAttn))) break;
          // the first product of an item overwrites the accumulators: the last item's have been read
          if (h == 0 && i == 0 && n > 0 &&
              !(ok = mbar_wait_warp(turn_bar<kAccTurns>(acc_empty, n - 1), turn_parity<kAccTurns>(n - 1), err,
                                    kErrTimeoutAttn)))
            break;
          tc_fence_after();
#pragma unroll
          for (int kk = 4 * h; kk < 4 * h + 4; ++kk) {  // 16 queries per step; A (P^T, dS^T) from TMEM
            const uint32_t acc = (i > 0 || kk > 0) ? 1u : 0u;
            umma_bf16_tmem_a_warp(tdV, ts + kk * 16, desc_advance(dd, kk * 2048), idesc_acc, acc);
            umma_bf16_tmem_a_warp(tdK, ts + kk * 16 + 8, desc_advance(qd, kk * 2048), idesc_acc, acc);
          }
        }
        if (!ok) break;
        if (i + 1 < total) {  // the last tile's stages are released once the gradients have left them
          umma_commit_warp(&q_empty[g % QS]);
          umma_commit_warp(&d_empty[g % DS]);
          // the next tile's second dP^T half over this tile's last P^T/dS^T pairs
          if (!(ok = dp_half(g + 1, 1))) break;
          umma_commit_warp(&sdp_full[1]);
          if (i + 2 == total) umma_commit_warp(kv_empty);
        } else {
          umma_commit_warp(acc_full);
        }
      }
      ++n;
    }
    mma_drain(drained);
  } else {
    const int sub = warp & 3;
    const int part = (warp - 2) >> 2;  // which kCols of each 64 query columns this warp takes
    const int row = sub * 32 + lane;
    const int elem = threadIdx.x - 64;
    const uint32_t tl = static_cast<uint32_t>(sub * 32) << 16;
    // A tile's hull and its query rows' spans (of this lane's column in each half) are loaded a tile
    // ahead, an item's first ones before the last item's gradients are stored: a load here costs
    // the block 800 cycles.
    struct Ahead {
      Hull hull;
      int2 seen[2];
    };
    auto look = [&](int b, int qt) -> Ahead {
      Ahead r;
      r.hull = a.hulls[static_cast<int64_t>(b) * n_t + qt];
#pragma unroll
      for (int h = 0; h < 2; ++h) r.seen[h] = fetch_span(a.spans, b, qt * 128 + h * 64 + part * kCols + lane, s);
      return r;
    };
    auto first_tile = [](const Item& x) { return x.first + (PARTIAL ? x.begin % x.count : 0); };
    Item it, next_it;
    Where next_w{0, 0, 0, 0};
    Ahead ahead{};
    bool ok = true, more = get_item_warp(ring, 0, next_it);
    if (more) {
      next_w = where(next_it.lin);
      if (next_it.steps > 0) ahead = look(next_w.b, first_tile(next_it));
    }
    for (int m = 1, n = 0, g = 0; ok && more; ++m) {
      it = next_it;
      const Where w = next_w;
      const int k0 = w.kt * 128, key = k0 + row;
      const int total = it.steps;
      int qt = it.first, hq = w.kvh * group;
      if (PARTIAL && total > 0) {
        qt += it.begin % it.count;
        hq += it.begin / it.count;
      }
      for (int i = 0; i < total && ok; ++i, ++g) {
        const int q0 = qt * 128;
        const bool all = sees_all(ahead.hull, k0, k0 + 128), padded = ahead.hull.max_lo == INT_MAX;
        uint32_t vis[2] = {~0u, ~0u};  // visible query columns of this thread's key, per half
        if (!all) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            vis[h] = warp_transpose(span_bits(clamp_span(ahead.seen[h], s), k0 + sub * 32), lane);
        }
        const float slope2 = BIAS ? __ldg(a.slopes + hq) * kLog2e : 0.f;
        if (++qt == it.first + it.count) {  // the walk of the group's next head
          qt = it.first;
          ++hq;
        }
        if (i + 1 < total) ahead = look(w.b, qt);
        uint8_t* dstage = sm + L::DO + (g % DS) * L::DSTAGE;
        const float4* lsd_s = reinterpret_cast<const float4*>(dstage + L::TILE);
        // the pairs were copied with the tile's dO: observe that copy before reading them
        if (!(ok = mbar_wait_warp(&d_full[g % DS], (g / DS) & 1, err, kErrTimeoutAttn))) break;
        const uint32_t ts = s_slot(g) + tl, td = d_slot(g) + tl;
#pragma unroll kUnroll
        for (int h = 0; h < 2; ++h) {
          if (!ok) break;
          if (!(ok = mbar_wait_warp(&sdp_full[h], g & 1, err, kErrTimeoutAttn))) break;
          tc_fence_after();
          const int cb = h * 64 + part * kCols;  // this warp's score columns [cb, cb + kCols)
          float sv[kCols], dv[kCols];
          tmem_ld_pair<kCols>(ts + cb, td + cb, sv, dv);
          if (h == 1) {  // every dP^T column of the tile is now in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(dp_free);
          }
          if constexpr (CAP) cap_tanh<kCols>(sv, a.score);
          const float d0 = static_cast<float>(q0 + cb - key);
#pragma unroll
          for (int k = 0; k < kCols / 2; ++k) {  // columns 2k, 2k+1: queries with (-lse2, -delta) in lv
            const float4 lv = lsd_s[cb / 2 + k];
            float2 x = make_float2(sv[2 * k], sv[2 * k + 1]), y = make_float2(dv[2 * k], dv[2 * k + 1]);
            const float2 dist = make_float2(fabsf(d0 + (2 * k)), fabsf(d0 + (2 * k + 1)));
            p_and_ds<CAP, BIAS>(x, y, make_float2(lv.x, lv.z), make_float2(lv.y, lv.w), dist, slope2, a.score);
            sv[2 * k] = x.x;
            sv[2 * k + 1] = x.y;
            dv[2 * k] = y.x;
            dv[2 * k + 1] = y.y;
          }
          if (!all) {
            const uint32_t seen = h ? vis[1] : vis[0];
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
              const bool keep = seen >> c & 1u;
              sv[c] = keep ? sv[c] : 0.f;
              dv[c] = keep ? dv[c] : 0.f;
            }
          }
          // P^T pairs then dS^T pairs over this warp's own kCols S^T columns, 16 at a time: the A operands of
          // K-steps cb / 16 and on of the accumulating MMAs
#pragma unroll
          for (int o = 0; o < kCols; o += 16) {
            store_pairs16<kCols>(ts + cb + o, sv, o);
            store_pairs16<kCols>(ts + cb + o + 8, dv, o);
          }
          tmem_st_wait();
          if (padded) {  // this half's Q and dO rows that are padding: no product may read them
            const int r = h * 64 + (elem & 63), which = elem >> 6;
            if (which < 2 * L::NSL && reinterpret_cast<const float2*>(lsd_s)[r].x == -INFINITY) {
              uint8_t* tile = which < L::NSL ? sm + L::Q + (g % QS) * L::TILE : dstage;
              zero_slice_row(tile + (which % L::NSL) * kSlice128, r);
            }
            fence_proxy_async_smem();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_half[h]);
        }
      }
      if (!ok) break;
      more = get_item_warp(ring, m, next_it);
      if (more) {
        next_w = where(next_it.lin);
        if (next_it.steps > 0) ahead = look(next_w.b, first_tile(next_it));
      }
      if (PARTIAL && total == 0) continue;  // the kernel that adds the parts writes the zeros
      if (total == 0) {
        const int64_t t = static_cast<int64_t>(w.b) * s + k0;
        zero_rows<HD>(a.dk + t * a.lddk + static_cast<int64_t>(w.kvh) * HD, a.lddk, min(128, s - k0), elem, R::kElem);
        zero_rows<HD>(a.dv + t * a.lddv + static_cast<int64_t>(w.kvh) * HD, a.lddv, min(128, s - k0), elem, R::kElem);
        continue;
      }
      if (!(ok = mbar_wait_warp(acc_full, n & 1, err, kErrTimeoutAttn))) break;
      tc_fence_after();
      if constexpr (PARTIAL) {
        const int64_t slot = ((static_cast<int64_t>(w.b) * nkv + w.kvh) * parts + w.part) * n_t + w.kt;
        float* p = a.partial + slot * (2 * 128 * HD);
        partial_cols<HD * 4 / EW>(tdK + tl, part * (HD * 4 / EW), p, row);
        partial_cols<HD * 4 / EW>(tdV + tl, part * (HD * 4 / EW), p + 128 * HD, row);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(turn_bar<kAccTurns>(acc_empty, n));
        ++n;
        continue;
      }
      uint8_t* out_k = sm + L::Q + ((g - 1) % QS) * L::TILE;
      uint8_t* out_v = sm + L::DO + ((g - 1) % DS) * L::DSTAGE;
      stage_cols<HD * 4 / EW>(tdK + tl, part * (HD * 4 / EW), a.score.scale, out_k, row);
      stage_cols<HD * 4 / EW>(tdV + tl, part * (HD * 4 / EW), 1.f, out_v, row);
      tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(turn_bar<kAccTurns>(acc_empty, n));
      ++n;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, 512);
}

// dK and dV of one key tile: the sums of its walk's parts, added in their order.
template <int HD>
__global__ void __launch_bounds__(256) span_join_kernel(const __grid_constant__ BwdArgs a, int n_t) {
  wait_for_previous();
  const int kt = blockIdx.x % n_t, hb = blockIdx.x / n_t;
  const int c = blockIdx.y * 2 + (threadIdx.x >> 7);  // 4 columns of dK, then of dV
  const int kvh = hb % a.nkv, b = hb / a.nkv, group = a.nh / a.nkv;
  const int row = threadIdx.x & 127, key = kt * 128 + row;
  if (key >= a.s) return;
  const int steps = group * walk_tiles(a.q_ranges[static_cast<int64_t>(b) * n_t + kt]);
  const int64_t part_size = static_cast<int64_t>(n_t) * (2 * 128 * HD);
  const float* p = a.partial + (static_cast<int64_t>(b) * a.nkv + kvh) * a.parts * part_size +
                   kt * static_cast<int64_t>(2 * 128 * HD);
  const int64_t t = static_cast<int64_t>(b) * a.s + key;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < a.parts; ++k) {
    if (steps < a.parts && part_begin(steps, k, a.parts) == part_begin(steps, k + 1, a.parts)) continue;  // no step
    const float4 x = reinterpret_cast<const float4*>(p + k * part_size)[c * 128 + row];
    sum = make_float4(sum.x + x.x, sum.y + x.y, sum.z + x.z, sum.w + x.w);
  }
  const bool is_k = c < HD / 4;
  const float m = is_k ? a.score.scale : 1.f;
  bf16* dst = is_k ? a.dk + t * a.lddk + kvh * static_cast<int64_t>(HD) + 4 * c
                   : a.dv + t * a.lddv + kvh * static_cast<int64_t>(HD) + 4 * (c - HD / 4);
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(sum.x * m, sum.y * m), pack_bf16(sum.z * m, sum.w * m));
}

// ------------------------------------------------------------------ dQ (Q-outer)
template <int HD>
struct SmemQ {
  static constexpr int NSL = HD / 64;
  static constexpr int KS = 3, VS = 2;               // K ring and V ring depths
  static constexpr int TILE = NSL * kSlice128;
  static constexpr int Q = 0;
  static constexpr int DO = Q + TILE;
  static constexpr int K = DO + TILE;                // KS tiles
  static constexpr int V = K + KS * TILE;            // VS tiles
  static constexpr int BAR = V + VS * TILE;
  static constexpr int BYTES = BAR + 320;            // the dynamic window is 1024-aligned (checked)
  static_assert(BYTES <= 232448, "dQ shared memory above the 227 KB per-CTA limit");
};

template <int HD, bool CAP, bool BIAS, int EW>
__global__ void __launch_bounds__(Roles<EW>::kThreads, 1)
    attn_span_dq_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do,
                        const __grid_constant__ CUtensorMap map_dq, const __grid_constant__ BwdArgs a) {
  using L = SmemQ<HD>;
  using R = Roles<EW>;
  constexpr int kUnroll = CAP ? 2 : 1;  // as in dK/dV
  constexpr int kCols = R::kCols;
  constexpr int KS = L::KS, VS = L::VS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  int* err = a.err;
  if (smem_addr(sm) & 1023) {  // the swizzled layouts need a 1024-byte aligned base
    if (threadIdx.x == 0) record_give_up(err, kErrTimeoutAttn);
    return;
  }
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint64_t* q_full = bar + 0;
  uint64_t* q_empty = bar + 1;           // every MMA that reads the item's Q and dO has completed
  uint64_t* k_full = bar + 2;            // [KS]
  uint64_t* k_empty = bar + 5;           // [KS]
  uint64_t* v_full = bar + 8;            // [VS]
  uint64_t* v_empty = bar + 10;          // [VS]
  uint64_t* sdp_full = bar + 12;         // the tile's S and dP are complete
  uint64_t* dp_free = bar + 13;          // every warp holds its dP columns in registers
  uint64_t* ds_first = bar + 14;         // every warp has written its first half of the tile's dS
  uint64_t* ds_last = bar + 15;          // [kLastHalfTurns]: and its second
  uint64_t* acc_full = bar + 17;         // the item's dQ MMAs have completed
  uint64_t* acc_empty = bar + 18;        // [kAccTurns]: every warp has read its part of dQ and staged it
  const ItemRing ring{bar + 20, bar + 22, reinterpret_cast<Item*>(bar + 25), err};
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + 24);
  uint64_t* drained = bar + 34;          // the MMA warp's last products have completed

  const int s = a.s, nh = a.nh;
  const int n_t = (s + 127) / 128, n_hb = nh * a.B;
  const int group = nh / a.nkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // item -> query tile (the last one sees the most keys under a causal mask), head, sequence
  struct Where {
    int qt, head, b;
  };
  auto where = [&](int lin) -> Where {
    const TileSlot slot = heavy_first_slot(lin, n_t, n_hb);
    return {n_t - 1 - slot.rank, slot.hb % nh, slot.hb / nh};
  };

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < KS; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    mbar_init(sdp_full, 1);
    mbar_init(dp_free, EW);
    mbar_init(ds_first, EW);
    for (int i = 0; i < kLastHalfTurns; ++i) mbar_init(&ds_last[i], EW);
    mbar_init(acc_full, 1);
    mbar_init(drained, 1);
    for (int i = 0; i < kAccTurns; ++i) mbar_init(&acc_empty[i], EW);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ring.full[i], 1);
      mbar_init(&ring.empty[i], R::kItemReaders);
    }
    fence_mbar_init();
    tma_prefetch_map(&map_q);
    tma_prefetch_map(&map_k);
    tma_prefetch_map(&map_v);
    tma_prefetch_map(&map_do);
  }
  if (warp == 1) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  wait_for_previous();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  const uint32_t tdP = tbase + 256, tdQ = tbase + 384;
  // g numbers the block's tiles across its items, n its items with a walk
  auto s_slot = [&](int g) { return tbase + (g & 1) * 128; };

  if (warp == 0) {
    // takes the items, each with the last loads of the one before, and loads the K ring
    if (lane == 0) {
      const int items = n_t * n_hb;
      auto take = [&](int lin) -> Item {
        Item it{-1, 0, 0, 0, 0, {0, 0, 0, 0}};
        if (lin < items) {
          const Where w = where(lin);
          it.lin = lin;
          it.hull = a.hulls[static_cast<int64_t>(w.b) * n_t + w.qt];
          it.first = it.hull.min_lo / 128;
          it.count = it.hull.max_hi > 0 ? (it.hull.max_hi + 127) / 128 - it.first : 0;
        }
        return it;
      };
      Item cur = take(blockIdx.x);
      bool ok = put_item(ring, 0, cur);
      int g = 0;
      for (int m = 1; ok && cur.lin >= 0; ++m) {
        const Where w = where(cur.lin);
        const int early = max(cur.count - kTakeAhead, 0);
        Item next;
        auto hand_on = [&] {
          next = take(gridDim.x + atomicAdd(a.taken, 1));
          return put_item(ring, m, next);
        };
        if (cur.count == 0 && !(ok = hand_on())) break;
        for (int j = 0; j < cur.count; ++j, ++g) {
          if (j == early && !(ok = hand_on())) break;
          const int st = g % KS;
          if (!(ok = mbar_wait(&k_empty[st], ((g / KS) & 1) ^ 1u, err, kErrTimeoutAttn))) break;
          mbar_arrive_expect_tx(&k_full[st], L::TILE);
          tma_load_4d(sm + L::K + st * L::TILE, &map_k, &k_full[st], 0, (cur.first + j) * 128,
                      w.head / group * (HD / 64), w.b);
        }
        cur = next;
      }
      ring_drain<KS>(k_full, g);
    }
  } else if (warp == R::kRingWarp) {
    if (lane == 0) {  // the V ring
      Item it;
      bool ok = true;
      int g = 0;
      for (int m = 0; ok && get_item(ring, m, it); ++m) {
        const Where w = where(it.lin);
        for (int j = 0; j < it.count; ++j, ++g) {
          const int st = g % VS;
          if (!(ok = mbar_wait(&v_empty[st], ((g / VS) & 1) ^ 1u, err, kErrTimeoutAttn))) break;
          mbar_arrive_expect_tx(&v_full[st], L::TILE);
          tma_load_4d(sm + L::V + st * L::TILE, &map_v, &v_full[st], 0, (it.first + j) * 128,
                      w.head / group * (HD / 64), w.b);
        }
      }
      ring_drain<VS>(v_full, g);
    }
  } else if (warp == R::kItemWarp) {
    // Q and dO, once per item, and the gradient of the item before, from the K stage of its last tile,
    // which is released when it has been read; first this block's share of the query ranges that dK/dV walks
    for (int64_t i = blockIdx.x; i < static_cast<int64_t>(a.B) * n_t; i += gridDim.x) {
      const Hull* hulls = a.hulls + i / n_t * n_t;
      const int k0 = static_cast<int>(i % n_t) * 128;
      int first = INT_MAX, last = -1;
      for (int q = lane; q < n_t; q += 32) {
        const Hull h = hulls[q];
        if (h.min_lo < k0 + 128 && h.max_hi > k0) {
          first = min(first, q);
          last = q;
        }
      }
      first = __reduce_min_sync(0xffffffffu, first);
      last = __reduce_max_sync(0xffffffffu, last);
      if (lane == 0) a.q_ranges[i] = make_int2(first, last);
    }
    if (lane == 0) {
      Item it;
      Where out{0, 0, 0};
      bool ok = true;
      auto store = [&](int n, int g) -> bool {  // item n, which ended with tile g
        if (!mbar_wait(turn_bar<kAccTurns>(acc_empty, n), turn_parity<kAccTurns>(n), err, kErrTimeoutAttn))
          return false;
        tma_store_4d(&map_dq, sm + L::K + (g % KS) * L::TILE, 0, out.qt * 128, out.head * (HD / 64), out.b);
        bulk_commit();
        bulk_wait_read();
        mbar_arrive(&k_empty[g % KS]);
        return true;
      };
      int n = 0, g = 0, stored = 0;
      for (int m = 0; ok && get_item(ring, m, it); ++m) {
        const Where w = where(it.lin);
        const int last = g - 1;
        if (it.count > 0) {
          if (!(ok = mbar_wait(q_empty, (n & 1) ^ 1u, err, kErrTimeoutAttn))) break;
          mbar_arrive_expect_tx(q_full, 2 * L::TILE);
          tma_load_4d(sm + L::Q, &map_q, q_full, 0, w.qt * 128, w.head * (HD / 64), w.b);
          tma_load_4d(sm + L::DO, &map_do, q_full, 0, w.qt * 128, w.head * (HD / 64), w.b);
        }
        if (stored < n) ok = store(stored++, last);
        if (it.count > 0) {
          out = w;
          g += it.count;
          ++n;
        }
      }
      if (ok && stored < n) store(stored, g - 1);
      if (n > 0) mbar_drain(q_full, (n - 1) & 1);
      bulk_wait();
    }
  } else if (warp == 1) {
    // the whole warp runs the issuing loop; elect.sync picks the lane that issues each MMA
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t idesc_acc = idesc_bf16_f32(128, HD, false, true);
    const uint64_t qd = smem_desc_sw128(smem_addr(sm + L::Q), 16, 1024);
    const uint64_t dd = smem_desc_sw128(smem_addr(sm + L::DO), 16, 1024);
    // S = Q K^T (dp = false) or dP = dO V^T of tile g into TMEM slot t, once its operand is in;
    // a V stage is released as soon as its dP has run
    auto scores = [&](int g, bool dp, uint32_t t) -> bool {
      uint64_t* full = dp ? &v_full[g % VS] : &k_full[g % KS];
      const uint32_t parity = dp ? (g / VS) & 1 : (g / KS) & 1;
      if (!mbar_wait_warp(full, parity, err, kErrTimeoutAttn)) return false;
      tc_fence_after();
      const uint64_t ad = dp ? dd : qd;
      const uint64_t bd =
          smem_desc_sw128(smem_addr(dp ? sm + L::V + (g % VS) * L::TILE : sm + L::K + (g % KS) * L::TILE), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        const uint32_t off = (kk >> 2) * kSlice128 + (kk & 3) * 32;
        umma_bf16_warp(t, desc_advance(ad, off), desc_advance(bd, off), idesc_s, kk > 0 ? 1u : 0u);
      }
      if (dp) umma_commit_warp(&v_empty[g % VS]);
      return true;
    };
    Item it;
    bool ok = true;
    for (int m = 0, n = 0, g = 0; ok && get_item_warp(ring, m, it); ++m) {
      const int total = it.count;
      if (total == 0) continue;
      // the item's first scores: its S slot was last read by products issued before, the dP slot is
      // free once every warp holds the last tile's columns
      if (!(ok = mbar_wait_warp(q_full, n & 1, err, kErrTimeoutAttn))) break;
      if (!(ok = scores(g, false, s_slot(g)))) break;
      if (g > 0 && !(ok = mbar_wait_warp(dp_free, (g - 1) & 1, err, kErrTimeoutAttn))) break;
      if (!(ok = scores(g, true, tdP))) break;
      umma_commit_warp(sdp_full);
      if (total == 1) umma_commit_warp(q_empty);
      for (int j = 0; j < total && ok; ++j, ++g) {
        // B operand of the dQ MMAs: the K tile read MN-major (16 keys per step)
        const uint64_t kd = smem_desc_sw128(smem_addr(sm + L::K + (g % KS) * L::TILE), kSlice128, 1024);
        // the next tile's S into the other S slot, whose dS was read by MMAs issued earlier
        if (j + 1 < total && !(ok = scores(g + 1, false, s_slot(g + 1)))) break;
        for (int h = 0; h < 2 && ok; ++h) {
          if (h == 1 && j + 1 < total) {  // the dP slot is free once every warp holds its columns
            if (!(ok = mbar_wait_warp(dp_free, g & 1, err, kErrTimeoutAttn))) break;
            tc_fence_after();
            if (!(ok = scores(g + 1, true, tdP))) break;
            umma_commit_warp(sdp_full);
            if (j + 2 == total) umma_commit_warp(q_empty);
          }
          if (!(ok = mbar_wait_warp(h ? turn_bar<kLastHalfTurns>(ds_last, g) : ds_first,
                                    h ? turn_parity<kLastHalfTurns>(g) : g & 1, err, kErrTimeoutAttn)))
            break;
          // the first product of an item overwrites the accumulator: the last item's has been read
          if (h == 0 && j == 0 && n > 0 &&
              !(ok = mbar_wait_warp(turn_bar<kAccTurns>(acc_empty, n - 1), turn_parity<kAccTurns>(n - 1), err,
                                    kErrTimeoutAttn)))
            break;
          tc_fence_after();
#pragma unroll
          for (int kk = 4 * h; kk < 4 * h + 4; ++kk)  // 16 keys per step; A (dS) from TMEM
            umma_bf16_tmem_a_warp(tdQ, s_slot(g) + kk * 16, desc_advance(kd, kk * 2048), idesc_acc,
                                  (j > 0 || kk > 0) ? 1u : 0u);
        }
        if (!ok) break;
        // the last tile's K stage is released once the gradient has left it
        if (j + 1 < total) umma_commit_warp(&k_empty[g % KS]);
        else umma_commit_warp(acc_full);
      }
      ++n;
    }
    mma_drain(drained);
  } else {
    const int sub = warp & 3;
    const int part = (warp - 2) >> 2;  // which kCols of each 64 key columns this warp takes
    const int row = sub * 32 + lane;
    const int elem = threadIdx.x - 64;
    const uint32_t tl = static_cast<uint32_t>(sub * 32) << 16;
    // a row's span and (-lse2, -delta) are loaded before the last item's gradient is stored
    struct Ahead {
      int2 seen;
      float2 lq;
    };
    auto look = [&](const Where& w) -> Ahead {
      const int q = w.qt * 128 + row;
      return {fetch_span(a.spans, w.b, q, s),
              a.lsd[(static_cast<int64_t>(w.b) * nh + w.head) * pad128(s) + q]};  // padded: q is inside
    };
    Item it, next_it;
    Where next_w{0, 0, 0};
    Ahead ahead{};
    bool ok = true, more = get_item_warp(ring, 0, next_it);
    if (more) {
      next_w = where(next_it.lin);
      ahead = look(next_w);
    }
    for (int m = 1, n = 0, g = 0; ok && more; ++m) {
      it = next_it;
      const Where w = next_w;
      const int q0 = w.qt * 128, q = q0 + row;
      const Hull hull = it.hull;
      const int2 seen = clamp_span(ahead.seen, s);
      const float2 nl2 = make_float2(ahead.lq.x, ahead.lq.x), ndl = make_float2(ahead.lq.y, ahead.lq.y);
      const float slope2 = BIAS ? a.slopes[w.head] * kLog2e : 0.f;
      const bool padded = hull.max_lo == INT_MAX;
      for (int j = 0; j < it.count && ok; ++j, ++g) {
        if (!(ok = mbar_wait_warp(sdp_full, g & 1, err, kErrTimeoutAttn))) break;
        tc_fence_after();
        const uint32_t ts = s_slot(g) + tl;
        const int key_tile = (it.first + j) * 128;
        const bool all = sees_all(hull, key_tile, key_tile + 128);
        // rows of K that nothing here may see: outside the hull, or padding among the tile's own rows
        const bool own = padded && key_tile == q0;
        const bool clean = own || key_tile < hull.min_lo || key_tile + 128 > hull.max_hi;
#pragma unroll kUnroll
        for (int h = 0; h < 2; ++h) {
          const int cb = h * 64 + part * kCols;
          float sv[kCols], dv[kCols];
          tmem_ld_pair<kCols>(ts + cb, tdP + tl + cb, sv, dv);
          if (h == 1) {  // every dP column of the tile is now in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(dp_free);
          }
          const int key0 = key_tile + cb;
          if constexpr (CAP) cap_tanh<kCols>(sv, a.score);
          const float d0 = static_cast<float>(q - key0);
#pragma unroll
          for (int k = 0; k < kCols / 2; ++k) {  // dS = P (dP - delta) z', two columns at a time
            float2 x = make_float2(sv[2 * k], sv[2 * k + 1]), y = make_float2(dv[2 * k], dv[2 * k + 1]);
            const float2 dist = make_float2(fabsf(d0 - (2 * k)), fabsf(d0 - (2 * k + 1)));
            p_and_ds<CAP, BIAS>(x, y, nl2, ndl, dist, slope2, a.score);
            dv[2 * k] = y.x;
            dv[2 * k + 1] = y.y;
          }
          if (!all) {
            const uint32_t vis = span_bits(seen, key0);
#pragma unroll
            for (int c = 0; c < kCols; ++c) dv[c] = vis >> c & 1u ? dv[c] : 0.f;
          }
          // dS goes back into TMEM over this warp's S columns (A operands of K-steps cb / 16 and on)
#pragma unroll
          for (int o = 0; o < kCols; o += 16) store_pairs16<kCols>(ts + cb + o, dv, o);
          tmem_st_wait();
          if (clean) {
            const int r = h * 64 + (elem & 63), which = elem >> 6, key = key_tile + r;
            bool gone = key < hull.min_lo || key >= hull.max_hi;
            if (own && !gone) {
              const int2 its = load_span(a.spans, w.b, key, s);  // key < max_hi <= s
              gone = its.x >= its.y;
            }
            if (which < L::NSL && gone) zero_slice_row(sm + L::K + (g % KS) * L::TILE + which * kSlice128, r);
            fence_proxy_async_smem();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(h ? turn_bar<kLastHalfTurns>(ds_last, g) : ds_first);
        }
      }
      if (!ok) break;
      more = get_item_warp(ring, m, next_it);
      if (more) {
        next_w = where(next_it.lin);
        ahead = look(next_w);
      }
      if (it.count == 0) {
        zero_rows<HD>(a.dq + (static_cast<int64_t>(w.b) * s + q0) * a.lddq + static_cast<int64_t>(w.head) * HD, a.lddq,
                      min(128, s - q0), elem, R::kElem);
        continue;
      }
      if (!(ok = mbar_wait_warp(acc_full, n & 1, err, kErrTimeoutAttn))) break;
      tc_fence_after();
      uint8_t* out = sm + L::K + ((g - 1) % KS) * L::TILE;
      stage_cols<HD * 4 / EW>(tdQ + tl, part * (HD * 4 / EW), a.score.scale, out, row);
      tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(turn_bar<kAccTurns>(acc_empty, n));
      ++n;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, 512);
}

template <int HD, bool CAP, bool BIAS>
cudaError_t launch(const AttnSpanArgs& g, const bf16* o, int64_t ldo, const float* lse, const bf16* dout, int64_t lddo,
                   BwdArgs a, float2* lsd, Hull* hulls, cudaStream_t st) {
  const int n_t = (g.s + 127) / 128;
  span_delta_kernel<HD><<<static_cast<unsigned>(n_t) * g.nh * g.B, 256, 0, st>>>(o, ldo, dout, lddo, lse, a.spans, lsd,
                                                                                 hulls, a.taken, g.s, g.nh, n_t);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  constexpr uint32_t nsl = HD / 64;  // one box carries every head_dim slice of a tile
  const int64_t s = g.s;
  const uint64_t qs = static_cast<uint64_t>(g.nh) * nsl, ks = static_cast<uint64_t>(g.nkv) * nsl;
  CUtensorMap mq, mk, mv, md, mdq, mdk, mdv;
  if (!tma_map_heads(&mq, g.q, s, g.B, g.ldq, s * g.ldq, qs, nsl, 128) ||
      !tma_map_heads(&mk, g.k, s, g.B, g.ldk, s * g.ldk, ks, nsl, 128) ||
      !tma_map_heads(&mv, g.v, s, g.B, g.ldv, s * g.ldv, ks, nsl, 128) ||
      !tma_map_heads(&md, dout, s, g.B, lddo, s * lddo, qs, nsl, 128) ||
      !tma_map_heads(&mdq, a.dq, s, g.B, a.lddq, s * a.lddq, qs, nsl, 128) ||
      !tma_map_heads(&mdk, a.dk, s, g.B, a.lddk, s * a.lddk, ks, nsl, 128) ||
      !tma_map_heads(&mdv, a.dv, s, g.B, a.lddv, s * a.lddv, ks, nsl, 128))
    return cudaErrorInvalidValue;
  constexpr int kQWarps = CAP ? 16 : 8, kKWarps = CAP ? 16 : 8;
  auto* dq = &attn_span_dq_kernel<HD, CAP, BIAS, kQWarps>;
  static std::atomic<uint64_t> dq_ready{0}, dkdv_ready[2] = {{0}, {0}};
  e = allow_smem(dq, SmemQ<HD>::BYTES, dq_ready);
  if (e != cudaSuccess) return e;
  const int sms = gemm_num_sms();
  const int64_t q_items = static_cast<int64_t>(n_t) * g.nh * g.B;
  const int64_t k_items = static_cast<int64_t>(n_t) * g.nkv * a.parts * g.B;
  e = launch_following(dq, dim3(static_cast<unsigned>(q_items < sms ? q_items : sms)), Roles<kQWarps>::kThreads,
                       SmemQ<HD>::BYTES, st, mq, mk, mv, md, mdq, a);
  if (e != cudaSuccess) return e;
  auto* dkdv = a.parts > 1 ? &attn_span_dkdv_kernel<HD, CAP, BIAS, kKWarps, true>
                         : &attn_span_dkdv_kernel<HD, CAP, BIAS, kKWarps, false>;
  e = allow_smem(dkdv, SmemKV<HD>::BYTES, dkdv_ready[a.parts > 1]);
  if (e != cudaSuccess) return e;
  e = launch_following(dkdv, dim3(static_cast<unsigned>(k_items < sms ? k_items : sms)), Roles<kKWarps>::kThreads,
                       SmemKV<HD>::BYTES, st, mq, mk, mv, md, mdk, mdv, a);
  if (e != cudaSuccess || a.parts == 1) return e;
  const dim3 join_grid(static_cast<unsigned>(n_t) * g.nkv * g.B, HD / 4);
  return launch_following(span_join_kernel<HD>, join_grid, 256, 0, st, a, n_t);
}

}  // namespace

// Parts that the walk of a key tile, its group's heads one after another, is cut into; each part is an
// item and leaves fp32 sums, which another kernel adds. With few key tiles the longest walk is the
// kernel's time: up to one an SM they are cut into about 512 (B 2, s 333, 4/1 heads: dK/dV 37 us in 6 blocks,
// 14 + 4 us in 24; 4096 tokens, 32/4 heads: the whole backward 578 us in 128 items, 388 in 256, 385 in 512;
// 8192, 16/2: 1104, 710, 691), unless more than one for two SMs are too short to pay for the sums, 1 KB a key and
// part written and read (whole backward, 128 items of up to 16 steps 75 us, in two 86, in four 91; 32 steps 107,
// 99, 109; 96 of up to 60 steps 162, 123, 121; 112 of up to 64, cut: 171, 132, 136). Up to two an SM are cut in
// two if they are very long (256 items, causal: of up to 160 steps 472 us, in two 479; 256 steps 705, 696; 384
// 1045, 1021; 512 1393 and 1359, 1353 and 1303 with 8/2 heads of 16384 tokens; 1024 2672, 2585). Both limits are
// above where the times cross, between 16 and 32 and between 160 and 256 steps.
static int walk_parts(int B, int s, int nh, int nkv) {
  const int group = nh / nkv;
  const int64_t n_t = pad128(s) / 128, items = n_t * nkv * B, longest = n_t * group;
  if (items > kSms) return items <= 2 * kSms && longest >= 512 && group > 1 ? 2 : 1;
  if (items > kSms / 2 && longest < 64) return 1;
  return static_cast<int>(std::min<int64_t>(group, (kPartItems + items / 2) / items));
}

uint64_t attn_span_bwd_scratch(int B, int s, int nh, int nkv, int hd) {
  const uint64_t sp = static_cast<uint64_t>(pad128(s));
  const uint64_t tile = sizeof(Hull) + sizeof(int2);
  const uint64_t lists = static_cast<uint64_t>(B) * (nh * sp * sizeof(float2) + sp / 128 * tile) + 16;
  const int parts = walk_parts(B, s, nh, nkv);
  const uint64_t sums = parts > 1 ? static_cast<uint64_t>(B) * nkv * parts * sp * 2 * hd * sizeof(float) : 0;
  return (lists + 15) / 16 * 16 + sums;
}

cudaError_t attn_span_bwd(const AttnSpanArgs& g, const bf16* o, int64_t ldo, const float* lse, const bf16* dout,
                          int64_t lddo, bf16* dq, int64_t lddq, bf16* dk, int64_t lddk, bf16* dv, int64_t lddv,
                          void* scratch, int* err, cudaStream_t st) {
  auto rows = [](const void* p, int64_t ld, int64_t cols) {
    return p && (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0 && ld >= cols && ld < (int64_t{1} << 31);
  };
  if (!attn_span_ok(g) || !lse || !err || !scratch || (reinterpret_cast<uintptr_t>(scratch) & 15))
    return cudaErrorInvalidValue;
  const int64_t qc = static_cast<int64_t>(g.nh) * g.hd, kc = static_cast<int64_t>(g.nkv) * g.hd;
  if (!rows(o, ldo, qc) || !rows(dout, lddo, qc) || !rows(dq, lddq, qc) || !rows(dk, lddk, kc) || !rows(dv, lddv, kc) ||
      static_cast<double>(g.s) * 2 * lddo >= 1e12 || static_cast<double>(g.s) * 2 * lddq >= 1e12 ||
      static_cast<double>(g.s) * 2 * lddk >= 1e12 || static_cast<double>(g.s) * 2 * lddv >= 1e12 ||
      ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(err)) & 3))
    return cudaErrorInvalidValue;
  // the walk of one key tile, up to ceil(s/128) tiles for each of its query heads at 2 to 3 us, stays well
  // below the limit of the waits for its end, and its steps below 2^19 (part_begin)
  if ((static_cast<int64_t>(g.s) + 127) / 128 * 128 * (g.nh / g.nkv) > kSpanMaxWalk) return cudaErrorInvalidValue;
  struct Columns {
    const bf16* p;
    int64_t ld, cols;
  };
  const Columns out[3] = {{dq, lddq, qc}, {dk, lddk, kc}, {dv, lddv, kc}};
  const Columns other[8] = {{g.q, g.ldq, qc}, {g.k, g.ldk, kc}, {g.v, g.ldv, kc}, {o, ldo, qc},
                            {dout, lddo, qc}, out[0], out[1], out[2]};
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < 5 + i; ++j)
      if (columns_overlap(out[i].p, out[i].ld, out[i].cols, other[j].p, other[j].ld, other[j].cols,
                          static_cast<int64_t>(g.B) * g.s))
        return cudaErrorInvalidValue;
  float2* lsd = static_cast<float2*>(scratch);
  Hull* hulls = reinterpret_cast<Hull*>(lsd + static_cast<int64_t>(g.B) * g.nh * pad128(g.s));
  const int64_t tiles = static_cast<int64_t>(g.B) * (pad128(g.s) / 128);
  int2* q_ranges = reinterpret_cast<int2*>(hulls + tiles);
  const uint64_t all = attn_span_bwd_scratch(g.B, g.s, g.nh, g.nkv, g.hd);
  const int parts = walk_parts(g.B, g.s, g.nh, g.nkv);
  const uint64_t sums = static_cast<uint64_t>(g.B) * g.nkv * parts * pad128(g.s) * 2 * g.hd * sizeof(float);
  float* partial = parts > 1 ? reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + (all - sums)) : nullptr;
  int* taken = reinterpret_cast<int*>(q_ranges + tiles);
  const BwdArgs a{{g.lo, g.hi}, g.slopes, lsd, hulls, q_ranges, taken, parts, partial, dq, dk, dv, lddq,
                  lddk, lddv, g.B, g.s, g.nh, g.nkv, score_args(g), err};
  return dispatch(g, [&](auto hd, auto cap, auto bias) {
    return launch<decltype(hd)::value, decltype(cap)::value, decltype(bias)::value>(g, o, ldo, lse, dout, lddo, a, lsd,
                                                                                    hulls, st);
  });
}

}  // namespace mt
