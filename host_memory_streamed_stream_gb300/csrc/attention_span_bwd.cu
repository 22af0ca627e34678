// Attention over spans, backward, on the tcgen05 tensor cores. Deterministic, no atomics.
//
// The kernels are those of the causal backward (attention_bwd_tc.cu): lsd pairs
// (-lse2, -delta) per query row; dK/dV with one CTA per (128-key tile, kv head, sequence) walking
// the 128-query tiles of its group's heads,
//     S^T = K Q^T, dP^T = V dO^T, P^T = 2^(z - lse2), dS^T = P^T (dP^T - delta) z',
//     dV += P^T dO, dK += dS^T Q;
// dQ with one CTA per (128-query tile, head, sequence) walking 128-key tiles, dQ += dS K; 128 x 128
// tiles, two 128-column score slots in TMEM, P and dS written back over the scores as bf16 pairs
// and read from TMEM, each in two halves of 64 columns. What differs:
//  * z is the capped and biased score and z' the cap's derivative 1 - tanh^2 = 4 r (1 - r);
//  * the delta kernel also writes each query tile's hull; a dQ CTA walks the key tiles of its hull,
//    a dK/dV CTA the query tiles from the first to the last whose hull meets its keys, and a tile
//    that meets nothing writes zeros;
//  * a tile that some row does not see whole is masked by words of 32 bits: a query row's span is a
//    run of bits over its key columns; in dK/dV, where a thread holds a key row, 32 lanes make the
//    runs of 32 query columns and transpose them through the warp;
//  * operand rows that must not count (padding rows, keys outside the hull) are zeroed in shared
//    memory before the products that sum over them, as 0 x NaN is NaN: padding may hold anything.
#include <cstdint>

#include "attention_span.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "tile_order.cuh"
#include "tma.h"

namespace mt {

namespace {

using namespace span;

constexpr int kThreads = 320;       // TMA warp, MMA warp, 8 elementwise warps
constexpr int kElem = 256;          // elementwise threads
constexpr int kCols = 32;           // score columns an elementwise warp takes per half tile
constexpr int kElemWarps = kElem / 32;  // arrivals per barrier phase (one elected lane per warp)
constexpr int kSlice128 = 128 * 128;  // bytes of a [128 rows][64 bf16] swizzle-atom-wide slice

__host__ __device__ __forceinline__ int pad128(int s) { return (s + 127) & ~127; }

// Pack the 16 values v[o .. o + 15] into 8 bf16 pairs and store them to 8 TMEM columns of this
// thread's lane (the A-operand layout: element k of a row in column k/2, even k in the low half).
__device__ __forceinline__ void store_pairs16(uint32_t taddr, const float (&v)[kCols], int o) {
  uint32_t w[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) w[c] = pack_bf16(v[o + 2 * c], v[o + 2 * c + 1]);
  tmem_st_8cols(taddr, w);
}

// Two 32-column TMEM loads (S and dP of one row) behind a single wait.
__device__ __forceinline__ void tmem_ld_2x32f(uint32_t ta, uint32_t tb, float (&a)[kCols], float (&b)[kCols]) {
  uint32_t ra[32], rb[32];
  tmem_ld_32cols(ta, ra);
  tmem_ld_32cols(tb, rb);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    a[i] = __uint_as_float(ra[i]);
    b[i] = __uint_as_float(rb[i]);
  }
}

// Half of one TMEM lane's fp32 row (columns [part*HD/2, +HD/2)), times `scale`, as bf16 to dst.
// acc = false: the accumulator was never written, the row is zero.
template <int HD>
__device__ __forceinline__ void half_row_out(uint32_t taddr, int part, float scale, bf16* dst, bool store, bool acc) {
#pragma unroll
  for (int c = 0; c < HD / 2; c += 32) {
    uint32_t r[32] = {};
    if (acc) {
      tmem_ld_32cols(taddr + part * (HD / 2) + c, r);
      tmem_ld_wait();
    }
    if (!store) continue;
    uint4* d = reinterpret_cast<uint4*>(dst + part * (HD / 2) + c);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      uint4 u;
      u.x = pack_bf16(__uint_as_float(r[8 * v + 0]) * scale, __uint_as_float(r[8 * v + 1]) * scale);
      u.y = pack_bf16(__uint_as_float(r[8 * v + 2]) * scale, __uint_as_float(r[8 * v + 3]) * scale);
      u.z = pack_bf16(__uint_as_float(r[8 * v + 4]) * scale, __uint_as_float(r[8 * v + 5]) * scale);
      u.w = pack_bf16(__uint_as_float(r[8 * v + 6]) * scale, __uint_as_float(r[8 * v + 7]) * scale);
      d[v] = u;
    }
  }
}

// ------------------------------------------------------------------ delta and hulls
// One block per 128 query rows of a (sequence, head): HD/8 lanes per row (16-byte loads). A row
// whose span is empty (or past the end, or without a finite score) gets (-inf, -0): every
// probability of it is 0. The blocks of head 0 also reduce their rows' spans to the tile's hull.
template <int HD>
__global__ void __launch_bounds__(256)
    span_delta_kernel(const bf16* __restrict__ o, int64_t ldo, const bf16* __restrict__ dout, int64_t lddo,
                      const float* __restrict__ lse, Spans spans, float2* __restrict__ lsd, Hull* __restrict__ hulls,
                      int s, int nh, int n_t) {
  constexpr int kLanes = HD / 8;  // lanes per row
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
  if (threadIdx.x == 0) hulls[static_cast<int64_t>(b) * n_t + tile] = join(join(parts[0], parts[1]), join(parts[2], parts[3]));
}

struct BwdArgs {
  Spans spans;
  const float* slopes;
  const float2* lsd;
  const Hull* hulls;
  bf16 *dq, *dk, *dv;
  int64_t lddq, lddk, lddv;
  int s, nh, nkv;
  ScoreArgs score;
  int* err;
};

// P and dS of one pair of columns: raw scores and dP in, P and dS out. nl = -lse2, nd = -delta of
// the columns' (or the row's) queries; dist = |i - j| where there is a bias.
template <bool CAP, bool BIAS>
__device__ __forceinline__ void p_and_ds(float2& sv, float2& dv, float2 nl, float2 nd, float2 dist, float slope2,
                                         const ScoreArgs& a) {
  float2 e, r;
  if constexpr (CAP) {
    r = make_float2(cap_r(sv.x, a), cap_r(sv.y, a));
    e = make_float2(cap_score(r.x, a), cap_score(r.y, a));
    if constexpr (BIAS) e = __ffma2_rn(make_float2(-slope2, -slope2), dist, e);
    e = __fadd2_rn(e, nl);
  } else {
    if constexpr (BIAS) nl = __ffma2_rn(make_float2(-slope2, -slope2), dist, nl);
    e = __ffma2_rn(sv, make_float2(a.scale_log2, a.scale_log2), nl);
  }
  const float2 p = make_float2(ex2(e.x), ex2(e.y));
  float2 d = __fmul2_rn(p, __fadd2_rn(dv, nd));
  if constexpr (CAP) {
    const float2 r4 = __fmul2_rn(r, make_float2(4.f, 4.f));
    d = __fmul2_rn(d, __ffma2_rn(make_float2(-r4.x, -r4.y), r, r4));
  }
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
  static constexpr int BYTES = BAR + 256;               // the dynamic window is 1024-aligned (checked)
  static_assert(BYTES <= 232448, "dK/dV shared memory above the 227 KB per-CTA limit");
};

template <int HD, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    attn_span_dkdv_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do,
                          const __grid_constant__ BwdArgs a) {
  using L = SmemKV<HD>;
  constexpr int QS = L::QS, DS = L::DS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  int* err = a.err;
  if (smem_addr(sm) & 1023) {  // the swizzled layouts need a 1024-byte aligned base
    if (threadIdx.x == 0) atomicCAS(err, 0, kErrTimeoutAttn);
    return;
  }
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint64_t* kv_full = bar + 0;
  uint64_t* q_full = bar + 1;            // [QS]
  uint64_t* q_empty = bar + 4;           // [QS]
  uint64_t* d_full = bar + 7;            // [DS]
  uint64_t* d_empty = bar + 9;           // [DS]
  uint64_t* sdp_full = bar + 11;         // [2]: the tile's S^T and that half of its dP^T are complete
  uint64_t* dp_free = bar + 13;          // every warp holds its dP^T columns in registers
  uint64_t* p_half = bar + 14;           // [2]: every warp has written P^T/dS^T of that half
  uint64_t* acc_done = bar + 16;         // the last tile's accumulating MMAs have completed
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + 17);
  int* q_range = reinterpret_cast<int*>(bar + 18);  // first and last query tile that meets the keys

  const int s = a.s, nh = a.nh, nkv = a.nkv;
  const int n_t = (s + 127) / 128;
  const TileSlot slot = heavy_first_slot(static_cast<int>(blockIdx.x), n_t, static_cast<int>(gridDim.x) / n_t);
  const int kt = slot.rank;  // the first key tile is seen by the most queries under a causal mask
  const int kvh = slot.hb % nkv, b = slot.hb / nkv;
  const int group = nh / nkv;
  const int k0 = kt * 128;
  const int sp = pad128(s);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Hull* hulls = a.hulls + static_cast<int64_t>(b) * n_t;

  if (threadIdx.x == 0) {
    q_range[0] = INT_MAX;
    q_range[1] = -1;
    mbar_init(kv_full, 1);
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
    mbar_init(dp_free, kElemWarps);
    mbar_init(&p_half[0], kElemWarps);
    mbar_init(&p_half[1], kElemWarps);
    mbar_init(acc_done, 1);
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
  __syncthreads();
  {
    int first = INT_MAX, last = -1;
    for (int i = threadIdx.x; i < n_t; i += kThreads) {
      const Hull h = hulls[i];
      if (h.min_lo < k0 + 128 && h.max_hi > k0) {
        first = min(first, i);
        last = i;
      }
    }
    first = __reduce_min_sync(0xffffffffu, first);
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0 && last >= 0) {
      atomicMin(&q_range[0], first);
      atomicMax(&q_range[1], last);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  const int qt0 = q_range[0];
  const int per_head = q_range[1] < 0 ? 0 : q_range[1] - qt0 + 1;
  const int total = group * per_head;
  const uint32_t tdV = tbase + 256, tdK = tbase + 256 + HD;
  auto s_slot = [&](int i) { return tbase + (i & 1) * 128; };        // S^T, then P^T | dS^T pairs
  auto d_slot = [&](int i) { return tbase + ((i & 1) ^ 1) * 128; };  // dP^T

  if (warp == 0) {
    // lane 0: K and V once, then the Q ring; lane 1: the dO ring with the (-lse2, -delta) pairs
    if (lane == 0 && total > 0) {
      mbar_arrive_expect_tx(kv_full, 2 * L::TILE);
      tma_load_4d(sm + L::K, &map_k, kv_full, 0, k0, kvh * (HD / 64), b);
      tma_load_4d(sm + L::V, &map_v, kv_full, 0, k0, kvh * (HD / 64), b);
      for (int i = 0; i < total; ++i) {
        const int st = i % QS;
        const int hq = kvh * group + i / per_head;
        const int q0 = (qt0 + i % per_head) * 128;
        if (!mbar_wait(&q_empty[st], ((i / QS) & 1) ^ 1u, err, kErrTimeoutAttn)) break;
        mbar_arrive_expect_tx(&q_full[st], L::TILE);
        tma_load_4d(sm + L::Q + st * L::TILE, &map_q, &q_full[st], 0, q0, hq * (HD / 64), b);
      }
    } else if (lane == 1) {
      for (int i = 0; i < total; ++i) {
        const int st = i % DS;
        const int hq = kvh * group + i / per_head;
        const int q0 = (qt0 + i % per_head) * 128;
        if (!mbar_wait(&d_empty[st], ((i / DS) & 1) ^ 1u, err, kErrTimeoutAttn)) break;
        mbar_arrive_expect_tx(&d_full[st], L::TILE + 1024);
        uint8_t* base = sm + L::DO + st * L::DSTAGE;
        tma_load_4d(base, &map_do, &d_full[st], 0, q0, hq * (HD / 64), b);
        bulk_load_1d(base + L::TILE, a.lsd + (static_cast<int64_t>(b) * nh + hq) * sp + q0, 1024, &d_full[st]);
      }
    }
  } else if (warp == 1) {
    // the whole warp runs the issuing loop; elect.sync picks the lane that issues each MMA
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t idesc_dh = idesc_bf16_f32(128, 64, false, false);
    constexpr uint32_t idesc_acc = idesc_bf16_f32(128, HD, false, true);
    const uint64_t kd = smem_desc_sw128(smem_addr(sm + L::K), 16, 1024);
    const uint64_t vd = smem_desc_sw128(smem_addr(sm + L::V), 16, 1024);
    bool ok = total > 0 && mbar_wait_warp(kv_full, 0, err, kErrTimeoutAttn);
    // S^T = K Q^T of tile i into TMEM slot t, once its Q tile is in
    auto s_scores = [&](int i, uint32_t t) -> bool {
      if (!mbar_wait_warp(&q_full[i % QS], (i / QS) & 1, err, kErrTimeoutAttn)) return false;
      tc_fence_after();
      const uint64_t bd = smem_desc_sw128(smem_addr(sm + L::Q + (i % QS) * L::TILE), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        const uint32_t off = (kk >> 2) * kSlice128 + (kk & 3) * 32;
        umma_bf16_warp(t, desc_advance(kd, off), desc_advance(bd, off), idesc_s, kk > 0 ? 1u : 0u);
      }
      return true;
    };
    // half h of dP^T = V dO^T of tile i into columns [64 h, 64 h + 64) of TMEM slot t
    auto dp_half = [&](int i, int h, uint32_t t) -> bool {
      if (!mbar_wait_warp(&d_full[i % DS], (i / DS) & 1, err, kErrTimeoutAttn)) return false;
      tc_fence_after();
      const uint64_t bd = smem_desc_sw128(smem_addr(sm + L::DO + (i % DS) * L::DSTAGE), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        const uint32_t off = (kk >> 2) * kSlice128 + (kk & 3) * 32;
        umma_bf16_warp(t + h * 64, desc_advance(vd, off), desc_advance(bd, off + h * 8192), idesc_dh,
                       kk > 0 ? 1u : 0u);
      }
      return true;
    };
    if (ok) ok = s_scores(0, s_slot(0)) && dp_half(0, 0, d_slot(0)) && dp_half(0, 1, d_slot(0));
    if (ok) {
      umma_commit_warp(&sdp_full[0]);
      umma_commit_warp(&sdp_full[1]);
    }
    for (int i = 0; i < total && ok; ++i) {
      // B operands of the accumulating MMAs: dO and Q tiles read MN-major (16 queries per step)
      const uint64_t qd = smem_desc_sw128(smem_addr(sm + L::Q + (i % QS) * L::TILE), kSlice128, 1024);
      const uint64_t dd = smem_desc_sw128(smem_addr(sm + L::DO + (i % DS) * L::DSTAGE), kSlice128, 1024);
      const uint32_t ts = s_slot(i);
      for (int h = 0; h < 2 && ok; ++h) {
        if (h == 1 && i + 1 < total) {
          // the next tile's first dP^T half over this tile's first P^T/dS^T pairs, after the MMAs
          // reading them; then the next S^T into the dP^T slot, free once every warp holds its columns
          if (!(ok = dp_half(i + 1, 0, d_slot(i + 1)))) break;
          if (!(ok = mbar_wait_warp(dp_free, i & 1, err, kErrTimeoutAttn))) break;
          tc_fence_after();
          if (!(ok = s_scores(i + 1, s_slot(i + 1)))) break;
          umma_commit_warp(&sdp_full[0]);
        }
        if (!(ok = mbar_wait_warp(&p_half[h], i & 1, err, kErrTimeoutAttn))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 4 * h; kk < 4 * h + 4; ++kk) {  // 16 queries per step; A (P^T, dS^T) from TMEM
          const uint32_t acc = (i > 0 || kk > 0) ? 1u : 0u;
          umma_bf16_tmem_a_warp(tdV, ts + kk * 16, desc_advance(dd, kk * 2048), idesc_acc, acc);
          umma_bf16_tmem_a_warp(tdK, ts + kk * 16 + 8, desc_advance(qd, kk * 2048), idesc_acc, acc);
        }
      }
      if (!ok) break;
      umma_commit_warp(&q_empty[i % QS]);
      umma_commit_warp(&d_empty[i % DS]);
      if (i + 1 < total) {
        // the next tile's second dP^T half over this tile's last P^T/dS^T pairs
        if (!(ok = dp_half(i + 1, 1, d_slot(i + 1)))) break;
        umma_commit_warp(&sdp_full[1]);
      } else {
        umma_commit_warp(acc_done);
      }
    }
  } else {
    const int sub = warp & 3;
    const int part = (warp - 2) >> 2;  // which 32 of each 64 query columns this warp takes
    const int row = sub * 32 + lane;
    const int key = k0 + row;
    const int elem = threadIdx.x - 64;
    const uint32_t tl = static_cast<uint32_t>(sub * 32) << 16;
    bool ok = true;
    Hull hull = total > 0 ? hulls[qt0] : Hull{0, 0, 0, 0};
    for (int i = 0; i < total && ok; ++i) {
      const int q0 = (qt0 + i % per_head) * 128;
      const bool all = sees_all(hull, k0, k0 + 128), padded = hull.max_lo == INT_MAX;
      if (i + 1 < total) hull = hulls[qt0 + (i + 1) % per_head];
      uint32_t vis[2] = {~0u, ~0u};  // visible query columns of this thread's key, per half
      if (!all) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int q = q0 + h * 64 + part * kCols + lane;
          const int2 seen = q < s ? load_span(a.spans, b, q, s) : make_int2(0, 0);
          vis[h] = warp_transpose(span_bits(seen, k0 + sub * 32), lane);
        }
      }
      const float slope2 = BIAS ? __ldg(a.slopes + kvh * group + i / per_head) * kLog2e : 0.f;
      uint8_t* dstage = sm + L::DO + (i % DS) * L::DSTAGE;
      const float4* lsd_s = reinterpret_cast<const float4*>(dstage + L::TILE);
      // the pairs were copied with the tile's dO: observe that copy before reading them
      if (!(ok = mbar_wait_warp(&d_full[i % DS], (i / DS) & 1, err, kErrTimeoutAttn))) break;
      const uint32_t ts = s_slot(i) + tl, td = d_slot(i) + tl;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!ok) break;
        if (!(ok = mbar_wait_warp(&sdp_full[h], i & 1, err, kErrTimeoutAttn))) break;
        tc_fence_after();
        const int cb = h * 64 + part * kCols;  // this warp's score columns [cb, cb + 32)
        float sv[kCols], dv[kCols];
        tmem_ld_2x32f(ts + cb, td + cb, sv, dv);
        if (h == 1) {  // every dP^T column of the tile is now in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(dp_free);
        }
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
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            const bool keep = vis[h] >> c & 1u;
            sv[c] = keep ? sv[c] : 0.f;
            dv[c] = keep ? dv[c] : 0.f;
          }
        }
        // P^T pairs then dS^T pairs over this warp's own 16 S^T columns: the A operands of
        // K-step cb / 16 of the accumulating MMAs
#pragma unroll
        for (int o = 0; o < kCols; o += 16) {
          store_pairs16(ts + cb + o, sv, o);
          store_pairs16(ts + cb + o + 8, dv, o);
        }
        tmem_st_wait();
        if (padded) {  // this half's Q and dO rows that are padding: no product may read them
          const int r = h * 64 + (elem & 63), which = elem >> 6;
          if (which < 2 * L::NSL && reinterpret_cast<const float2*>(lsd_s)[r].x == -INFINITY) {
            uint8_t* tile = which < L::NSL ? sm + L::Q + (i % QS) * L::TILE : dstage;
            zero_slice_row(tile + (which % L::NSL) * kSlice128, r);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_half[h]);
      }
    }
    if (ok && (total == 0 || mbar_wait_warp(acc_done, 0, err, kErrTimeoutAttn))) {
      tc_fence_after();
      const int64_t t = static_cast<int64_t>(b) * s + key;
      half_row_out<HD>(tdK + tl, part, a.score.scale, a.dk + t * a.lddk + static_cast<int64_t>(kvh) * HD, key < s,
                       total > 0);
      half_row_out<HD>(tdV + tl, part, 1.f, a.dv + t * a.lddv + static_cast<int64_t>(kvh) * HD, key < s, total > 0);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, 512);
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
  static constexpr int BYTES = BAR + 256;            // the dynamic window is 1024-aligned (checked)
  static_assert(BYTES <= 232448, "dQ shared memory above the 227 KB per-CTA limit");
};

template <int HD, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1)
    attn_span_dq_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do,
                        const __grid_constant__ BwdArgs a) {
  using L = SmemQ<HD>;
  constexpr int KS = L::KS, VS = L::VS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  int* err = a.err;
  if (smem_addr(sm) & 1023) {  // the swizzled layouts need a 1024-byte aligned base
    if (threadIdx.x == 0) atomicCAS(err, 0, kErrTimeoutAttn);
    return;
  }
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint64_t* q_full = bar + 0;
  uint64_t* k_full = bar + 1;            // [KS]
  uint64_t* k_empty = bar + 4;           // [KS]
  uint64_t* v_full = bar + 7;            // [VS]
  uint64_t* v_empty = bar + 9;           // [VS]
  uint64_t* sdp_full = bar + 11;         // the tile's S and dP are complete
  uint64_t* dp_free = bar + 12;          // every warp holds its dP columns in registers
  uint64_t* ds_half = bar + 13;          // [2]
  uint64_t* dq_done = bar + 15;          // the last tile's dQ MMAs have completed
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + 16);
  uint32_t* empty_rows = reinterpret_cast<uint32_t*>(bar + 18);  // [4] bit r: row r of the 32 is padding

  const int s = a.s, nh = a.nh;
  const int n_t = (s + 127) / 128;
  const TileSlot slot = heavy_first_slot(static_cast<int>(blockIdx.x), n_t, static_cast<int>(gridDim.x) / n_t);
  const int qt = n_t - 1 - slot.rank;  // the last query tile sees the most keys under a causal mask
  const int head = slot.hb % nh, b = slot.hb / nh;
  const int kvh = head / (nh / a.nkv);
  const int q0 = qt * 128;
  const Hull hull = a.hulls[static_cast<int64_t>(b) * n_t + qt];
  const int j0 = hull.min_lo / 128;
  const int n_kv = hull.max_hi > 0 ? (hull.max_hi + 127) / 128 - j0 : 0;  // key tiles j0 .. j0 + n_kv - 1
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp & 3;
  const int part = (warp - 2) >> 2;  // which 32 of each 64 key columns this elementwise warp takes
  const int row = sub * 32 + lane;
  const int q = q0 + row;
  int2 seen = make_int2(0, 0);
  if (warp >= 2) {
    if (q < s) seen = load_span(a.spans, b, q, s);
    const uint32_t none = __ballot_sync(0xffffffffu, seen.x >= seen.y);
    if (lane == 0 && part == 0) empty_rows[sub] = none;
  }

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < KS; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    mbar_init(sdp_full, 1);
    mbar_init(dp_free, kElemWarps);
    mbar_init(&ds_half[0], kElemWarps);
    mbar_init(&ds_half[1], kElemWarps);
    mbar_init(dq_done, 1);
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  const uint32_t tdP = tbase + 256, tdQ = tbase + 384;
  auto s_slot = [&](int j) { return tbase + (j & 1) * 128; };

  if (warp == 0) {
    // lane 0: Q and dO once, then the K ring; lane 1: the V ring
    if (lane == 0 && n_kv > 0) {
      mbar_arrive_expect_tx(q_full, 2 * L::TILE);
      tma_load_4d(sm + L::Q, &map_q, q_full, 0, q0, head * (HD / 64), b);
      tma_load_4d(sm + L::DO, &map_do, q_full, 0, q0, head * (HD / 64), b);
      for (int j = 0; j < n_kv; ++j) {
        const int st = j % KS;
        if (!mbar_wait(&k_empty[st], ((j / KS) & 1) ^ 1u, err, kErrTimeoutAttn)) break;
        mbar_arrive_expect_tx(&k_full[st], L::TILE);
        tma_load_4d(sm + L::K + st * L::TILE, &map_k, &k_full[st], 0, (j0 + j) * 128, kvh * (HD / 64), b);
      }
    } else if (lane == 1) {
      for (int j = 0; j < n_kv; ++j) {
        const int st = j % VS;
        if (!mbar_wait(&v_empty[st], ((j / VS) & 1) ^ 1u, err, kErrTimeoutAttn)) break;
        mbar_arrive_expect_tx(&v_full[st], L::TILE);
        tma_load_4d(sm + L::V + st * L::TILE, &map_v, &v_full[st], 0, (j0 + j) * 128, kvh * (HD / 64), b);
      }
    }
  } else if (warp == 1) {
    // the whole warp runs the issuing loop; elect.sync picks the lane that issues each MMA
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t idesc_acc = idesc_bf16_f32(128, HD, false, true);
    const uint64_t qd = smem_desc_sw128(smem_addr(sm + L::Q), 16, 1024);
    const uint64_t dd = smem_desc_sw128(smem_addr(sm + L::DO), 16, 1024);
    bool ok = n_kv > 0 && mbar_wait_warp(q_full, 0, err, kErrTimeoutAttn);
    // S = Q K^T (dp = false) or dP = dO V^T of tile j into TMEM slot t, once its operand is in;
    // a V stage is released as soon as its dP has run
    auto scores = [&](int j, bool dp, uint32_t t) -> bool {
      uint64_t* full = dp ? &v_full[j % VS] : &k_full[j % KS];
      const uint32_t parity = dp ? (j / VS) & 1 : (j / KS) & 1;
      if (!mbar_wait_warp(full, parity, err, kErrTimeoutAttn)) return false;
      tc_fence_after();
      const uint64_t ad = dp ? dd : qd;
      const uint64_t bd =
          smem_desc_sw128(smem_addr(dp ? sm + L::V + (j % VS) * L::TILE : sm + L::K + (j % KS) * L::TILE), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        const uint32_t off = (kk >> 2) * kSlice128 + (kk & 3) * 32;
        umma_bf16_warp(t, desc_advance(ad, off), desc_advance(bd, off), idesc_s, kk > 0 ? 1u : 0u);
      }
      if (dp) umma_commit_warp(&v_empty[j % VS]);
      return true;
    };
    if (ok) ok = scores(0, false, s_slot(0)) && scores(0, true, tdP);
    if (ok) umma_commit_warp(sdp_full);
    for (int j = 0; j < n_kv && ok; ++j) {
      // B operand of the dQ MMAs: the K tile read MN-major (16 keys per step)
      const uint64_t kd = smem_desc_sw128(smem_addr(sm + L::K + (j % KS) * L::TILE), kSlice128, 1024);
      // the next tile's S into the other S slot, whose dS was read by MMAs issued earlier
      if (j + 1 < n_kv && !(ok = scores(j + 1, false, s_slot(j + 1)))) break;
      for (int h = 0; h < 2 && ok; ++h) {
        if (h == 1 && j + 1 < n_kv) {  // the dP slot is free once every warp holds its columns
          if (!(ok = mbar_wait_warp(dp_free, j & 1, err, kErrTimeoutAttn))) break;
          tc_fence_after();
          if (!(ok = scores(j + 1, true, tdP))) break;
          umma_commit_warp(sdp_full);
        }
        if (!(ok = mbar_wait_warp(&ds_half[h], j & 1, err, kErrTimeoutAttn))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 4 * h; kk < 4 * h + 4; ++kk)  // 16 keys per step; A (dS) from TMEM
          umma_bf16_tmem_a_warp(tdQ, s_slot(j) + kk * 16, desc_advance(kd, kk * 2048), idesc_acc,
                                (j > 0 || kk > 0) ? 1u : 0u);
      }
      if (!ok) break;
      umma_commit_warp(&k_empty[j % KS]);
      if (j == n_kv - 1) umma_commit_warp(dq_done);
    }
  } else {
    const int elem = threadIdx.x - 64;
    const bool padded = (empty_rows[0] | empty_rows[1] | empty_rows[2] | empty_rows[3]) != 0;
    const uint32_t tl = static_cast<uint32_t>(sub * 32) << 16;
    const float2 lq = a.lsd[(static_cast<int64_t>(b) * nh + head) * pad128(s) + q];  // padded: q is inside
    const float2 nl2 = make_float2(lq.x, lq.x), ndl = make_float2(lq.y, lq.y);
    const float slope2 = BIAS ? a.slopes[head] * kLog2e : 0.f;
    bool ok = true;
    for (int j = 0; j < n_kv && ok; ++j) {
      if (!(ok = mbar_wait_warp(sdp_full, j & 1, err, kErrTimeoutAttn))) break;
      tc_fence_after();
      const uint32_t ts = s_slot(j) + tl;
      const int key_tile = (j0 + j) * 128;
      const bool all = sees_all(hull, key_tile, key_tile + 128);
      // rows of K that nothing here may see: outside the hull, or padding among the tile's own rows
      const bool own = padded && key_tile == q0;
      const bool clean = own || key_tile < hull.min_lo || key_tile + 128 > hull.max_hi;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int cb = h * 64 + part * kCols;
        float sv[kCols], dv[kCols];
        tmem_ld_2x32f(ts + cb, tdP + tl + cb, sv, dv);
        if (h == 1) {  // every dP column of the tile is now in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(dp_free);
        }
        const int key0 = key_tile + cb;
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
        // dS goes back into TMEM over this warp's S columns (A operand of K-step cb / 16)
#pragma unroll
        for (int o = 0; o < kCols; o += 16) store_pairs16(ts + cb + o, dv, o);
        tmem_st_wait();
        if (clean) {
          const int r = h * 64 + (elem & 63), which = elem >> 6, key = key_tile + r;
          const bool pad = own && (empty_rows[r >> 5] >> (r & 31) & 1u);
          if (which < L::NSL && (key < hull.min_lo || key >= hull.max_hi || pad))
            zero_slice_row(sm + L::K + (j % KS) * L::TILE + which * kSlice128, r);
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ds_half[h]);
      }
    }
    if (ok && (n_kv == 0 || mbar_wait_warp(dq_done, 0, err, kErrTimeoutAttn))) {
      tc_fence_after();
      half_row_out<HD>(tdQ + tl, part, a.score.scale,
                       a.dq + (static_cast<int64_t>(b) * s + q) * a.lddq + static_cast<int64_t>(head) * HD, q < s,
                       n_kv > 0);
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
                                                                                 hulls, g.s, g.nh, n_t);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  constexpr uint32_t nsl = HD / 64;  // one box carries every head_dim slice of a tile
  const int64_t s = g.s;
  const uint64_t qs = static_cast<uint64_t>(g.nh) * nsl, ks = static_cast<uint64_t>(g.nkv) * nsl;
  CUtensorMap mq, mk, mv, md;
  if (!tma_map_heads(&mq, g.q, s, g.B, g.ldq, s * g.ldq, qs, nsl, 128) ||
      !tma_map_heads(&mk, g.k, s, g.B, g.ldk, s * g.ldk, ks, nsl, 128) ||
      !tma_map_heads(&mv, g.v, s, g.B, g.ldv, s * g.ldv, ks, nsl, 128) ||
      !tma_map_heads(&md, dout, s, g.B, lddo, s * lddo, qs, nsl, 128))
    return cudaErrorInvalidValue;
  auto* dq = &attn_span_dq_kernel<HD, CAP, BIAS>;
  e = cudaFuncSetAttribute(dq, cudaFuncAttributeMaxDynamicSharedMemorySize, SmemQ<HD>::BYTES);
  if (e != cudaSuccess) return e;
  dq<<<static_cast<unsigned>(n_t) * g.nh * g.B, kThreads, SmemQ<HD>::BYTES, st>>>(mq, mk, mv, md, a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  auto* dkdv = &attn_span_dkdv_kernel<HD, CAP, BIAS>;
  e = cudaFuncSetAttribute(dkdv, cudaFuncAttributeMaxDynamicSharedMemorySize, SmemKV<HD>::BYTES);
  if (e != cudaSuccess) return e;
  dkdv<<<static_cast<unsigned>(n_t) * g.nkv * g.B, kThreads, SmemKV<HD>::BYTES, st>>>(mq, mk, mv, md, a);
  return cudaGetLastError();
}

}  // namespace

uint64_t attn_span_bwd_scratch(int B, int s, int nh) {
  const uint64_t sp = static_cast<uint64_t>(pad128(s));
  return static_cast<uint64_t>(B) * (nh * sp * sizeof(float2) + sp / 128 * sizeof(Hull));
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
      static_cast<double>(g.s) * 2 * lddo >= 1e12)
    return cudaErrorInvalidValue;
  float2* lsd = static_cast<float2*>(scratch);
  Hull* hulls = reinterpret_cast<Hull*>(lsd + static_cast<int64_t>(g.B) * g.nh * pad128(g.s));
  const BwdArgs a{{g.lo, g.hi}, g.slopes, lsd, hulls, dq, dk, dv, lddq, lddk, lddv, g.s, g.nh, g.nkv, score_args(g), err};
  return dispatch(g, [&](auto hd, auto cap, auto bias) {
    return launch<decltype(hd)::value, decltype(cap)::value, decltype(bias)::value>(g, o, ldo, lse, dout, lddo, a, lsd,
                                                                                    hulls, st);
  });
}

}  // namespace mt
