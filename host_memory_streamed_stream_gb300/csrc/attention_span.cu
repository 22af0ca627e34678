// Attention over spans, forward, on the tcgen05 tensor cores: every query row sees its own range of
// keys, scores may be capped by a tanh and lowered by a distance bias, q, k and v are separate
// column ranges with their own strides.
//
// The pipeline is that of the causal kernel (attention_tc.cu): one CTA per (128-query tile, query
// head, sequence), two CTAs per SM; warp 0 loads Q once and K and V tiles of 64 keys into two
// rings, warp 1 issues S_j = Q K_j^T into one of two TMEM score buffers and O += P_j V_j, warps
// 2..5 hold one query row per thread (or, see kBounded, warps 2..9 half a row). What differs:
//  * the softmax warps first reduce their rows' spans to the tile's hull; the key tiles that are
//    loaded and multiplied are those of [min_lo, max_hi), the masked path is taken where some row
//    does not see the whole tile, and a tile of empty rows writes zeros and loads nothing;
//  * a row may see nothing in a tile, or at all: its running maximum is then -inf, which enters the
//    exponentials as 0 (all of them are 2^-inf = 0), and at the end o = 0 and lse = -inf;
//  * rows of V that no query row of the tile may see (keys outside the hull, padding rows inside
//    the tile's own range) are zeroed in shared memory before the product, as 0 x NaN is NaN:
//    padding may hold anything.
//
// Measured (head size 128): two 4096-token sequences of 32 heads, packed documents of 700 tokens on
// average, 108 us (1.28 times the visible scores are computed in the tiles, at 890 TFLOP/s: blocks are
// eleven tiles long, two of five tiles take the masked path, and the longest blocks end last); the same
// sequences causal 209 us, 1310 TFLOP/s; 16384 tokens, 8/2 heads, causal 352 us, 1560 TFLOP/s, capped with
// a prefix 598 us, 980 TFLOP/s, bound by the elementwise warps' instructions. Blocks that go on to further
// items (taken over from the grid) instead of ending came out slower, 135 us for the packed documents:
// the look-ahead costs the tile loop more than the second CTA of an SM leaves uncovered.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attention_span.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "tile_order.cuh"
#include "tma.h"

namespace mt {

namespace {

using namespace span;

constexpr int kKeys = 64;              // keys per tile
constexpr int kSlice128 = 128 * 128;   // [128 rows][64 bf16]: one 128-byte swizzle atom wide
constexpr int kSlice64 = 64 * 128;     // [64 rows][64 bf16]
constexpr float kLazyRescale = 8.f;    // log2 units
// Capped scores lie in [-c log2(e), c log2(e)]. Up to kBounded log2 units (c <= 50.5) the exponentials
// need no running maximum: 2^(z - kBoundedRef) stays between 2^-81 and 2^65, so the sums over 2^22 keys
// stay within fp32 for values between 2^-40 and 2^40. Without it a row's two halves of a tile have nothing to tell
// each other, so two threads share a row (eight softmax warps): the tanh's polynomial is long, and
// four warps a block left the FMA units idle half of the time (16384 tokens, 8/2 heads, capped:
// 691 us with the running maximum and one thread a row).
constexpr float kBounded = 73.f, kBoundedRef = 8.f;
constexpr int kKStages = 3;            // K ring depth
constexpr int kVStages = 2;            // V ring depth

template <int HD>
struct Smem {
  static constexpr int NSL = HD / 64;               // 64-wide slices of head_dim
  static constexpr int Q = 0;                       // NSL x [128 queries][64]
  static constexpr int TILE = NSL * kSlice64;       // one K or V tile: NSL x [64 keys][64]
  static constexpr int K = Q + NSL * kSlice128;     // kKStages K tiles
  static constexpr int V = K + kKStages * TILE;     // kVStages V tiles
  static constexpr int BAR = V + kVStages * TILE;   // barriers, TMEM address, hulls, padding rows
  static constexpr int BYTES = BAR + 256;           // the dynamic window is 1024-aligned (checked)
  static_assert(2 * (BYTES + 1024) <= 233472, "two CTAs no longer fit an SM");
};

struct FwdArgs {
  Spans spans;
  const float* slopes;
  bf16* o;
  int64_t ldo;
  float* lse;
  int s, nh, nkv, head_group;
  ScoreArgs score;
  int* err;
};

template <int HD, bool CAP, bool BIAS, bool BOUNDED>
__global__ void __launch_bounds__(BOUNDED ? 320 : 192, 2)
    attn_span_fwd_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v, const __grid_constant__ FwdArgs a) {
  using L = Smem<HD>;
  constexpr int kCols = BOUNDED ? 32 : 64;      // score columns of a softmax thread
  constexpr int kSoftmax = BOUNDED ? 256 : 128;  // softmax threads
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  int* err = a.err;
  if (smem_addr(sm) & 1023) {  // the swizzled layouts need a 1024-byte aligned base
    if (threadIdx.x == 0) record_give_up(err, kErrTimeoutAttn);
    return;
  }
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR);
  uint64_t* q_full = bar + 0;
  uint64_t* k_full = bar + 1;    // [kKStages]
  uint64_t* k_empty = bar + 4;   // [kKStages]
  uint64_t* v_full = bar + 7;    // [kVStages]
  uint64_t* v_empty = bar + 9;   // [kVStages]
  uint64_t* s_full = bar + 11;   // [2]
  uint64_t* p_full = bar + 13;   // [2]
  uint64_t* pv_done = bar + 15;  // one phase per O += P_j V_j (the lazy rescale waits on it)
  uint64_t* o_done = bar + 16;   // once: every O += P_j V_j of the tile has completed
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + 17);
  Hull* hulls = reinterpret_cast<Hull*>(bar + 18);               // [4] of the softmax warps
  uint32_t* empty_rows = reinterpret_cast<uint32_t*>(bar + 26);  // [4] bit r: the warp's row r is padding
  uint64_t* drained = bar + 28;  // the MMA warp's last products have completed

  const int s = a.s, nh = a.nh;
  const int n_qt = (s + 127) / 128;
  const TileSlot slot = heavy_first_slot(static_cast<int>(blockIdx.x), n_qt, static_cast<int>(gridDim.x) / n_qt,
                                         a.head_group);
  const int qt = n_qt - 1 - slot.rank;  // the last query tile sees the most keys under a causal mask
  const int head = slot.hb % nh, b = slot.hb / nh;
  const int kvh = head / (nh / a.nkv);
  const int q0 = qt * 128;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp & 3;
  const int row = sub * 32 + lane;  // of the softmax warps
  const int q = q0 + row;

  int2 seen = make_int2(0, 0);
  if (warp >= 2) {
    if (q < s) seen = load_span(a.spans, b, q, s);
    const Hull h = warp_hull(row_hull(seen, q < s));
    const uint32_t none = __ballot_sync(0xffffffffu, seen.x >= seen.y);
    if (lane == 0 && warp < 6) {
      hulls[sub] = h;
      empty_rows[sub] = none;
    }
  }
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kSoftmax);
    }
    mbar_init(pv_done, 1);
    mbar_init(o_done, 1);
    mbar_init(drained, 1);
    fence_mbar_init();
    tma_prefetch_map(&map_q);
    tma_prefetch_map(&map_k);
    tma_prefetch_map(&map_v);
  }
  if (warp == 1) {
    tmem_alloc(tslot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  const uint32_t tS0 = tbase, tO = tbase + 2 * kKeys;
  const Hull hull = join(join(hulls[0], hulls[1]), join(hulls[2], hulls[3]));
  const int j0 = hull.min_lo / kKeys;
  const int n_kv = hull.max_hi > 0 ? (hull.max_hi + kKeys - 1) / kKeys - j0 : 0;  // key tiles j0 .. j0 + n_kv - 1

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producers
    if (lane == 0 && n_kv > 0) {
      mbar_arrive_expect_tx(q_full, L::NSL * kSlice128);
      tma_load_4d(sm + L::Q, &map_q, q_full, 0, q0, head * (HD / 64), b);  // all head_dim slices at once
      int j = 0;
      for (; j < n_kv; ++j) {
        const int st = j % kKStages;
        if (!mbar_wait(&k_empty[st], ((j / kKStages) & 1) ^ 1u, err, kErrTimeoutAttn)) break;
        mbar_arrive_expect_tx(&k_full[st], L::TILE);
        tma_load_4d(sm + L::K + st * L::TILE, &map_k, &k_full[st], 0, (j0 + j) * kKeys, kvh * (HD / 64), b);
      }
      mbar_drain(q_full, 0);
      ring_drain<kKStages>(k_full, j);
    } else if (lane == 1) {
      int j = 0;
      for (; j < n_kv; ++j) {
        const int st = j % kVStages;
        if (!mbar_wait(&v_empty[st], ((j / kVStages) & 1) ^ 1u, err, kErrTimeoutAttn)) break;
        mbar_arrive_expect_tx(&v_full[st], L::TILE);
        tma_load_4d(sm + L::V + st * L::TILE, &map_v, &v_full[st], 0, (j0 + j) * kKeys, kvh * (HD / 64), b);
      }
      ring_drain<kVStages>(v_full, j);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, kKeys, false, false);
    constexpr uint32_t idesc_o = idesc_bf16_f32(128, HD, false, true);
    const uint64_t qd = smem_desc_sw128(smem_addr(sm + L::Q), 16, 1024);
    bool ok = n_kv > 0 && mbar_wait_warp(q_full, 0, err, kErrTimeoutAttn);
    // score buffer j&1 last held P_{j-2}, read by O += P_{j-2} V_{j-2}, which was issued
    // before S_j: MMAs run in issue order, so no wait is needed.
    auto issue_s = [&](int j) -> bool {
      const int st = j & 1, ks = j % kKStages;
      if (!mbar_wait_warp(&k_full[ks], (j / kKStages) & 1, err, kErrTimeoutAttn)) return false;
      tc_fence_after();
      const uint64_t kd = smem_desc_sw128(smem_addr(sm + L::K + ks * L::TILE), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        const uint32_t a_off = (kk >> 2) * kSlice128 + (kk & 3) * 32;
        const uint32_t b_off = (kk >> 2) * kSlice64 + (kk & 3) * 32;
        umma_bf16_warp(tS0 + st * kKeys, desc_advance(qd, a_off), desc_advance(kd, b_off), idesc_s, kk > 0 ? 1u : 0u);
      }
      umma_commit_warp(&s_full[st]);
      umma_commit_warp(&k_empty[ks]);
      return true;
    };
    if (ok) ok = issue_s(0);
    for (int j = 0; j < n_kv && ok; ++j) {
      if (j + 1 < n_kv && !(ok = issue_s(j + 1))) break;
      const int st = j & 1, vs = j % kVStages;
      if (!(ok = mbar_wait_warp(&p_full[st], (j >> 1) & 1, err, kErrTimeoutAttn))) break;
      if (!(ok = mbar_wait_warp(&v_full[vs], (j / kVStages) & 1, err, kErrTimeoutAttn))) break;
      tc_fence_after();
      const uint64_t vd = smem_desc_sw128(smem_addr(sm + L::V + vs * L::TILE), kSlice64, 1024);
#pragma unroll
      for (int kk = 0; kk < kKeys / 16; ++kk)  // A = P_j from TMEM: 16 keys = 8 columns per step
        umma_bf16_tmem_a_warp(tO, tS0 + st * kKeys + (16 * kk / kCols) * kCols + 16 * kk % kCols / 2,
                              desc_advance(vd, kk * 2048), idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
      umma_commit_warp(&v_empty[vs]);
      umma_commit_warp(pv_done);
      if (j == n_kv - 1) umma_commit_warp(o_done);
    }
    mma_drain(drained);
  } else {
    // ------------------------------------------------------------ softmax (warps 2..5, or 2..9)
    const uint32_t tl = static_cast<uint32_t>(sub * 32) << 16;
    const int part = (warp - 2) >> 2;  // which kCols of a tile's columns (0 with one thread a row)
    const int elem = threadIdx.x - 64;
    const bool padded = (empty_rows[0] | empty_rows[1] | empty_rows[2] | empty_rows[3]) != 0;
    const float slope2 = BIAS ? a.slopes[head] * kLog2e : 0.f;
    const float to_log2 = CAP ? a.score.cap_log2 : a.score.scale_log2;  // a score times this: log2 units
    float m_ref = BOUNDED ? kBoundedRef : -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n_kv; ++j) {
      const int st = j & 1;
      const int key0 = (j0 + j) * kKeys;
      // this thread's scores and, over them, its part of P as bf16 pairs (key 2c in the low half of
      // column c): a thread overwrites only columns that it has read
      const uint32_t tS = tS0 + tl + st * kKeys + part * kCols;
      if (!(ok = mbar_wait_warp(&s_full[st], (j >> 1) & 1, err, kErrTimeoutAttn))) break;
      tc_fence_after();
      float sc[kCols];
#pragma unroll
      for (int c4 = 0; c4 < kCols / 32; ++c4) {
        uint32_t r[32];
        tmem_ld_32cols(tS + c4 * 32, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) sc[c4 * 32 + i] = __uint_as_float(r[i]);
      }
      if constexpr (CAP) cap_tanh<kCols>(sc, a.score);
      if constexpr (BIAS) {
        const float d0 = static_cast<float>(q - key0);
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          sc[c] = fmaf(-slope2, fabsf(d0 - static_cast<float>(c)), sc[c] * to_log2);
      }
      if (!sees_all(hull, key0, key0 + kKeys)) {
#pragma unroll
        for (int c4 = 0; c4 < kCols / 32; ++c4) {
          const uint32_t vis = span_bits(seen, key0 + part * kCols + c4 * 32);
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!(vis >> c & 1u)) sc[c4 * 32 + c] = -INFINITY;
        }
      }
      if constexpr (!BOUNDED) {
        float r = sc[0];
#pragma unroll
        for (int c = 1; c + 1 < kCols; c += 2) r = fmax3(r, sc[c], sc[c + 1]);
        const float mx = fmaxf(r, sc[kCols - 1]) * (BIAS ? 1.f : to_log2);
        const bool need = mx > m_ref + kLazyRescale;
        const float m_new = need ? mx : m_ref;
        // rescale O only when a row's max grew past the lazy threshold; O += P_{j-1} V_{j-1} must
        // have finished first (P_j may be written before it has: it goes to the other buffer)
        if (j > 0 && __any_sync(0xffffffffu, need)) {
          if (!(ok = mbar_wait_warp(pv_done, (j - 1) & 1, err, kErrTimeoutAttn))) break;
          tc_fence_after();
          const float factor = need ? ex2(m_ref - m_new) : 1.f;  // 0 where nothing was seen before
#pragma unroll
          for (int c4 = 0; c4 < HD / 32; ++c4) {
            uint32_t w[32];
            tmem_ld_32cols(tO + tl + c4 * 32, w);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * factor);
            tmem_st_32cols(tO + tl + c4 * 32, w);
          }
          tmem_st_wait();
          l *= factor;
        }
        m_ref = m_new;
      }
      uint32_t pw[kCols / 2];
      const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
      const float2 sl = make_float2(to_log2, to_log2), nm = make_float2(neg_m, neg_m);
      float2 acc = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < kCols / 2; ++c) {
        const float2 x = make_float2(sc[2 * c], sc[2 * c + 1]);
        const float2 v = BIAS ? __fadd2_rn(x, nm) : __ffma2_rn(x, sl, nm);
        const float2 pp = make_float2(ex2(v.x), ex2(v.y));
        acc = __fadd2_rn(acc, pp);
        pw[c] = pack_bf16(pp.x, pp.y);
      }
      if constexpr (kCols == 64) tmem_st_32cols(tS, pw);
      else tmem_st_16cols(tS, pw);
      tmem_st_wait();
      l += acc.x + acc.y;
      // rows of V that nothing here may see: outside the hull, or padding among the tile's own rows
      const bool own = padded && key0 < q0 + 128 && key0 + kKeys > q0;
      if (key0 < hull.min_lo || key0 + kKeys > hull.max_hi || own) {
        if (!(ok = mbar_wait_warp(&v_full[j % kVStages], (j / kVStages) & 1, err, kErrTimeoutAttn))) break;
        const int kr = elem & 63, key = key0 + kr, which = elem >> 6;
        const bool pad = own && key >= q0 && key < q0 + 128 && (empty_rows[(key - q0) >> 5] >> ((key - q0) & 31) & 1u);
        if ((key < hull.min_lo || key >= hull.max_hi || pad) && which < L::NSL)
          zero_slice_row(sm + L::V + (j % kVStages) * L::TILE + which * kSlice64, kr);
        fence_proxy_async_smem();
      }
      tc_fence_before();
      mbar_arrive(&p_full[st]);
    }
    // the output waits on its own barrier: a parity wait on pv_done could not tell the last
    // product's phase from the one two before it
    ok = ok && (n_kv == 0 || mbar_wait_warp(o_done, 0, err, kErrTimeoutAttn));
    tc_fence_after();
    if constexpr (BOUNDED) {  // the row's two sums, through Q's memory (every product has run)
      float* sums = reinterpret_cast<float*>(sm + L::Q);
      if (ok) sums[part * 128 + row] = l;
      asm volatile("bar.sync 1, %0;" ::"n"(kSoftmax) : "memory");
      if (ok) l += sums[(part ^ 1) * 128 + row];
    }
    if (ok) {
      const bool some = l != 0.f;  // NaN counts as something
      const float inv = 1.f / l;
      // the warp's 32 rows and this part's columns, up to 64 at a time
      constexpr int kOut = BOUNDED ? HD / 2 : HD, kStep = kOut < 64 ? kOut : 64;
      bf16* o0 = a.o + (static_cast<int64_t>(b) * s + q0 + sub * 32) * a.ldo + static_cast<int64_t>(head) * HD +
                 part * kOut;
#pragma unroll
      for (int c = 0; c < kOut; c += kStep) {
        uint4 out[kStep / 8];
#pragma unroll
        for (int c4 = 0; c4 < kStep / 32; ++c4) {
          uint32_t r[32] = {};
          if (n_kv > 0) {
            tmem_ld_32cols(tO + tl + part * kOut + c + c4 * 32, r);
            tmem_ld_wait();
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = some ? __float_as_uint(__uint_as_float(r[i]) * inv) : 0u;
#pragma unroll
          for (int v = 0; v < 4; ++v)
            out[4 * c4 + v] = make_uint4(pack_bf16(__uint_as_float(r[8 * v + 0]), __uint_as_float(r[8 * v + 1])),
                                         pack_bf16(__uint_as_float(r[8 * v + 2]), __uint_as_float(r[8 * v + 3])),
                                         pack_bf16(__uint_as_float(r[8 * v + 4]), __uint_as_float(r[8 * v + 5])),
                                         pack_bf16(__uint_as_float(r[8 * v + 6]), __uint_as_float(r[8 * v + 7])));
        }
        store_rows<kStep / 8>(o0 + c, a.ldo, s - q0 - sub * 32, out, lane);
      }
      if (q < s && part == 0)
        a.lse[(static_cast<int64_t>(b) * nh + head) * s + q] = some ? m_ref + log2f(l) : -INFINITY;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, 256);
}

template <int HD, bool CAP, bool BIAS>
cudaError_t launch(const AttnSpanArgs& g, bf16* o, int64_t ldo, float* lse, int* err, cudaStream_t st) {
  using L = Smem<HD>;
  CUtensorMap mq, mk, mv;
  const int64_t s = g.s;
  if (!tma_map_heads(&mq, g.q, s, g.B, g.ldq, s * g.ldq, static_cast<uint64_t>(g.nh) * L::NSL, L::NSL, 128) ||
      !tma_map_heads(&mk, g.k, s, g.B, g.ldk, s * g.ldk, static_cast<uint64_t>(g.nkv) * L::NSL, L::NSL, kKeys) ||
      !tma_map_heads(&mv, g.v, s, g.B, g.ldv, s * g.ldv, static_cast<uint64_t>(g.nkv) * L::NSL, L::NSL, kKeys))
    return cudaErrorInvalidValue;
  // Blocks go heaviest first over as many (head, sequence) pairs as keep their K and V in half of the L2,
  // 16 at least: the more pairs, the less the last ones' long blocks stand alone at the end, until
  // the pairs' keys push one another out. (16, 32, 64 pairs: 4096 tokens, 40/8 heads, 0.4 MB of K and V a
  // pair of them, 144, 147, 134 us, capped 223, 221, 195; two sequences of 32 heads, 2 MB a pair, 214, 212,
  // 217, as packed documents 110, 109, 108.)
  constexpr int64_t kGroupBytes = 64 << 20;
  const int64_t fit = kGroupBytes / (s * HD * 4) * (g.nh / g.nkv), pairs = static_cast<int64_t>(g.nh) * g.B;
  const int head_group = static_cast<int>(std::max<int64_t>(std::min(fit, pairs), kHeadGroup));
  const FwdArgs a{{g.lo, g.hi}, g.slopes, o, ldo, lse, g.s, g.nh, g.nkv, head_group, score_args(g), err};
  auto run = [&](auto bounded) {
    auto* kernel = &attn_span_fwd_kernel<HD, CAP, BIAS, decltype(bounded)::value>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = allow_smem(kernel, L::BYTES, ready);
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>((s + 127) / 128 * g.nh * g.B), decltype(bounded)::value ? 320 : 192, L::BYTES, st>>>(
        mq, mk, mv, a);
    return cudaGetLastError();
  };
  if constexpr (CAP && !BIAS)
    if (a.score.cap_log2 <= kBounded) return run(std::true_type{});
  return run(std::false_type{});
}

}  // namespace

bool attn_span_ok(const AttnSpanArgs& g) {
  auto rows = [](const void* p, int64_t ld, int64_t cols) {
    return p && (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0 && ld >= cols && ld < (int64_t{1} << 31);
  };
  if (g.B <= 0 || g.s <= 0 || g.s > kSpanMaxSeq || g.nh <= 0 || g.nkv <= 0 || g.nh % g.nkv ||
      (g.hd != 64 && g.hd != 128))
    return false;
  const int64_t nh = g.nh, nkv = g.nkv;
  if (!rows(g.q, g.ldq, nh * g.hd) || !rows(g.k, g.ldk, nkv * g.hd) || !rows(g.v, g.ldv, nkv * g.hd)) return false;
  if ((reinterpret_cast<uintptr_t>(g.lo) | reinterpret_cast<uintptr_t>(g.hi) | reinterpret_cast<uintptr_t>(g.slopes)) & 3)
    return false;
  if (!std::isfinite(g.scale) || !(g.scale > 0.f) || !std::isfinite(g.cap) || g.cap < 0.f) return false;
  if (g.cap > 0.f && (!std::isnormal(g.cap) || !std::isfinite(g.scale / g.cap) || !std::isfinite(kLog2e * g.cap)))
    return false;
  if (!std::isfinite(kLog2e * g.scale)) return false;
  // batch * tiles * heads blocks, and tensor-map strides below 2^40 bytes
  return (g.s + 127) / 128 * nh * g.B <= INT_MAX && static_cast<double>(g.s) * 2 * g.ldq < 1e12 &&
         static_cast<double>(g.s) * 2 * g.ldk < 1e12 && static_cast<double>(g.s) * 2 * g.ldv < 1e12;
}

cudaError_t attn_span_fwd(const AttnSpanArgs& g, bf16* o, int64_t ldo, float* lse, int* err, cudaStream_t st) {
  const int64_t qc = static_cast<int64_t>(g.nh) * g.hd, kc = static_cast<int64_t>(g.nkv) * g.hd;
  const int64_t T = static_cast<int64_t>(g.B) * g.s;
  if (!attn_span_ok(g) || !o || !lse || !err || (reinterpret_cast<uintptr_t>(o) & 15) || ldo % 8 || ldo < qc ||
      ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(err)) & 3) ||
      columns_overlap(o, ldo, qc, g.q, g.ldq, qc, T) || columns_overlap(o, ldo, qc, g.k, g.ldk, kc, T) ||
      columns_overlap(o, ldo, qc, g.v, g.ldv, kc, T))
    return cudaErrorInvalidValue;
  return dispatch(g, [&](auto hd, auto cap, auto bias) {
    return launch<decltype(hd)::value, decltype(cap)::value, decltype(bias)::value>(g, o, ldo, lse, err, st);
  });
}

}  // namespace mt
