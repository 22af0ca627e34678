// Rotary positions beyond the layer template's (explicit positions, part of the head, both pair
// layouts, scaled frequencies) and the norms of queries and keys fused with the rotation.
//
// All of it is bound by HBM (a few operations per 2-byte element), so each kernel moves every
// element once, in 16-byte accesses. A head's row of hd columns is cut into hd/16 units of two
// 16-byte vectors, one unit per thread: in the rotated part columns [8u, 8u+8) and [rot/2 + 8u, +8),
// which are 8 whole rotation pairs in either layout (half: indices [8u, 8u+8); interleaved: [4u, 4u+4)
// and [rot/4 + 4u, +4)), so the rotation needs no exchange between threads, and a thread keeps the
// same unit, and so the same cosines and sines, for every head of its token. Neighbouring threads
// read neighbouring vectors in both accesses (with 16 adjacent columns per thread instead, every
// access covers half of each 32-byte sector: 53 us instead of 51 for 8192 x 64 interleaved heads).
// Measured (head size 128; a plain copy reaches 6.77 TB/s): rotation of 8192 x 64 heads 43.1 us, 6.3
// TB/s; norm forward of 4096 x 48 heads 24.6 us (21 us of it on the device, where its start and tail
// show), its backward of 8192 x 64 heads 74.7 us, 5.4 TB/s. A single token takes 3 us on the device and is bound by the call.
#include <cmath>
#include <cstdint>

#include "follow.cuh"
#include "kernels.h"
#include "mt_kernels.h"
#include "ptx.cuh"

namespace mt {

namespace {

constexpr int kRotThreads = 256;
constexpr double kTwoPi = 6.283185307179586476925286766559;

// A unit's 16 values in fp32, arranged for the rotation: a[i] pairs with b[i], i < 8. In the half layout
// a is the first vector and b the second; in the interleaved one a holds the even elements of both
// and b the odd ones. Two neighbouring i at a time go through the packed fp32 units: with scalar
// arithmetic these kernels are bound by instructions (19 to 27 an element for the norms), not HBM.
struct Row16 {
  float2 a[4], b[4];
};
__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
template <bool INTER>
__device__ __forceinline__ Row16 unpack(const uint4& v0, const uint4& v1) {
  const uint32_t x[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  Row16 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (INTER) {
      r.a[i] = make_float2(bf_lo(x[2 * i]), bf_lo(x[2 * i + 1]));
      r.b[i] = make_float2(bf_hi(x[2 * i]), bf_hi(x[2 * i + 1]));
    } else {
      r.a[i] = make_float2(bf_lo(x[i]), bf_hi(x[i]));
      r.b[i] = make_float2(bf_lo(x[4 + i]), bf_hi(x[4 + i]));
    }
  }
  return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
template <bool INTER>
__device__ __forceinline__ void pack(const Row16& r, uint4& v0, uint4& v1) {
  uint32_t x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (INTER) {
      x[2 * i] = pack2(r.a[i].x, r.b[i].x);
      x[2 * i + 1] = pack2(r.a[i].y, r.b[i].y);
    } else {
      x[i] = pack2(r.a[i].x, r.a[i].y);
      x[4 + i] = pack2(r.b[i].x, r.b[i].y);
    }
  }
  v0 = make_uint4(x[0], x[1], x[2], x[3]);
  v1 = make_uint4(x[4], x[5], x[6], x[7]);
}
// Column (within the unit's vectors) of value i of a (half 0) or b (half 1): vector, element.
__device__ __forceinline__ int2 place_of(int half, int i, bool interleaved) {
  return interleaved ? make_int2(i >> 2, 2 * (i & 3) + half) : make_int2(half, i);
}

// Where a unit's two vectors lie in the head's row, and whether it is rotated.
struct Unit {
  int c0, c1;
  bool rotated;
};
__device__ __forceinline__ Unit unit_of(int u, int hd, int rot) {
  if (16 * u < rot) return {8 * u, rot / 2 + 8 * u, true};
  const int c = rot / 2 + 8 * u;  // rot + 8 (u - rot / 16)
  return {c, c + (hd - rot) / 2, false};
}

// Cosines and sines of the unit's 8 rotation indices, in pairs like Row16.
struct Angles {
  float2 c[4], s[4];
};
struct RawAngles {
  float4 r[4];
};
__device__ __forceinline__ Angles angles_of(const RawAngles& w) {
  Angles g;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    g.c[k] = make_float2(w.r[k].x, w.r[k].z);
    g.s[k] = make_float2(w.r[k].y, w.r[k].w);
  }
  return g;
}

struct Rotation {
  const float* cs;
  const int32_t* positions;
  int n_pos, rot;
  int* err;
};
// Position of token t (T stays below 2^31); not checked against the table.
__device__ __forceinline__ int position_of(const Rotation& q, uint32_t t) {
  return q.positions ? q.positions[t] : static_cast<int>(t % static_cast<uint32_t>(q.n_pos));
}
// The unit's angles at a position; one outside the table raises the error flag and leaves the token
// as it is (angle 0).
template <bool INTER>
__device__ __forceinline__ RawAngles load_angles(const Rotation& q, int p, int u) {
  RawAngles w;
  if (p < 0 || p >= q.n_pos) {
    atomicCAS(q.err, 0, kErrBadPosition);
#pragma unroll
    for (int k = 0; k < 4; ++k) w.r[k] = make_float4(1.f, 0.f, 1.f, 0.f);
    return w;
  }
  const float* row = q.cs + static_cast<int64_t>(p) * q.rot + (INTER ? 8 : 16) * u;
  const int second = INTER ? q.rot / 2 : 8;  // floats to the angles of the unit's last 4 pairs
#pragma unroll
  for (int k = 0; k < 4; ++k) w.r[k] = __ldg(reinterpret_cast<const float4*>(row + (k >> 1) * second) + (k & 1));
  return w;
}

// a' = a c - b s, b' = b c + a s; INVERSE the transpose.
template <bool INVERSE>
__device__ __forceinline__ void rotate(Row16& v, const Angles& g) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 as = __fmul2_rn(v.a[k], g.s[k]), bs = __fmul2_rn(v.b[k], g.s[k]);
    const float2 neg_as = make_float2(-as.x, -as.y), neg_bs = make_float2(-bs.x, -bs.y);
    v.a[k] = __ffma2_rn(v.a[k], g.c[k], INVERSE ? bs : neg_bs);
    v.b[k] = __ffma2_rn(v.b[k], g.c[k], INVERSE ? neg_as : as);
  }
}

// How a block's threads take rows: unit (fastest), head slot, token slot. A thread takes the heads of its
// slot in turns and keeps its token's angles for them.
struct RowSplit {
  int units, head_slots, token_slots;
  __host__ __device__ int rows() const { return head_slots * token_slots; }
};
// The split that leaves the fewest threads idle over the turns; among equals the one with the most
// turns, up to most_turns, for angles loaded once a token. 8192 x 64 heads rotated in 4 turns 43.1 us, in
// 8 44.8, in 2 45.4; 4096 x 48 heads normed in up to 8 turns 24.6 us, in up to 4 28.6. Below 16 tokens an SM
// two turns at most, to spread them (40/8 heads, norm forward, backward: 64 tokens 10.8, 14.8 us in up to 8
// turns, 8.7, 10.8 in two; 608 tokens 12.8, 18.9 and 10.7, 18.9; 2048 the same; 4096 27.5, 44.3 and 30, 49.7).
RowSplit row_split(int T, int heads, int hd, int most_turns) {
  RowSplit s{hd / 16, 1, 1};
  const int slots = kRotThreads / s.units;
  if (T < kSms * 16) most_turns = 2;
  double best = -1.0;
  for (int hs = heads < slots ? heads : slots; hs >= 1; --hs) {
    const int turns = (heads + hs - 1) / hs;
    if (turns > most_turns && best >= 0.0) break;
    const int ts = slots / hs;
    const double used = static_cast<double>(heads) * ts / (static_cast<double>(turns) * slots);
    if (used >= best) {
      best = used;
      s.head_slots = hs;
      s.token_slots = ts;
    }
  }
  return s;
}

// Sum over the HD/16 threads of a head's row (consecutive lanes).
template <int HD>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = HD / 32; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct RowArgs {
  const bf16* x;
  int64_t ldx;
  bf16* y;
  int64_t ldy;
  int T, heads, hd;
  RowSplit split;
  Rotation rotation;
  // the norms'
  int nh;
  const bf16 *gq, *gk;
  float* rstd;
  float eps;
};

// One pass over rows: the rotation (HD = 0: any head size), or, with HD, y = R(x rstd g), rstd =
// 1/sqrt(mean x^2 + eps), one row per head. A block takes token_slots tokens, a thread two heads a
// turn: both rows' loads are in flight together, the first ones before the token's position and
// angles, which depend on each other. What hides the rest of the latency is the number of threads, so
// the gains are read again for every row (from L1) and the registers kept to four blocks an SM.
// Threads past the last head or token stay for the row sums.
constexpr int kHeadsPerTurn = 2;
template <int HD, bool INTER, bool INVERSE>
__global__ void __launch_bounds__(kRotThreads, 4) row_kernel(const __grid_constant__ RowArgs p) {
  const int units = HD ? HD / 16 : p.split.units, hd = HD ? HD : p.hd, head_slots = p.split.head_slots;
  const int u = threadIdx.x % units, slot = threadIdx.x / units;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * p.split.token_slots + slot / head_slots;
  const Unit w = unit_of(u, hd, p.rotation.rot);
  const bool live = t < p.T && slot < p.split.rows() && (HD || w.rotated || p.x != p.y);
  if (!HD && !live) return;
  const int h0 = slot % head_slots;
  const int64_t step = static_cast<int64_t>(head_slots) * hd;
  const bf16* xr = p.x + t * p.ldx + static_cast<int64_t>(h0) * hd;
  bf16* yr = p.y + t * p.ldy + static_cast<int64_t>(h0) * hd;
  uint4 v0[kHeadsPerTurn], v1[kHeadsPerTurn];
  auto load = [&](int h) {
#pragma unroll
    for (int k = 0; k < kHeadsPerTurn; ++k) {
      v0[k] = v1[k] = make_uint4(0u, 0u, 0u, 0u);
      if (live && h + k * head_slots < p.heads) {
        v0[k] = *reinterpret_cast<const uint4*>(xr + k * step + w.c0);
        v1[k] = *reinterpret_cast<const uint4*>(xr + k * step + w.c1);
      }
    }
    xr += kHeadsPerTurn * step;
  };
  load(h0);
  Angles ang{};
  if (live && w.rotated) {
    const int pos = position_of(p.rotation, static_cast<uint32_t>(t));
    ang = angles_of(load_angles<INTER>(p.rotation, pos, u));
  }
  for (int hb = 0; hb < p.heads; hb += kHeadsPerTurn * head_slots) {  // the same turns in every thread
    if (hb > 0) load(hb + h0);
#pragma unroll
    for (int k = 0; k < kHeadsPerTurn; ++k) {
      const int h = hb + h0 + k * head_slots;
      const bool on = live && h < p.heads;
      if constexpr (HD > 0) {
        Row16 v = unpack<INTER>(v0[k], v1[k]);
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = __ffma2_rn(v.a[i], v.a[i], __ffma2_rn(v.b[i], v.b[i], ss));
        const float rs = rsqrtf(row_sum<HD>(ss.x + ss.y) * (1.f / HD) + p.eps);
        const bf16* gain = h < p.nh ? p.gq : p.gk;
        const Row16 g = unpack<INTER>(__ldg(reinterpret_cast<const uint4*>(gain + w.c0)),
                                      __ldg(reinterpret_cast<const uint4*>(gain + w.c1)));
        const float2 rs2 = make_float2(rs, rs);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v.a[i] = __fmul2_rn(__fmul2_rn(v.a[i], rs2), g.a[i]);
          v.b[i] = __fmul2_rn(__fmul2_rn(v.b[i], rs2), g.b[i]);
        }
        if (w.rotated) rotate<false>(v, ang);
        pack<INTER>(v, v0[k], v1[k]);
        if (on && p.rstd && u == 0) p.rstd[t * p.heads + h] = rs;
      } else if (w.rotated) {
        Row16 v = unpack<INTER>(v0[k], v1[k]);
        rotate<INVERSE>(v, ang);
        pack<INTER>(v, v0[k], v1[k]);
      }
      if (on) {
        *reinterpret_cast<uint4*>(yr + k * step + w.c0) = v0[k];
        *reinterpret_cast<uint4*>(yr + k * step + w.c1) = v1[k];
      }
    }
    yr += kHeadsPerTurn * step;
  }
}

template <int HD>
cudaError_t launch_rows(const RowArgs& a, bool interleaved, bool inverse, cudaStream_t s) {
  const int64_t slots = a.split.token_slots;
  const unsigned blocks = static_cast<unsigned>((a.T + slots - 1) / slots);
  auto* kernel = interleaved ? (inverse ? row_kernel<HD, true, HD == 0> : row_kernel<HD, true, false>)
                             : (inverse ? row_kernel<HD, false, HD == 0> : row_kernel<HD, false, false>);
  kernel<<<blocks, (a.split.units * a.split.rows() + 31) / 32 * 32, 0, s>>>(a);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ backward of the query/key norms
// Blocks take either query heads or key heads: blocks [0, q.blocks) the former, the rest the latter, in
// proportion to the heads. A thread then has one gain, kept in registers, and one gain gradient.
struct NormSide {
  RowSplit split;
  int blocks;
};
struct NormSplit {
  NormSide q, k;
};
NormSplit norm_split(int T, int nh, int nkv, int hd) {
  constexpr int blocks = kQkNormParts;
  NormSplit s{{row_split(T, nh, hd, 8), 0}, {row_split(T, nkv, hd, 8), 0}};
  auto most = [T](const RowSplit& r) { return (T - 1) / r.token_slots + 1; };
  const int share = static_cast<int>(static_cast<int64_t>(blocks) * nh / (nh + nkv)), q = share > 0 ? share : 1;
  const int k = blocks > q ? blocks - q : 1;
  s.q.blocks = most(s.q.split) < q ? most(s.q.split) : q;
  s.k.blocks = most(s.k.split) < k ? most(s.k.split) : k;
  return s;
}

struct BwdArgs {
  const bf16 *x, *dy;
  int64_t ldx, lddy;
  bf16* dx;
  int64_t lddx;
  const bf16 *gq, *gk;
  const float* rstd;
  float* partial;
  int T, nh, heads;
  Rotation rotation;
};

// One row's operands as loaded, a turn ahead of their use.
struct RawRow {
  uint4 x0, x1, d0, d1;
  float rs;
};

// With u = R^T dy and n = x rstd: dx = rstd (u g - n mean(u g n)) per head row, and the block's share
// of dg = sum over its rows of u n: a thread keeps its 16 columns for every row it takes, so the sums
// stay in registers; at the end they are added over the block's slots in slot order and written to the
// block's row of `partial` [blocks][HD]: fixed order, no atomics.
// The next row and, with a new token, its angles are loaded before the current row is worked on, and
// the position of the token after that.
template <int HD, bool INTER>
__global__ void __launch_bounds__(kRotThreads, 2)
    qk_norm_bwd_kernel(const __grid_constant__ BwdArgs p, const __grid_constant__ NormSplit bs) {
  constexpr int kUnits = HD / 16;
  __shared__ float sums[kRotThreads][17];
  let_next_start();
  const bool is_q = static_cast<int>(blockIdx.x) < bs.q.blocks;
  const NormSide& side = is_q ? bs.q : bs.k;
  const int head_slots = side.split.head_slots, token_slots = side.split.token_slots;
  const int heads = is_q ? p.nh : p.heads - p.nh, first = is_q ? 0 : p.nh;
  const int block = is_q ? blockIdx.x : blockIdx.x - bs.q.blocks;
  const int u = threadIdx.x % kUnits, slot = threadIdx.x / kUnits;
  const int h0 = slot % head_slots;
  const bool in = slot < head_slots * token_slots;
  const Unit w = unit_of(u, HD, p.rotation.rot);
  const bool turns_on = in && w.rotated;
  const uint32_t T = static_cast<uint32_t>(p.T);
  const bf16* gain = is_q ? p.gq : p.gk;
  const Row16 g = unpack<INTER>(__ldg(reinterpret_cast<const uint4*>(gain + w.c0)),
                                __ldg(reinterpret_cast<const uint4*>(gain + w.c1)));
  Row16 acc;
#pragma unroll
  for (int k = 0; k < 4; ++k) acc.a[k] = acc.b[k] = make_float2(0.f, 0.f);

  uint32_t t = static_cast<uint32_t>(block) * token_slots + slot / head_slots;  // the row being loaded: token,
  int hb = 0;                                                                 // head - h0
  const uint32_t step = static_cast<uint32_t>(side.blocks) * token_slots;
  const int turns = (heads + head_slots - 1) / head_slots;
  const uint32_t tokens = (T - 1 - static_cast<uint32_t>(block) * token_slots) / step + 1;  // >= 1
  auto load = [&](RawRow& r) {
    r.x0 = r.x1 = r.d0 = r.d1 = make_uint4(0u, 0u, 0u, 0u);
    r.rs = 0.f;
    if (in && t < T && hb + h0 < heads) {
      const int64_t col = static_cast<int64_t>(first + hb + h0) * HD;
      const bf16* xr = p.x + t * p.ldx + col;
      r.x0 = *reinterpret_cast<const uint4*>(xr + w.c0);
      r.x1 = *reinterpret_cast<const uint4*>(xr + w.c1);
      const bf16* dr = p.dy + t * p.lddy + col;
      r.d0 = *reinterpret_cast<const uint4*>(dr + w.c0);
      r.d1 = *reinterpret_cast<const uint4*>(dr + w.c1);
      r.rs = p.rstd[static_cast<int64_t>(t) * p.heads + first + hb + h0];
    }
  };
  RawRow next;
  RawAngles raw{};
  Angles ang{};
  int pos = turns_on && t < T ? position_of(p.rotation, t) : 0;
  load(next);
  if (turns_on && t < T) raw = load_angles<INTER>(p.rotation, pos, u);
  if (turns_on && t + step < T) pos = position_of(p.rotation, t + step);
  for (uint32_t it = 0; it < tokens; ++it) {
    ang = angles_of(raw);
    for (int turn = 0; turn < turns; ++turn) {
      const RawRow cur = next;
      const uint32_t tc = t;
      const int hc = hb + h0;
      const bool on = in && t < T && hc < heads;
      hb += head_slots;
      if (turn + 1 == turns) {
        hb = 0;
        t += step;
        if (turns_on && t < T) {
          raw = load_angles<INTER>(p.rotation, pos, u);
          if (t + step < T) pos = position_of(p.rotation, t + step);
        }
      }
      load(next);
      Row16 n = unpack<INTER>(cur.x0, cur.x1);
      Row16 d = unpack<INTER>(cur.d0, cur.d1);
      if (w.rotated) rotate<true>(d, ang);
      const float2 rs2 = make_float2(cur.rs, cur.rs);
      float2 dot = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        n.a[k] = __fmul2_rn(n.a[k], rs2);
        n.b[k] = __fmul2_rn(n.b[k], rs2);
        acc.a[k] = __ffma2_rn(d.a[k], n.a[k], acc.a[k]);
        acc.b[k] = __ffma2_rn(d.b[k], n.b[k], acc.b[k]);
        d.a[k] = __fmul2_rn(d.a[k], g.a[k]);
        d.b[k] = __fmul2_rn(d.b[k], g.b[k]);
        dot = __ffma2_rn(d.a[k], n.a[k], __ffma2_rn(d.b[k], n.b[k], dot));
      }
      const float m = row_sum<HD>(dot.x + dot.y) * (-1.f / HD);
      const float2 m2 = make_float2(m, m);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        n.a[k] = __fmul2_rn(rs2, __ffma2_rn(n.a[k], m2, d.a[k]));
        n.b[k] = __fmul2_rn(rs2, __ffma2_rn(n.b[k], m2, d.b[k]));
      }
      if (on) {
        bf16* o = p.dx + tc * p.lddx + static_cast<int64_t>(first + hc) * HD;
        uint4 v0, v1;
        pack<INTER>(n, v0, v1);
        *reinterpret_cast<uint4*>(o + w.c0) = v0;
        *reinterpret_cast<uint4*>(o + w.c1) = v1;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sums[threadIdx.x][i] = (i & 1) ? acc.a[i / 2].y : acc.a[i / 2].x;
    sums[threadIdx.x][8 + i] = (i & 1) ? acc.b[i / 2].y : acc.b[i / 2].x;
  }
  __syncthreads();
  if (threadIdx.x < HD) {  // one thread per (unit, value) pair
    const int un = threadIdx.x / 16, i = threadIdx.x % 16;
    float s = 0.f;
    for (int k = 0; k < head_slots * token_slots; ++k) s += sums[k * kUnits + un][i];
    const Unit q = unit_of(un, HD, p.rotation.rot);
    const int2 at = place_of(i >> 3, i & 7, INTER);
    p.partial[static_cast<int64_t>(blockIdx.x) * HD + (at.x ? q.c1 : q.c0) + at.y] = s;
  }
}

// Block 0: dgq[j] = sum of the query blocks' partial[p][j], block 1: dgk from the key blocks': the
// rows dealt to 1024/HD groups of threads (group g: rows g, g + groups, ...), then the groups added
// in order. One latency after another is all it is: with ten loads in flight a lone backward call takes 102
// us instead of 105 (8192 x 64 heads).
template <int HD>
__global__ void __launch_bounds__(1024)
    qk_gain_reduce_kernel(const float* __restrict__ partial, int blocks_q, int blocks_k, bf16* __restrict__ dgq,
                          bf16* __restrict__ dgk) {
  constexpr int kGroups = 1024 / HD;
  __shared__ float acc[kGroups][HD];
  const int j = threadIdx.x % HD, g = threadIdx.x / HD;
  const int p0 = blockIdx.x ? blocks_q : 0, p1 = blockIdx.x ? blocks_q + blocks_k : blocks_q;
  float s = 0.f;
  wait_for_previous();
  constexpr int kAhead = 10;  // loads in flight; the sum keeps its order
  for (int p = p0 + g; p < p1; p += kAhead * kGroups) {
    float v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      v[k] = p + k * kGroups < p1 ? partial[static_cast<int64_t>(p + k * kGroups) * HD + j] : 0.f;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) s += v[k];
  }
  acc[g][j] = s;
  __syncthreads();
  if (g == 0) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) s += acc[k][j];
    (blockIdx.x ? dgk : dgq)[j] = __float2bfloat16_rn(s);
  }
}

// Rotation table. An angle is kept in turns as a 64-bit fraction: with F = the frequency in turns
// per position times 2^64, p F mod 2^64 is the angle of position p without the whole turns, exact
// for every p up to the rounding of F itself (2^-53 of the frequency), where p f in fp32 would lose
// all of it for far positions and fp64 arithmetic is slow on this part. The top 32 bits, less the
// nearest quarter turn, convert to fp32 with an error below 2^-26 turns. The kernel is bound by
// instructions (two scalar series an angle): 131072 x 64 angles take 14 us, 4.8 TB/s, below the 20 us of the
// host's calls.
struct TurnTable {
  uint64_t turns[kRotaryMaxPairs];
};

// cos and sin of phase / 2^64 turns. Within an eighth of a turn of the nearest quarter the Taylor
// series to y^9 and y^10 leave out less than 2e-9 and 2e-10.
__device__ __forceinline__ float2 cos_sin_turns(uint64_t phase, float amp) {
  const uint32_t top = static_cast<uint32_t>(phase >> 32);
  const uint32_t quarter = (top + (1u << 29)) >> 30;
  const float y = static_cast<float>(static_cast<int32_t>(top - (quarter << 30))) * static_cast<float>(kTwoPi * 0x1p-32);
  const float y2 = y * y;
  const float s = y * fmaf(y2, fmaf(y2, fmaf(y2, fmaf(y2, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), 1.f);
  const float c = fmaf(y2, fmaf(y2, fmaf(y2, fmaf(y2, fmaf(y2, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f),
                                -0.5f), 1.f);
  const float a = (quarter & 1) ? s : c, b = (quarter & 1) ? c : s;
  return make_float2((quarter == 1 || quarter == 2) ? -a * amp : a * amp, (quarter & 2) ? -b * amp : b * amp);
}

// Thread x takes the pairs 2x and 2x + 1 (one 16-byte store a position) of every gridDim-th group of
// blockDim.y positions; its phases advance by a constant, which wraps as it should.
__global__ void __launch_bounds__(kRotThreads)
    rotary_table_kernel(const __grid_constant__ TurnTable f, float2* __restrict__ out, int n_pos, int pairs, float amp) {
  const int i = 2 * threadIdx.x;
  int64_t p = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
  const uint64_t f0 = f.turns[i], f1 = f.turns[i + 1];  // i + 1 < kRotaryMaxPairs: zero past the last
  uint64_t a0 = p * f0, a1 = p * f1;
  for (; p < n_pos; p += step, a0 += step * f0, a1 += step * f1) {
    float2* o = out + p * pairs + i;
    const float2 u = cos_sin_turns(a0, amp);
    if (pairs % 2 == 0) {  // every row starts on 16 bytes
      const float2 v = cos_sin_turns(a1, amp);
      *reinterpret_cast<float4*>(o) = make_float4(u.x, u.y, v.x, v.y);
    } else {
      o[0] = u;
      if (i + 1 < pairs) o[1] = cos_sin_turns(a1, amp);
    }
  }
}

// Heads that the kernels index with 32 bits.
bool heads_ok(int64_t heads) { return heads > 0 && heads <= kRotaryMaxHeads; }
bool vec_aligned(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0; }
bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
// Whether y may be written while x is read: they are one row matrix, or share nothing.
bool may_write(const bf16* y, int64_t ldy, const bf16* x, int64_t ldx, int64_t cols, int T) {
  return (x == y && ldx == ldy) || !columns_overlap(x, ldx, cols, y, ldy, cols, T);
}

bool rotation_ok(int hd, int rot, const float* cs, int n_pos, const int32_t* positions, const int* err) {
  if (rot < 0 || rot > hd || rot % 16) return false;
  if (rot == 0) return true;
  return cs && aligned(cs, 16) && aligned(positions, 4) && n_pos > 0 && err && aligned(err, 4);
}

}  // namespace

bool rotary_inv_freq(int rot, double theta, int scaling, double factor, double original, double low, double high,
                     double* inv_freq) {
  auto positive = [](double v) { return std::isfinite(v) && v > 0.0; };
  if (!inv_freq || rot <= 0 || rot % 2 || rot / 2 > kRotaryMaxPairs || !positive(theta)) return false;
  if (scaling < MTK_ROTARY_PLAIN || scaling > MTK_ROTARY_BANDS) return false;
  if (scaling != MTK_ROTARY_PLAIN && !positive(factor)) return false;
  if (scaling == MTK_ROTARY_BASE && rot == 2) return false;
  if (scaling == MTK_ROTARY_BANDS &&
      (!positive(original) || !std::isfinite(low) || !std::isfinite(high) || !(high > low)))
    return false;
  const double base = scaling == MTK_ROTARY_BASE ? theta * std::pow(factor, rot / (rot - 2.0)) : theta;
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == MTK_ROTARY_LINEAR) f /= factor;
    if (scaling == MTK_ROTARY_BANDS) {
      double w = (original * f / kTwoPi - low) / (high - low);
      w = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
      f *= w + (1.0 - w) / factor;
    }
    if (!std::isfinite(f)) return false;
    inv_freq[i] = f;
  }
  return true;
}

cudaError_t rotary_table(const double* inv_freq, int rot, int n_pos, double amp, float* out, cudaStream_t s) {
  if (rot <= 0 || rot % 2 || rot / 2 > kRotaryMaxPairs || n_pos <= 0 || (reinterpret_cast<uintptr_t>(out) & 15) ||
      !std::isfinite(static_cast<float>(amp)))
    return cudaErrorInvalidValue;
  TurnTable f{};
  for (int i = 0; i < rot / 2; ++i) {
    if (!std::isfinite(inv_freq[i])) return cudaErrorInvalidValue;
    double turn = inv_freq[i] / kTwoPi;
    turn -= std::floor(turn);
    f.turns[i] = turn < 1.0 ? static_cast<uint64_t>(std::ldexp(turn, 64)) : 0;
  }
  const int pairs = rot / 2;
  const dim3 threads((pairs + 1) / 2, kRotThreads / ((pairs + 1) / 2));
  const unsigned groups = (static_cast<unsigned>(n_pos) + threads.y - 1) / threads.y;
  rotary_table_kernel<<<groups < kSms * 8 ? groups : kSms * 8, threads, 0, s>>>(
      f, reinterpret_cast<float2*>(out), n_pos, pairs, static_cast<float>(amp));
  return cudaGetLastError();
}

cudaError_t rotary(const bf16* x, int64_t ldx, bf16* y, int64_t ldy, int T, int heads, int hd, int rot,
                   bool interleaved, const int32_t* positions, const float* cs, int n_pos, bool inverse, int* err,
                   cudaStream_t s) {
  if (T <= 0 || !heads_ok(heads) || hd <= 0 || hd % 16 || hd > 16 * kRotThreads || rot == 0 ||
      !rotation_ok(hd, rot, cs, n_pos, positions, err))
    return cudaErrorInvalidValue;
  const int64_t cols = static_cast<int64_t>(heads) * hd;
  if (!vec_aligned(x, ldx) || !vec_aligned(y, ldy) || ldx < cols || ldy < cols || !may_write(y, ldy, x, ldx, cols, T))
    return cudaErrorInvalidValue;
  const RowArgs a{x, ldx, y, ldy, T, heads, hd, row_split(T, heads, hd, 4), {cs, positions, n_pos, rot, err},
                  0, nullptr, nullptr, nullptr, 0.f};
  return launch_rows<0>(a, interleaved, inverse, s);
}

namespace {
bool norm_ok(int T, int nh, int nkv, int hd, int rot, const float* cs, int n_pos, const int32_t* positions,
             const bf16* gq, const bf16* gk, const int* err) {
  return T > 0 && nh > 0 && nkv > 0 && heads_ok(static_cast<int64_t>(nh) + nkv) && (hd == 64 || hd == 128) &&
         rotation_ok(hd, rot, cs, n_pos, positions, err) && vec_aligned(gq, 0) && vec_aligned(gk, 0);
}
}  // namespace

cudaError_t qk_norm_rope(const bf16* x, int64_t ldx, const bf16* gq, const bf16* gk, bf16* y, int64_t ldy, float* rstd,
                         int T, int nh, int nkv, int hd, int rot, bool interleaved, float eps,
                         const int32_t* positions, const float* cs, int n_pos, int* err, cudaStream_t s) {
  if (!norm_ok(T, nh, nkv, hd, rot, cs, n_pos, positions, gq, gk, err)) return cudaErrorInvalidValue;
  const int heads = nh + nkv;
  const int64_t cols = static_cast<int64_t>(heads) * hd;
  if (!vec_aligned(x, ldx) || !vec_aligned(y, ldy) || ldx < cols || ldy < cols || !aligned(rstd, 4) ||
      !may_write(y, ldy, x, ldx, cols, T))
    return cudaErrorInvalidValue;
  const RowArgs a{x, ldx, y, ldy, T, heads, hd, row_split(T, heads, hd, 8), {cs, positions, n_pos, rot, err},
                  nh, gq, gk, rstd, eps};
  return hd == 64 ? launch_rows<64>(a, interleaved, false, s) : launch_rows<128>(a, interleaved, false, s);
}

int qk_norm_rope_bwd_parts(int T, int nh, int nkv, int hd) {
  const NormSplit s = norm_split(T, nh, nkv, hd);
  return s.q.blocks + s.k.blocks;
}

cudaError_t qk_norm_rope_bwd(const bf16* dy, int64_t lddy, const bf16* x, int64_t ldx, const bf16* gq, const bf16* gk,
                             const float* rstd, bf16* dx, int64_t lddx, float* partial, bf16* dgq, bf16* dgk, int T,
                             int nh, int nkv, int hd, int rot, bool interleaved, const int32_t* positions,
                             const float* cs, int n_pos, int* err, cudaStream_t s) {
  if (!norm_ok(T, nh, nkv, hd, rot, cs, n_pos, positions, gq, gk, err)) return cudaErrorInvalidValue;
  const int heads = nh + nkv;
  const int64_t cols = static_cast<int64_t>(heads) * hd;
  if (!vec_aligned(dy, lddy) || !vec_aligned(x, ldx) || !vec_aligned(dx, lddx) || lddy < cols || ldx < cols ||
      lddx < cols || !aligned(rstd, 4) || !aligned(partial, 4) || !aligned(dgq, 2) || !aligned(dgk, 2) ||
      !may_write(dx, lddx, dy, lddy, cols, T) || !may_write(dx, lddx, x, ldx, cols, T))
    return cudaErrorInvalidValue;
  const NormSplit sp = norm_split(T, nh, nkv, hd);
  const BwdArgs a{x, dy, ldx, lddy, dx, lddx, gq, gk, rstd, partial, T, nh, heads, {cs, positions, n_pos, rot, err}};
  auto* kernel = hd == 64 ? (interleaved ? qk_norm_bwd_kernel<64, true> : qk_norm_bwd_kernel<64, false>)
                          : (interleaved ? qk_norm_bwd_kernel<128, true> : qk_norm_bwd_kernel<128, false>);
  kernel<<<sp.q.blocks + sp.k.blocks, kRotThreads, 0, s>>>(a, sp);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_following(hd == 64 ? qk_gain_reduce_kernel<64> : qk_gain_reduce_kernel<128>, dim3(2), 1024, 0, s,
                          partial, sp.q.blocks, sp.k.blocks, dgq, dgk);
}

}  // namespace mt
