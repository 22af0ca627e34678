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
#include <cmath>
#include <cstdint>

#include "kernels.h"
#include "mt_kernels.h"
#include "ptx.cuh"

namespace mt {

namespace {

constexpr int kRotThreads = 256;
constexpr double kTwoPi = 6.283185307179586476925286766559;

struct Vec16 {  // 16 columns of one head's row, as loaded
  uint4 a, b;
};

__device__ __forceinline__ void unpack8(const uint4& w, float* v) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(x[j] << 16);
    v[2 * j + 1] = __uint_as_float(x[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
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

// Cosine and sine of the unit's 8 rotation indices at a token's position; a position outside the
// table raises the error flag and leaves the token as it is (angle 0).
__device__ __forceinline__ void load_angles(const float* __restrict__ cs, const int32_t* __restrict__ positions,
                                            int64_t t, int n_pos, int rot, bool interleaved, int u, int* err,
                                            float4 (&r)[4]) {
  const int p = positions ? positions[t] : static_cast<int>(t % n_pos);
  if (p < 0 || p >= n_pos) {
    atomicCAS(err, 0, kErrBadPosition);
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = make_float4(1.f, 0.f, 1.f, 0.f);
    return;
  }
  const float* q = cs + static_cast<int64_t>(p) * rot + (interleaved ? 8 : 16) * u;
  const int second = interleaved ? rot / 2 : 8;  // floats to the angles of the unit's last 4 pairs
#pragma unroll
  for (int k = 0; k < 4; ++k) r[k] = __ldg(reinterpret_cast<const float4*>(q + (k >> 1) * second) + (k & 1));
}

// The rotation on the unit's 16 values (v[0..8) from the first vector); sgn -1 for the transpose.
__device__ __forceinline__ void rotate(float (&v)[16], const float4 (&r)[4], bool interleaved, float sgn) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = (i & 1) ? r[i / 2].z : r[i / 2].x;
    const float s = sgn * ((i & 1) ? r[i / 2].w : r[i / 2].y);
    if (interleaved) {
      const float a = v[2 * i], b = v[2 * i + 1];
      v[2 * i] = a * c - b * s;
      v[2 * i + 1] = b * c + a * s;
    } else {
      const float a = v[i], b = v[8 + i];
      v[i] = a * c - b * s;
      v[8 + i] = b * c + a * s;
    }
  }
}

// Threads of a block: unit (fastest), head slot, token slot. A thread takes the heads of its slot one
// after the other; the slots are as few as give that many turns, so that the turns are even (48
// heads of 8 units: 24 slots, two turns, not 32 and a half-empty second turn).
struct RowSplit {
  int units, head_slots, token_slots;
  int rows() const { return units * head_slots * token_slots; }
  int threads() const { return (rows() + 31) / 32 * 32; }  // whole warps, for the row sums
};
RowSplit row_split(int heads, int hd) {
  RowSplit s;
  s.units = hd / 16;
  const int slots = kRotThreads / s.units;
  const int turns = (heads + slots - 1) / slots;
  s.head_slots = (heads + turns - 1) / turns;
  s.token_slots = slots / s.head_slots;
  return s;
}

// Two heads a turn: both rows' loads are in flight together, and before the angles are needed.
constexpr int kHeadsPerTurn = 2;

__global__ void __launch_bounds__(kRotThreads)
    rotary_kernel(const bf16* x, int64_t ldx, bf16* y, int64_t ldy, int T, int heads, int hd, int rot, bool interleaved,
                  const int32_t* __restrict__ positions, const float* __restrict__ cs, int n_pos, float sgn, int units,
                  int head_slots, int token_slots, int* err) {
  const int u = threadIdx.x % units, slot = threadIdx.x / units;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * token_slots + slot / head_slots;
  if (t >= T || slot >= head_slots * token_slots) return;
  const Unit w = unit_of(u, hd, rot);
  if (!w.rotated && x == y) return;
  float4 r[4];
  if (w.rotated) load_angles(cs, positions, t, n_pos, rot, interleaved, u, err, r);
  for (int h = slot % head_slots; h < heads; h += kHeadsPerTurn * head_slots) {
    uint4 a[kHeadsPerTurn], b[kHeadsPerTurn];
#pragma unroll
    for (int k = 0; k < kHeadsPerTurn; ++k) {
      if (h + k * head_slots >= heads) break;
      const bf16* xr = x + t * ldx + static_cast<int64_t>(h + k * head_slots) * hd;
      a[k] = *reinterpret_cast<const uint4*>(xr + w.c0);
      b[k] = *reinterpret_cast<const uint4*>(xr + w.c1);
    }
#pragma unroll
    for (int k = 0; k < kHeadsPerTurn; ++k) {
      if (h + k * head_slots >= heads) break;
      if (w.rotated) {
        float v[16];
        unpack8(a[k], v);
        unpack8(b[k], v + 8);
        rotate(v, r, interleaved, sgn);
        a[k] = pack8(v);
        b[k] = pack8(v + 8);
      }
      bf16* yr = y + t * ldy + static_cast<int64_t>(h + k * head_slots) * hd;
      *reinterpret_cast<uint4*>(yr + w.c0) = a[k];
      *reinterpret_cast<uint4*>(yr + w.c1) = b[k];
    }
  }
}

// Sum over the HD/16 threads of a head's row (consecutive lanes).
template <int HD>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = HD / 32; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// y = R(x rstd g), rstd = 1/sqrt(mean x^2 + eps), one row per head. Threads past the last head or
// token stay for the row sums (their rows are empty).
template <int HD>
__global__ void __launch_bounds__(kRotThreads)
    qk_norm_rope_kernel(const bf16* x, int64_t ldx, const bf16* __restrict__ gq, const bf16* __restrict__ gk, bf16* y,
                        int64_t ldy, float* __restrict__ rstd, int T, int nh, int heads, int rot, bool interleaved,
                        float eps, const int32_t* __restrict__ positions, const float* __restrict__ cs, int n_pos,
                        int head_slots, int token_slots, int* err) {
  constexpr int kUnits = HD / 16;
  const int u = threadIdx.x % kUnits, slot = threadIdx.x / kUnits;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * token_slots + slot / head_slots;
  const bool live = t < T && slot < head_slots * token_slots;
  const Unit w = unit_of(u, HD, rot);
  const int h0 = slot % head_slots;
  float4 r[4];
  if (live && w.rotated) load_angles(cs, positions, t, n_pos, rot, interleaved, u, err, r);
  for (int hb = 0; hb < heads; hb += kHeadsPerTurn * head_slots) {  // the same trip count in every thread
    uint4 a[kHeadsPerTurn], b[kHeadsPerTurn];
#pragma unroll
    for (int k = 0; k < kHeadsPerTurn; ++k) {
      const int h = hb + h0 + k * head_slots;
      a[k] = b[k] = make_uint4(0u, 0u, 0u, 0u);
      if (live && h < heads) {
        const bf16* xr = x + t * ldx + static_cast<int64_t>(h) * HD;
        a[k] = *reinterpret_cast<const uint4*>(xr + w.c0);
        b[k] = *reinterpret_cast<const uint4*>(xr + w.c1);
      }
    }
#pragma unroll
    for (int k = 0; k < kHeadsPerTurn; ++k) {
      const int h = hb + h0 + k * head_slots;
      float v[16];
      unpack8(a[k], v);
      unpack8(b[k], v + 8);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss += v[i] * v[i];
      const float rs = rsqrtf(row_sum<HD>(ss) * (1.f / HD) + eps);
      if (!(live && h < heads)) continue;
      const bf16* gain = h < nh ? gq : gk;
      float g[16];
      unpack8(__ldg(reinterpret_cast<const uint4*>(gain + w.c0)), g);
      unpack8(__ldg(reinterpret_cast<const uint4*>(gain + w.c1)), g + 8);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = v[i] * rs * g[i];
      if (w.rotated) rotate(v, r, interleaved, 1.f);
      bf16* yr = y + t * ldy + static_cast<int64_t>(h) * HD;
      *reinterpret_cast<uint4*>(yr + w.c0) = pack8(v);
      *reinterpret_cast<uint4*>(yr + w.c1) = pack8(v + 8);
      if (rstd && u == 0) rstd[t * heads + h] = rs;
    }
  }
}

// The backward's blocks take either query heads or key heads: blocks [0, blocks_q) the former, the
// rest the latter, in proportion to the heads. A thread then sums one gain gradient only.
struct BwdSide {
  RowSplit split;
  int blocks;
};
struct BwdSplit {
  BwdSide q, k;
};
BwdSplit bwd_split(int T, int nh, int nkv, int hd) {
  BwdSplit s{{row_split(nh, hd), 0}, {row_split(nkv, hd), 0}};
  auto most = [T](const RowSplit& r) { return (T - 1) / r.token_slots + 1; };
  const int share = static_cast<int>(static_cast<int64_t>(kQkNormParts) * nh / (nh + nkv)), q = share > 0 ? share : 1;
  const int k = kQkNormParts > q ? kQkNormParts - q : 1;
  s.q.blocks = most(s.q.split) < q ? most(s.q.split) : q;
  s.k.blocks = most(s.k.split) < k ? most(s.k.split) : k;
  return s;
}

// One row's operands as loaded, a turn ahead of their use.
struct RowPair {
  uint4 d0, d1, x0, x1;
  float rs;
};

// With u = R^T dy and n = x rstd: dx = rstd (u g - n mean(u g n)) per head row, and each block's
// share of dg = sum over tokens and heads of u n. A thread keeps its 16 columns for every row it
// takes, so the gain sums stay in registers; at the end they are added over the block's slots in
// slot order and written to the block's row of `partial` [blocks][HD]: fixed order, no atomics. The
// next row and, with a new token, its angles are loaded before the current row is worked on.
template <int HD>
__global__ void __launch_bounds__(kRotThreads, 2)
    qk_norm_rope_bwd_kernel(const bf16* dy, int64_t lddy, const bf16* x, int64_t ldx, const bf16* __restrict__ gq,
                            const bf16* __restrict__ gk, const float* __restrict__ rstd, bf16* dx, int64_t lddx,
                            float* __restrict__ partial, int T, int nh, int all_heads, int rot, bool interleaved,
                            const int32_t* __restrict__ positions, const float* __restrict__ cs, int n_pos,
                            const __grid_constant__ BwdSplit bs, int* err) {
  constexpr int kUnits = HD / 16;
  __shared__ float sums[kRotThreads][17];
  const bool is_q = static_cast<int>(blockIdx.x) < bs.q.blocks;
  const BwdSide& side = is_q ? bs.q : bs.k;
  const int head_slots = side.split.head_slots, token_slots = side.split.token_slots;
  const int heads = is_q ? nh : all_heads - nh, first = is_q ? 0 : nh;
  const int block = is_q ? blockIdx.x : blockIdx.x - bs.q.blocks;
  const int u = threadIdx.x % kUnits, slot = threadIdx.x / kUnits;
  const bool in = slot < head_slots * token_slots;
  const Unit w = unit_of(u, HD, rot);
  const int h0 = slot % head_slots, tslot = slot / head_slots;
  const uint4 g0 = __ldg(reinterpret_cast<const uint4*>((is_q ? gq : gk) + w.c0));
  const uint4 g1 = __ldg(reinterpret_cast<const uint4*>((is_q ? gq : gk) + w.c1));
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;

  int64_t t = static_cast<int64_t>(block) * token_slots + tslot;  // the row being loaded
  int hb = 0;
  const int64_t step = static_cast<int64_t>(side.blocks) * token_slots;
  const int turns = (heads + head_slots - 1) / head_slots;
  const int64_t token_turns = (T - 1 - static_cast<int64_t>(block) * token_slots) / step + 1;  // >= 1
  auto load = [&](RowPair& p) {
    p.d0 = p.d1 = p.x0 = p.x1 = make_uint4(0u, 0u, 0u, 0u);
    p.rs = 0.f;
    if (in && t < T && hb + h0 < heads) {
      const int64_t col = static_cast<int64_t>(first + hb + h0) * HD;
      const bf16 *dr = dy + t * lddy + col, *xr = x + t * ldx + col;
      p.d0 = *reinterpret_cast<const uint4*>(dr + w.c0);
      p.d1 = *reinterpret_cast<const uint4*>(dr + w.c1);
      p.x0 = *reinterpret_cast<const uint4*>(xr + w.c0);
      p.x1 = *reinterpret_cast<const uint4*>(xr + w.c1);
      p.rs = rstd[t * all_heads + first + hb + h0];
    }
  };
  float4 r[4], r_next[4];
  RowPair next;
  load(next);
  if (in && t < T && w.rotated) load_angles(cs, positions, t, n_pos, rot, interleaved, u, err, r_next);
  for (int64_t it = 0; it < token_turns * turns; ++it) {
    const RowPair cur = next;
    const int64_t tc = t;
    const int hc = hb + h0;
    const bool on = in && t < T && hc < heads;
    if (hb == 0) {
#pragma unroll
      for (int k = 0; k < 4; ++k) r[k] = r_next[k];
    }
    hb += head_slots;
    if (hb >= heads) {
      hb = 0;
      t += step;
      if (in && t < T && w.rotated) load_angles(cs, positions, t, n_pos, rot, interleaved, u, err, r_next);
    }
    load(next);
    float d[16], n[16], g[16];
    unpack8(cur.d0, d);
    unpack8(cur.d1, d + 8);
    unpack8(cur.x0, n);
    unpack8(cur.x1, n + 8);
    unpack8(g0, g);
    unpack8(g1, g + 8);
    if (on && w.rotated) rotate(d, r, interleaved, -1.f);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      n[i] *= cur.rs;
      acc[i] += d[i] * n[i];
      d[i] *= g[i];
      dot += d[i] * n[i];
    }
    const float m = row_sum<HD>(dot) * (1.f / HD);
    if (!on) continue;
#pragma unroll
    for (int i = 0; i < 16; ++i) d[i] = cur.rs * (d[i] - n[i] * m);
    bf16* o = dx + tc * lddx + static_cast<int64_t>(first + hc) * HD;
    *reinterpret_cast<uint4*>(o + w.c0) = pack8(d);
    *reinterpret_cast<uint4*>(o + w.c1) = pack8(d + 8);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) sums[threadIdx.x][i] = acc[i];
  __syncthreads();
  if (threadIdx.x < HD) {  // one thread per (unit, value) pair
    const int un = threadIdx.x / 16, i = threadIdx.x % 16;
    float s = 0.f;
    for (int k = 0; k < head_slots * token_slots; ++k) s += sums[k * kUnits + un][i];
    const Unit q = unit_of(un, HD, rot);
    partial[static_cast<int64_t>(blockIdx.x) * HD + (i < 8 ? q.c0 + i : q.c1 + i - 8)] = s;
  }
}

// Block 0: dgq[j] = sum of the query blocks' partial[p][j], block 1: dgk from the key blocks': the
// rows dealt to 1024/HD groups of threads (group g: rows g, g + groups, ...), then the groups added
// in order.
template <int HD>
__global__ void __launch_bounds__(1024)
    qk_gain_reduce_kernel(const float* __restrict__ partial, int blocks_q, int blocks_k, bf16* __restrict__ dgq,
                          bf16* __restrict__ dgk) {
  constexpr int kGroups = 1024 / HD;
  __shared__ float acc[kGroups][HD];
  const int j = threadIdx.x % HD, g = threadIdx.x / HD;
  const int p0 = blockIdx.x ? blocks_q : 0, p1 = blockIdx.x ? blocks_q + blocks_k : blocks_q;
  float s = 0.f;
  for (int p = p0 + g; p < p1; p += kGroups) s += partial[static_cast<int64_t>(p) * HD + j];
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
// nearest quarter turn, convert to fp32 with an error below 2^-26 turns.
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

bool rotation_ok(int hd, int rot, const float* cs, int n_pos, const int32_t* positions, const int* err) {
  if (rot < 0 || rot > hd || rot % 16) return false;
  if (rot == 0) return true;
  return cs && (reinterpret_cast<uintptr_t>(cs) & 15) == 0 && (reinterpret_cast<uintptr_t>(positions) & 3) == 0 &&
         n_pos > 0 && err;
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
  if (rot <= 0 || rot % 2 || rot / 2 > kRotaryMaxPairs || n_pos <= 0 || (reinterpret_cast<uintptr_t>(out) & 15))
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
  rotary_table_kernel<<<groups < 152 * 8 ? groups : 152 * 8, threads, 0, s>>>(f, reinterpret_cast<float2*>(out), n_pos,
                                                                             pairs, static_cast<float>(amp));
  return cudaGetLastError();
}

cudaError_t rotary(const bf16* x, int64_t ldx, bf16* y, int64_t ldy, int T, int heads, int hd, int rot,
                   bool interleaved, const int32_t* positions, const float* cs, int n_pos, bool inverse, int* err,
                   cudaStream_t s) {
  if (T <= 0 || !heads_ok(heads) || hd <= 0 || hd % 16 || hd > 16 * kRotThreads || rot == 0 ||
      !rotation_ok(hd, rot, cs, n_pos, positions, err))
    return cudaErrorInvalidValue;
  if (!vec_aligned(x, ldx) || !vec_aligned(y, ldy) || ldx < static_cast<int64_t>(heads) * hd ||
      ldy < static_cast<int64_t>(heads) * hd || (x == y && ldx != ldy))
    return cudaErrorInvalidValue;
  const RowSplit sp = row_split(heads, hd);
  const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(T) + sp.token_slots - 1) / sp.token_slots);
  rotary_kernel<<<blocks, sp.threads(), 0, s>>>(x, ldx, y, ldy, T, heads, hd, rot, interleaved, positions, cs, n_pos,
                                                inverse ? -1.f : 1.f, sp.units, sp.head_slots, sp.token_slots, err);
  return cudaGetLastError();
}

cudaError_t qk_norm_rope(const bf16* x, int64_t ldx, const bf16* gq, const bf16* gk, bf16* y, int64_t ldy, float* rstd,
                         int T, int nh, int nkv, int hd, int rot, bool interleaved, float eps,
                         const int32_t* positions, const float* cs, int n_pos, int* err, cudaStream_t s) {
  if (T <= 0 || nh <= 0 || nkv <= 0 || !heads_ok(static_cast<int64_t>(nh) + nkv) || (hd != 64 && hd != 128) || !rotation_ok(hd, rot, cs, n_pos, positions, err))
    return cudaErrorInvalidValue;
  const int heads = nh + nkv;
  if (!vec_aligned(x, ldx) || !vec_aligned(y, ldy) || !vec_aligned(gq, 0) || !vec_aligned(gk, 0) ||
      ldx < static_cast<int64_t>(heads) * hd || ldy < static_cast<int64_t>(heads) * hd || (x == y && ldx != ldy))
    return cudaErrorInvalidValue;
  const RowSplit sp = row_split(heads, hd);
  const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(T) + sp.token_slots - 1) / sp.token_slots);
  (hd == 64 ? qk_norm_rope_kernel<64> : qk_norm_rope_kernel<128>)<<<blocks, sp.threads(), 0, s>>>(
      x, ldx, gq, gk, y, ldy, rstd, T, nh, heads, rot, interleaved, eps, positions, cs, n_pos, sp.head_slots,
      sp.token_slots, err);
  return cudaGetLastError();
}

int qk_norm_rope_bwd_parts(int T, int nh, int nkv, int hd) {
  const BwdSplit s = bwd_split(T, nh, nkv, hd);
  return s.q.blocks + s.k.blocks;
}

cudaError_t qk_norm_rope_bwd(const bf16* dy, int64_t lddy, const bf16* x, int64_t ldx, const bf16* gq, const bf16* gk,
                             const float* rstd, bf16* dx, int64_t lddx, float* partial, bf16* dgq, bf16* dgk, int T,
                             int nh, int nkv, int hd, int rot, bool interleaved, const int32_t* positions,
                             const float* cs, int n_pos, int* err, cudaStream_t s) {
  if (T <= 0 || nh <= 0 || nkv <= 0 || !heads_ok(static_cast<int64_t>(nh) + nkv) || (hd != 64 && hd != 128) || !rotation_ok(hd, rot, cs, n_pos, positions, err))
    return cudaErrorInvalidValue;
  const int heads = nh + nkv;
  const int64_t cols = static_cast<int64_t>(heads) * hd;
  if (!vec_aligned(dy, lddy) || !vec_aligned(x, ldx) || !vec_aligned(dx, lddx) || !vec_aligned(gq, 0) ||
      !vec_aligned(gk, 0) || lddy < cols || ldx < cols || lddx < cols || (dx == dy && lddx != lddy) ||
      (dx == x && lddx != ldx))
    return cudaErrorInvalidValue;
  const BwdSplit sp = bwd_split(T, nh, nkv, hd);
  (hd == 64 ? qk_norm_rope_bwd_kernel<64> : qk_norm_rope_bwd_kernel<128>)<<<sp.q.blocks + sp.k.blocks, kRotThreads, 0,
                                                                            s>>>(
      dy, lddy, x, ldx, gq, gk, rstd, dx, lddx, partial, T, nh, heads, rot, interleaved, positions, cs, n_pos, sp, err);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  (hd == 64 ? qk_gain_reduce_kernel<64> : qk_gain_reduce_kernel<128>)<<<2, 1024, 0, s>>>(
      partial, sp.q.blocks, sp.k.blocks, dgq, dgk);
  return cudaGetLastError();
}

}  // namespace mt
