// Rotary positions beyond the layer template's (explicit positions, part of the head, both pair
// layouts, scaled frequencies) and the norms of queries and keys fused with the rotation.
//
// All of it is bound by HBM (a few operations per 2-byte element), so each kernel moves every
// element once, in 16-byte accesses. A head's row of hd columns is cut into hd/16 units of two
// 16-byte vectors, one unit per thread: a unit of the rotated part holds 8 whole rotation pairs in
// either layout (half: columns [8u, 8u+8) and [rot/2 + 8u, +8); interleaved: columns
// [16u, 16u+16); both are rotation indices [8u, 8u+8)), so the rotation needs no exchange between
// threads, and a thread keeps the same unit, and so the same cosines and sines, for every head of
// its token.
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
__device__ __forceinline__ Unit unit_of(int u, int rot, bool interleaved) {
  if (16 * u >= rot || interleaved) return {16 * u, 16 * u + 8, 16 * u < rot};
  return {8 * u, rot / 2 + 8 * u, true};
}

// Cosine and sine of the unit's 8 rotation indices at a token's position; a position outside the
// table raises the error flag and leaves the token as it is (angle 0).
__device__ __forceinline__ void load_angles(const float* __restrict__ cs, const int32_t* __restrict__ positions,
                                            int64_t t, int n_pos, int rot, int u, int* err, float4 (&r)[4]) {
  const int p = positions ? positions[t] : static_cast<int>(t % n_pos);
  if (p < 0 || p >= n_pos) {
    atomicCAS(err, 0, kErrBadPosition);
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = make_float4(1.f, 0.f, 1.f, 0.f);
    return;
  }
  const float4* q = reinterpret_cast<const float4*>(cs + static_cast<int64_t>(p) * rot + 16 * u);
#pragma unroll
  for (int k = 0; k < 4; ++k) r[k] = __ldg(q + k);
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

// Threads of a block: unit (fastest), head slot, token slot.
struct RowSplit {
  int units, head_slots, token_slots;
  int threads() const { return units * head_slots * token_slots; }
};
RowSplit row_split(int heads, int hd) {
  RowSplit s;
  s.units = hd / 16;
  const int slots = kRotThreads / s.units;
  s.head_slots = heads < slots ? heads : slots;
  s.token_slots = slots / s.head_slots;
  return s;
}

__global__ void __launch_bounds__(kRotThreads)
    rotary_kernel(const bf16* x, int64_t ldx, bf16* y, int64_t ldy, int T, int heads, int hd, int rot, bool interleaved,
                  const int32_t* __restrict__ positions, const float* __restrict__ cs, int n_pos, float sgn, int units,
                  int head_slots, int token_slots, int* err) {
  const int u = threadIdx.x % units, slot = threadIdx.x / units;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * token_slots + slot / head_slots;
  if (t >= T) return;
  const Unit w = unit_of(u, rot, interleaved);
  if (!w.rotated && x == y) return;
  float4 r[4];
  if (w.rotated) load_angles(cs, positions, t, n_pos, rot, u, err, r);
  for (int h = slot % head_slots; h < heads; h += head_slots) {
    const bf16* xr = x + t * ldx + static_cast<int64_t>(h) * hd;
    bf16* yr = y + t * ldy + static_cast<int64_t>(h) * hd;
    uint4 a = *reinterpret_cast<const uint4*>(xr + w.c0), b = *reinterpret_cast<const uint4*>(xr + w.c1);
    if (w.rotated) {
      float v[16];
      unpack8(a, v);
      unpack8(b, v + 8);
      rotate(v, r, interleaved, sgn);
      a = pack8(v);
      b = pack8(v + 8);
    }
    *reinterpret_cast<uint4*>(yr + w.c0) = a;
    *reinterpret_cast<uint4*>(yr + w.c1) = b;
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
  const Unit w = unit_of(u, rot, interleaved);
  float4 r[4];
  if (live && w.rotated) load_angles(cs, positions, t, n_pos, rot, u, err, r);
  const int h0 = slot % head_slots;
  for (int hb = 0; hb < heads; hb += head_slots) {  // the same trip count in every thread
    const int h = hb + h0;
    const bool on = live && h < heads;
    float v[16];
    if (on) {
      const bf16* xr = x + t * ldx + static_cast<int64_t>(h) * HD;
      unpack8(*reinterpret_cast<const uint4*>(xr + w.c0), v);
      unpack8(*reinterpret_cast<const uint4*>(xr + w.c1), v + 8);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.f;
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss += v[i] * v[i];
    const float rs = rsqrtf(row_sum<HD>(ss) * (1.f / HD) + eps);
    if (!on) continue;
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

// With u = R^T dy and n = x rstd: dx = rstd (u g - n mean(u g n)) per head row, and each block's
// share of dg = sum over tokens and heads of u n. A thread keeps its 16 columns for every row it
// takes, so the gain sums stay in registers; at the end they are added over the block's slots in
// slot order and written to the block's row of `partial`, [2][HD] (q, k): fixed order, no atomics.
template <int HD>
__global__ void __launch_bounds__(kRotThreads)
    qk_norm_rope_bwd_kernel(const bf16* dy, int64_t lddy, const bf16* x, int64_t ldx, const bf16* __restrict__ gq,
                            const bf16* __restrict__ gk, const float* __restrict__ rstd, bf16* dx, int64_t lddx,
                            float* __restrict__ partial, int T, int nh, int heads, int rot, bool interleaved,
                            const int32_t* __restrict__ positions, const float* __restrict__ cs, int n_pos,
                            int head_slots, int token_slots, int* err) {
  constexpr int kUnits = HD / 16;
  __shared__ float sums[kRotThreads][17];
  const int u = threadIdx.x % kUnits, slot = threadIdx.x / kUnits;
  const bool in = slot < head_slots * token_slots;
  const Unit w = unit_of(u, rot, interleaved);
  const int h0 = slot % head_slots, tslot = slot / head_slots;
  float accq[16], acck[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) accq[i] = acck[i] = 0.f;
  for (int64_t tb = static_cast<int64_t>(blockIdx.x) * token_slots; tb < T;
       tb += static_cast<int64_t>(gridDim.x) * token_slots) {
    const int64_t t = tb + tslot;
    const bool live = in && t < T;
    float4 r[4];
    if (live && w.rotated) load_angles(cs, positions, t, n_pos, rot, u, err, r);
    for (int hb = 0; hb < heads; hb += head_slots) {
      const int h = hb + h0;
      const bool on = live && h < heads;
      float d[16], n[16], g[16];
      float rs = 0.f;
      if (on) {
        const bf16* dr = dy + t * lddy + static_cast<int64_t>(h) * HD;
        const bf16* xr = x + t * ldx + static_cast<int64_t>(h) * HD;
        unpack8(*reinterpret_cast<const uint4*>(dr + w.c0), d);
        unpack8(*reinterpret_cast<const uint4*>(dr + w.c1), d + 8);
        unpack8(*reinterpret_cast<const uint4*>(xr + w.c0), n);
        unpack8(*reinterpret_cast<const uint4*>(xr + w.c1), n + 8);
        rs = rstd[t * heads + h];
        const bf16* gain = h < nh ? gq : gk;
        unpack8(__ldg(reinterpret_cast<const uint4*>(gain + w.c0)), g);
        unpack8(__ldg(reinterpret_cast<const uint4*>(gain + w.c1)), g + 8);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) d[i] = n[i] = g[i] = 0.f;
      }
      if (on && w.rotated) rotate(d, r, interleaved, -1.f);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        n[i] *= rs;
        const float un = d[i] * n[i];
        if (h < nh)
          accq[i] += un;
        else
          acck[i] += un;
        d[i] *= g[i];
        dot += d[i] * n[i];
      }
      const float m = row_sum<HD>(dot) * (1.f / HD);
      if (!on) continue;
#pragma unroll
      for (int i = 0; i < 16; ++i) d[i] = rs * (d[i] - n[i] * m);
      bf16* o = dx + t * lddx + static_cast<int64_t>(h) * HD;
      *reinterpret_cast<uint4*>(o + w.c0) = pack8(d);
      *reinterpret_cast<uint4*>(o + w.c1) = pack8(d + 8);
    }
  }
  for (int part = 0; part < 2; ++part) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) sums[threadIdx.x][i] = part ? acck[i] : accq[i];
    __syncthreads();
    if (threadIdx.x < HD) {  // one thread per (unit, value) pair
      const int un = threadIdx.x / 16, i = threadIdx.x % 16;
      float s = 0.f;
      for (int k = 0; k < static_cast<int>(blockDim.x) / kUnits; ++k) s += sums[k * kUnits + un][i];
      const Unit q = unit_of(un, rot, interleaved);
      partial[(static_cast<int64_t>(blockIdx.x) * 2 + part) * HD + (i < 8 ? q.c0 + i : q.c1 + i - 8)] = s;
    }
  }
}

// dg[part][j] = sum of partial[p][part][j] over p: one block per gain, the rows dealt to 1024/HD
// groups of threads (group g: rows g, g + groups, ...), then the groups added in order.
template <int HD>
__global__ void __launch_bounds__(1024)
    qk_gain_reduce_kernel(const float* __restrict__ partial, int parts, bf16* __restrict__ dgq, bf16* __restrict__ dgk) {
  constexpr int kGroups = 1024 / HD;
  __shared__ float acc[kGroups][HD];
  const int j = threadIdx.x % HD, g = threadIdx.x / HD;
  float s = 0.f;
  for (int p = g; p < parts; p += kGroups) s += partial[(static_cast<int64_t>(p) * 2 + blockIdx.x) * HD + j];
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

__device__ __forceinline__ float2 cos_sin_turns(uint64_t phase, float amp) {
  const uint32_t top = static_cast<uint32_t>(phase >> 32);
  const uint32_t quarter = (top + (1u << 29)) >> 30;
  const float half_turns = static_cast<float>(static_cast<int32_t>(top - (quarter << 30))) * 0x1p-31f;
  float s, c;
  sincospif(half_turns, &s, &c);
  const float a = (quarter & 1) ? s : c, b = (quarter & 1) ? c : s;
  return make_float2((quarter == 1 || quarter == 2) ? -a * amp : a * amp, (quarter & 2) ? -b * amp : b * amp);
}

__global__ void rotary_table_kernel(const __grid_constant__ TurnTable f, float2* __restrict__ out, int64_t total,
                                    int pairs, float amp) {
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x)
    out[i] = cos_sin_turns(static_cast<uint64_t>(i / pairs) * f.turns[i % pairs], amp);
}

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
  const int64_t total = static_cast<int64_t>(n_pos) * (rot / 2);
  const int64_t blocks = (total + 255) / 256;
  rotary_table_kernel<<<static_cast<unsigned>(blocks < 152 * 32 ? blocks : 152 * 32), 256, 0, s>>>(
      f, reinterpret_cast<float2*>(out), total, rot / 2, static_cast<float>(amp));
  return cudaGetLastError();
}

cudaError_t rotary(const bf16* x, int64_t ldx, bf16* y, int64_t ldy, int T, int heads, int hd, int rot,
                   bool interleaved, const int32_t* positions, const float* cs, int n_pos, bool inverse, int* err,
                   cudaStream_t s) {
  if (T <= 0 || heads <= 0 || hd <= 0 || hd % 16 || hd > 16 * kRotThreads || rot == 0 ||
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
  const int heads = nh + nkv;
  if (T <= 0 || nh <= 0 || nkv <= 0 || (hd != 64 && hd != 128) || !rotation_ok(hd, rot, cs, n_pos, positions, err))
    return cudaErrorInvalidValue;
  if (!vec_aligned(x, ldx) || !vec_aligned(y, ldy) || !vec_aligned(gq, 0) || !vec_aligned(gk, 0) ||
      ldx < static_cast<int64_t>(heads) * hd || ldy < static_cast<int64_t>(heads) * hd || (x == y && ldx != ldy))
    return cudaErrorInvalidValue;
  const RowSplit sp = row_split(heads, hd);
  const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(T) + sp.token_slots - 1) / sp.token_slots);
  (hd == 64 ? qk_norm_rope_kernel<64> : qk_norm_rope_kernel<128>)<<<blocks, kRotThreads, 0, s>>>(
      x, ldx, gq, gk, y, ldy, rstd, T, nh, heads, rot, interleaved, eps, positions, cs, n_pos, sp.head_slots,
      sp.token_slots, err);
  return cudaGetLastError();
}

int qk_norm_rope_bwd_parts(int T, int nh, int nkv, int hd) {
  const RowSplit sp = row_split(nh + nkv, hd);
  const int64_t blocks = (static_cast<int64_t>(T) + sp.token_slots - 1) / sp.token_slots;
  return static_cast<int>(blocks < kQkNormParts ? blocks : kQkNormParts);
}

cudaError_t qk_norm_rope_bwd(const bf16* dy, int64_t lddy, const bf16* x, int64_t ldx, const bf16* gq, const bf16* gk,
                             const float* rstd, bf16* dx, int64_t lddx, float* partial, bf16* dgq, bf16* dgk, int T,
                             int nh, int nkv, int hd, int rot, bool interleaved, const int32_t* positions,
                             const float* cs, int n_pos, int* err, cudaStream_t s) {
  const int heads = nh + nkv;
  if (T <= 0 || nh <= 0 || nkv <= 0 || (hd != 64 && hd != 128) || !rotation_ok(hd, rot, cs, n_pos, positions, err))
    return cudaErrorInvalidValue;
  const int64_t cols = static_cast<int64_t>(heads) * hd;
  if (!vec_aligned(dy, lddy) || !vec_aligned(x, ldx) || !vec_aligned(dx, lddx) || !vec_aligned(gq, 0) ||
      !vec_aligned(gk, 0) || lddy < cols || ldx < cols || lddx < cols || (dx == dy && lddx != lddy) ||
      (dx == x && lddx != ldx))
    return cudaErrorInvalidValue;
  const RowSplit sp = row_split(heads, hd);
  const int parts = qk_norm_rope_bwd_parts(T, nh, nkv, hd);
  (hd == 64 ? qk_norm_rope_bwd_kernel<64> : qk_norm_rope_bwd_kernel<128>)<<<parts, kRotThreads, 0, s>>>(
      dy, lddy, x, ldx, gq, gk, rstd, dx, lddx, partial, T, nh, heads, rot, interleaved, positions, cs, n_pos,
      sp.head_slots, sp.token_slots, err);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  (hd == 64 ? qk_gain_reduce_kernel<64> : qk_gain_reduce_kernel<128>)<<<2, 1024, 0, s>>>(partial, parts, dgq, dgk);
  return cudaGetLastError();
}

}  // namespace mt
