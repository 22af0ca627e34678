// Rows of fp32 or bf16 numbers, eight columns at a time: 16-byte accesses, arithmetic in fp32. Shared by the
// kernels of the losses, the layer norm and the embedding.
#pragma once
#include <cstdint>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace mt {

// Eight neighbouring columns. A thread's loads are issued first and unpacked where they are used.
template <class T>
struct Raw8;
template <>
struct Raw8<float> {
  uint4 a, b;
};
template <>
struct Raw8<bf16> {
  uint4 a;
};

__device__ __forceinline__ Raw8<float> load8(const float* p) {
  const uint4* q = reinterpret_cast<const uint4*>(p);
  return {q[0], q[1]};
}
__device__ __forceinline__ Raw8<bf16> load8(const bf16* p) { return {*reinterpret_cast<const uint4*>(p)}; }

__device__ __forceinline__ void unpack8(const uint4& u, float* v) {
  const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(x[i] << 16);
    v[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<bf16>& r, float* v) { unpack8(r.a, v); }
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float* v) {
  const uint32_t x[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(x[i]);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store8(bf16* p, const float* v) { *reinterpret_cast<uint4*>(p) = pack8(v); }
__device__ __forceinline__ void store8(float* p, const float* v) {
  float4* q = reinterpret_cast<float4*>(p);
  q[0] = make_float4(v[0], v[1], v[2], v[3]);
  q[1] = make_float4(v[4], v[5], v[6], v[7]);
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16 x) { return __bfloat162float(x); }

// A token id outside the vocabulary: a data error, which does not replace another code.
__device__ __forceinline__ void record_bad_token(int* err) {
  if (err) atomicCAS(err, 0, kErrBadToken);
}

// Element types of the entries that take more than one (MTK_F32, MTK_BF16 of the C ABI).
enum RowType : int { kRowF32 = 0, kRowBf16 = 1 };
inline bool row_type_ok(int t) { return t == kRowF32 || t == kRowBf16; }
inline int row_type_bytes(int t) { return t == kRowF32 ? 4 : 2; }

// A matrix of `rows` rows that the kernels take in 16-byte accesses.
inline bool rows_ok(const void* p, int64_t ld, int64_t cols) {
  return p && (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld >= cols && ld % 8 == 0;
}
inline bool vec_ok(const void* p, uintptr_t bytes) { return p && (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
// Whether two matrices share memory, from the first to the last element of each.
inline bool spans_overlap(const void* a, int64_t lda, int esz_a, const void* b, int64_t ldb, int esz_b, int64_t rows,
                          int64_t cols) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  const uintptr_t a1 = a0 + ((rows - 1) * lda + cols) * esz_a, b1 = b0 + ((rows - 1) * ldb + cols) * esz_b;
  return a0 < b1 && b0 < a1;
}

inline bool ranges_overlap(const void* a, uint64_t bytes_a, const void* b, uint64_t bytes_b) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + bytes_b && b0 < a0 + bytes_a;
}

}  // namespace mt
