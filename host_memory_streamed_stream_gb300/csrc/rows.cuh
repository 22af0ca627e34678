// Rows of fp32 or bf16 numbers, eight columns at a time: 16-byte accesses, arithmetic in fp32. Shared by the
// kernels of the losses, the layer norm and the embedding.
#pragma once
#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace mt {

__device__ __forceinline__ void unpack8(const uint4& u, float* v) {
  const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(x[i] << 16);
    v[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16 x) { return __bfloat162float(x); }

// W neighbouring columns, in 8 or 16 bytes.
__device__ __forceinline__ void unpack2(uint32_t x, float* v) {
  v[0] = __uint_as_float(x << 16);
  v[1] = __uint_as_float(x & 0xffff0000u);
}
template <class T, int W>
__device__ __forceinline__ void read_cols(const T* p, float* v) {
  if constexpr (sizeof(T) == 4) {
    static_assert(W == 4, "16 bytes");
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else if constexpr (W == 4) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    unpack2(q.x, v);
    unpack2(q.y, v + 2);
  } else {
    unpack8(*reinterpret_cast<const uint4*>(p), v);
  }
}
template <class T, int W>
__device__ __forceinline__ void write_cols(T* p, const float* v) {
  if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else if constexpr (W == 4) *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  else *reinterpret_cast<uint4*>(p) = pack8(v);
}

// cp.async: 16 bytes (or 8) of global memory to shared memory. A thread waits for its own copies by groups.
__device__ __forceinline__ void cp_async_chunk(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_half(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_end_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most n of this thread's groups are in flight. Rings of 4 rows need n <= 3; the other cases make a jump table
// of the switch, whose pace suits the layer norm's fp32 backward at 8192 x 4096 (97 us, 102 as a chain of tests), but
// not at 8000 x 5120 (138, 113).
__device__ __forceinline__ void cp_async_wait_groups(int n) {
#define MT_WAIT(N) \
  case N: asm volatile("cp.async.wait_group " #N ";" ::: "memory"); break;
  switch (n) {
    MT_WAIT(1) MT_WAIT(2) MT_WAIT(3) MT_WAIT(4) MT_WAIT(5) MT_WAIT(6) MT_WAIT(7) MT_WAIT(8) MT_WAIT(9) MT_WAIT(10)
    MT_WAIT(11) MT_WAIT(12) MT_WAIT(13) MT_WAIT(14) MT_WAIT(15) MT_WAIT(16) MT_WAIT(17) MT_WAIT(18) MT_WAIT(19)
    MT_WAIT(20) MT_WAIT(21) MT_WAIT(22) MT_WAIT(23) MT_WAIT(24)
    default: asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
#undef MT_WAIT
}

// Bulk copies of shared memory to global memory: both 16-byte aligned, a multiple of 16 bytes. What was written to
// shared memory before is fenced first; the source stays as it is until the copies have read it.
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void bulk_store(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_store_end_group() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// The blocks of a cluster.
__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned cluster_blocks() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Also between the start of the blocks and their first access to each other's shared memory.
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

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
// Whether two matrices may share an element: not if one ends before the other begins, nor if they lie beside each other
// in rows of one buffer, the same number of bytes apart. What else interleaves counts as sharing.
inline bool spans_overlap(const void* a, int64_t lda, int esz_a, const void* b, int64_t ldb, int esz_b, int64_t rows,
                          int64_t cols) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  const uintptr_t a1 = a0 + ((rows - 1) * lda + cols) * esz_a, b1 = b0 + ((rows - 1) * ldb + cols) * esz_b;
  if (a1 <= b0 || b1 <= a0) return false;
  const uintptr_t row = lda * esz_a, wide_a = cols * esz_a, wide_b = cols * esz_b;
  if (row != static_cast<uintptr_t>(ldb * esz_b)) return true;
  // from the start of a row of a on to the next one of b
  const uintptr_t gap = b0 >= a0 ? (b0 - a0) % row : row - 1 - (a0 - b0 - 1) % row;
  return gap < wide_a || gap + wide_b > row;
}

inline bool ranges_overlap(const void* a, uint64_t bytes_a, const void* b, uint64_t bytes_b) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + bytes_b && b0 < a0 + bytes_a;
}

}  // namespace mt
