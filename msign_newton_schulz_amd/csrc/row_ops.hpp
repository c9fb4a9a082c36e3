// Helpers of the kernels that work on rows: 16-byte chunks of a row as
// fp32 values, and reductions over a workgroup.
#pragma once

#include "common.hpp"

namespace msign {
namespace rows {

// A 16-byte access at any element's address: rows of odd length start
// anywhere, and gfx950's vector memory path takes such addresses.
typedef u32x4 u32x4_any __attribute__((aligned(2)));

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

template <typename T> struct Raw { using type = uint16_t; };
template <> struct Raw<float> { using type = uint32_t; };

// Elements i .. i + CE - 1 of a row of n, `fill` bits past its end.
template <typename T>
__device__ __forceinline__ u32x4 load_chunk(const void* row, int i, int n, uint32_t fill) {
  using R = typename Raw<T>::type;
  constexpr int CE = 16 / Elem<T>::size;
  const R* p = static_cast<const R*>(row) + i;
  if (i + CE <= n) return *reinterpret_cast<const u32x4_any*>(p);
  u32x4 v;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if constexpr (CE == 8) {
      const uint32_t lo = i + 2 * w < n ? p[2 * w] : fill;
      const uint32_t hi = i + 2 * w + 1 < n ? p[2 * w + 1] : fill;
      v[w] = lo | (hi << 16);
    } else {
      v[w] = i + w < n ? p[w] : fill;
    }
  }
  return v;
}

template <typename T>
__device__ __forceinline__ void store_chunk(void* row, int i, int n, const u32x4& v) {
  using R = typename Raw<T>::type;
  constexpr int CE = 16 / Elem<T>::size;
  R* p = static_cast<R*>(row) + i;
  if (i + CE <= n) {
    *reinterpret_cast<u32x4_any*>(p) = v;
    return;
  }
#pragma unroll
  for (int e = 0; e < CE; ++e)
    if (i + e < n) p[e] = CE == 8 ? (R)(v[e >> 1] >> (16 * (e & 1))) : (R)v[e & 3];
}

template <typename T>
__device__ __forceinline__ void unpack(const u32x4& v, float (&f)[16 / Elem<T>::size]) {
  if constexpr (Elem<T>::size == 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __builtin_bit_cast(f32x4, v)[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint16_t h = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
      f[e] = Elem<T>::dt == DT_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
    }
  }
}

template <typename T>
__device__ __forceinline__ u32x4 pack(const float (&f)[16 / Elem<T>::size]) {
  u32x4 v;
  if constexpr (Elem<T>::size == 4) {
    const f32x4 t = {f[0], f[1], f[2], f[3]};
    v = __builtin_bit_cast(u32x4, t);
  } else {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const f32x2 t = {f[2 * w], f[2 * w + 1]};
      if constexpr (Elem<T>::dt == DT_BF16) v[w] = __builtin_bit_cast(uint32_t, __builtin_convertvector(t, bf16x2));
      else v[w] = __builtin_bit_cast(uint32_t, __builtin_convertvector(t, f16x2));
    }
  }
  return v;
}

// Rows held by a workgroup.  Chunk c of a thread is chunk c NT + t of the row's `whole` 16-byte chunks
// (its last n % CE elements are taken one by one, by the first threads).  A
// thread past the end takes the last chunk: it loads it and stores the
// same result as the chunk's own thread, and only the sums leave it out.  So the
// passes over a row have no branch, which lets the compiler count the loads in
// flight instead of waiting for all of them.  This holds for what is loaded before
// any of the row's stores: where an output takes an input's place, a pass that
// loads between its stores leaves these threads out.
template <int NT>
__device__ __forceinline__ uint32_t chunk_offset(int c, int t, int whole) {
  const int i = c * NT + t;
  return (uint32_t)(i < whole ? i : whole - 1) * 16u;
}

__device__ __forceinline__ u32x4 load_at(const char* row, uint32_t off) {
  return *reinterpret_cast<const u32x4_any*>(row + off);
}

__device__ __forceinline__ void store_at(char* row, uint32_t off, const u32x4& v) {
  *reinterpret_cast<u32x4_any*>(row + off) = v;
}

// Sum over a workgroup of NT threads in a fixed order, in every thread.
// `slots`: NT / 64 floats of LDS that no other wave still reads.
template <int NT>
__device__ __forceinline__ float block_sum(float v, float* slots) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) v += slots[w];
  }
  return v;
}

}  // namespace rows
}  // namespace msign
