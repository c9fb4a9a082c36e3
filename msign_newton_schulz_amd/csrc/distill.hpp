// Distillation on a teacher's top logits: loss and gradient of a row of
// logits z against the teacher's distribution p over `top` of its entries.
//
// With m = max z, S = sum exp((z - m) / tau):
//     log q_i = (z_i - m) / tau - log S
//     loss    = tau^2 sum_k p_k (log p_k - log q_{i_k})
//     dz_j    = tau grad (exp((z_j - m) / tau) / S - p_j)
// z - m is formed before the division, so that rows of the type's lowest
// value do not overflow.  A workgroup takes a row and reads it once where it
// fits its registers (C chunks of 16 bytes a thread), keeping the running
// maximum and sum of a softmax; longer rows are read again for the gradient.
// The gradient is written as if p were 0 and the at most `top` elements with a
// teacher's entry are then written once more, each from the fp32 value.
//
// Bound by memory.  Measured with the gradient (one read, one write): bf16, 8192
// x 131072, 4.3 GB in 880 to 925 us, 4.6 to 4.9 TB/s; f32, 1001 x 50021, rows off
// 16 bytes, 98 us, 4.1 TB/s.  A form whose row in registers spilled took 2446 us
// for the first; loading the next row into the registers that this row's
// gradient leaves, with no branch, so that loads are counted, made the rest.  The
// loss alone: 256 MB of rows of 32768 47 us, 5.7 TB/s; 32 rows of 32000 6.9 us,
// latency.  The teacher's entries are compared with one another for equal indices,
// which long lists pay for (bf16, us with the gradient, 8 / 64 / 128 / 256 / 512 /
// 1024 entries: 16384 x 8192 127 / 145 / 183 / 271 / 802 / 2911; 4194 x 32000 114 /
// 131 / 147 / 182 / 419 / 1407; 1024 x 131072 124 / 128 / 142 / 169 / 237 / 549; the
// loss alone 67 to 126, 51 to 92, 51 to 65).
#pragma once

#include "gemm_nt.hpp"
#include "row_ops.hpp"

#include <cfloat>

namespace msign {
namespace distill {

using namespace rows;

constexpr int kMaxTop = 1024;

struct Args {
  const void* z;
  int64_t ldz;
  const void* idx;
  const void* teacher;
  const float* grad;
  int64_t grad_stride;
  float* loss;
  void* dz;
  int64_t rows;
  int32_t idx64, teacher_dtype, vocab, top;
  float tau;
};

// A maximum and the sum of exp((v - max) / tau) over some values.
struct MaxSum {
  float m, s;
};

__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.f : m; }

// k = log2(e) / tau
__device__ __forceinline__ MaxSum join(const MaxSum& a, const MaxSum& b, float k) {
  const float m = fmaxf(a.m, b.m), r = finite_or_zero(m);
  return {m, a.s * __builtin_amdgcn_exp2f((a.m - r) * k) + b.s * __builtin_amdgcn_exp2f((b.m - r) * k)};
}

template <typename T>
__device__ __forceinline__ void add_chunk(MaxSum& a, const u32x4& v, float k, bool in) {
  constexpr int CE = 16 / Elem<T>::size;
  float f[CE];
  unpack<T>(v, f);
  float m = a.m;
#pragma unroll
  for (int e = 0; e < CE; e += 2) m = fmaxf(fmaxf(f[e], f[e + 1]), m);  // (one instruction)
  const float r = finite_or_zero(m);
  float s = a.s * __builtin_amdgcn_exp2f((a.m - r) * k);
#pragma unroll
  for (int e = 0; e < CE; ++e) s += __builtin_amdgcn_exp2f((f[e] - r) * k);
  a.m = in ? m : a.m;
  a.s = in ? s : a.s;
}

// Over a wave, in every lane: the maximum first, so that each lane rescales
// its sum once and the butterfly adds.
__device__ __forceinline__ MaxSum wave_join(const MaxSum& a, float k) {
  float m = a.m;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
  float s = a.s * __builtin_amdgcn_exp2f((a.m - finite_or_zero(m)) * k);
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off);
  return {m, s};
}

// Of the W waves' values in LDS.
template <int W>
__device__ __forceinline__ MaxSum join_waves(const MaxSum* w, float k) {
  MaxSum v[W];
  float m = -INFINITY, s = 0.f;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    v[i] = w[i];
    m = fmaxf(m, v[i].m);
  }
  const float r = finite_or_zero(m);
#pragma unroll
  for (int i = 0; i < W; ++i) s += v[i].s * __builtin_amdgcn_exp2f((v[i].m - r) * k);
  return {m, s};
}

// The teacher's entries of a row that a thread takes (entry e NT + t): index
// (-1: padding) and teacher's logit.
template <int NT>
struct Entries {
  static constexpr int E = (kMaxTop + NT - 1) / NT;
  int i[E];
  float t[E];

  __device__ __forceinline__ void load(const Args& a, int64_t row) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int s = e * NT + (int)threadIdx.x;
      i[e] = -1;
      t[e] = -INFINITY;
      if (s >= a.top) continue;
      const int64_t at = row * a.top + s;
      const int64_t j = a.idx64 ? static_cast<const int64_t*>(a.idx)[at] : static_cast<const int32_t*>(a.idx)[at];
      const float v = load_as_f32(a.teacher, at, a.teacher_dtype);
      if (j >= 0 && j < a.vocab) {
        i[e] = (int)j;
        t[e] = v;
      }
    }
  }
};

// A workgroup takes rows blockIdx, blockIdx + gridDim, ...  With C > 0 (and a
// gradient) the row is in registers, C chunks a thread: chunk c of the next
// row is loaded as soon as this row's gradient of chunk c is stored, so that
// memory works through both passes over the registers.  With C = 0 rows are
// streamed, twice for a gradient.
//
// OCC: waves per SIMD that the registers have to allow.  Several workgroups on
// a CU cover each other's reductions.
template <typename T, int NT, int C, bool GRAD, int OCC>
__global__ void __launch_bounds__(NT, OCC) row_kernel(const Args a) {
  constexpr int CE = 16 / Elem<T>::size, W = NT / 64, E = Entries<NT>::E;
  __shared__ float p_k[kMaxTop], z_k[GRAD ? kMaxTop : 1];
  __shared__ int i_k[kMaxTop];
  __shared__ MaxSum join_z[W], join_t[W];
  __shared__ float slots[W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = a.vocab;
  const int whole = n / CE, tail = n % CE;  // chunks and single elements
  // (finite at any tau: the largest logit's difference is 0 and stays 0)
  const float k = fminf(1.44269504f / a.tau, FLT_MAX);
  auto zrow = [&](int64_t row) { return static_cast<const char*>(a.z) + row * a.ldz * Elem<T>::size; };

  constexpr int KEEP = C > 0 ? C : 1;
  u32x4 v[KEEP];
  Entries<NT> ent;
  int64_t row = blockIdx.x;
  if constexpr (C > 0) {
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = load_at(zrow(row), chunk_offset<NT>(c, tid, whole));
  }
  // The next row's maximum and sum over chunks 0 .. C - LAG - 1, taken LAG
  // chunks behind its loads, while this row's gradient is stored.
  constexpr int LAG = C < 8 ? C : 8;
  MaxSum ahead = {-INFINITY, 0.f};
  if constexpr (C > LAG) {
    static_for<C - LAG>([&](auto I) {
      constexpr int c = decltype(I)::value;
      add_chunk<T>(ahead, v[c], k, c * NT + tid < whole);
      __builtin_amdgcn_sched_barrier(0);
    });
  }
  ent.load(a, row);
  for (; row < a.rows; row += gridDim.x) {
    // the thread's number, new to the compiler in every row: it would else keep
    // C addresses in registers from row to row
    int ot = tid;
    asm volatile("" : "+v"(ot));
    const char* z = zrow(row);
    float zt[E];  // the student's logits at the entries
#pragma unroll
    for (int e = 0; e < E; ++e) zt[e] = ent.i[e] >= 0 ? load_as_f32(z, ent.i[e], Elem<T>::dt) : 0.f;
    const float last = tid < tail ? load_as_f32(z, whole * CE + tid, Elem<T>::dt) : -INFINITY;
    MaxSum q = {-INFINITY, 0.f}, t = {-INFINITY, 0.f};
    if constexpr (C > 0) {
      q = ahead;
      static_for<LAG>([&](auto I) {
        constexpr int c = C - LAG + decltype(I)::value;
        add_chunk<T>(q, v[c], k, c * NT + ot < whole);
        __builtin_amdgcn_sched_barrier(0);  // (chunks unpacked ahead of their turn do not fit the registers)
      });
    } else {
      constexpr int U = 4;
      for (int c0 = 0; c0 * NT < whole; c0 += U) {
        u32x4 u[U];
#pragma unroll
        for (int c = 0; c < U; ++c) u[c] = load_at(z, chunk_offset<NT>(c0 + c, tid, whole));
#pragma unroll
        for (int c = 0; c < U; ++c) add_chunk<T>(q, u[c], k, (c0 + c) * NT + tid < whole);
      }
    }
    q = join(q, MaxSum{last, last == -INFINITY ? 0.f : 1.f}, k);
#pragma unroll
    for (int e = 0; e < E; ++e) t = join(t, MaxSum{ent.t[e], ent.t[e] == -INFINITY ? 0.f : 1.f}, k);
    q = wave_join(q, k);
    t = wave_join(t, k);
    if constexpr (W > 1) {
      if (lane == 0) {
        join_z[wave] = q;
        join_t[wave] = t;
      }
      __syncthreads();
      q = join_waves<W>(join_z, k);
      t = join_waves<W>(join_t, k);
    } else {
      __syncthreads();  // (the last row's entries have been read)
    }
    const float mz = finite_or_zero(q.m), mt = finite_or_zero(t.m);
    const bool any = t.s != 0.f;  // (NaN counts as something)
    const float log_st = a.tau * (logf(q.s) - logf(t.s)), inv_t = 1.f / t.s;
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int s = e * NT + tid;
      float p = 0.f;
      if (any && ent.i[e] >= 0 && ent.t[e] != -INFINITY) {
        const float d = ent.t[e] - mt;
        p = __builtin_amdgcn_exp2f(d * k) * inv_t;
        // tau (log p - log q); q = 0 at a logit of minus infinity, also where
        // every logit is
        const float r = zt[e] == -INFINITY ? INFINITY : d - (zt[e] - mz) + log_st;
        if (!(p == 0.f)) sum = fmaf(p, r, sum);
      }
      if (s < a.top) {
        p_k[s] = p;
        i_k[s] = ent.i[e];
        if constexpr (GRAD) z_k[s] = zt[e];
      }
    }
    sum = block_sum<NT>(sum, slots);
    if (tid == 0) a.loss[row] = a.tau * sum;
    const int64_t next = row + gridDim.x;
    if constexpr (!GRAD) {
      if (next < a.rows) ent.load(a, next);
      __syncthreads();  // (the slots are free)
    } else {
      const float scale = any ? a.tau * a.grad[row * a.grad_stride] : 0.f;
      const bool zero = scale == 0.f;
      const float f = q.s == 0.f ? 0.f : scale / q.s;
      char* dz = static_cast<char*>(a.dz) + row * n * Elem<T>::size;
      if (next < a.rows) ent.load(a, next);
      auto gradient = [&](const u32x4& raw) {
        float x[CE];
        unpack<T>(raw, x);
#pragma unroll
        for (int e = 0; e < CE; ++e) x[e] = f * __builtin_amdgcn_exp2f((x[e] - mz) * k);
        const u32x4 o = pack<T>(x);
        return zero ? u32x4{0u, 0u, 0u, 0u} : o;
      };
      if constexpr (C > 0) {
        // (without a next row: one chunk, which nobody uses)
        const char* znext = next < a.rows ? zrow(next) : z;
        const int whole_next = next < a.rows ? whole : 1;
        ahead = {-INFINITY, 0.f};
        static_for<C>([&](auto I) {
          constexpr int c = decltype(I)::value;
          // new to the compiler, which would else keep the first pass's
          // unpacked values for this one
          asm volatile("" : "+v"(v[c]));
          store_at(dz, chunk_offset<NT>(c, ot, whole), gradient(v[c]));
          v[c] = load_at(znext, chunk_offset<NT>(c, ot, whole_next));
          if constexpr (c >= LAG) add_chunk<T>(ahead, v[c - LAG], k, (c - LAG) * NT + ot < whole_next);
          __builtin_amdgcn_sched_barrier(0);
        });
      } else {
#pragma unroll 2
        for (int c = 0; c * NT < whole; ++c) {
          const uint32_t off = chunk_offset<NT>(c, tid, whole);
          const u32x4 x = load_at(z, off);
          if (c * NT + tid < whole) store_at(dz, off, gradient(x));
        }
      }
      if (tid < tail)
        store_from_f32(dz, whole * CE + tid, Elem<T>::dt, zero ? 0.f : f * __builtin_amdgcn_exp2f((last - mz) * k));
      __syncthreads();
      // the entries' elements once more; those of the same index all write the
      // same value
      for (int s = tid; s < a.top; s += NT) {
        const int i = i_k[s];
        if (i < 0) continue;
        float p = 0.f;
#pragma unroll 4
        for (int o = 0; o < a.top; ++o) p += i_k[o] == i ? p_k[o] : 0.f;
        const float qi = q.s == 0.f ? 0.f : __builtin_amdgcn_exp2f((z_k[s] - mz) * k) / q.s;
        store_from_f32(dz, i, Elem<T>::dt, zero ? 0.f : scale * (qi - p));
      }
    }
  }
}

}  // namespace distill
}  // namespace msign
