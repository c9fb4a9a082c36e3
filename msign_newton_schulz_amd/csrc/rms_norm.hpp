// Root-mean-square norm with the residual's addition, forward and backward.
//
// One read of every input and one write of every output: a workgroup walks
// over rows b, b + gridDim, ... and holds a row in registers, C chunks of 16
// bytes a thread.  Each thread has the same columns in all rows, so it keeps
// the weight, and in the backward pass sums the weight's gradient in
// registers; the workgroups' sums are added by a second kernel in a fixed
// order.  The next row is loaded before this one is reduced (HOLD; wide rows
// leave no registers for that and read the weight again each time).  Bound by
// memory.  Measured, bf16, 16384 x 4096, four sets of tensors in turn: forward, two
// reads and two writes of 134 MB, 98 us, 5.5 TB/s (a large copy 5.2); backward,
// three and one, 108 us, 5.0 TB/s; rows off 16 bytes, f16, 5001 x 4099, 46 us, 3.6
// TB/s, 5 of them the second kernel's.  One row of 4096: 2.9 us, a launch and two
// rounds of latency.  Without HOLD the backward pass waits for each row's loads, and
// reads dh and the weight between its stores: 24000 columns of 16 bits 86 us for
// 268 MB, 3.1 TB/s.
#pragma once

#include "row_ops.hpp"

namespace msign {
namespace norm {

using namespace rows;

// CE weights from column i on; columns past dim read the last one.
template <int CE>
__device__ __forceinline__ void load_weights(const void* w, int32_t dt, int i, int dim, float (&f)[CE]) {
  if (dt == DT_F32) {
#pragma unroll
    for (int q = 0; q < CE / 4; ++q) {
      if (i + 4 * q + 4 <= dim) {
        float t[4];
        unpack<float>(load_at(static_cast<const char*>(w), (uint32_t)(i + 4 * q) * 4u), t);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[4 * q + e] = t[e];
      }
    }
  } else if (CE == 8 && i + CE <= dim) {
    const u32x4 v = load_at(static_cast<const char*>(w), (uint32_t)i * 2u);
    float t[8];
    if (dt == DT_BF16) unpack<bf16_t>(v, t);
    else unpack<f16_t>(v, t);
#pragma unroll
    for (int e = 0; e < CE; ++e) f[e] = t[e];
  } else {
#pragma unroll
    for (int e = 0; e < CE; ++e) f[e] = load_as_f32(w, i + e < dim ? i + e : dim - 1, dt);
  }
}

// The same values, new to the compiler: it would else keep what it derived from
// them (unpacked rows from pass to pass, addresses and weights from row to
// row) in more registers than there are.
__device__ __forceinline__ void renew(int& v) { asm volatile("" : "+v"(v)); }
template <int C>
__device__ __forceinline__ void renew(u32x4 (&v)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) asm volatile("" : "+v"(v[c]));
}

struct ForwardArgs {
  const void *x, *r, *w;
  void *y, *h;
  float* rstd;
  int64_t ldx, ldr, rows;
  int32_t dim, w_dtype;
  float eps;
};

template <typename T, int NT, int C, bool HOLD>
__global__ void __launch_bounds__(NT, 4) forward_kernel(const ForwardArgs a) {
  constexpr int CE = 16 / Elem<T>::size, ESZ = Elem<T>::size;
  __shared__ float slots[2][NT / 64];
  const int tid = threadIdx.x, n = a.dim, whole = n / CE, tail = n % CE, last = whole * CE + tid;
  const bool has_r = a.r != nullptr, has_tail = tid < tail;
  const float inv = 1.f / (float)n;
  int ot = tid;  // see renew()
  auto at = [&](int c) { return chunk_offset<NT>(c, ot, whole); };
  auto xrow = [&](int64_t row) { return static_cast<const char*>(a.x) + row * a.ldx * ESZ; };
  auto rrow = [&](int64_t row) { return static_cast<const char*>(a.r) + row * a.ldr * ESZ; };
  float w[HOLD ? C : 1][CE], w_tail = has_tail ? load_as_f32(a.w, last, a.w_dtype) : 0.f;
  if constexpr (HOLD) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (whole > 0) load_weights<CE>(a.w, a.w_dtype, (int)(at(c) / ESZ), n, w[c]);
  }
  u32x4 xv[C], rv[C];
  float xt = 0.f, rt = 0.f;
  auto load = [&](int64_t row, u32x4 (&xo)[C], u32x4 (&ro)[C], float& xe, float& re) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      ro[c] = u32x4{0u, 0u, 0u, 0u};
      if (whole > 0) xo[c] = load_at(xrow(row), at(c));
      if (whole > 0 && has_r) ro[c] = load_at(rrow(row), at(c));
    }
    if (has_tail) {
      xe = load_as_f32(xrow(row), last, Elem<T>::dt);
      if (has_r) re = load_as_f32(rrow(row), last, Elem<T>::dt);
    }
  };
  int64_t row = blockIdx.x;
  load(row, xv, rv, xt, rt);
  for (int turn = 0; row < a.rows; row += gridDim.x, turn ^= 1) {
    if constexpr (!HOLD) renew(ot);
    u32x4 xn[HOLD ? C : 1], rn[HOLD ? C : 1];
    float xtn = 0.f, rtn = 0.f;
    const int64_t next = row + gridDim.x;
    if constexpr (HOLD) load(next < a.rows ? next : row, xn, rn, xtn, rtn);
    float sum = (xt + rt) * (xt + rt);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float f[CE], g[CE], s = 0.f;
      unpack<T>(xv[c], f);
      unpack<T>(rv[c], g);
#pragma unroll
      for (int e = 0; e < CE; ++e) s = fmaf(f[e] + g[e], f[e] + g[e], s);
      sum += c * NT + tid < whole ? s : 0.f;
    }
    // (two sets of slots: one barrier a row)
    sum = block_sum<NT>(sum, slots[turn]);
    const float s = 1.f / sqrtf(sum * inv + a.eps);
    if (tid == 0) a.rstd[row] = s;
    char* y = static_cast<char*>(a.y) + row * n * ESZ;
    char* h = static_cast<char*>(a.h) + row * n * ESZ;
    renew(xv);
    renew(rv);
    if (whole > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float f[CE], g[CE], o[CE], wc[CE];
        unpack<T>(xv[c], f);
        unpack<T>(rv[c], g);
        if constexpr (!HOLD) load_weights<CE>(a.w, a.w_dtype, (int)(at(c) / ESZ), n, wc);
#pragma unroll
        for (int e = 0; e < CE; ++e) {
          f[e] += g[e];
          o[e] = f[e] * s * (HOLD ? w[HOLD ? c : 0][e] : wc[e]);
        }
        store_at(y, at(c), pack<T>(o));
        if (has_r) store_at(h, at(c), pack<T>(f));
      }
    }
    if (has_tail) {
      store_from_f32(y, last, Elem<T>::dt, (xt + rt) * s * w_tail);
      if (has_r) store_from_f32(h, last, Elem<T>::dt, xt + rt);
    }
    if constexpr (HOLD) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        xv[c] = xn[c];
        rv[c] = rn[c];
      }
      xt = xtn;
      rt = rtn;
    } else if (next < a.rows) {
      load(next, xv, rv, xt, rt);
    }
  }
}

struct BackwardArgs {
  const void *dy, *h, *w, *dh;
  const float* rstd;
  void* dx;
  float* partial;  // [gridDim][dim] sums of dy n
  int64_t ld_dy, ldh, ld_dh, rows;
  int32_t dim, w_dtype;
};

// G: rows that a workgroup takes at once, NT threads each (only rows of one
// wave: G waves then leave one partial sum).
template <typename T, int NT, int C, bool HOLD, int G>
__global__ void __launch_bounds__(NT * G, C <= 2 ? 3 : 2) backward_kernel(const BackwardArgs a) {
  static_assert(G == 1 || NT == 64, "only single waves share a workgroup");
  constexpr int CE = 16 / Elem<T>::size, ESZ = Elem<T>::size;
  __shared__ float slots[2][NT / 64];
  const int tid = threadIdx.x % NT, group = threadIdx.x / NT, n = a.dim, whole = n / CE, tail = n % CE, last = whole * CE + tid;
  const bool has_dh = a.dh != nullptr, has_tail = tid < tail;
  const float inv = 1.f / (float)n;
  int ot = tid;  // see renew()
  auto at = [&](int c) { return chunk_offset<NT>(c, ot, whole); };
  auto dyrow = [&](int64_t row) { return static_cast<const char*>(a.dy) + row * a.ld_dy * ESZ; };
  auto hrow = [&](int64_t row) { return static_cast<const char*>(a.h) + row * a.ldh * ESZ; };
  auto dhrow = [&](int64_t row) { return static_cast<const char*>(a.dh) + row * a.ld_dh * ESZ; };
  float w[HOLD ? C : 1][CE], dw[C][CE], w_tail = has_tail ? load_as_f32(a.w, last, a.w_dtype) : 0.f, dw_tail = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if constexpr (HOLD) {
      if (whole > 0) load_weights<CE>(a.w, a.w_dtype, (int)(at(c) / ESZ), n, w[c]);
    }
#pragma unroll
    for (int e = 0; e < CE; ++e) dw[c][e] = 0.f;
  }
  struct Row {
    u32x4 dy[C], h[C];
    float dy_t, h_t, rstd;
  };
  auto load = [&](int64_t row, Row& o) {
    o.rstd = a.rstd[row];
    if (whole > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        o.dy[c] = load_at(dyrow(row), at(c));
        o.h[c] = load_at(hrow(row), at(c));
      }
    }
    o.dy_t = o.h_t = 0.f;
    if (has_tail) {
      o.dy_t = load_as_f32(dyrow(row), last, Elem<T>::dt);
      o.h_t = load_as_f32(hrow(row), last, Elem<T>::dt);
    }
  };
  Row cur;
  const int64_t stride = (int64_t)gridDim.x * G;
  int64_t row = (int64_t)blockIdx.x * G + group;
  load(row < a.rows ? row : a.rows - 1, cur);
  for (int turn = 0; row < a.rows; row += stride, turn ^= 1) {
    if constexpr (!HOLD) renew(ot);
    const int64_t next = row + stride;
    u32x4 gv[HOLD ? C : 1];
    float g_t = 0.f;
#pragma unroll
    for (int c = 0; c < (HOLD ? C : 1); ++c) gv[c] = u32x4{0u, 0u, 0u, 0u};
    if (has_dh) {
      if (HOLD && whole > 0) {
#pragma unroll
        for (int c = 0; c < (HOLD ? C : 1); ++c) gv[c] = load_at(dhrow(row), at(c));
      }
      if (has_tail) g_t = load_as_f32(dhrow(row), last, Elem<T>::dt);
    }
    Row nxt;
    if constexpr (HOLD) load(next < a.rows ? next : row, nxt);
    const float s = cur.rstd;
    float sum = cur.dy_t * (cur.h_t * s);
    dw_tail += sum;
    sum *= w_tail;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float y[CE], x[CE], wc[CE], part = 0.f;
      unpack<T>(cur.dy[c], y);
      unpack<T>(cur.h[c], x);
      if constexpr (!HOLD) load_weights<CE>(a.w, a.w_dtype, (int)(at(c) / ESZ), n, wc);
#pragma unroll
      for (int e = 0; e < CE; ++e) {
        const float yn = y[e] * (x[e] * s);
        dw[c][e] += yn;
        part = fmaf(yn, HOLD ? w[HOLD ? c : 0][e] : wc[e], part);
      }
      sum += c * NT + tid < whole ? part : 0.f;
    }
    const float mean = block_sum<NT>(sum, slots[turn]) * inv;
    char* dx = static_cast<char*>(a.dx) + row * n * ESZ;
    renew(cur.dy);
    renew(cur.h);
    if constexpr (!HOLD) renew(ot);
    if (whole > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float y[CE], x[CE], g[CE], o[CE], wc[CE];
        unpack<T>(cur.dy[c], y);
        unpack<T>(cur.h[c], x);
        if constexpr (!HOLD) {
          // dx may be dh itself, and its other chunks have been stored by now: only
          // a chunk's own thread reads it here
          if (c * NT + tid >= whole) continue;
          gv[0] = has_dh ? load_at(dhrow(row), at(c)) : u32x4{0u, 0u, 0u, 0u};
          load_weights<CE>(a.w, a.w_dtype, (int)(at(c) / ESZ), n, wc);
        }
        unpack<T>(gv[HOLD ? c : 0], g);
#pragma unroll
        for (int e = 0; e < CE; ++e)
          o[e] = fmaf(s, fmaf(-mean, x[e] * s, y[e] * (HOLD ? w[HOLD ? c : 0][e] : wc[e])), g[e]);
        store_at(dx, at(c), pack<T>(o));
      }
    }
    if (has_tail)
      store_from_f32(dx, last, Elem<T>::dt, fmaf(s, fmaf(-mean, cur.h_t * s, cur.dy_t * w_tail), g_t));
    if constexpr (HOLD) cur = nxt;
    else if (next < a.rows) load(next, cur);
  }
  float* out = a.partial + (int64_t)blockIdx.x * n;
  if constexpr (G > 1) {  // the waves' sums, in wave order
    __shared__ float sums[G - 1][64 * (C * CE + 1)];
    if (group > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < CE; ++e) sums[group - 1][(c * CE + e) * 64 + tid] = dw[c][e];
      sums[group - 1][C * CE * 64 + tid] = dw_tail;
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 0; g < G - 1; ++g) {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < CE; ++e) dw[c][e] += sums[g][(c * CE + e) * 64 + tid];
      dw_tail += sums[g][C * CE * 64 + tid];
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (c * NT + tid >= whole) continue;
#pragma unroll
    for (int q = 0; q < CE / 4; ++q) {
      const float t[4] = {dw[c][4 * q], dw[c][4 * q + 1], dw[c][4 * q + 2], dw[c][4 * q + 3]};
      store_at(reinterpret_cast<char*>(out), at(c) * (4 / ESZ) + q * 16u, pack<float>(t));
    }
  }
  if (has_tail) out[last] = dw_tail;
}

// dweight[i] = sum of partial[b][i] over b, 64 columns a workgroup: wave v
// adds b = v, v + 16, ... and the waves' sums are added in wave order.
__global__ void __launch_bounds__(1024) weight_sum_kernel(const float* partial, int32_t nb, void* dweight,
                                                          int32_t dim, int32_t w_dtype) {
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (i < dim) {
#pragma unroll 16
    for (int b = wave; b < nb; b += 16) s += partial[(int64_t)b * dim + i];
  }
  part[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && i < dim) {
    s = part[0][lane];
#pragma unroll
    for (int v = 1; v < 16; ++v) s += part[v][lane];
    store_from_f32(dweight, i, w_dtype, s);
  }
}

}  // namespace norm
}  // namespace msign
