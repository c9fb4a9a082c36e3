// The feed-forward block's forward products for a few tokens (gfx950).
//
// With at most 32 tokens the products are bound by the weights' bytes: each is
// read once, by one wave, straight into the registers that the matrix
// instruction takes (lane l holds 16 bytes of weight row l % 16 at K chunk
// l / 16), with no LDS on the way; the tokens' fragments come from the caches.
// The waves of a workgroup share 16 rows of a weight matrix (gated: of both) and
// split the sum over K; their sums meet in LDS in wave order.  Against tiles this
// saves the passes that join parts and, in fp32, the 128 rows that a tile
// multiplies.  Measured with both products (weights once): bf16, 1 token, 1024 x
// 4096 5.6 and 7.0 us, the second with 64 workgroups for 256 CUs; 4096 x 8192 38 us
// a call, 5.3 TB/s; fp32, 1
// token, 4096 x 14336 136 us, 5.2 TB/s, 16 tokens 180 us, where the tokens'
// fragments take as much cache bandwidth as the weights.  Two groups of rows a
// workgroup, to share them, took 165 us there and 44 us in the bf16 case, for
// want of workgroups: left out.
#pragma once

#include "ffn_gemm.hpp"

namespace msign {
namespace ffn {

constexpr int kSkinnyTokens = 32;

struct SkinnyArgs {
  const void* x;      // [tokens, K], pitch ldx: the tokens' side
  const void* w[2];   // [N, K]: weights (gated: gate and up)
  int64_t ldx, ldw[2];
  int32_t tokens, N, K;  // K a multiple of 16 bytes
  void* out;          // plain: y, gated: h
  int64_t ldo;
  int32_t out_cols;   // columns that exist in out (gated: those past N become zeros)
  void *gate, *up;    // gated: may be null
  int64_t ld_act;
  int32_t activation;
};

// MT groups of 16 tokens, W waves.
template <typename T, int MT, int W, bool GATED>
__global__ void __launch_bounds__(W * 64) skinny_kernel(const SkinnyArgs a) {
  constexpr int ESZ = Elem<T>::size, CE = 16 / ESZ, KS = 4 * CE;  // k values of a step
  constexpr int NB = GATED ? 2 : 1;
  constexpr int U = NB + MT <= 3 ? 4 : 2;  // steps of a batch; one to two batches are in flight
  __shared__ f32x4 part[W][NB * MT][64];
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16;
  const int steps = (a.K + KS - 1) / KS;
  const int s0 = (int)((int64_t)wave * steps / W), s1 = (int)((int64_t)(wave + 1) * steps / W);

  // rows past the last read the last one: their products are not stored
  const char *wp[NB], *xp[MT];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int row = n0 + r;
    wp[b] = static_cast<const char*>(a.w[b]) + (int64_t)(row < a.N ? row : a.N - 1) * a.ldw[b] * ESZ;
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = m * 16 + r;
    xp[m] = static_cast<const char*>(a.x) + (int64_t)(row < a.tokens ? row : a.tokens - 1) * a.ldx * ESZ;
  }
  f32x4 acc[NB][MT];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[b][m] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Batch i: steps s0 + i U ...  Steps past the wave's last read that one again,
  // chunks past the rows' end the last chunk: no load has a branch, and the
  // loads of one batch are counted while the other's are waited for.
  struct Batch { u32x4 w[U][NB], x[U][MT]; };
  auto fetch = [&](int i, Batch& v) {
    uint32_t at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int st = s0 + i * U + u, k = (st < s1 ? st : s1 - 1) * KS + g * CE;
      at[u] = (uint32_t)(k < a.K ? k : a.K - CE) * ESZ;
    }
    // (a row's consecutive steps one after the other: they share cache lines)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int u = 0; u < U; ++u) v.w[u][b] = *reinterpret_cast<const u32x4*>(wp[b] + at[u]);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int u = 0; u < U; ++u) v.x[u][m] = *reinterpret_cast<const u32x4*>(xp[m] + at[u]);
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  auto multiply = [&](int i, Batch& v, auto last) {
    if constexpr (decltype(last)::value) {  // (both sides are cleared: 0 times infinity is NaN)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int st = s0 + i * U + u;
        const bool in = st < s1 && st * KS + g * CE < a.K;
#pragma unroll
        for (int b = 0; b < NB; ++b) v.w[u][b] = in ? v.w[u][b] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int m = 0; m < MT; ++m) v.x[u][m] = in ? v.x[u][m] : u32x4{0u, 0u, 0u, 0u};
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int m = 0; m < MT; ++m) Mma<T>::run(acc[b][m], v.w[u][b], v.x[u][m]);
  };
  const int batches = (s1 - s0 + U - 1) / U;
  if (batches > 0) {
    Batch v0, v1;
    fetch(0, v0);
    int i = 0;
    for (; i + 2 < batches; i += 2) {
      fetch(i + 1, v1);
      multiply(i, v0, I0{});
      fetch(i + 2, v0);
      multiply(i + 1, v1, I0{});
    }
    if (i + 1 < batches) {
      fetch(i + 1, v1);
      multiply(i, v0, I0{});
      multiply(i + 1, v1, I1{});
    } else {
      multiply(i, v0, I1{});
    }
  }

#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int m = 0; m < MT; ++m) part[wave][b * MT + m][lane] = acc[b][m];
  __syncthreads();
  // wave v finishes tokens 16 v ..: lane l holds token l % 16 and four
  // consecutive columns
  if (wave < MT) {
    const int m = wave, token = m * 16 + r, n = n0 + 4 * g;
    auto total = [&](int f) {
      f32x4 t = part[0][f][lane];
#pragma unroll
      for (int q = 1; q < W; ++q) t += part[q][f][lane];
      return t;
    };
    auto put = [&](void* base, int64_t ld, int cols, const float (&o)[4]) {
      const int64_t at = (int64_t)token * ld + n;
      if (n + 3 < cols) {  // four elements at any alignment
        struct __attribute__((packed, aligned(ESZ))) Four { typename rows::Raw<T>::type v[4]; };
        Four f;
        store_vec4(&f, 0, Elem<T>::dt, o);
        *reinterpret_cast<Four*>(static_cast<char*>(base) + at * ESZ) = f;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < cols) store_from_f32(base, at + e, Elem<T>::dt, o[e]);
      }
    };
    const f32x4 t0 = total(m);
    float o[4] = {t0[0], t0[1], t0[2], t0[3]};
    if constexpr (GATED) {
      const f32x4 t1 = total(MT + m);
      const float up[4] = {t1[0], t1[1], t1[2], t1[3]};
      if (token < a.tokens && a.gate != nullptr) {
        put(a.gate, a.ld_act, a.N, o);
        put(a.up, a.ld_act, a.N, up);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float s = a.activation == 0 ? gate<0>(o[e]) : gate<1>(o[e]);
        o[e] = n + e < a.N ? o[e] * s * up[e] : 0.f;
      }
    }
    if (token < a.tokens) put(a.out, a.ldo, a.out_cols, o);
  }
}

// Launches a product of at most kSkinnyTokens tokens.
hipError_t launch_skinny(int32_t dtype, bool gated, const SkinnyArgs& a, hipStream_t st);
hipError_t launch_skinny_bf16(bool gated, const SkinnyArgs& a, hipStream_t st);
hipError_t launch_skinny_f16(bool gated, const SkinnyArgs& a, hipStream_t st);
hipError_t launch_skinny_f32(bool gated, const SkinnyArgs& a, hipStream_t st);

template <typename T, int MT, int W, bool GATED>
hipError_t skinny_cfg(const SkinnyArgs& a, hipStream_t st) {
  const int64_t blocks = (a.N + 15) / 16;
  if (blocks == 0 || a.tokens == 0) return hipSuccess;
  skinny_kernel<T, MT, W, GATED><<<dim3((unsigned)blocks), W * 64, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t skinny_typed(bool gated, const SkinnyArgs& a, hipStream_t st) {
  const bool two = a.tokens > 16;
  if (gated) return two ? skinny_cfg<T, 2, 8, true>(a, st) : skinny_cfg<T, 1, 8, true>(a, st);
  return two ? skinny_cfg<T, 2, 16, false>(a, st) : skinny_cfg<T, 1, 16, false>(a, st);
}

}  // namespace ffn
}  // namespace msign
