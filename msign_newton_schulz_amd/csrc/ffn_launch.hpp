// Launches of the feed-forward block's products for one element type; each
// type is a translation unit of its own, so that they compile in parallel.
#pragma once

#include "ffn_gemm.hpp"

#include <climits>
#include <cstring>

namespace msign {
namespace ffn {

// The arguments of ng problems as tiles of C; `blocks` of them.
template <typename C>
hipError_t fill(const Plan& plan, const Args<kMaxProblems>& in, int ng, Args<C::NG>& a, int64_t& blocks) {
  if (ng < 1 || ng > C::NG) return hipErrorInvalidValue;
  std::memset(&a, 0, sizeof(a));
  int64_t tiles = 0;
  for (int i = 0; i < C::NG; ++i) {
    a.bstart[i] = INT32_MAX;
    if (i >= ng) continue;
    a.g[i] = in.g[i];
    Problem& p = a.g[i];
    p.tiles_m = (p.M + C::BM - 1) / C::BM;
    p.tiles_n = (p.N + C::CN - 1) / C::CN;
    a.bstart[i] = (int32_t)(tiles * plan.split);
    tiles += (int64_t)p.tiles_m * p.tiles_n;
    if (tiles * plan.split > INT32_MAX / 2) return hipErrorInvalidValue;
  }
  if (plan.split > 1 && ng != 1) return hipErrorInvalidValue;
  a.split = plan.split;
  a.partial = in.partial;
  a.activation = in.activation;
  a.gate = in.gate; a.up = in.up; a.ld_act = in.ld_act;
  a.h = in.h; a.dg = in.dg; a.du = in.du; a.ldh = in.ldh;
  blocks = tiles * plan.split;
  return hipSuccess;
}

// Joins the parts of a launch's tiles, if there are any.
template <typename C>
hipError_t join_parts(const Args<C::NG>& a, int64_t blocks, hipStream_t st) {
  if (a.split == 1 || blocks == 0) return hipSuccess;
  reduce_kernel<C><<<dim3((unsigned)(blocks / a.split * C::FM)), C::NT, 0, st>>>(a);
  return hipGetLastError();
}

template <typename C>
hipError_t launch_tile(const Plan& plan, const Args<kMaxProblems>& in, int ng, hipStream_t st) {
  Args<C::NG> a;
  int64_t blocks = 0;
  hipError_t e = fill<C>(plan, in, ng, a, blocks);
  if (e != hipSuccess || blocks == 0) return e;
  tile_kernel<C><<<dim3((unsigned)blocks), C::NT, 0, st>>>(a);
  e = hipGetLastError();
  return e == hipSuccess ? join_parts<C>(a, blocks, st) : e;
}

// Both products in one launch, the one with the longer blocks first.
template <typename CX, typename CW>
hipError_t launch_pair(const Plan& plan_dx, const Plan& plan_dw, const Args<kMaxProblems>& dx,
                       const Args<kMaxProblems>& dw, hipStream_t st) {
  Pair<CX, CW> p;
  std::memset(&p, 0, sizeof(p));
  int64_t nx = 0, nw = 0;
  hipError_t e = fill<CX>(plan_dx, dx, 1, p.a, nx);
  if (e == hipSuccess) e = fill<CW>(plan_dw, dw, kMaxProblems, p.b, nw);
  if (e != hipSuccess || nx + nw == 0) return e;
  p.na = (int32_t)nx;
  p.nb = (int32_t)nw;
  p.b_first = plan_dw.block_us > plan_dx.block_us ? 1 : 0;
  pair_kernel<CX, CW><<<dim3((unsigned)(nx + nw)), CX::NT, 0, st>>>(p);
  e = hipGetLastError();
  return e == hipSuccess ? join_parts<CX>(p.a, nx, st) : e;
}

template <typename T, bool AKM, bool BKM, int EPI, int NG, int NSEG = 1>
hipError_t launch_variant(const Plan& plan, const Args<kMaxProblems>& a, int ng, hipStream_t st) {
  if constexpr (Elem<T>::size == 4) {
    return launch_tile<Tile<T, 64, 128, 2, 2, 8, AKM, BKM, EPI, NG, NSEG>>(plan, a, ng, st);
  } else {
    if (plan.rows == 256) return launch_tile<Tile<T, 256, 256, 2, 2, 8, AKM, BKM, EPI, NG, NSEG>>(plan, a, ng, st);
    if (plan.cpr == 16) return launch_tile<Tile<T, 128, 128, 2, 2, 16, AKM, BKM, EPI, NG, NSEG>>(plan, a, ng, st);
    return launch_tile<Tile<T, 128, 128, 2, 2, 8, AKM, BKM, EPI, NG, NSEG>>(plan, a, ng, st);
  }
}

template <typename T>
hipError_t launch_typed(Kind kind, const Plan& plan, const Args<kMaxProblems>& a, int ng, hipStream_t st) {
  switch (kind) {
    case K_GATED: return launch_variant<T, false, false, EPI_GATED, 1>(plan, a, ng, st);
    case K_DOWN: return launch_variant<T, false, false, EPI_PLAIN, 1>(plan, a, ng, st);
    default: return launch_variant<T, false, true, EPI_DGATED, 1>(plan, a, ng, st);
  }
}

// In one launch where both take the same number of workgroups a CU: at few
// rounds one's blocks fill the CUs that the other's last round leaves, at many
// rounds it makes no difference.  (bf16, us of the backward pass in one launch
// and in two, by rounds of their blocks: one, 400 tokens of 1000 x 1000 32 and 35;
// two, 1000 of 600 x 700 42 and 49, 1024 of 1024 x 4096 79 and 85, 4096 of them
// 222 and 230, 16384 of them 797 and 789; four, 4096 of 2048 x 7168 642 and 641;
// twelve, 4096 of 4096 x 14336 2261 and 2262; thirteen, 8192 of them 4457 and
// 4465.)
// Of tiles of two kinds a CU would hold one workgroup where it can hold two of
// the smaller kind: in one launch if all the blocks are two rounds or less, for
// the gaps saved, else one after the other.  (X 8 for dx in 128-tiles of 8 chunks
// and so on.  Two rounds or less: X 8 and W 16, 2767 tokens of 16 x 477 47 and 53;
// X 16 and W 8, 13 of 700 x 900 36 and 40; X 8 and W 256, 417 of 9335 x 338 82 and
// 90; X 256 and W 8, 2192 of 4531 x 376 115 and 126.  More: X 8 and W 16, 8625 of
// 8174 x 18 337 and 334; X 16 and W 8, 64 of 4096 x 14336 281 and 228; X 8 and W
// 256, 900 of 1500 x 3300 130 and 130; X 256 and W 8, 2942 of 380 x 11706 325 and
// 298.)
template <typename T>
hipError_t launch_dx_dw_typed(const Plan& px, const Plan& pw, const Args<kMaxProblems>& dx,
                              const Args<kMaxProblems>& dw, hipStream_t st) {
  if constexpr (Elem<T>::size == 4) {
    return launch_pair<Tile<T, 64, 128, 2, 2, 8, false, true, EPI_PLAIN, 1, 2>,
                       Tile<T, 64, 128, 2, 2, 8, true, true, EPI_PLAIN, kMaxProblems, 1>>(px, pw, dx, dw, st);
  } else {
    using X256 = Tile<T, 256, 256, 2, 2, 8, false, true, EPI_PLAIN, 1, 2>;
    using X16 = Tile<T, 128, 128, 2, 2, 16, false, true, EPI_PLAIN, 1, 2>;
    using X8 = Tile<T, 128, 128, 2, 2, 8, false, true, EPI_PLAIN, 1, 2>;
    using W256 = Tile<T, 256, 256, 2, 2, 8, true, true, EPI_PLAIN, kMaxProblems, 1>;
    using W16 = Tile<T, 128, 128, 2, 2, 16, true, true, EPI_PLAIN, kMaxProblems, 1>;
    using W8 = Tile<T, 128, 128, 2, 2, 8, true, true, EPI_PLAIN, kMaxProblems, 1>;
    const bool two_x = px.rows == 128 && px.cpr == 8, two_w = pw.rows == 128 && pw.cpr == 8;
    if (two_x && two_w) return launch_pair<X8, W8>(px, pw, dx, dw, st);
    if (!two_x && !two_w) {
      if (px.rows == 256) {
        return pw.rows == 256 ? launch_pair<X256, W256>(px, pw, dx, dw, st)
                              : launch_pair<X256, W16>(px, pw, dx, dw, st);
      }
      return pw.rows == 256 ? launch_pair<X16, W256>(px, pw, dx, dw, st) : launch_pair<X16, W16>(px, pw, dx, dw, st);
    }
    if (px.blocks + pw.blocks <= 512) {
      if (two_x)
        return pw.rows == 256 ? launch_pair<X8, W256>(px, pw, dx, dw, st) : launch_pair<X8, W16>(px, pw, dx, dw, st);
      return px.rows == 256 ? launch_pair<X256, W8>(px, pw, dx, dw, st) : launch_pair<X16, W8>(px, pw, dx, dw, st);
    }
    const hipError_t e = two_x             ? launch_tile<X8>(px, dx, 1, st)
                         : px.rows == 256 ? launch_tile<X256>(px, dx, 1, st)
                                          : launch_tile<X16>(px, dx, 1, st);
    if (e != hipSuccess) return e;
    return two_w             ? launch_tile<W8>(pw, dw, kMaxProblems, st)
           : pw.rows == 256 ? launch_tile<W256>(pw, dw, kMaxProblems, st)
                            : launch_tile<W16>(pw, dw, kMaxProblems, st);
  }
}

}  // namespace ffn
}  // namespace msign
