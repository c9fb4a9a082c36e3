// Host side of the training-block operators (include/msign_train.h): argument
// checks, workspace layout and launches.
#include "../../include/msign_train.h"
#include "distill.hpp"
#include "ffn_gemm.hpp"
#include "ffn_skinny.hpp"
#include "rms_norm.hpp"

#include <cmath>
#include <cstring>
#include <string>

using namespace msign;

namespace {

thread_local std::string g_err;

msign_status_t fail(msign_status_t st, const char* msg) {
  g_err = msg;
  return st;
}

msign_status_t hip_fail(hipError_t e, const char* what) {
  g_err = std::string(what) + ": " + hipGetErrorString(e);
  return MSIGN_ERR_HIP;
}

constexpr int64_t kMaxDim = int64_t(1) << 20, kMaxTokens = int64_t(1) << 24, kMaxPitch = int64_t(1) << 21;
constexpr int64_t kMaxNormDim = 32768;
// The products' offsets inside a tile have 32 bits, so kMaxPitch; the row
// operators' have 64: here the bytes of kMaxTokens rows still do not overflow.
constexpr int64_t kMaxRowPitch = int64_t(1) << 36;
constexpr size_t kInvalid = (size_t)-1;

bool dt_valid(int32_t dt) { return dt == MSIGN_F32 || dt == MSIGN_BF16 || dt == MSIGN_F16; }
int64_t dt_size(int32_t dt) { return dt == MSIGN_F32 ? 4 : 2; }
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// A [rows, cols] matrix in memory, for overlap checks.
struct Range {
  const char* p;
  int64_t bytes;
};

Range range(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size) {
  if (p == nullptr || rows <= 0 || cols <= 0) return {nullptr, 0};
  return {static_cast<const char*>(p), ((rows - 1) * ld + cols) * size};
}

bool overlap(const Range& a, const Range& b) {
  return a.p != nullptr && b.p != nullptr && a.p < b.p + b.bytes && b.p < a.p + a.bytes;
}

// Whether an output meets an input or another output.
template <int NO, int NI>
bool outputs_overlap(const Range (&out)[NO], const Range (&in)[NI]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
    for (int j = 0; j < NI; ++j)
      if (overlap(out[i], in[j])) return true;
  }
  return false;
}

struct Carver {
  size_t off = 0;
  size_t take(int64_t bytes) {
    const size_t o = off;
    off += (size_t)round_up(bytes, 256);
    return o;
  }
};

// ------------------------------------------------ feed-forward block ------

// An operand as the products read it: the caller's matrix, or a copy with
// rows padded to 16 bytes.
struct Operand {
  const void* src;
  int64_t ld, rows, cols;
  bool copy;
  size_t off;
  int64_t ldc;  // pitch of the copy
};

Operand operand(const void* p, int64_t ld, int64_t rows, int64_t cols, int64_t size, Carver& c) {
  Operand o = {p, ld, rows, cols, false, 0, 0};
  const int64_t ce = 16 / size;
  o.copy = !aligned(p, 16) || ld % ce != 0 || cols % ce != 0;
  if (o.copy) {
    o.ldc = round_up(cols, 64);
    o.off = c.take(rows * o.ldc * size);
  }
  return o;
}

// The tile, the slice's length and the parts of the sum over K of `count` m x n
// products with `segments` sums over k: the fewest microseconds by a model of
// rounds of resident workgroups.  Its constants are fitted to products of 64 to
// 8192 tokens.  In 16 bits a 256-tile takes 1.25 us a slice of 128 bytes, a
// 128-tile 0.66 us as a CU's only workgroup and 1.25 us as one of two, and 1.1 us
// for a slice of 256 bytes, which leaves room for one workgroup; a tile's start
// and end take 12, 4 and 5 us, the pass that joins parts 9 and 4.5 us and its
// bytes.  Both sides, bf16, 4096 x 14336: 64 tokens' forward 75 us with slices of
// 256 bytes and 86 without, 256 tokens' 120 and 134; 1024 tokens' 280 us in
// 256-tiles, the down product alone 122 in 128-tiles and 102 in 256-tiles; 1024
// x 4096 with 1024 tokens, gated product, 22 us in two workgroups a CU, 29 in
// slices of 256 bytes.  fp32 products, bound by the matrix instruction, have
// tiles of 64 x 128 in slices of 128 bytes, 1 us each: twice the workgroups of
// 128 x 128, so fewer parts (1024 x 4096, 250 tokens 59 and 70 us, 64 tokens 36
// and 51; the same from 1024 tokens on).
ffn::Plan plan_product(int64_t m, int64_t n, int64_t count, int64_t k, int64_t segments, int32_t dtype,
                       bool may_split) {
  struct Variant {
    int rows, cols, cpr;
    double slice_us, slice_us_shared, start_us, join_us;
    int64_t slots;
  };
  static const Variant kVariants[] = {{256, 256, 8, 1.25, 1.25, 12.0, 9.0, 256},
                                      {128, 128, 8, 0.66, 1.25, 4.0, 4.5, 512},
                                      {128, 128, 16, 1.1, 1.1, 5.0, 4.5, 256}};
  static const Variant kVariantF32 = {64, 128, 8, 1.0, 1.0, 4.0, 4.5, 256};
  ffn::Plan best = {0, 8, 1, 0, 0, 0.0};
  double best_us = 1e30;
  auto consider = [&](const Variant& v, int64_t kte) {
    const int64_t t = count * ((m + v.rows - 1) / v.rows) * ((n + v.cols - 1) / v.cols);
    const int64_t slices = (k + kte - 1) / kte * segments;
    for (int split = 1; split <= 16 && (split == 1 || (may_split && slices * v.cpr >= 32 * split)); ++split) {
      const int64_t blocks = t * split;
      const int64_t part = ((slices + 1) / 2 + split - 1) / split * 2;
      const int64_t rounds = (blocks + v.slots - 1) / v.slots;
      const size_t bytes = split > 1 ? (size_t)blocks * v.rows * v.cols * 4 : 0;
      const double block_us = part * (blocks <= 256 ? v.slice_us : v.slice_us_shared) + v.start_us;
      const double us = rounds * block_us + (split > 1 ? v.join_us + bytes / 1.0e7 : 0.0);
      if (us < best_us) {
        best_us = us;
        best = {v.rows, v.cpr, split, bytes, blocks, block_us};
      }
    }
  };
  if (dtype == MSIGN_F32)
    consider(kVariantF32, kVariantF32.cpr * 4);
  else
    for (const Variant& v : kVariants) consider(v, v.cpr * 8);
  return best;
}

struct ForwardPlan {
  Operand x, wg, wu, wd;
  size_t h, total;
  int64_t ldh;
  bool few;  // the kernels for a few tokens; else:
  size_t partial;
  ffn::Plan gated, down;
};

// Whether the forward pass takes the kernels for a few tokens: up to 16 tokens,
// and up to 32 of small weights.  Beyond, the tokens' fragments, read from the
// caches beside every weight, cost more than the passes that join tiles' parts;
// in 16 bits they do so at large weights whatever the tokens.  (Us here and in
// tiles.  bf16, 1024 x 4096: 1 token 17 and 24, 32 tokens 20 and 25; 2048 x 7168:
// 1 token 24 and 29, 16 tokens 32 and 30, 32 tokens 41 and 31; 4096 x 8192: 16
// tokens 45 and 45; 4096 x 14336: 16 tokens 85 and 71.  fp32, 512 x 2048: 32
// tokens 20 and 26; 1024 x 4096: 1 token 21 and 33, 32 tokens 36 and 35; 4096 x
// 14336: 16 tokens 180 and 189.)
bool skinny(const ffn_block_t& b) {
  const bool f32 = b.dtype == MSIGN_F32;
  const int64_t weights = b.dim * b.hidden;
  if (b.tokens <= 16) return f32 || weights <= (int64_t(1) << 25);
  return b.tokens <= ffn::kSkinnyTokens && weights <= (int64_t(1) << (f32 ? 20 : 23));
}

ForwardPlan plan_forward(const ffn_block_t& b) {
  const int64_t size = dt_size(b.dtype);
  ForwardPlan p = {};
  Carver c;
  p.x = operand(b.x, b.ldx, b.tokens, b.dim, size, c);
  p.wg = operand(b.w_gate, b.ld_gate, b.hidden, b.dim, size, c);
  p.wu = operand(b.w_up, b.ld_up, b.hidden, b.dim, size, c);
  p.wd = operand(b.w_down, b.ld_down, b.dim, b.hidden, size, c);
  p.ldh = round_up(b.hidden, 64);
  p.h = c.take(b.tokens * p.ldh * size);
  p.few = skinny(b);
  if (!p.few) {
    p.gated = plan_product(b.tokens, 2 * b.hidden, 1, b.dim, 1, b.dtype, true);
    p.down = plan_product(b.tokens, b.dim, 1, b.hidden, 1, b.dtype, true);
    p.partial = c.take((int64_t)(p.gated.partial_bytes > p.down.partial_bytes ? p.gated.partial_bytes
                                                                              : p.down.partial_bytes));
  }
  p.total = c.off;
  return p;
}

struct BackwardPlan {
  Operand x, wg, wu, wd, dy;
  size_t h, dg, du, partial, total;
  int64_t ldh;
  ffn::Plan dgated, dx, dw;
};

BackwardPlan plan_backward(const ffn_block_t& b, const void* dy, int64_t ld_dy) {
  const int64_t size = dt_size(b.dtype);
  BackwardPlan p;
  Carver c;
  p.x = operand(b.x, b.ldx, b.tokens, b.dim, size, c);
  p.wg = operand(b.w_gate, b.ld_gate, b.hidden, b.dim, size, c);
  p.wu = operand(b.w_up, b.ld_up, b.hidden, b.dim, size, c);
  p.wd = operand(b.w_down, b.ld_down, b.dim, b.hidden, size, c);
  p.dy = operand(dy, ld_dy, b.tokens, b.dim, size, c);
  p.ldh = round_up(b.hidden, 64);
  p.h = c.take(b.tokens * p.ldh * size);
  p.dg = c.take(b.tokens * p.ldh * size);
  p.du = c.take(b.tokens * p.ldh * size);
  p.dgated = plan_product(b.tokens, b.hidden, 1, b.dim, 1, b.dtype, true);
  p.dx = plan_product(b.tokens, b.dim, 1, b.hidden, 2, b.dtype, true);
  p.dw = plan_product(b.hidden, b.dim, 3, b.tokens, 1, b.dtype, false);
  p.partial = c.take((int64_t)(p.dgated.partial_bytes > p.dx.partial_bytes ? p.dgated.partial_bytes
                                                                           : p.dx.partial_bytes));
  p.total = c.off;
  return p;
}

bool block_valid(const ffn_block_t* b) {
  return b != nullptr && dt_valid(b->dtype) && b->tokens >= 0 && b->dim >= 0 && b->hidden >= 0 &&
         b->tokens <= kMaxTokens && b->dim <= kMaxDim && b->hidden <= kMaxDim;
}

msign_status_t check_block(const ffn_block_t* b) {
  if (b == nullptr) return fail(MSIGN_ERR_ARG, "block must be non-null");
  if (!dt_valid(b->dtype)) return fail(MSIGN_ERR_DTYPE, "dtype must be MSIGN_F32, MSIGN_BF16 or MSIGN_F16");
  if (!block_valid(b)) return fail(MSIGN_ERR_SHAPE, "tokens must be in 0..2^24, dim and hidden in 0..2^20");
  if (b->activation != FFN_SILU && b->activation != FFN_GELU)
    return fail(MSIGN_ERR_ARG, "activation must be FFN_SILU or FFN_GELU");
  return MSIGN_OK;
}

// A matrix argument: given, aligned to its elements, with a possible pitch.
bool matrix_ok(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size, int64_t most = kMaxPitch) {
  if (rows == 0 || cols == 0) return true;
  return p != nullptr && aligned(p, (size_t)size) && ld >= cols && ld <= most;
}

// The same for the operators that take one row at a time.
bool rows_ok(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t size) {
  return matrix_ok(p, rows, cols, ld, size, kMaxRowPitch);
}

// A vector argument with n elements.
bool vector_ok(const void* p, int64_t n, int64_t size) { return n == 0 || (p != nullptr && aligned(p, (size_t)size)); }

msign_status_t check_block_operands(const ffn_block_t& b) {
  const int64_t s = dt_size(b.dtype);
  if (!matrix_ok(b.x, b.tokens, b.dim, b.ldx, s) || !matrix_ok(b.w_gate, b.hidden, b.dim, b.ld_gate, s) ||
      !matrix_ok(b.w_up, b.hidden, b.dim, b.ld_up, s) || !matrix_ok(b.w_down, b.dim, b.hidden, b.ld_down, s))
    return fail(MSIGN_ERR_ARG, "x and the weights must be non-null, aligned to their elements, with pitches of at "
                               "least a row and at most 2^21 elements");
  return MSIGN_OK;
}

msign_status_t check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return MSIGN_OK;
  if (ws == nullptr || bytes < need || !aligned(ws, 256))
    return fail(MSIGN_ERR_WORKSPACE, "workspace is null, smaller than required or not 256-byte aligned");
  return MSIGN_OK;
}

// The operand's address and pitch for the products, after its copy if it
// needs one.
struct View {
  const void* p;
  int64_t ld;
};

template <typename T>
hipError_t pad_copy(const Operand& o, char* dst, hipStream_t st) {
  const int64_t chunks = o.rows * (o.ldc * (int64_t)sizeof(T) / 16);
  const int64_t blocks = (chunks + 255) / 256;
  ffn::pad_copy_kernel<T><<<dim3((unsigned)(blocks < 8192 ? blocks : 8192)), 256, 0, st>>>(
      static_cast<const T*>(o.src), o.ld, reinterpret_cast<T*>(dst), o.ldc, o.rows, (int32_t)o.cols);
  return hipGetLastError();
}

hipError_t resolve(const Operand& o, int64_t size, char* ws, hipStream_t st, View* v) {
  if (!o.copy || o.rows == 0 || o.cols == 0) {
    *v = {o.src, o.ld};
    return hipSuccess;
  }
  *v = {ws + o.off, o.ldc};
  return size == 4 ? pad_copy<uint32_t>(o, ws + o.off, st) : pad_copy<uint16_t>(o, ws + o.off, st);
}

ffn::Problem problem(int64_t m, int64_t n, int64_t k, int64_t size) {
  ffn::Problem p;
  std::memset(&p, 0, sizeof(p));
  p.M = (int32_t)m;
  p.N = (int32_t)n;
  p.K = (int32_t)round_up(k, 16 / size);
  p.kvalid = (int32_t)k;
  return p;
}

void set_c(ffn::Problem& p, void* c, int64_t ldc) {
  p.C = c;
  p.ldc = ldc;
}

}  // namespace

namespace msign {
namespace ffn {

hipError_t launch(int32_t dtype, Kind kind, const Plan& plan, Args<kMaxProblems> args, int ng, hipStream_t st) {
  switch (dtype) {
    case MSIGN_BF16: return launch_bf16(kind, plan, args, ng, st);
    case MSIGN_F16: return launch_f16(kind, plan, args, ng, st);
    default: return launch_f32(kind, plan, args, ng, st);
  }
}

hipError_t launch_dx_dw(int32_t dtype, const Plan& plan_dx, const Plan& plan_dw, const Args<kMaxProblems>& dx,
                        const Args<kMaxProblems>& dw, hipStream_t st) {
  switch (dtype) {
    case MSIGN_BF16: return launch_dx_dw_bf16(plan_dx, plan_dw, dx, dw, st);
    case MSIGN_F16: return launch_dx_dw_f16(plan_dx, plan_dw, dx, dw, st);
    default: return launch_dx_dw_f32(plan_dx, plan_dw, dx, dw, st);
  }
}

hipError_t launch_skinny(int32_t dtype, bool gated, const SkinnyArgs& a, hipStream_t st) {
  switch (dtype) {
    case MSIGN_BF16: return launch_skinny_bf16(gated, a, st);
    case MSIGN_F16: return launch_skinny_f16(gated, a, st);
    default: return launch_skinny_f32(gated, a, st);
  }
}

}  // namespace ffn
}  // namespace msign

extern "C" {

const char* msign_train_last_error(void) { return g_err.c_str(); }

size_t ffn_forward_workspace_bytes(const ffn_block_t* b) {
  if (!block_valid(b)) return kInvalid;
  return plan_forward(*b).total;
}

size_t ffn_backward_workspace_bytes(const ffn_block_t* b, const void* dy, int64_t ld_dy) {
  if (!block_valid(b)) return kInvalid;
  return plan_backward(*b, dy, ld_dy).total;
}

msign_status_t ffn_forward(const ffn_block_t* bp, void* y, int64_t ldy, void* gate, void* up, int64_t ld_act,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
  msign_status_t st = check_block(bp);
  if (st != MSIGN_OK) return st;
  const ffn_block_t& b = *bp;
  const int64_t s = dt_size(b.dtype);
  if ((st = check_block_operands(b)) != MSIGN_OK) return st;
  if ((gate == nullptr) != (up == nullptr)) return fail(MSIGN_ERR_ARG, "gate and up must both be given or both null");
  if (!matrix_ok(y, b.tokens, b.dim, ldy, s) ||
      (gate != nullptr && (!matrix_ok(gate, b.tokens, b.hidden, ld_act, s) ||
                           !matrix_ok(up, b.tokens, b.hidden, ld_act, s))))
    return fail(MSIGN_ERR_ARG, "y, gate and up must be non-null, aligned to their elements, with pitches of at least "
                               "a row and at most 2^21 elements");
  const ForwardPlan p = plan_forward(b);
  if ((st = check_workspace(workspace, workspace_bytes, p.total)) != MSIGN_OK) return st;
  const Range out[] = {range(y, b.tokens, b.dim, ldy, s), range(gate, b.tokens, b.hidden, ld_act, s),
                       range(up, b.tokens, b.hidden, ld_act, s), {static_cast<char*>(workspace), (int64_t)p.total}};
  const Range in[] = {range(b.x, b.tokens, b.dim, b.ldx, s), range(b.w_gate, b.hidden, b.dim, b.ld_gate, s),
                      range(b.w_up, b.hidden, b.dim, b.ld_up, s), range(b.w_down, b.dim, b.hidden, b.ld_down, s)};
  if (outputs_overlap(out, in)) return fail(MSIGN_ERR_ALIAS, "an output overlaps an input, another output or the workspace");
  if (b.tokens == 0) return MSIGN_OK;

  char* ws = static_cast<char*>(workspace);
  View x, wg, wu, wd;
  hipError_t e;
  if ((e = resolve(p.x, s, ws, stream, &x)) != hipSuccess || (e = resolve(p.wg, s, ws, stream, &wg)) != hipSuccess ||
      (e = resolve(p.wu, s, ws, stream, &wu)) != hipSuccess || (e = resolve(p.wd, s, ws, stream, &wd)) != hipSuccess)
    return hip_fail(e, "pad_copy_kernel");

  if (p.few) {
    const int64_t ce = 16 / s;
    ffn::SkinnyArgs k;
    std::memset(&k, 0, sizeof(k));
    k.tokens = (int32_t)b.tokens;
    k.activation = b.activation;
    k.x = x.p; k.ldx = x.ld;
    k.w[0] = wg.p; k.ldw[0] = wg.ld;
    k.w[1] = wu.p; k.ldw[1] = wu.ld;
    k.N = (int32_t)b.hidden;
    k.K = (int32_t)round_up(b.dim, ce);
    k.out = ws + p.h; k.ldo = p.ldh; k.out_cols = (int32_t)round_up(b.hidden, ce);
    k.gate = gate; k.up = up; k.ld_act = ld_act;
    if ((e = ffn::launch_skinny(b.dtype, true, k, stream)) != hipSuccess) return hip_fail(e, "gated product");
    k.x = ws + p.h; k.ldx = p.ldh;
    k.w[0] = wd.p; k.ldw[0] = wd.ld;
    k.N = (int32_t)b.dim;
    k.K = (int32_t)round_up(b.hidden, ce);
    k.out = y; k.ldo = ldy; k.out_cols = (int32_t)b.dim;
    if ((e = ffn::launch_skinny(b.dtype, false, k, stream)) != hipSuccess) return hip_fail(e, "down product");
    return MSIGN_OK;
  }

  ffn::Args<ffn::kMaxProblems> a;
  std::memset(&a, 0, sizeof(a));
  a.activation = b.activation;
  a.partial = reinterpret_cast<float*>(ws + p.partial);
  a.h = ws + p.h;
  a.ldh = p.ldh;
  a.gate = gate;
  a.up = up;
  a.ld_act = ld_act;
  a.g[0] = problem(b.tokens, b.hidden, b.dim, s);
  a.g[0].A[0] = x.p; a.g[0].lda[0] = x.ld;
  a.g[0].B[0] = wg.p; a.g[0].ldb[0] = wg.ld;
  a.g[0].B[1] = wu.p; a.g[0].ldb[1] = wu.ld;
  if ((e = ffn::launch(b.dtype, ffn::K_GATED, p.gated, a, 1, stream)) != hipSuccess) return hip_fail(e, "gated product");

  a.g[0] = problem(b.tokens, b.dim, b.hidden, s);
  a.g[0].A[0] = a.h; a.g[0].lda[0] = p.ldh;
  a.g[0].B[0] = wd.p; a.g[0].ldb[0] = wd.ld;
  set_c(a.g[0], y, ldy);
  if ((e = ffn::launch(b.dtype, ffn::K_DOWN, p.down, a, 1, stream)) != hipSuccess) return hip_fail(e, "down product");
  return MSIGN_OK;
}

msign_status_t ffn_backward(const ffn_block_t* bp, const void* dy, int64_t ld_dy, const void* gate, const void* up,
                            int64_t ld_act, void* dx, void* dw_gate, void* dw_up, void* dw_down, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
  msign_status_t st = check_block(bp);
  if (st != MSIGN_OK) return st;
  const ffn_block_t& b = *bp;
  const int64_t s = dt_size(b.dtype);
  if ((st = check_block_operands(b)) != MSIGN_OK) return st;
  if (!matrix_ok(dy, b.tokens, b.dim, ld_dy, s) || !matrix_ok(gate, b.tokens, b.hidden, ld_act, s) ||
      !matrix_ok(up, b.tokens, b.hidden, ld_act, s) || !matrix_ok(dx, b.tokens, b.dim, b.dim, s) ||
      !matrix_ok(dw_gate, b.hidden, b.dim, b.dim, s) || !matrix_ok(dw_up, b.hidden, b.dim, b.dim, s) ||
      !matrix_ok(dw_down, b.dim, b.hidden, b.hidden, s))
    return fail(MSIGN_ERR_ARG, "dy, gate, up and the gradients must be non-null, aligned to their elements, with "
                               "pitches of at least a row and at most 2^21 elements");
  const BackwardPlan p = plan_backward(b, dy, ld_dy);
  if ((st = check_workspace(workspace, workspace_bytes, p.total)) != MSIGN_OK) return st;
  const Range out[] = {range(dx, b.tokens, b.dim, b.dim, s), range(dw_gate, b.hidden, b.dim, b.dim, s),
                       range(dw_up, b.hidden, b.dim, b.dim, s), range(dw_down, b.dim, b.hidden, b.hidden, s),
                       {static_cast<char*>(workspace), (int64_t)p.total}};
  const Range in[] = {range(b.x, b.tokens, b.dim, b.ldx, s), range(b.w_gate, b.hidden, b.dim, b.ld_gate, s),
                      range(b.w_up, b.hidden, b.dim, b.ld_up, s), range(b.w_down, b.dim, b.hidden, b.ld_down, s),
                      range(dy, b.tokens, b.dim, ld_dy, s), range(gate, b.tokens, b.hidden, ld_act, s),
                      range(up, b.tokens, b.hidden, ld_act, s)};
  if (outputs_overlap(out, in)) return fail(MSIGN_ERR_ALIAS, "an output overlaps an input, another output or the workspace");

  char* ws = static_cast<char*>(workspace);
  View x, wg, wu, wd, vdy;
  hipError_t e;
  if ((e = resolve(p.x, s, ws, stream, &x)) != hipSuccess || (e = resolve(p.wg, s, ws, stream, &wg)) != hipSuccess ||
      (e = resolve(p.wu, s, ws, stream, &wu)) != hipSuccess || (e = resolve(p.wd, s, ws, stream, &wd)) != hipSuccess ||
      (e = resolve(p.dy, s, ws, stream, &vdy)) != hipSuccess)
    return hip_fail(e, "pad_copy_kernel");

  ffn::Args<ffn::kMaxProblems> a;
  std::memset(&a, 0, sizeof(a));
  a.activation = b.activation;
  a.partial = reinterpret_cast<float*>(ws + p.partial);
  a.h = ws + p.h;
  a.dg = ws + p.dg;
  a.du = ws + p.du;
  a.ldh = p.ldh;
  a.gate = const_cast<void*>(gate);
  a.up = const_cast<void*>(up);
  a.ld_act = ld_act;
  // dh = dy Wd, turned into dg, du and h
  a.g[0] = problem(b.tokens, b.hidden, b.dim, s);
  a.g[0].A[0] = vdy.p; a.g[0].lda[0] = vdy.ld;
  a.g[0].B[0] = wd.p; a.g[0].ldb[0] = wd.ld;
  if ((e = ffn::launch(b.dtype, ffn::K_DGATED, p.dgated, a, 1, stream)) != hipSuccess)
    return hip_fail(e, "gated gradient product");
  // dx = dg Wg + du Wu
  a.g[0] = problem(b.tokens, b.dim, b.hidden, s);
  a.g[0].A[0] = a.dg; a.g[0].lda[0] = p.ldh;
  a.g[0].A[1] = a.du; a.g[0].lda[1] = p.ldh;
  a.g[0].B[0] = wg.p; a.g[0].ldb[0] = wg.ld;
  a.g[0].B[1] = wu.p; a.g[0].ldb[1] = wu.ld;
  set_c(a.g[0], dx, b.dim);
  const ffn::Args<ffn::kMaxProblems> dx_args = a;
  // dWg = dg^T x, dWu = du^T x, dWd = dy^T h
  for (int i = 0; i < 2; ++i) {
    a.g[i] = problem(b.hidden, b.dim, b.tokens, s);
    a.g[i].A[0] = i == 0 ? a.dg : a.du; a.g[i].lda[0] = p.ldh;
    a.g[i].B[0] = x.p; a.g[i].ldb[0] = x.ld;
    set_c(a.g[i], i == 0 ? dw_gate : dw_up, b.dim);
  }
  a.g[2] = problem(b.dim, b.hidden, b.tokens, s);
  a.g[2].A[0] = vdy.p; a.g[2].lda[0] = vdy.ld;
  a.g[2].B[0] = a.h; a.g[2].ldb[0] = p.ldh;
  set_c(a.g[2], dw_down, b.hidden);
  if ((e = ffn::launch_dx_dw(b.dtype, p.dx, p.dw, dx_args, a, stream)) != hipSuccess)
    return hip_fail(e, "gradient products");
  return MSIGN_OK;
}

}  // extern "C"

// --------------------------------------------------------------- norm -----

namespace {

// The forward pass: the workgroups of NT threads that the 256 CUs hold at four
// waves per SIMD; three where 256 threads hold two chunks each, which then
// have enough loads in flight (three and four a CU: bf16, 16384 x 4096 97 and 102
// us; with one chunk, 16384 x 2048, 43 and 41 us).
template <typename T, int NT, int C, bool HOLD>
hipError_t norm_forward_cfg(const norm::ForwardArgs& a, hipStream_t st) {
  constexpr int64_t resident = 256 * (NT == 256 && C == 2 ? 3 : 16 * 64 / NT);
  const int64_t blocks = a.rows < resident ? a.rows : resident;
  norm::forward_kernel<T, NT, C, HOLD><<<dim3((unsigned)blocks), NT, 0, st>>>(a);
  return hipGetLastError();
}

// The backward pass: the workgroups that the 256 CUs hold, three of 256 threads
// (three waves per SIMD are the most that the registers allow; two with more than
// two chunks a thread), one of 512.  With 1024 workgroups a part of the
// rows waits for a second turn, and there are more partial sums of the weight's
// gradient to write and add (bf16, dh and dy one tensor: 16384 x 4096 84 and 96 us;
// 8192 x 8192 in 512 threads 92 and 99 us).
constexpr int64_t kNormBackwardBlocks = 256 * 3;

template <typename T, int NT, int C, bool HOLD>
hipError_t norm_backward_cfg(const norm::BackwardArgs& a, int64_t& blocks, hipStream_t st) {
  constexpr int G = NT == 64 ? 4 : 1;
  constexpr int64_t per_cu = NT * G > 256 ? 1 : C > 2 ? 2 : 3, resident = 256 * per_cu;
  static_assert(resident <= kNormBackwardBlocks, "partial sums");
  const int64_t most = (a.rows + G - 1) / G;
  blocks = most < resident ? most : resident;
  norm::backward_kernel<T, NT, C, HOLD, G><<<dim3((unsigned)blocks), NT * G, 0, st>>>(a);
  return hipGetLastError();
}

// The smallest configuration whose threads hold the whole 16-byte chunks of a
// row of `dim` T: f(NT, C, HOLD).  The backward pass takes more chunks a thread,
// in two workgroups a CU instead of one, or the next row held instead of the
// weight read again (bf16, 268 MB in all, us here and in the forward pass's
// configuration: dim 4104 57 and 77, 5120 54 and 66, 8192 55 and 57, 8200 66 and
// 82, 16384 61 and 62, 24000 90 and 112, both while threads past a row's end took
// part in its last pass, 86 since).  In the forward pass 256 threads with three or
// four chunks are slower (5120: 59 and 45; 8192: 83 and 44).
template <typename T, bool BACKWARD, typename F>
hipError_t norm_config(int64_t dim, F&& f) {
  using std::integral_constant;
  using Yes = std::true_type;
  using No = std::false_type;
  const int64_t chunks = dim / (16 / Elem<T>::size);
  if (chunks <= 64) return f(integral_constant<int, 64>{}, integral_constant<int, 1>{}, Yes{});
  if (chunks <= 128) return f(integral_constant<int, 64>{}, integral_constant<int, 2>{}, Yes{});
  if (chunks <= 256) return f(integral_constant<int, 256>{}, integral_constant<int, 1>{}, Yes{});
  if (chunks <= 512) return f(integral_constant<int, 256>{}, integral_constant<int, 2>{}, Yes{});
  if constexpr (BACKWARD) {
    if (chunks <= 768) return f(integral_constant<int, 256>{}, integral_constant<int, 3>{}, Yes{});
    if (chunks <= 1024) return f(integral_constant<int, 256>{}, integral_constant<int, 4>{}, Yes{});
    if (chunks <= 2048) return f(integral_constant<int, 512>{}, integral_constant<int, 4>{}, Yes{});
    if (chunks <= 4096) return f(integral_constant<int, 512>{}, integral_constant<int, 8>{}, No{});
    if constexpr (Elem<T>::size == 4) return f(integral_constant<int, 512>{}, integral_constant<int, 16>{}, No{});
  } else {
    if (chunks <= 1024) return f(integral_constant<int, 512>{}, integral_constant<int, 2>{}, Yes{});
    if (chunks <= 2048) return f(integral_constant<int, 1024>{}, integral_constant<int, 2>{}, No{});
    if (chunks <= 4096) return f(integral_constant<int, 1024>{}, integral_constant<int, 4>{}, No{});
    if constexpr (Elem<T>::size == 4) return f(integral_constant<int, 1024>{}, integral_constant<int, 8>{}, No{});
  }
  return hipErrorInvalidValue;  // (dim is at most 32768)
}

// Rows of partial sums of the weight's gradient: at most one per workgroup.
int64_t norm_backward_blocks(int64_t tokens) { return tokens < kNormBackwardBlocks ? tokens : kNormBackwardBlocks; }

msign_status_t check_norm(int64_t tokens, int64_t dim, int32_t dtype, int32_t w_dtype) {
  if (!dt_valid(dtype) || !dt_valid(w_dtype))
    return fail(MSIGN_ERR_DTYPE, "dtype and w_dtype must be MSIGN_F32, MSIGN_BF16 or MSIGN_F16");
  if (tokens < 0 || tokens > kMaxTokens || dim < 0 || dim > kMaxNormDim)
    return fail(MSIGN_ERR_SHAPE, "tokens must be in 0..2^24 and dim in 0..32768");
  return MSIGN_OK;
}

}  // namespace

extern "C" {

msign_status_t add_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                            void* y, void* h_out, float* rstd, int64_t tokens, int64_t dim, int32_t dtype,
                            int32_t w_dtype, float eps, hipStream_t stream) {
  msign_status_t st = check_norm(tokens, dim, dtype, w_dtype);
  if (st != MSIGN_OK) return st;
  if (!(eps > 0.f) || !std::isfinite(eps)) return fail(MSIGN_ERR_ARG, "eps must be positive and finite");
  if (tokens == 0 || dim == 0) return MSIGN_OK;
  const int64_t s = dt_size(dtype);
  if (!rows_ok(x, tokens, dim, ldx, s) || !rows_ok(y, tokens, dim, dim, s) ||
      !vector_ok(weight, dim, dt_size(w_dtype)) || !vector_ok(rstd, tokens, 4) ||
      (residual != nullptr && (!rows_ok(residual, tokens, dim, ldr, s) || !rows_ok(h_out, tokens, dim, dim, s))))
    return fail(MSIGN_ERR_ARG, "tensors must be non-null, aligned to their elements, with pitches of at least a row "
                               "and at most 2^36 elements");
  const Range hr = residual != nullptr ? range(h_out, tokens, dim, dim, s) : Range{nullptr, 0};
  const Range xr = range(x, tokens, dim, ldx, s), rr = range(residual, tokens, dim, ldr, s);
  const Range wr = range(weight, 1, dim, dim, dt_size(w_dtype));
  const Range out[] = {range(y, tokens, dim, dim, s), hr, range(rstd, 1, tokens, tokens, 4)};
  // h may take the place of x or of the residual: each element is read before it is written
  const bool same_x = h_out == x && ldx == dim, same_r = h_out == residual && ldr == dim;
  const Range in_y[] = {xr, rr, wr}, in_h[] = {same_x ? Range{nullptr, 0} : xr, same_r ? Range{nullptr, 0} : rr, wr};
  const Range only_y[] = {out[0], out[2]}, only_h[] = {hr};
  const Range none[] = {{nullptr, 0}};
  if (outputs_overlap(out, none) || outputs_overlap(only_y, in_y) || outputs_overlap(only_h, in_h))
    return fail(MSIGN_ERR_ALIAS, "an output overlaps an input or another output");
  const norm::ForwardArgs a = {x, residual, weight, y, h_out, rstd, ldx, ldr, tokens, (int32_t)dim, w_dtype, eps};
  auto run = [&](auto t) {
    using T = decltype(t);
    return norm_config<T, false>(dim, [&](auto NT, auto C, auto HOLD) {
      return norm_forward_cfg<T, NT(), C(), HOLD()>(a, stream);
    });
  };
  const hipError_t e = dtype == MSIGN_BF16 ? run(bf16_t{}) : dtype == MSIGN_F16 ? run(f16_t{}) : run(0.f);
  return e == hipSuccess ? MSIGN_OK : hip_fail(e, "forward_kernel");
}

size_t add_rms_norm_backward_workspace_bytes(int64_t tokens, int64_t dim) {
  if (tokens < 0 || tokens > kMaxTokens || dim < 0 || dim > kMaxNormDim) return kInvalid;
  return (size_t)round_up(norm_backward_blocks(tokens) * dim * 4, 256);
}

msign_status_t add_rms_norm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ldh, const float* rstd,
                                     const void* weight, const void* dh, int64_t ld_dh, void* dx, void* dweight,
                                     int64_t tokens, int64_t dim, int32_t dtype, int32_t w_dtype, void* workspace,
                                     size_t workspace_bytes, hipStream_t stream) {
  msign_status_t st = check_norm(tokens, dim, dtype, w_dtype);
  if (st != MSIGN_OK) return st;
  if (dim == 0) return MSIGN_OK;
  const int64_t s = dt_size(dtype), w = dt_size(w_dtype);
  if (!rows_ok(dy, tokens, dim, ld_dy, s) || !rows_ok(h, tokens, dim, ldh, s) ||
      !vector_ok(rstd, tokens, 4) || !vector_ok(weight, dim, w) ||
      !vector_ok(dweight, dim, w) || !rows_ok(dx, tokens, dim, dim, s) ||
      (dh != nullptr && !rows_ok(dh, tokens, dim, ld_dh, s)))
    return fail(MSIGN_ERR_ARG, "tensors must be non-null, aligned to their elements, with pitches of at least a row "
                               "and at most 2^36 elements");
  const size_t need = add_rms_norm_backward_workspace_bytes(tokens, dim);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MSIGN_OK) return st;
  const Range dyr = range(dy, tokens, dim, ld_dy, s), dhr = range(dh, tokens, dim, ld_dh, s);
  const Range hr = range(h, tokens, dim, ldh, s), sr = range(rstd, 1, tokens, tokens, 4);
  const Range wr = range(weight, 1, dim, dim, w), none = {nullptr, 0};
  const Range dxr = range(dx, tokens, dim, dim, s);
  const Range others[] = {range(dweight, 1, dim, dim, w), {static_cast<char*>(workspace), (int64_t)need}};
  // dx may take the place of dy or dh: each element is read before it is written
  const Range in_dx[] = {dx == dy && ld_dy == dim ? none : dyr, dx == dh && ld_dh == dim ? none : dhr, hr, sr, wr,
                         others[0], others[1]};
  const Range in[] = {dyr, dhr, hr, sr, wr};
  const Range only[] = {dxr};
  if (outputs_overlap(only, in_dx) || outputs_overlap(others, in))
    return fail(MSIGN_ERR_ALIAS, "an output overlaps an input, another output or the workspace");
  float* partial = static_cast<float*>(workspace);
  int64_t blocks = norm_backward_blocks(tokens);
  if (blocks > 0) {
    const norm::BackwardArgs a = {dy, h, weight, dh, rstd, dx, partial, ld_dy, ldh, ld_dh, tokens, (int32_t)dim,
                                  w_dtype};
    auto run = [&](auto t) {
      using T = decltype(t);
      return norm_config<T, true>(dim, [&](auto NT, auto C, auto HOLD) {
        return norm_backward_cfg<T, NT(), C(), HOLD()>(a, blocks, stream);
      });
    };
    const hipError_t e = dtype == MSIGN_BF16 ? run(bf16_t{}) : dtype == MSIGN_F16 ? run(f16_t{}) : run(0.f);
    if (e != hipSuccess) return hip_fail(e, "backward_kernel");
  }
  norm::weight_sum_kernel<<<dim3((unsigned)((dim + 63) / 64)), 1024, 0, stream>>>(partial, (int32_t)blocks, dweight,
                                                                                 (int32_t)dim, w_dtype);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? MSIGN_OK : hip_fail(e, "weight_sum_kernel");
}

}  // extern "C"

// -------------------------------------------------------- distillation ----

namespace {

static_assert(distill::kMaxTop == DISTILL_MAX_TOP, "entries per row");

// OCC: waves per SIMD, so 4 OCC / (NT / 64) workgroups on each of the 256 CUs
template <typename T, int NT, int C, bool GRAD, int OCC>
hipError_t distill_cfg(const distill::Args& a, hipStream_t st) {
  constexpr int64_t resident = 256 * (4 * OCC / (NT / 64));
  static_assert(resident > 0, "workgroups");
  distill::row_kernel<T, NT, C, GRAD, OCC>
      <<<dim3((unsigned)(a.rows < resident ? a.rows : resident)), NT, 0, st>>>(a);
  return hipGetLastError();
}

// The loss alone streams its rows: 256 threads a row, 1024 where few long rows
// would leave the card idle (bf16, 4096 rows of 32768: 47 and 89 us; 64 rows of
// 160000: 15 and 13 us).  With the gradient a row stays in registers between its
// two passes, in the smallest configuration whose chunks of 16 bytes hold it, and
// longer rows are read twice.  Us of bf16 rows, 256 MB of them, in the one taken
// and in the next one that holds them, or read twice (by 256 threads up to 2^15,
// else by 1024):
//   vocabulary    4096   8192  16384  32768  65536  98304  131072  160000
//   taken          138    117    110    113    111    132     124     149
//   next           208    171    156    151    170    151     140       -
//   read twice     247    157    137    143    138    146     138     151
template <typename T>
hipError_t distill_typed(const distill::Args& a, hipStream_t st) {
  const int64_t chunks = a.vocab / (16 / Elem<T>::size);
  if (a.dz == nullptr) {
    if (chunks <= 1024 || a.rows >= 512) return distill_cfg<T, 256, 0, false, 7>(a, st);
    return distill_cfg<T, 1024, 0, false, 4>(a, st);
  }
  if (chunks == 0) return distill_cfg<T, 256, 0, true, 4>(a, st);
  if (chunks <= 512) return distill_cfg<T, 64, 8, true, 3>(a, st);
  if (chunks <= 1024) return distill_cfg<T, 256, 4, true, 5>(a, st);
  if (chunks <= 2048) return distill_cfg<T, 256, 8, true, 4>(a, st);
  if (chunks <= 4096) return distill_cfg<T, 256, 16, true, 3>(a, st);
  if (chunks <= 8192) return distill_cfg<T, 512, 16, true, 4>(a, st);
  if (chunks <= 12288) return distill_cfg<T, 512, 24, true, 2>(a, st);
  if (chunks <= 16384) return distill_cfg<T, 512, 32, true, 2>(a, st);
  if (chunks <= 20480) return distill_cfg<T, 512, 40, true, 2>(a, st);
  return distill_cfg<T, 1024, 0, true, 4>(a, st);
}

}  // namespace

extern "C" {

msign_status_t distill_topk(const void* logits, int64_t ld_logits, const void* indices, int32_t indices_64,
                            const void* teacher, int32_t teacher_dtype, const float* grad, int64_t grad_stride,
                            float* loss, void* dlogits, int64_t rows, int64_t vocab, int64_t top, float tau,
                            int32_t dtype, hipStream_t stream) {
  if (!dt_valid(dtype) || !dt_valid(teacher_dtype))
    return fail(MSIGN_ERR_DTYPE, "dtype and teacher_dtype must be MSIGN_F32, MSIGN_BF16 or MSIGN_F16");
  if (rows < 0 || rows > kMaxTokens || vocab < 1 || vocab > kMaxPitch || top < 0 || top > DISTILL_MAX_TOP)
    return fail(MSIGN_ERR_SHAPE, "rows must be in 0..2^24, vocab in 1..2^21 and top in 0..1024");
  if (!(tau > 0.f) || !std::isfinite(tau)) return fail(MSIGN_ERR_ARG, "tau must be positive and finite");
  if (indices_64 != 0 && indices_64 != 1) return fail(MSIGN_ERR_ARG, "indices_64 must be 0 or 1");
  if (grad_stride < 0 || grad_stride > kMaxRowPitch) return fail(MSIGN_ERR_ARG, "grad_stride must be in 0..2^36");
  if (rows == 0) return MSIGN_OK;
  const int64_t s = dt_size(dtype), is = indices_64 ? 8 : 4, ts = dt_size(teacher_dtype);
  if (!rows_ok(logits, rows, vocab, ld_logits, s) || !rows_ok(indices, rows, top, top, is) ||
      !rows_ok(teacher, rows, top, top, ts) || !vector_ok(loss, rows, 4) ||
      (dlogits != nullptr && (!rows_ok(dlogits, rows, vocab, vocab, s) || grad == nullptr || !aligned(grad, 4))))
    return fail(MSIGN_ERR_ARG, "tensors must be non-null, aligned to their elements, with a pitch of at least a row "
                               "and at most 2^36 elements; dlogits needs grad");
  const Range zr = range(logits, rows, vocab, ld_logits, s), none = {nullptr, 0};
  const Range lossr = range(loss, 1, rows, rows, 4), dzr = range(dlogits, rows, vocab, vocab, s);
  const Range gr = dlogits != nullptr ? range(grad, rows, 1, grad_stride, 4) : none;
  const Range ir = range(indices, rows, top, top, is), tr = range(teacher, rows, top, top, ts);
  const Range only_loss[] = {lossr}, only_dz[] = {dzr};
  // dlogits may take the place of the logits: an element is read before it is written
  const Range in_loss[] = {zr, ir, tr, gr, dzr};
  const Range in_dz[] = {dlogits == logits && ld_logits == vocab ? none : zr, ir, tr, gr};
  if (outputs_overlap(only_loss, in_loss) || outputs_overlap(only_dz, in_dz))
    return fail(MSIGN_ERR_ALIAS, "an output overlaps an input or another output");
  const distill::Args a = {logits, ld_logits, indices, teacher, grad, grad_stride, loss, dlogits, rows,
                           indices_64, teacher_dtype, (int32_t)vocab, (int32_t)top, tau};
  hipError_t e;
  switch (dtype) {
    case MSIGN_BF16: e = distill_typed<bf16_t>(a, stream); break;
    case MSIGN_F16: e = distill_typed<f16_t>(a, stream); break;
    default: e = distill_typed<float>(a, stream);
  }
  return e == hipSuccess ? MSIGN_OK : hip_fail(e, "row_kernel");
}

}  // extern "C"
