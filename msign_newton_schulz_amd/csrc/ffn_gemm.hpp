// Matrix products of the gated feed-forward block (gfx950).
//
// One tile kernel computes C = A B^T (M x N, summed over K) for every product
// of the block's forward and backward pass:
//   g, u, h     A = x            B = Wg and Wu    both read along K = dim; the
//                                activation and h = a(g) u in the epilogue
//   y           A = h            B = Wd           both along K = hidden
//   dh          A = dy           B = Wd           B stored K-major (rows are k);
//                                the epilogue turns dh into dg, du and h
//   dx          A = dg | du      B = Wg | Wu      B K-major; the sum over K runs
//                                over the two pairs one after the other
//   dWg,dWu,dWd A = dg, du, dy   B = x, x, h      both K-major, K = tokens, three
//                                products, in one launch with dx
//
// Tiles: 256 x 256 by four waves of 128 x 128, one workgroup a CU (128 KB of
// LDS), or 128 x 128 by four waves of 64 x 64, with K slices of 128 bytes (two
// workgroups a CU) or 256 (one).  A slice of both operands goes from global
// memory straight into one of two LDS stages (buffer_load ... lds).  Chunks of
// 16 bytes are XOR-swizzled so that neither fragment reads along K
// (ds_read_b128) nor transpose reads of K-major tiles (ds_read_b64_tr_b16)
// meet bank conflicts (the counter reads 0).  A 128 x 128 wave tile reads 32 KB
// of LDS a slice for 128 matrix instructions, half of the LDS rate, and its
// accumulators fill the accumulation registers; 64 x 64 waves need all of the
// rate, and reach 860 TFLOP/s, 1010 with slices of 256 bytes, which have half
// the barriers.  They serve products with too few 256-tiles for the card.
//
// Measured, bf16, 4096 x 14336 (a library's products of these shapes: 1441 to
// 1652 TFLOP/s both along K, 1267 to 1435 with B K-major, 905 to 921 with both):
//   8192 tokens: gated 1435 us, 1341 TFLOP/s; down 665 us, 1447 TFLOP/s
//   4096 tokens: dgated 458 us, 1050 TFLOP/s; dx and the three weight gradients
//   in one launch 1766 us, 1362 TFLOP/s (apart 650 and 1092; timed in turn, the
//   whole pass takes the same either way, 2261 and 2262 us)
//   16 tokens: gated 42 us, 5.6 TB/s; down 23 us, 5.1 TB/s, bound by memory
// Bound by the matrix instructions at the clock that the power limit leaves
// (down: busy 80 % of the time at 1.77 GHz, gated 72 % at 1.72 GHz).  dgated
// reads two and writes three matrices of its size in its epilogue: while a CU's
// only workgroup is there, its matrix units rest.  An earlier form of 8 waves of
// 128 x 64 took 1722, 777, 735, 964 and 1896 us.  fp32 has tiles of 64 x 128, two
// or more workgroups a CU, and reaches 148 TFLOP/s (a library's: 139 to 142).
//
// The wave's tile is computed in four quadrants, A halves x B halves, so that
// the fragments of the next quadrant are read while the current one is
// multiplied; see tile_block.  The matrix instruction gets B as its first operand:
// a lane then holds four consecutive columns of one row of C.
#pragma once

#include "gemm_nt.hpp"
#include "row_ops.hpp"

namespace msign {
namespace ffn {

enum Epilogue : int { EPI_PLAIN = 0, EPI_GATED = 1, EPI_DGATED = 2 };

struct Problem {
  // K segments 0 and 1 (EPI_GATED: B[0] = Wg and B[1] = Wu of one segment)
  const void* A[2];
  const void* B[2];
  int64_t lda[2], ldb[2];
  int32_t M, N;       // EPI_GATED, EPI_DGATED: N = hidden
  int32_t K;          // per segment; row-major operands: a multiple of 16 bytes
  int32_t kvalid;     // rows of a K-major operand that exist (at most K)
  void* C;            // EPI_PLAIN
  int64_t ldc;
  int32_t tiles_m, tiles_n;
};

constexpr int kMaxProblems = 3;

template <int NG>
struct Args {
  Problem g[NG];
  int32_t bstart[NG];   // first block of each problem
  int32_t split;        // parts of the sum over K, one block each
  float* partial;       // fp32 sums of the parts (split > 1)
  int32_t activation;
  // EPI_GATED: outputs gate, up (may be null) and h.  EPI_DGATED: inputs gate
  // and up, outputs dg, du, h.  dg, du and h: pitch ldh, a multiple of 16
  // bytes, with columns N .. round_up(N, 16 bytes) written as zeros.
  void *gate, *up;
  int64_t ld_act;
  void *h, *dg, *du;
  int64_t ldh;
};

// s(w), with a(g) = g s(w): silu's w is g; gelu's tanh form has w = 2 sqrt(2/pi)
// (g + c g^3).  Kind is compile-time: chosen per value it took a third more
// instructions.
constexpr float kGelu = 1.5957691216057308f, kGelu3 = 0.044715f * kGelu;  // 2 sqrt(2 / pi), and c times it
constexpr float kLog2e = 1.44269504f;

template <int KIND>
__device__ __forceinline__ float gate(float g) {
  const float w = KIND == 0 ? -kLog2e * g : g * fmaf(-kLog2e * kGelu3, g * g, -kLog2e * kGelu);
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(w));
}

// a(g) and a'(g) = s + g w' s (1 - s).  Beyond |g| = 128 (silu) or 16 (gelu) s
// is 0 or 1 in fp32, so g is held there, and g w' stays finite.
template <int KIND>
__device__ __forceinline__ void activate(float g, float& a, float& da) {
  const float s = gate<KIND>(g);
  a = g * s;
  const float lim = KIND == 0 ? 128.f : 16.f, h = __builtin_amdgcn_fmed3f(g, -lim, lim);
  const float gw = KIND == 0 ? h : h * fmaf(3.f * kGelu3, h * h, kGelu);
  da = s * fmaf(gw, 1.f - s, 1.f);
}

// Tile (ti, tj) of the L-th tile: groups of GM tile rows are walked column by
// column, so that tiles running together share operand strips in L2.
__device__ __forceinline__ void tile_at(const Problem& p, int L, int& ti, int& tj) {
  constexpr int GM = 8;
  const int per = GM * p.tiles_n, g = L / per, first = g * GM;
  const int gm = p.tiles_m - first < GM ? p.tiles_m - first : GM;
  const int rr = L - g * per;
  ti = first + rr % gm;
  tj = rr / gm;
}

template <typename T, int BM_, int BN_, int WGM_, int WGN_, int CPR_, bool AKM_, bool BKM_, int EPI_, int NG_,
          int NSEG_>
struct Tile {
  using type = T;
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, EPI = EPI_, NG = NG_, NSEG = NSEG_;
  static constexpr bool AKM = AKM_, BKM = BKM_;  // operand stored K-major
  static constexpr int NT = WGM * WGN * 64;
  static constexpr int WM = BM / WGM, WN = BN / WGN, FM = WM / 16, FN = WN / 16;
  static constexpr int ESZ = Elem<T>::size, CE = 16 / ESZ;
  static constexpr int CPR = CPR_, KTE = CPR * CE;  // a K slice: CPR chunks of 16 bytes
  static constexpr int KSUB = CPR / 4;              // matrix instruction K steps per slice
  static constexpr int ACH = BM * CPR / NT, BCH = BN * CPR / NT;
  static constexpr int LDS = 2 * (BM + BN) * CPR;  // chunks: two stages
  static constexpr bool DUAL = EPI == EPI_GATED;
  // columns of C per tile: a gated tile holds as many gate as up columns
  static constexpr int CN = DUAL ? BN / 2 : BN;
  static_assert(FM % 2 == 0 && FN % 2 == 0 && NT % (8 * CPR) == 0 && (CPR == 8 || CPR == 16), "tile");
  static_assert(!DUAL || (!BKM && (WN / 2) % 8 == 0), "gated tiles read B along K");
};

// 16 bytes per lane from byte `off` of a buffer, zeros past its end, into 64
// consecutive chunks of LDS at `dst` (uniform over the wave).  Written as
// assembly, which has no result in registers: from the builtin the compiler
// cannot tell which later LDS reads depend on it and makes them wait for the
// loads in flight.  loads_barrier's wait is the one that counts.
// (dst = base + OFF chunks.)
template <int OFF>
__device__ __forceinline__ void load_lds(const u32x4& rsrc, int off, uint32_t base) {
  asm volatile("s_add_u32 m0, %0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(base), "v"(off), "s"(rsrc), "n"(OFF * 16) : "memory", "m0", "scc");
}

__device__ __forceinline__ u32x4 make_rsrc(const char* base, int bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  return u32x4{(uint32_t)b, (uint32_t)(b >> 32) & 0xffffu, (uint32_t)bytes, 0x00020000u};
}

// Moves a buffer's start (its length stays).
__device__ __forceinline__ void advance(u32x4& rsrc, int64_t bytes) {
  const uint64_t b = (((uint64_t)rsrc[1] << 32) | rsrc[0]) + (uint64_t)bytes;
  rsrc[0] = (uint32_t)b;
  rsrc[1] = (uint32_t)(b >> 32);
}

// acc += A B with the accumulator kept in place.  (From the builtin the
// compiler moves accumulators on to other registers, which costs copies and
// spills next to a full register file.)  The instruction's wait states are
// kept by the callers: an accumulator comes up again only after the other
// fragments of its quadrant, and settle() stands before it is read.
template <typename T>  // bf16_t or f16_t
__device__ __forceinline__ void mma(f32x4& acc, const u32x4& a, const u32x4& b) {
  if constexpr (std::is_same<T, bf16_t>::value)
    asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
  else
    asm("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}

// fp32: one of the four products of a fragment.
__device__ __forceinline__ void mma_f32(f32x4& acc, float a, float b) {
  asm("v_mfma_f32_16x16x4_f32 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}

// Wait states between writing accumulators and mma(), and between mma() and
// reading its results.
template <int M, int N>
__device__ __forceinline__ void settle(f32x4 (&acc)[M][N]) {
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) asm volatile("" : "+a"(acc[i][j]));
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) asm volatile("" : "+a"(acc[i][j]));
  __builtin_amdgcn_sched_barrier(0);
}

// Waits until at most N of this wave's loads into LDS are in flight, then for
// the other waves.
template <int N>
__device__ __forceinline__ void loads_barrier() {
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" :: "n"(N) : "memory");
}

// Waits for this wave's LDS reads, then for the other waves.
__device__ __forceinline__ void reads_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Chunk position in a row-major LDS row.  A wave's 16-byte reads go 16 lanes at
// once, of 16 rows and two chunks: rows of 16 chunks, which all start at the
// same bank, change halves with the row's parity, as rows of 8 chunks do by
// themselves.
template <int CPR>
__device__ __forceinline__ int swz_row(int row, int ch) {
  return CPR == 16 ? ch ^ ((row & 7) | ((row & 1) << 3)) : ch ^ (row & 7);
}

// Moves one operand's K slices into LDS, one after the other.  Row-major (KM
// false): LDS rows are the tile's rows, CPR chunks each, swizzled by the row.
// K-major: LDS rows are the slice's k, ROWS / CE chunks each.  Reads past the
// operand's rows, columns or last k get an offset past the buffer's end and
// return zeros, so slices past the last one may be asked for.
template <typename C, int ROWS, bool KM, bool IS_B>
struct Loader {
  static constexpr int N = ROWS * C::CPR / C::NT;    // loads per thread and slice
  static constexpr int CPRK = ROWS / C::CE;          // chunks of a K-major row
  static constexpr int RSTEP = KM ? C::NT / CPRK : C::NT / C::CPR;
  static constexpr bool DUAL = IS_B && C::DUAL;
  // gated tiles: a load instruction of all waves reads Wg or Wu, or (each wave
  // always the same rows of the waves' parts) a wave reads one of them only
  static constexpr int H = C::WN / 2;
  static constexpr int ND = DUAL && RSTEP <= H ? 2 : 1;
  static_assert(!DUAL || (ND == 2 ? H % RSTEP == 0 : RSTEP % C::WN == 0), "rows of a load");
  static constexpr int kOutside = 0x7fffffff;
  u32x4 rsrc[ND];       // from the next slice's first byte on
  int32_t off[N];       // this thread's chunks
  int32_t left;         // k values from the next slice's start on
  int32_t kch;          // row-major: first k of this thread's chunk in a slice
  int32_t pitch, cols;  // K-major: bytes of a row, and of the columns from the tile's first on
  const char* ptr1;     // segment 1's first slice
  int32_t full, pitch1, off1[KM && C::NSEG > 1 ? N : 1];

  static __device__ __forceinline__ int k_offset(int s, int pitch, int cols) {
    const int kr = (int)threadIdx.x / CPRK + s * RSTEP;
    const int ch = swz_t<C::ESZ, CPRK>(kr, (int)threadIdx.x % CPRK);
    return ch * 16 < cols ? kr * pitch + ch * 16 : kOutside;
  }

  __device__ __forceinline__ void row_offsets(const Problem& p) {
#pragma unroll
    for (int s = 0; s < N; ++s) {
      int row = (int)threadIdx.x / C::CPR + s * RSTEP;
      int64_t ld = IS_B ? p.ldb[0] : p.lda[0];  // (both segments of a row-major operand have one pitch)
      if constexpr (DUAL) {
        ld = p.ldb[row % C::WN / H ? 1 : 0];
        row = row / C::WN * H + row % H;
      }
      off[s] = (row * (int)ld + kch) * C::ESZ;
    }
  }

  // first: the tile's first row; slice k0 of segment seg comes first
  __device__ __forceinline__ void init(const Problem& p, int first, int seg, int k0) {
    const int tid = threadIdx.x;
    const int uw = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int total = IS_B ? p.N : p.M;
    const char* b0 = static_cast<const char*>(IS_B ? p.B[0] : p.A[0]);
    const char* b1 = static_cast<const char*>(IS_B ? p.B[1] : p.A[1]);
    const int64_t ld0 = (IS_B ? p.ldb[0] : p.lda[0]) * C::ESZ, ld1 = (IS_B ? p.ldb[1] : p.lda[1]) * C::ESZ;
    if constexpr (KM) {
      cols = ((total + C::CE - 1) / C::CE * C::CE - first) * C::ESZ;
      left = p.kvalid - k0;
      pitch = (int)(seg ? ld1 : ld0);
      rsrc[0] = make_rsrc((seg ? b1 : b0) + k0 * (int64_t)pitch + first * (int64_t)C::ESZ, 0);
#pragma unroll
      for (int s = 0; s < N; ++s) off[s] = k_offset(s, pitch, cols);
      if constexpr (C::NSEG > 1) {
        ptr1 = b1 + first * (int64_t)C::ESZ;
        pitch1 = (int)ld1;
#pragma unroll
        for (int s = 0; s < N; ++s) off1[s] = k_offset(s, pitch1, cols);
      }
    } else {
      kch = swz_row<C::CPR>(tid / C::CPR, tid % C::CPR) * C::CE;
      left = p.K - k0;
      const int rows = total - first < ROWS ? total - first : ROWS;
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        // LDS rows of a gated tile's WN: the first half from Wg, the second from Wu
        const int which = !DUAL ? seg : ND == 2 ? d : (uw * (64 / C::CPR) % C::WN) / H;
        const int64_t ld = which ? ld1 : ld0;
        // a row past the last starts past the buffer's end, whatever its k
        rsrc[d] = make_rsrc((which ? b1 : b0) + first * ld + k0 * (int64_t)C::ESZ,
                            (int)((rows - 1) * ld + p.K * (int64_t)C::ESZ));
      }
      row_offsets(p);
      if constexpr (C::NSEG > 1) {
        ptr1 = b1 + first * ld1;
        full = (int)rsrc[0][2];
      }
    }
  }

  // Before a slice's loads.  to_segment1: segment 1 begins with it.  (Uniform
  // branches, taken where a segment ends.)
  __device__ __forceinline__ void begin(const Problem& p, bool to_segment1) {
    if constexpr (C::NSEG > 1) {
      if (to_segment1) {
        rsrc[0] = make_rsrc(ptr1, KM ? 0 : full);
        left = KM ? p.kvalid : p.K;
        if constexpr (KM) {
          pitch = pitch1;
#pragma unroll
          for (int s = 0; s < N; ++s) off[s] = off1[s];
        } else {
          row_offsets(p);
        }
      }
    }
    if constexpr (KM) {
      const int rows = left < C::KTE ? left : C::KTE;
      rsrc[0][2] = rows > 0 ? (rows - 1) * pitch + cols : 0;
    } else if (left < C::KTE) {
      // chunks past the last k
      const bool in = kch < left;
#pragma unroll
      for (int s = 0; s < N; ++s) off[s] = in ? off[s] : kOutside;
    }
  }

  // Load instruction S of the next slice into the stage at `base` (this wave's
  // first chunk of the operand's part).
  template <int S>
  __device__ __forceinline__ void load(uint32_t base) const {
    load_lds<S * C::NT>(rsrc[ND == 1 ? 0 : S * RSTEP % C::WN / H], off[S], base);
  }

  // Goes on to the next slice.
  __device__ __forceinline__ void next() {
#pragma unroll
    for (int d = 0; d < ND; ++d) advance(rsrc[d], KM ? (int64_t)C::KTE * pitch : (int64_t)C::KTE * C::ESZ);
    left -= C::KTE;
  }
};

// Reads a wave's fragments of one operand from an LDS stage: W rows of the
// wave tile, in two halves.  Every address is the lane's own offset with
// constants added (K steps, and rows of row-major tiles) or exclusive-ored
// (the swizzle's chunks).
template <typename C, int W, int ROWS, bool KM>
struct Reader {
  static constexpr int F = W / 32;            // fragments of a half
  static constexpr int CPRK = ROWS / C::CE;
  uint32_t lane_off;

  __device__ __forceinline__ void init(int w) {
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int row0 = w * W;
    if constexpr (!KM) {
      lane_off = (row0 + r) * (C::CPR * 16) + swz_row<C::CPR>(r, g) * 16;
    } else if constexpr (C::ESZ == 2) {
      // transpose reads: lane (g, r) ends with column r at k = 32 kk + 8 g + 0..7
      const int m = row0 + 4 * (r & 3), k = 8 * g + (r >> 2);
      lane_off = k * CPRK * 16 + swz_t<2, CPRK>(k, m >> 3) * 16 + (m & 7) * 2;
    } else {
      const int m = row0 + r, k = 4 * g;
      lane_off = k * CPRK * 16 + swz_t<4, CPRK>(k, m >> 2) * 16 + (m & 3) * 4;
    }
  }

  // The lane's offset, new to the compiler: it would else keep every address
  // of the loop in a register of its own.
  __device__ __forceinline__ void refresh() { asm volatile("" : "+v"(lane_off)); }

  // fragment f of half `half` at K step kk, into out[kk F + f]
  template <int HALF, int I>
  __device__ __forceinline__ void read(const u32x4* tile, u32x4 (&out)[F * C::KSUB]) const {
    constexpr int half = HALF, kk = I / F, f = I % F;
    const char* t = reinterpret_cast<const char*>(tile);
    {
      if constexpr (!KM) {
        const uint32_t o = lane_off ^ (kk * 64);
        out[kk * F + f] = *reinterpret_cast<const u32x4*>(t + o + (half * (W / 2) + f * 16) * (C::CPR * 16));
      } else if constexpr (C::ESZ == 2) {
        const uint32_t o = lane_off ^ ((half * (W / 2) + f * 16) * 2);
        out[kk * F + f] = lds_read_tr16_pair(t + o, kk * 32 * CPRK * 16, (kk * 32 + 4) * CPRK * 16);
      } else {
        const uint32_t o = lane_off ^ ((half * (W / 2) + f * 16) * 4);
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const float*>(t + o + (kk * 16 + e) * CPRK * 16);
        out[kk * F + f] = __builtin_bit_cast(u32x4, v);
      }
    }
  }
};

// ---- epilogue ----
//
// A wave's accumulators go through its part of the LDS (free after the K loop)
// as fp32, PR rows at a time, and come back by rows: 16 bytes of output per
// lane, whole lines per row, where the accumulators' own layout would store 8
// bytes to each of 16 rows.  Rows of WN floats; chunks of four floats are
// exclusive-ored with the row, which keeps both ways free of bank conflicts.

// Fragment row `acc` (FN fragments) as rows row0 .. row0 + 15 of the stage.
template <typename C>
__device__ __forceinline__ void stage_rows(float* stage, int row0, const f32x4 (&acc)[C::FN]) {
  const int lane = threadIdx.x & 63, m = lane & 15;
#pragma unroll
  for (int fn = 0; fn < C::FN; ++fn)
    *reinterpret_cast<f32x4*>(stage + (row0 + m) * C::WN + ((fn * 4 + (lane >> 4)) ^ m) * 4) = acc[fn];
}

template <typename C>
__device__ __forceinline__ void read_row(const float* stage, int row, int col, float (&v)[C::CE]) {
#pragma unroll
  for (int q = 0; q < C::CE / 4; ++q) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(stage + row * C::WN + ((col / 4 + q) ^ (row & 15)) * 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * q + e] = x[e];
  }
}

// Stores columns n .. n + CE - 1 (those below `cols`) of a row, at any
// alignment.
template <typename T, int CE>
__device__ __forceinline__ void put(void* base, int64_t row_at, int n, int cols, const float (&v)[CE]) {
  rows::store_chunk<T>(static_cast<char*>(base) + row_at * Elem<T>::size, n, cols, rows::pack<T>(v));
}

// The outputs of NP times PR rows from m0 on, columns n0 .. of a wave tile.
// fill(i) brings rows i PR .. of the wave tile into its stage (i is a constant:
// the accumulators are registers).  Lane l: CE
// columns from (l % LPR) CE on, of row l / LPR of 64 / LPR.
template <typename C, int PR, int NP, int KIND, typename Fill>
__device__ __forceinline__ void finish_rows(const Args<C::NG>& a, const Problem& p, int m0, int n0,
                                            const float* stage, Fill fill) {
  using T = typename C::type;
  constexpr int CE = C::CE, W = C::DUAL ? C::WN / 2 : C::WN, LPR = W / CE, RPI = 64 / LPR, IT = PR / RPI;
  const int lane = threadIdx.x & 63, r0 = lane / LPR, c = lane % LPR * CE;
  const int n = n0 + c;
  if constexpr (C::EPI == EPI_PLAIN) {
    static_for<NP>([&](auto P) {
      constexpr int ph = decltype(P)::value;
      fill(P);
      if (n >= p.N) return;
#pragma unroll 2
      for (int it = 0; it < IT; ++it) {
        const int r = it * RPI + r0, m = m0 + ph * PR + r;
        float v[CE];
        read_row<C>(stage, r, c, v);
        if (m < p.M) put<T, CE>(p.C, (int64_t)m * p.ldc, n, p.N, v);
      }
    });
  } else if constexpr (C::EPI == EPI_GATED) {
    static_for<NP>([&](auto P) {
      constexpr int ph = decltype(P)::value;
      fill(P);
      if (n >= p.N) return;
#pragma unroll 2
      for (int it = 0; it < IT; ++it) {
        const int r = it * RPI + r0, m = m0 + ph * PR + r;
        float g[CE], u[CE], h[CE];
        read_row<C>(stage, r, c, g);
        read_row<C>(stage, r, c + W, u);
        if (m >= p.M) continue;
#pragma unroll
        for (int e = 0; e < CE; ++e) h[e] = g[e] * gate<KIND>(g[e]) * u[e];
        if (n + CE > p.N) {
#pragma unroll
          for (int e = 0; e < CE; ++e) h[e] = n + e < p.N ? h[e] : 0.f;
        }
        *reinterpret_cast<u32x4*>(static_cast<char*>(a.h) + ((int64_t)m * a.ldh + n) * C::ESZ) = rows::pack<T>(h);
        if (a.gate != nullptr) {
          put<T, CE>(a.gate, (int64_t)m * a.ld_act, n, p.N, g);
          put<T, CE>(a.up, (int64_t)m * a.ld_act, n, p.N, u);
        }
      }
    });
  } else {
    // outputs of row r of a phase from its chunks of gate and up
    auto emit = [&](int ph, int r, const u32x4& gv, const u32x4& uv) {
      const int m = m0 + ph * PR + r;
      float dh[CE], g[CE], u[CE], dg[CE], du[CE], h[CE];
      read_row<C>(stage, r, c, dh);
      rows::unpack<T>(gv, g);
      rows::unpack<T>(uv, u);
      if (n + CE > p.N) {  // columns past N are other rows' values
#pragma unroll
        for (int e = 0; e < CE; ++e) dh[e] = n + e < p.N ? dh[e] : 0.f;
      }
#pragma unroll
      for (int e = 0; e < CE; ++e) {
        float act, d;
        activate<KIND>(g[e], act, d);
        du[e] = dh[e] * act;
        dg[e] = dh[e] * u[e] * d;
        h[e] = act * u[e];
      }
      if (m >= p.M) return;
      const int64_t at = ((int64_t)m * a.ldh + n) * C::ESZ;
      *reinterpret_cast<u32x4*>(static_cast<char*>(a.dg) + at) = rows::pack<T>(dg);
      *reinterpret_cast<u32x4*>(static_cast<char*>(a.du) + at) = rows::pack<T>(du);
      *reinterpret_cast<u32x4*>(static_cast<char*>(a.h) + at) = rows::pack<T>(h);
    };
    const char *gate = static_cast<const char*>(a.gate), *up = static_cast<const char*>(a.up);
    if (__builtin_amdgcn_ballot_w64(n + CE > p.N) == 0) {
      // Whole chunks in every lane: U rows' loads in flight while the U rows
      // before them are worked on, in batches over all phases.  Rows past the
      // last read the last one, so that the loads have no branch and are
      // counted.
      constexpr int U = IT < 4 ? IT : 4, NBP = IT / U, NB = NP * NBP;
      auto fetch = [&](int b, u32x4 (&gv)[U], u32x4 (&uv)[U]) {
        const int mb = m0 + (b < NB ? b : NB - 1) * U * RPI + r0;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int m = mb + i * RPI;
          const int64_t at = ((int64_t)(m < p.M ? m : p.M - 1) * a.ld_act + n) * C::ESZ;
          gv[i] = *reinterpret_cast<const rows::u32x4_any*>(gate + at);
          uv[i] = *reinterpret_cast<const rows::u32x4_any*>(up + at);
        }
      };
      auto batch = [&](int b, const u32x4 (&gv)[U], const u32x4 (&uv)[U]) {
#pragma unroll
        for (int i = 0; i < U; ++i) emit(b / NBP, (b % NBP * U + i) * RPI + r0, gv[i], uv[i]);
      };
      u32x4 g0[U], u0[U], g1[U], u1[U];
      fetch(0, g0, u0);
      static_assert(NB == 1 || NBP % 2 == 0, "pairs of batches");
      static_for<NP>([&](auto P) {
        fill(P);
        if constexpr (NB == 1) {
          batch(0, g0, u0);
        } else {
#pragma unroll 1
          for (int b = decltype(P)::value * NBP; b < (decltype(P)::value + 1) * NBP; b += 2) {
            fetch(b + 1, g1, u1);
            batch(b, g0, u0);
            fetch(b + 2, g0, u0);
            batch(b + 1, g1, u1);
          }
        }
      });
      return;
    }
    static_for<NP>([&](auto P) {
      constexpr int ph = decltype(P)::value;
      fill(P);
      if (n >= p.N) return;
#pragma unroll 1
      for (int it = 0; it < IT; ++it) {
        const int r = it * RPI + r0, m = m0 + ph * PR + r;
        if (m >= p.M) break;
        const int64_t at = (int64_t)m * a.ld_act * C::ESZ;
        emit(ph, r, rows::load_chunk<T>(gate + at, n, p.N, 0), rows::load_chunk<T>(up + at, n, p.N, 0));
      }
    });
  }
}

template <typename C, int PR, int NP, typename Fill>
__device__ __forceinline__ void finish(const Args<C::NG>& a, const Problem& p, int m0, int n0, const float* stage,
                                       Fill fill) {
  if (C::EPI == EPI_PLAIN || a.activation == 0) finish_rows<C, PR, NP, 0>(a, p, m0, n0, stage, fill);
  else finish_rows<C, PR, NP, 1>(a, p, m0, n0, stage, fill);
}

// Block b of a problem's nblocks.  lds: C::LDS chunks.
template <typename C>
__device__ __forceinline__ void tile_block(const Args<C::NG>& a, const Problem& p, int b, int nblocks,
                                           u32x4* const lds) {
  using T = typename C::type;
  constexpr int FMH = C::FM / 2, FNH = C::FN / 2;
  constexpr int NA = C::BM * C::CPR, NB = C::BN * C::CPR;  // chunks of a stage
  u32x4* const lds_a[2] = {lds, lds + NA};
  u32x4* const lds_b[2] = {lds + 2 * NA, lds + 2 * NA + NB};
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave / C::WGN, wn = wave % C::WGN;

  const int unit = xcd_contiguous(b, nblocks);
  const int L = unit / a.split, part = unit % a.split;
  int ti, tj;
  tile_at(p, L, ti, tj);
  const int m0 = ti * C::BM, n0 = tj * C::CN;

  const int kt = (p.K + C::KTE - 1) / C::KTE;  // slices per segment
  const int all = kt * C::NSEG;
  // parts of whole pairs of slices, as the loop takes them: a slice after the
  // last one is past the operands' end
  const int pairs = (all + 1) / 2;
  const int s0 = 2 * (int)((int64_t)part * pairs / a.split), s1 = 2 * (int)((int64_t)(part + 1) * pairs / a.split);
  const int nk = s1 - s0;
  Loader<C, C::BM, C::AKM, false> la;
  Loader<C, C::BN, C::BKM, true> lb;
  const int seg0 = C::NSEG > 1 && s0 >= kt ? 1 : 0;
  la.init(p, m0, seg0, (s0 - seg0 * kt) * C::KTE);
  lb.init(p, n0, seg0, (s0 - seg0 * kt) * C::KTE);
  int to_switch = C::NSEG > 1 && seg0 == 0 ? kt - s0 : -1;  // slices before segment 1

  f32x4 acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // load instruction i of a slice into stage S, A's and then B's
  const uint32_t lds0_a = (uint32_t)(uintptr_t)MSIGN_LDS(&lds_a[0][wave * 64]);
  const uint32_t lds0_b = (uint32_t)(uintptr_t)MSIGN_LDS(&lds_b[0][wave * 64]);
  auto load = [&](auto I, auto S) {
    constexpr int i = decltype(I)::value, st = decltype(S)::value;
    if constexpr (i < C::ACH) la.template load<i>(lds0_a + st * NA * 16);
    else if constexpr (i < C::ACH + C::BCH) lb.template load<i - C::ACH>(lds0_b + st * NB * 16);
  };
  auto begin = [&] {
    const bool sw = C::NSEG > 1 && to_switch == 0;
    la.begin(p, sw);
    lb.begin(p, sw);
    --to_switch;
  };
  auto next = [&] {
    la.next();
    lb.next();
  };
  auto issue = [&](auto S) {
    begin();
    static_for<C::ACH + C::BCH>([&](auto I) { load(I, S); });
    next();
  };
  Reader<C, C::WM, C::BM, C::AKM> ra;
  Reader<C, C::WN, C::BN, C::BKM> rb;
  ra.init(wm);
  rb.init(wn);
  // Quadrant (hm, hn): after each of its products at most one step of
  // between(i), i = 0, 1, ..., and nothing else: the order is kept as written.
  // (fp32: a fragment is four products, each over all fragments before the
  // next, so that none waits for the one before it)
  constexpr int E = C::ESZ == 4 ? 4 : 1;
  constexpr int MQ = FMH * FNH * C::KSUB * E;
  auto multiply = [&](auto HM, auto HN, const u32x4 (&fa)[FMH * C::KSUB], const u32x4 (&fb)[FNH * C::KSUB],
                      auto between) {
    constexpr int hm = decltype(HM)::value, hn = decltype(HN)::value;
    static_for<MQ>([&](auto I) {
      constexpr int i = decltype(I)::value, kk = i / (E * FMH * FNH), e = i / (FMH * FNH) % E, fn = i / FMH % FNH,
                    fm = i % FMH;
      f32x4& c = acc[hm * FMH + fm][hn * FNH + fn];
      const u32x4 &b = fb[kk * FNH + fn], &a = fa[kk * FMH + fm];
      if constexpr (E == 1) mma<T>(c, b, a);
      else mma_f32(c, __builtin_bit_cast(f32x4, b)[e], __builtin_bit_cast(f32x4, a)[e]);
      between(I);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  auto nothing = [](auto) {};
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;

  // Slice j lies in stage j & 1, and its quadrants (A half, B half) are
  // multiplied in the order (0,0), (0,1), (1,1), (1,0).  The last one's
  // fragments are in registers while the next slice's first halves are read
  // (B's into y, free by then: x and y change places every slice); the second
  // halves are read during the first quadrant.  Two barriers a slice:
  //   - early in the second quadrant, when every wave has read all of the
  //     slice: its stage takes the slice after the next, whose loads are spread
  //     over this quadrant and the next two (in a burst they stall the wave at
  //     the memory pipe's rate of one load per 16 cycles and CU);
  //   - after the third quadrant, when every wave's loads of the next slice
  //     have landed: those older than the ones issued in this slice.
  u32x4 a0[FMH * C::KSUB], a1[FMH * C::KSUB], bx[FNH * C::KSUB], by[FNH * C::KSUB];
  constexpr int RA = FMH * C::KSUB, RB = FNH * C::KSUB;  // reads of a half
  constexpr int V = C::ACH + C::BCH, V2 = V / 3, V3 = V - 2 * V2;  // loads in the second, third (and fourth) quadrant
  constexpr int RS = MQ / (RA + RB);                              // products per read
  constexpr int BAR = MQ / 8;                                     // products before the second quadrant's barrier
  static_assert(RS >= 1 && V3 <= MQ - BAR, "reads and loads of a quadrant");
  // At product i of MQ: the n-th of `count` loads, evenly from product `from` on.
  auto spread = [&](auto I, auto From, auto Count, auto First, auto S) {
    constexpr int i = decltype(I)::value, from = decltype(From)::value, count = decltype(Count)::value;
    constexpr int step = (MQ - from) / count, n = (i - from) / step;
    if constexpr (i >= from && (i - from) % step == 0 && n < count)
      load(std::integral_constant<int, decltype(First)::value + n>{}, S);
  };
  // quadrants (0,0), (0,1), (1,1) of the slice in stage S
  auto three = [&](auto S, u32x4 (&b0)[FNH * C::KSUB], u32x4 (&b1)[FNH * C::KSUB]) {
    constexpr int st = decltype(S)::value;
    multiply(I0{}, I0{}, a0, b0, [&](auto I) {
      constexpr int i = decltype(I)::value;
      if constexpr (i % RS == 0) {
        if constexpr (i / RS < RB) rb.template read<1, i / RS>(lds_b[st], b1);
        else if constexpr (i / RS - RB < RA) ra.template read<1, i / RS - RB>(lds_a[st], a1);
      }
    });
    multiply(I0{}, I1{}, a0, b1, [&](auto I) {
      constexpr int i = decltype(I)::value;
      if constexpr (i == BAR - 1) {
        reads_barrier();
        begin();
      }
      spread(I, std::integral_constant<int, BAR>{}, std::integral_constant<int, V2>{}, I0{}, S);
    });
    multiply(I1{}, I1{}, a1, b1, [&](auto I) {
      spread(I, I0{}, std::integral_constant<int, V3>{}, std::integral_constant<int, V2>{}, S);
    });
    loads_barrier<V2 + V3>();
  };
  // read i of the first halves of the slice in stage S, in the order of their use
  auto first_half = [&](auto I, auto S, u32x4 (&b)[FNH * C::KSUB]) {
    constexpr int i = decltype(I)::value, kk = i / (FMH + FNH), f = i % (FMH + FNH), st = decltype(S)::value;
    if constexpr (kk >= C::KSUB) return;
    else if constexpr (f < FMH) ra.template read<0, kk * FMH + f>(lds_a[st], a0);
    else rb.template read<0, kk * FNH + f - FMH>(lds_b[st], b);
  };
  // the last quadrant of the slice before, then those of the one in stage S
  auto trip = [&](auto S, u32x4 (&x)[FNH * C::KSUB], u32x4 (&y)[FNH * C::KSUB]) {
    using Before = std::integral_constant<int, 1 - decltype(S)::value>;
    ra.refresh();
    rb.refresh();
    multiply(I1{}, I0{}, a1, x, [&](auto I) {
      constexpr int i = decltype(I)::value;
      if constexpr (i % RS == 0) first_half(std::integral_constant<int, i / RS>{}, S, y);
      spread(I, std::integral_constant<int, MQ / 8>{}, std::integral_constant<int, V2>{},
             std::integral_constant<int, V2 + V3>{}, Before{});
    });
    next();
    three(S, y, x);
  };
  if (nk > 0) {
    issue(I0{});
    issue(I1{});
    loads_barrier<V>();
    static_for<RA + RB>([&](auto I) { first_half(I, I0{}, bx); });
    settle(acc);
    three(I0{}, bx, by);
    // (slices come in pairs; the last one may be past the end: all zeros)
    trip(I1{}, bx, by);
    for (int j = 2; j < nk; j += 2) {
      trip(I0{}, by, bx);
      trip(I1{}, bx, by);
    }
    multiply(I1{}, I0{}, a1, by, nothing);
    settle(acc);
    loads_barrier<0>();  // the slices past the end
  }

  if (a.split > 1) {
    // [tile][part][fragment row][fragment][thread]
    f32x4* dst = reinterpret_cast<f32x4*>(a.partial) + ((int64_t)L * a.split + part) * (C::FM * C::FN * C::NT) +
                 threadIdx.x;
#pragma unroll
    for (int fm = 0; fm < C::FM; ++fm) {
      if (m0 + wm * C::WM + fm * 16 >= p.M) break;  // (the reduce pass skips these rows too)
#pragma unroll
      for (int fn = 0; fn < C::FN; ++fn) dst[(fm * C::FN + fn) * C::NT] = acc[fm][fn];
    }
    return;
  }
  constexpr int PR = C::WM < 64 ? C::WM : 64;
  static_assert(C::NT / 64 * PR * C::WN * 4 <= C::LDS * 16, "stage");
  float* stage = reinterpret_cast<float*>(lds) + wave * (PR * C::WN);
  constexpr int NP = C::WM / PR;
  finish<C, PR, NP>(a, p, m0 + wm * C::WM, n0 + wn * (C::DUAL ? C::WN / 2 : C::WN), stage, [&](auto P) {
    static_for<PR / 16>([&](auto I) {
      constexpr int i = decltype(I)::value;
      stage_rows<C>(stage, i * 16, acc[decltype(P)::value * (PR / 16) + i]);
    });
  });
}

// Block b of all problems.
template <typename C>
__device__ __forceinline__ void problem_block(const Args<C::NG>& a, int b, int nblocks, u32x4* lds) {
  int gi = 0;
#pragma unroll
  for (int i = 1; i < C::NG; ++i) gi += b >= a.bstart[i] ? 1 : 0;
  const int first = a.bstart[gi];
  const int next = gi + 1 < C::NG ? a.bstart[gi + 1] : nblocks;
  tile_block<C>(a, a.g[gi], b - first, next - first, lds);
}

template <typename C>
__global__ void __launch_bounds__(C::NT) tile_kernel(const Args<C::NG> args) {
  __shared__ u32x4 lds[C::LDS];
  // read in place: indexing the by-value argument would copy it to scratch
  const Args<C::NG>& a = *(const Args<C::NG>*)__builtin_amdgcn_kernarg_segment_ptr();
  problem_block<C>(a, blockIdx.x, gridDim.x, lds);
}

// Two independent launches in one, so that one's blocks fill the CUs that the
// other's last round leaves (f16, 777 tokens of 1000 x 2730: 43 us, one after the
// other 51).
template <typename CA, typename CB>
struct Pair {
  Args<CA::NG> a;
  Args<CB::NG> b;
  int32_t na, nb;   // blocks
  int32_t b_first;  // b's blocks come first
};

template <typename CA, typename CB>
__global__ void __launch_bounds__(CA::NT) pair_kernel(const Pair<CA, CB> args) {
  static_assert(CA::NT == CB::NT, "threads");
  __shared__ u32x4 lds[CA::LDS > CB::LDS ? CA::LDS : CB::LDS];
  const Pair<CA, CB>& p = *(const Pair<CA, CB>*)__builtin_amdgcn_kernarg_segment_ptr();
  const int b = blockIdx.x, first = p.b_first ? p.nb : p.na;
  if ((b < first) == (p.b_first != 0)) problem_block<CB>(p.b, p.b_first ? b : b - first, p.nb, lds);
  else problem_block<CA>(p.a, p.b_first ? b - first : b, p.na, lds);
}

// Adds the parts of split tiles in part order and runs the epilogue: block
// (tile, fragment row).  One problem only.
template <typename C>
__global__ void __launch_bounds__(C::NT) reduce_kernel(const Args<C::NG> a) {
  const Problem& p = a.g[0];
  const int L = blockIdx.x / C::FM, fm = blockIdx.x % C::FM;
  __shared__ float stages[C::NT / 64][16 * C::WN];
  const int wave = threadIdx.x >> 6;
  const int wm = wave / C::WGN, wn = wave % C::WGN;
  int ti, tj;
  tile_at(p, L, ti, tj);
  const int row0 = ti * C::BM + wm * C::WM + fm * 16;
  if (row0 >= p.M) return;  // whole waves; there is no barrier below
  constexpr int STEP = C::FM * C::FN * C::NT;
  const f32x4* src = reinterpret_cast<const f32x4*>(a.partial) + (int64_t)L * a.split * STEP +
                     fm * C::FN * C::NT + threadIdx.x;
  f32x4 acc[C::FN];
#pragma unroll
  for (int fn = 0; fn < C::FN; ++fn) acc[fn] = src[fn * C::NT];
  int s = 1;
  for (; s + 4 <= a.split; s += 4) {  // four parts in flight
    f32x4 t[4][C::FN];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int fn = 0; fn < C::FN; ++fn) t[q][fn] = src[(int64_t)(s + q) * STEP + fn * C::NT];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int fn = 0; fn < C::FN; ++fn) acc[fn] += t[q][fn];
  }
  for (; s < a.split; ++s)
#pragma unroll
    for (int fn = 0; fn < C::FN; ++fn) acc[fn] += src[(int64_t)s * STEP + fn * C::NT];
  float* stage = stages[wave];
  finish<C, 16, 1>(a, p, row0, tj * C::CN + wn * (C::DUAL ? C::WN / 2 : C::WN), stage,
                   [&](auto) { stage_rows<C>(stage, 0, acc); });
}

// Copies a [rows, cols] matrix into rows of `ldo` elements (a multiple of 16
// bytes, at least cols), zeros in the columns from cols on.
template <typename T>
__global__ void __launch_bounds__(256) pad_copy_kernel(const T* src, int64_t ld, T* dst, int64_t ldo, int64_t rows,
                                                       int32_t cols) {
  constexpr int CE = 16 / (int)sizeof(T);
  const int64_t per = ldo / CE;
  const int64_t total = rows * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per;
    const int c = (int)(i - r * per) * CE;
    T v[CE];
#pragma unroll
    for (int e = 0; e < CE; ++e) v[e] = c + e < cols ? src[r * ld + c + e] : T(0);
    u32x4 w;
    __builtin_memcpy(&w, v, 16);
    *reinterpret_cast<u32x4*>(dst + r * ldo + c) = w;
  }
}

// ---- launch plan (host) ----

// One product launch: rows of a tile, chunks of 16 bytes in a K slice and parts
// of the sum over K.
struct Plan {
  int rows, cpr;
  int split;
  size_t partial_bytes;
  int64_t blocks;
  double block_us;  // the model's time of a block
};

// Products by their operands' layout and epilogue.
enum Kind : int { K_GATED = 0, K_DOWN = 1, K_DGATED = 2 };

// Runs ng problems (tiles_* are filled in here); args holds everything else.
hipError_t launch(int32_t dtype, Kind kind, const Plan& plan, Args<kMaxProblems> args, int ng, hipStream_t st);
// Runs the product of dx (one problem) and those of the weights' gradients (three).
hipError_t launch_dx_dw(int32_t dtype, const Plan& plan_dx, const Plan& plan_dw, const Args<kMaxProblems>& dx,
                        const Args<kMaxProblems>& dw, hipStream_t st);
hipError_t launch_dx_dw_bf16(const Plan& plan_dx, const Plan& plan_dw, const Args<kMaxProblems>& dx,
                             const Args<kMaxProblems>& dw, hipStream_t st);
hipError_t launch_dx_dw_f16(const Plan& plan_dx, const Plan& plan_dw, const Args<kMaxProblems>& dx,
                            const Args<kMaxProblems>& dw, hipStream_t st);
hipError_t launch_dx_dw_f32(const Plan& plan_dx, const Plan& plan_dw, const Args<kMaxProblems>& dx,
                            const Args<kMaxProblems>& dw, hipStream_t st);
hipError_t launch_bf16(Kind kind, const Plan& plan, const Args<kMaxProblems>& args, int ng, hipStream_t st);
hipError_t launch_f16(Kind kind, const Plan& plan, const Args<kMaxProblems>& args, int ng, hipStream_t st);
hipError_t launch_f32(Kind kind, const Plan& plan, const Args<kMaxProblems>& args, int ng, hipStream_t st);

}  // namespace ffn
}  // namespace msign
