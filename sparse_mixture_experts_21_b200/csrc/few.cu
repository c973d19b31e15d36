// A whole MoE layer for few tokens (1 .. 64), in one launch: router, top-k, routed and
// shared experts, weighted sum.
//
//   y_t = sum_j w_tj W2_e (silu(W1_e x_t) * (W3_e x_t)) + shared(x_t)
//
// Bound: the bytes of the weights of the experts that at least one token picks (and of the
// router and the shared expert); every weight is read once from HBM, or once for each 32 of an
// expert's tokens (all CTAs' tiles together outgrow the L2 before the next 32 need them).
//
// One cooperative launch, one CTA per SM, barriers over the grid:
//   logits     spread over the grid in K slices; arrive at barrier 1
//   shared     the shared experts' gate/up rows, cut evenly over the grid: they do not
//              depend on the routing
//   selection  meanwhile one warp waits at barrier 1, selects (token t on CTA t; one or two
//              tokens on every CTA) and builds the experts' token lists
//   gate/up    the met experts' hidden units, cut evenly over the grid
//   -- barrier 2 --
//   down       each CTA takes rows of W2 of all met experts, so a token's sum over its
//              experts stays inside one CTA: fixed order, no atomics, no second pass
//
// One warp streams the weights through a ring of shared-memory stages with TMA, 8 or 32 rows by
// 512 bytes a copy (at 512 bytes a copy, the engine's ~57 cycles for one would hold the stream
// to 2.5 TB/s), and runs ahead of the phases: the first down stages' weights are in
// flight while the CTA waits at barrier 2 for the hidden rows.  Two warps gather the same
// columns of the expert's tokens with cp.async.  Sixteen warps multiply with mma.sync
// m16n8k16: 16 weight rows by 8 tokens, which leaves nothing to gain from tcgen05 (its
// smallest tile is 128 rows, and no tensor pipe is near its limit: at 8 tokens a weight is
// used 8 times, two orders below what the pipes need to be the bound).  The order of k
// inside a fragment is free as long as both operands use it, so a thread feeds the MMA with
// its own 16-byte loads and no shuffles.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "few_common.cuh"

namespace moe {

namespace few {

constexpr int WARPS = WORKERS;                  // consumer warps
constexpr int X_WARPS = 2;                      // warps that gather tokens' columns
constexpr int W_WARP = WARPS, X_WARP0 = WARPS + 1, SELECT_WARP = X_WARP0 + X_WARPS;
constexpr int CONSUMERS = 32 * WARPS, THREADS = 32 * (SELECT_WARP + 1);

struct Maps {
  CUtensorMap m[6][2][2];  // boxes of a stage's columns (for 16 tokens, for 32) by 8 and by 32 rows
};

// Per weight type W (fp32 and bf16: x and weights; Mxfp4: bf16 x).  nt: 8-token columns of a
// pass (1, 2 or 4); seg(nt): columns of a stage.  A stage holds up to 64 weight rows as TMA
// leaves them (fp32, bf16: row by row, 32 gate rows before 32 up rows; MXFP4, in groups of 8
// rows: by 64-byte column chunks, the chunk's 8 rows, 64-byte swizzle, so that the 16 bytes
// that a quad takes of each of 8 rows fall into different banks), then the tokens' rows, 64 mod 128 bytes apart so that a quarter warp's
// 16-byte reads meet every bank once, then MXFP4's scales, 36 bytes a row.
// WK warps split a stage's columns, WARPS / WK its 16-row tiles.
struct Mxfp4 {};
template <typename W>
struct Cfg {
  using XT = W;
  static constexpr bool MX = false, SPLIT = true;
  static constexpr int STAGES = 4, WK = 4, RED = 2, GATE_UNITS = 4, PASS = 32, EB = sizeof(W);
  static __host__ __device__ constexpr int seg(int nt) { return (nt == 4 ? 256 : 512) / EB; }
  static __host__ __device__ constexpr int wbytes(int c) { return EB * c; }
};
template <>
struct Cfg<Mxfp4> {
  using XT = __nv_bfloat16;
  static constexpr bool MX = true, SPLIT = false;
  static constexpr int STAGES = 3, WK = 16, RED = 1, GATE_UNITS = 4, PASS = 32, EB = 2;
  static __host__ __device__ constexpr int seg(int nt) { return nt == 1 ? 1024 : 512; }
  static __host__ __device__ constexpr int wbytes(int c) { return c / 2; }
};
constexpr int SF_LD = 36;
template <class C> __host__ __device__ constexpr int wstride(int nt) { return C::wbytes(C::seg(nt)); }
template <class C> __host__ __device__ constexpr int xstride(int nt) { return C::EB * C::seg(nt) + 64; }
template <class C> __host__ __device__ constexpr int stage_use(int nt) {
  return SLOTS * wstride<C>(nt) + 8 * nt * xstride<C>(nt) + (C::MX ? SLOTS * SF_LD : 0);
}
template <class C> __host__ __device__ constexpr int stage_bytes() {
  int n = stage_use<C>(1) > stage_use<C>(2) ? stage_use<C>(1) : stage_use<C>(2);
  n = n > stage_use<C>(4) ? n : stage_use<C>(4);
  if (C::SPLIT) {                               // two ranges of 16 rows
    const int m = 32 * wstride<C>(1) + 8 * (2 * C::EB * C::seg(1) + 64);
    n = n > m ? n : m;
  }
  return (n + 511) / 512 * 512;
}
constexpr int RED_LD = SLOTS + 4;               // partial sums [token][row], padded: 32 banks
template <class C> __host__ __device__ constexpr int red_floats() { return C::WK * 8 * RED_LD; }
constexpr int YACC = MAX_T * SLOTS;             // a down tile's outputs
template <class C>
constexpr int smem_bytes() {
  return 1024 + C::STAGES * stage_bytes<C>() + (C::RED * red_floats<C>() + YACC) * 4 + (int)sizeof(Tables);
}
static_assert(alignof(Tables) == 16 && red_floats<Cfg<__nv_bfloat16>>() % 4 == 0 && red_floats<Cfg<Mxfp4>>() % 4 == 0 &&
              YACC % 4 == 0, "16-byte copies into the tables");
static_assert(smem_bytes<Cfg<__nv_bfloat16>>() <= 232448 && smem_bytes<Cfg<float>>() <= 232448 &&
              smem_bytes<Cfg<Mxfp4>>() <= 232448, "shared memory per CTA");
static_assert(8 * ROUTE_COLS <= 2 * red_floats<Cfg<float>>() + YACC && 8 * ROUTE_COLS <= red_floats<Cfg<Mxfp4>>() + YACC,
              "the router's tokens lie over the partial sums and the output tile");

// Row (within the expert) of slot s (0 .. 63) of a stage, or -1.  Down: 64 rows in order;
// gate/up: 8 gate rows, then the same 8 units' up rows, four times.
template <bool DOWN>
__device__ __forceinline__ int slot_row(const Tile& t, int s) {
  const int r = DOWN ? s : 8 * (s >> 4) + (s & 7);
  return r < 8 * t.nu ? t.base + r : -1;
}

// Weights of the stage at column k0, by one thread, in boxes of 32 rows and of 8 (MXFP4: 8);
// m[0], m[1]: the 8-row and the 32-row map.  Columns past K arrive as zeros and count as bytes.
// The thread's own steps would bound the stream (eight 8-row copies a stage took 5% longer
// than two 32-row ones), so there are few and none in loops where the tile is full.
template <class C>
__device__ __forceinline__ void load_box(const CUtensorMap* m, uint8_t* dst, uint64_t* bar, int k0, int row,
                                         uint64_t policy) {
  if (C::MX) tma_load_3d(m, dst, bar, 0, row, k0 >> 7, policy);
  else tma_load_2d(m, dst, bar, k0, row, policy);
}
template <class C, bool DOWN>
__device__ __forceinline__ void issue_w(const CUtensorMap* ma, const CUtensorMap* mb, const Tile& t, int k0, int box,
                                        uint8_t* dst, uint64_t* bar, uint64_t policy) {
  const int row = t.erow + t.base;
  if (DOWN) {
    mbar_arrive_expect_tx(bar, t.sub * t.nu * box);
    if (C::SPLIT && t.sub == 2) {                // one or two boxes, two column ranges
      load_box<C>(ma, dst, bar, k0, row, policy);
      load_box<C>(ma, dst + t.nu * box, bar, k0 + C::seg(1), row, policy);
      if (t.nu == 2) {
        load_box<C>(ma, dst + box, bar, k0, row + 8, policy);
        load_box<C>(ma, dst + 3 * box, bar, k0 + C::seg(1), row + 8, policy);
      }
      return;
    }
    int i = 0;
    if (!C::MX && t.nu >= 4) {
      load_box<C>(ma + 1, dst, bar, k0, row, policy);
      i = 4;
      if (t.nu == 8) {
        load_box<C>(ma + 1, dst + 4 * box, bar, k0, row + 32, policy);
        i = 8;
      }
    }
#pragma unroll 1
    for (; i < t.nu; ++i) load_box<C>(ma, dst + i * box, bar, k0, row + 8 * i, policy);
  } else {
    mbar_arrive_expect_tx(bar, 2 * t.nu * box);
    // gate and up rows: MXFP4 8 and 8 in turn, else 32 after 32
    if (!C::MX && t.nu == 4) {
      load_box<C>(ma + 1, dst, bar, k0, row, policy);
      load_box<C>(mb + 1, dst + 4 * box, bar, k0, row, policy);
    } else if (C::MX && t.nu == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        load_box<C>(ma, dst + 2 * i * box, bar, k0, row + 8 * i, policy);
        load_box<C>(mb, dst + (2 * i + 1) * box, bar, k0, row + 8 * i, policy);
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < t.nu; ++i) {
        load_box<C>(ma, dst + (C::MX ? 2 * i : i) * box, bar, k0, row + 8 * i, policy);
        load_box<C>(mb, dst + (C::MX ? 2 * i + 1 : i + 4) * box, bar, k0, row + 8 * i, policy);
      }
    }
  }
}
__device__ __forceinline__ void cp_async4(uint32_t smem_dst, const void* gsrc) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_dst), "l"(gsrc) : "memory");
}
// With 8 tokens or fewer, the down pass gives every token its own column whatever the expert:
// a warp then keeps the weighted sum over the experts in its registers and the warps' sums
// meet once a tile instead of once an expert.  Row of token c of the expert, or -1.
__device__ __forceinline__ bool by_token(const Args& a) { return a.T <= 8; }
__device__ __forceinline__ int row_of_token(const Tables& tb, const Tile& t, int c) {
  if (t.sh) return c < t.n ? c : -1;
  int r = -1;
  for (int i = 0; i < t.n; ++i)
    if (tb.row_tok[t.row + i] == c) r = i;
  return r;
}

// The token warps' part of a pass, set up once per tile so that a stage costs few instructions
// (each is a warp's dependent step of five cycles or so, against the ~700 to 1400 cycles that
// a stage takes from HBM): the same columns of the pass's tokens (x gathered by token, or
// hidden rows) and, for MXFP4, the weight rows' scales.
template <class C, bool DOWN>
struct Gather {
  static constexpr int NTOK = 8 / X_WARPS, NSF = SLOTS / (4 * X_WARPS);
  const uint8_t* tok[NTOK];              // this warp's first tokens: xw, xw + X_WARPS, ..
  const uint8_t* sf[C::MX ? NSF : 1];    // this lane's weight rows' scales, column block lane % 8; null: none
  int xs_ld;
  uint32_t xs, sd;                       // offsets in the stage

  __device__ __forceinline__ const uint8_t* token(const Args& a, const Tables& tb, const Tile& t, int i) const {
    using XT = typename C::XT;
    if (DOWN)
      return reinterpret_cast<const uint8_t*>(static_cast<const XT*>(a.h) + (t.sh ? (size_t)a.T * a.k * a.f : 0) +
                                              (size_t)(t.row + i) * t.K);
    return reinterpret_cast<const uint8_t*>(static_cast<const XT*>(C::MX ? a.x16 : a.x) +
                                            (size_t)(t.sh ? t.row + i : tb.row_tok[t.row + i]) * t.K);
  }
  __device__ __forceinline__ void tile(const Args& a, const Tables& tb, const Tile& t, int xw, int lane) {
    xs_ld = C::EB * t.seg + 64;
    // after the weights: 64 rows, or two ranges of 16
    xs = t.sub == 2 ? 32 * C::wbytes(t.seg / 2) : SLOTS * C::wbytes(t.seg);
#pragma unroll
    for (int m = 0; m < NTOK; ++m) {
      const int c = xw + X_WARPS * m;            // the stage's token row
      const int i = DOWN && by_token(a) ? row_of_token(tb, t, c) : c < t.n ? c : -1;
      tok[m] = i >= 0 ? token(a, tb, t, i) + 16 * lane : nullptr;
    }
    xs += xw * xs_ld + 16 * lane;
    if (C::MX) {
      const int s0 = 4 * xw + (lane >> 3), kb = lane & 7;
      sd = SLOTS * C::wbytes(t.seg) + 8 * t.nt * xs_ld + SF_LD * s0 + 4 * kb;
#pragma unroll
      for (int m = 0; m < NSF; ++m) {
        const int s = s0 + 4 * X_WARPS * m, r = slot_row<DOWN>(t, s), row = t.erow + r;
        sf[m] = r < 0 ? nullptr
                      : a.sf[(DOWN || !(s & 8)) ? t.ma : t.mb] + mx::atom_byte(row >> 7, t.K / 128, kb, row & 127, 0);
      }
    }
  }
  __device__ __forceinline__ void stage(const Args& a, const Tables& tb, const Tile& t, int k0, uint32_t st, int xw,
                                        int lane) const {
    const int cols = min(t.seg, t.K - k0), bytes = cols * C::EB, off = k0 * C::EB;
#pragma unroll
    for (int m = 0; m < NTOK; ++m)
      if (tok[m])
        for (int c = 0; c + 16 * lane < bytes; c += 512)
          cp_async16(st + xs + m * X_WARPS * xs_ld + c, tok[m] + off + c);
    for (int i = xw + 8; i < t.n; i += X_WARPS) {
      const uint8_t* p = token(a, tb, t, i) + 16 * lane + off;
      for (int c = 0; c + 16 * lane < bytes; c += 512) cp_async16(st + xs + (i - xw) * xs_ld + c, p + c);
    }
    if (C::MX && (lane & 7) < cols / 128) {
      const int at = k0 * 4;                      // 512 bytes per 128 columns
#pragma unroll
      for (int m = 0; m < NSF; ++m)
        if (sf[m]) cp_async4(st + sd + 4 * X_WARPS * SF_LD * m, sf[m] + at);
    }
  }
};

// ------------------------------------------------------------------ products
// Plain loads and MMAs without side effects: the compiler may move a tile's loads over the
// products before them.
__device__ __forceinline__ uint4 lds16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ uint32_t lds4(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }
__device__ __forceinline__ uint32_t lds2(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }
__device__ __forceinline__ uint32_t lds1(const uint8_t* p) { return *p; }
// D += A B, 16 x 8 x 16, fp32 accumulators: rows g and g + 8, columns 2t and 2t + 1 of lane 4g + t.
__device__ __forceinline__ void mma_bf16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// D = A B + C in fp16.
__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void gather_sync() { asm volatile("bar.sync 2, %0;" ::"n"(32 * X_WARPS) : "memory"); }
// Two bf16 to fp16, times a power of two.
__device__ __forceinline__ uint32_t scaled_f16(uint32_t v, float s) {
  const __half2 h = __floats2half2_rn(__uint_as_float(v << 16) * s, __uint_as_float(v & 0xffff0000u) * s);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Scale bytes of two blocks to 2^(byte - 127) as two bf16: byte 0 to the subnormal 2^-127; 255
// (NaN) to an infinity, which times the zero codes of such a block is NaN.
__device__ __forceinline__ uint32_t scale_pair(uint32_t s) {
  return __vmaxu2(__byte_perm(s, 0, 0x4140) << 7, 0x00400040u);
}
// fp16 holds bf16's eight significant bits but not its range: a row goes to fp16 times the
// power of two that brings its largest value (given as bits) to [2^14, 2^15).  What falls
// below fp16's subnormals is then under 2^-39 of the row's largest.  The sum is multiplied by
// the inverse, exactly.
__device__ __forceinline__ float row_scale(uint32_t amax) {
  return __uint_as_float((uint32_t)min(268 - (int)(amax >> 23), 253) << 23);
}
__device__ __forceinline__ float inverse_pow2(float s) {
  return __uint_as_float((254u - (__float_as_uint(s) >> 23)) << 23);
}
// Scale of token i of the pass.
template <bool DOWN>
__device__ __forceinline__ float token_scale(const Tile& t, const Tables& tb, int i) {
  if (DOWN) return tb.hs[t.sh ? MAX_T * MAX_K + t.row + i : t.row + i];
  return tb.xs[t.sh ? t.row + i : tb.row_tok[t.row + i]];
}

// MXFP4: token t to fp16 on CTA t, once for all that multiply with it (in every product it was
// a sixth of their instructions), by the warps that gather.
__device__ __forceinline__ void x_to_f16(const Args& a, Tables& tb, int xw, int lane) {
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const uint4* row = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) + (size_t)t * a.d);
    uint4* out = reinterpret_cast<uint4*>(static_cast<__half*>(a.x16) + (size_t)t * a.d);
    uint32_t m = 0;
#pragma unroll 7
    for (int c = 32 * xw + lane; c < a.d / 8; c += 32 * X_WARPS) {
      const uint4 v = ldg_nc16(row + c);
      m = __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                               __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
    }
    m = __reduce_max_sync(0xffffffffu, max(m << 16, m & 0xffff0000u));
    if (lane == 0) tb.xmax[xw] = m;
    gather_sync();
    const float s = row_scale(max(tb.xmax[0], tb.xmax[1]));
#pragma unroll 7
    for (int c = 32 * xw + lane; c < a.d / 8; c += 32 * X_WARPS) {
      const uint4 v = ldg_nc16(row + c);
      out[c] = make_uint4(scaled_f16(v.x, s), scaled_f16(v.y, s), scaled_f16(v.z, s), scaled_f16(v.w, s));
    }
    if (xw == 0 && lane == 0) a.xscale[t] = s;
    __threadfence();
    gather_sync();
    if (xw == 0 && lane == 0) grid_arrive(a.bar + BAR_X);
  }
  if (lane == 0) grid_wait(a.bar + BAR_X, a.T, tb);
  __syncwarp();
}

// This warp's sums over a pass: a 16-row tile by 8 NT tokens on its share of the columns.
// result(q, n, c): 16-row tile q of the warp's, column n, laid out as mma.sync's accumulators.
// fold: adds the pass, times the weights of its columns' tokens, to the sum over passes, for
// the columns (of this lane's two) that hold a token: a weight that is not a number stays with
// its own expert's tokens.  cols: bits of the columns that hold a token.
template <typename W, bool DOWN, int NT>
struct Product {
  using C = Cfg<W>;
  static constexpr int QT = 1;
  float acc[NT][4], sum[1][4] = {};
  bool on[NT];                             // column 8 n + g
  __device__ __forceinline__ void init(const Tile&, const Tables&, int lane, uint32_t cols) {
#pragma unroll
    for (int i = 0; i < NT * 4; ++i) acc[0][i] = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) on[n] = (cols >> (8 * n + (lane >> 2))) & 1u;
  }
  __device__ __forceinline__ void fold(float w0, float w1, bool on0, bool on1, int) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i & 1 ? on1 : on0) sum[0][i] = fmaf(i & 1 ? w1 : w0, acc[0][i], sum[0][i]);
  }
  __device__ __forceinline__ void stage(const Tile& t, int k0, const uint8_t* st, int warp, int lane) {
    constexpr int SEG = C::seg(NT), WS = wstride<C>(NT), XS = xstride<C>(NT);
    const int q = warp & 3, kq = warp >> 2, g = lane >> 2, tq = lane & 3;
    int cols = t.K - k0, xs = XS;
    constexpr int UP = (DOWN ? 8 : 32) * WS;      // to the row of the tile's lower half
    const uint8_t *wa = st + ((DOWN ? 16 : 8) * q + g) * WS, *xa = st + SLOTS * WS;
    if (DOWN && NT == 1 && t.sub == 2) {         // tile row 0 for all: q takes a column range
      if (q > 1) return;
      cols -= q * SEG;
      wa = st + (8 * t.nu * q + g) * WS;
      xs = 2 * C::EB * SEG + 64;
      xa = st + 32 * WS + q * C::EB * SEG;
    } else if ((DOWN ? 2 : 1) * q >= t.nu) {
      return;
    }
    xa += g * xs;
#pragma unroll
    for (int kk = 0; kk < SEG / 4; kk += 32) {
      const int c = kq * (SEG / 4) + kk + 8 * tq;
      const uint4 z = make_uint4(0, 0, 0, 0);
      const bool ok = c < cols;
      const uint4 a0 = ok ? lds16(wa + 2 * c) : z, a1 = ok ? lds16(wa + UP + 2 * c) : z;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 b = ok && on[n] ? lds16(xa + n * 8 * xs + 2 * c) : z;
        mma_bf16(acc[n], a0.x, a1.x, a0.y, a1.y, b.x, b.y);
        mma_bf16(acc[n], a0.z, a1.z, a0.w, a1.w, b.z, b.w);
      }
    }
  }
  __device__ __forceinline__ void result(int, int n, int, float* c) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = acc[n][i];
  }
};

// fp32: no tensor form keeps its bits.  A lane multiplies its 4 columns of rows g and g + 8 by
// all 8 tokens; the quad's partial sums meet at the tile's end.
template <bool DOWN, int NT>
struct Product<float, DOWN, NT> {
  using C = Cfg<float>;
  static constexpr int QT = 1;
  float acc[2][NT][8], sum[1][4] = {};
  uint32_t on;
  __device__ __forceinline__ void init(const Tile&, const Tables&, int, uint32_t cols) {
#pragma unroll
    for (int i = 0; i < 2 * NT * 8; ++i) acc[0][0][i] = 0.f;
    on = cols;
  }
  __device__ __forceinline__ void fold(float w0, float w1, bool on0, bool on1, int lane) {
    float c[4];
    result(0, 0, lane, c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i & 1 ? on1 : on0) sum[0][i] = fmaf(i & 1 ? w1 : w0, c[i], sum[0][i]);
  }
  __device__ __forceinline__ void stage(const Tile& t, int k0, const uint8_t* st, int warp, int lane) {
    constexpr int SEG = C::seg(NT), WS = wstride<C>(NT), XS = xstride<C>(NT);
    const int q = warp & 3, kq = warp >> 2, g = lane >> 2, tq = lane & 3;
    int cols = t.K - k0, xs = XS;
    constexpr int UP = (DOWN ? 8 : 32) * WS;      // to the row of the tile's lower half
    const uint8_t *wa = st + ((DOWN ? 16 : 8) * q + g) * WS, *xa = st + SLOTS * WS;
    if (DOWN && NT == 1 && t.sub == 2) {         // tile row 0 for all: q takes a column range
      if (q > 1) return;
      cols -= q * SEG;
      wa = st + (8 * t.nu * q + g) * WS;
      xs = 2 * C::EB * SEG + 64;
      xa = st + 32 * WS + q * C::EB * SEG;
    } else if ((DOWN ? 2 : 1) * q >= t.nu) {
      return;
    }
#pragma unroll 1
    for (int kk = 0; kk < SEG / 4; kk += 16) {
      const int c = kq * (SEG / 4) + kk + 4 * tq;
      if (c >= cols) continue;
      float w0[4], w1[4];
      unpack16(lds16(wa + 4 * c), w0, 0.f);
      unpack16(lds16(wa + UP + 4 * c), w1, 0.f);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (!((on >> (8 * n + j)) & 1u)) continue;
          float x[4];
          unpack16(lds16(xa + (8 * n + j) * xs + 4 * c), x, 0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[0][n][j] = fmaf(w0[i], x[i], acc[0][n][j]);
            acc[1][n][j] = fmaf(w1[i], x[i], acc[1][n][j]);
          }
        }
    }
  }
  __device__ __forceinline__ void result(int, int n, int lane, float* c) const {
    const int tq = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float v = acc[r][n][j];
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        if ((j >> 1) == tq) c[2 * r + (j & 1)] = v;
      }
  }
};

// MXFP4: a warp takes all four 16-row tiles on its share of the columns, so that a token's
// conversion to fp16 serves them all.  Codes go to fp16 exactly; a block's two MMAs make a
// sum of 32 columns, which the row's block scale multiplies in fp32.  About 35 instructions for
// the 512 codes of a 16-row tile's block, 16 of them the conversion of 4-bit codes; at HBM's rate
// a block arrives every 47 issue slots of an SM.  They would fit, but the warps issue in only 51%
// of the slots (24 tokens, 64 experts of 2048, d = 7168) with no pipe full: they wait for shared
// memory and for one another at the tiles' ends.  Without the products the call with 256 experts
// takes 575 us, with them 1 ms.  The block-scaled tensor cores take the codes as they are, but
// with the weights as the 128-row operand an M = 128 x K = 32 MMA costs ~200 cycles however few
// tokens there are, 800 for the 8.7 KB of codes that HBM brings in 357 (1.93 ms for 24 tokens);
// the weights as the 256-column operand are untried.
template <bool DOWN, int NT>
struct Product<Mxfp4, DOWN, NT> {
  using C = Cfg<Mxfp4>;
  static constexpr int QT = 4;
  float acc[4][NT][4], sum[DOWN && NT == 1 ? 4 : 1][4] = {};
  float ts[NT];                            // scale of column 8 n + g's token; 0: none
  __device__ __forceinline__ void init(const Tile& t, const Tables& tb, int lane, uint32_t) {
#pragma unroll
    for (int i = 0; i < 4 * NT * 4; ++i) acc[0][0][i] = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) ts[n] = 8 * n + (lane >> 2) < t.n ? token_scale<DOWN>(t, tb, 8 * n + (lane >> 2)) : 0.f;
  }
  // the sums of columns 2 tq and 2 tq + 1 without their rows' scales
  __device__ __forceinline__ void unscale(float s0, float s1) {
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i >> 2][0][i & 3] *= i & 1 ? s1 : s0;
  }
  // columns by token: row i (or -1) of column g
  __device__ __forceinline__ void scale_of(const Tile& t, const Tables& tb, int i) {
    ts[0] = i >= 0 ? token_scale<DOWN>(t, tb, i) : 0.f;
  }
  __device__ __forceinline__ void fold(float w0, float w1, bool on0, bool on1, int) {
#pragma unroll
    for (int q = 0; q < (DOWN && NT == 1 ? 4 : 1); ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i & 1 ? on1 : on0) sum[q][i] = fmaf(i & 1 ? w1 : w0, acc[q][0][i], sum[q][i]);
  }
  __device__ __forceinline__ void stage(const Tile& t, int k0, const uint8_t* st, int warp, int lane) {
    constexpr int SEG = C::seg(NT), WS = wstride<C>(NT), XS = xstride<C>(NT), BLOCKS = SEG / WARPS / 32;
    const int g = lane >> 2, tq = lane & 3;
    const int c0 = warp * (SEG / WARPS);
    if (c0 >= t.K - k0) return;              // whole 128-column blocks: uniform over the warp
    // 64-byte chunk c0 / 128 of the group's rows; its 16-byte unit (c0 / 32) % 4, swizzled
    const int unit = (c0 >> 5) & 3;
    const uint8_t *wa = st + 512 * (c0 >> 7) + 64 * g + 4 * tq;
    const uint8_t* xa = st + SLOTS * WS + g * XS + 16 * tq + 2 * c0;
    const uint8_t* sa = st + SLOTS * WS + 8 * NT * XS + SF_LD * g + (c0 >> 5);
    uint32_t b[BLOCKS][NT][4];
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 v = lds16(xa + n * 8 * XS + 64 * k);
        // a column without a token holds whatever the stage held before: zeros instead
        const bool on = ts[n] > 0.f;
        b[k][n][0] = !on ? 0u : DOWN ? scaled_f16(v.x, ts[n]) : v.x;
        b[k][n][1] = !on ? 0u : DOWN ? scaled_f16(v.y, ts[n]) : v.y;
        b[k][n][2] = !on ? 0u : DOWN ? scaled_f16(v.z, ts[n]) : v.z;
        b[k][n][3] = !on ? 0u : DOWN ? scaled_f16(v.w, ts[n]) : v.w;
      }
    const uint8_t* wu[BLOCKS];
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k) wu[k] = wa + 16 * ((unit + k) ^ ((g >> 1) & 3));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // scale bytes of this row and the one 8 below, for the warp's one or two blocks
      const uint32_t s0 = scale_pair(BLOCKS == 2 ? lds2(sa + 16 * SF_LD * q) : lds1(sa + 16 * SF_LD * q));
      const uint32_t s1 = scale_pair(BLOCKS == 2 ? lds2(sa + (16 * q + 8) * SF_LD) : lds1(sa + (16 * q + 8) * SF_LD));
#pragma unroll
      for (int k = 0; k < BLOCKS; ++k) {
        uint32_t a0[4], a1[4];
        mx4::e2m1_f16(lds4(wu[k] + 16 * q * WS), a0);
        mx4::e2m1_f16(lds4(wu[k] + (16 * q + 8) * WS), a1);
        const float f0 = __uint_as_float(k ? s0 & 0xffff0000u : s0 << 16);
        const float f1 = __uint_as_float(k ? s1 & 0xffff0000u : s1 << 16);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float p[4];
          mma_f16(p, a0[0], a1[0], a0[1], a1[1], b[k][n][0], b[k][n][1], 0.f, 0.f, 0.f, 0.f);
          mma_f16(p, a0[2], a1[2], a0[3], a1[3], b[k][n][2], b[k][n][3], p[0], p[1], p[2], p[3]);
          acc[q][n][0] = fmaf(p[0], f0, acc[q][n][0]);
          acc[q][n][1] = fmaf(p[1], f0, acc[q][n][1]);
          acc[q][n][2] = fmaf(p[2], f1, acc[q][n][2]);
          acc[q][n][3] = fmaf(p[3], f1, acc[q][n][3]);
        }
      }
    }
  }
  __device__ __forceinline__ void result(int q, int n, int, float* c) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = acc[q][n][i];
  }
};

// ------------------------------------------------------------------ range (MXFP4)
// The products multiply a row that is scaled to [2^14, 2^15) by the block scales and divide by the
// row's scale at the end: under block scales from about 2^105 the sum leaves fp32 on the way
// although it may be an ordinary number.  Dividing first would cost each block of each product
// four multiplications.  So what came out not finite is formed again when the phase is over, the
// factors in an order that leaves fp32 only where the sum does; finite results cost a comparison
// each.  (A scale byte 255 is NaN here; the products, for which it is an infinity, end up here
// with it.)  A row that holds an infinity or a NaN itself keeps what the products gave.
__device__ __forceinline__ bool finite_row(float scale) {        // row_scale(255 << 23): exponent field 13
  return (__float_as_uint(scale) >> 23) != 13u;
}
// Row `row` of a stack times v, whose scale is s, by one warp.
__device__ __noinline__ float dot_in_range(const uint8_t* q, const uint8_t* sf, int row, int K, const __nv_bfloat16* v,
                                           float s) {
  const int lane = threadIdx.x & 31;
  const float inv = inverse_pow2(s);
  const uint4* codes = reinterpret_cast<const uint4*>(q + (size_t)row * (K / 2));
  const uint4* x = reinterpret_cast<const uint4*>(v);
  float sum = 0.f;
#pragma unroll 1
  for (int b = lane; b < K / 32; b += 32) {
    const uint4 w = ldg_nc16(codes + b);
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
    float p = 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint32_t c[4];
      mx4::e2m1_f16(words[u], c);
      float xf[8];
      unpack16(__ldcg(x + 4 * b + u), xf, __nv_bfloat16());
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 cf = __half22float2(*reinterpret_cast<const __half2*>(&c[i]));
        p = fmaf(cf.x, xf[2 * i] * s, p);
        p = fmaf(cf.y, xf[2 * i + 1] * s, p);
      }
    }
    const uint32_t sb = sf[mx::atom_byte(row >> 7, K / 128, b >> 2, row & 127, b & 3)];
    sum = fmaf(p, mx4::e8m0_value(sb) * fminf(inv, 1.f), sum);
  }
  return warp_sum(sum) * fmaxf(inv, 1.f);
}
__device__ __forceinline__ float swiglu(float gate, float up) { return gate / (1.f + expf(-gate)) * up; }

// This CTA's hidden units of the shared or the routed part that are not finite, by the consumer
// warps (a token each); their share of the rows' maxima, which the tiles left out.
__device__ __noinline__ void hidden_in_range(const Args& a, const Tables& tb, bool shared) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t routed = (size_t)a.T * a.k * a.f;
  Tile t;
  for (Walk<Cfg<Mxfp4>, false> w(a, tb, shared); w.next(t);)
    for (int i = warp; i < t.n; i += WARPS) {
      const int tok = t.sh ? t.row + i : tb.row_tok[t.row + i];
      const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x) + (size_t)tok * a.d;
      __nv_bfloat16* h = static_cast<__nv_bfloat16*>(a.h) + (t.sh ? routed : 0) +
                         (size_t)(t.row + i) * (t.sh ? a.fs : a.f) + t.base;
      static_assert(8 * Cfg<Mxfp4>::GATE_UNITS == 32, "a lane per unit");
      float v = lane < 8 * t.nu ? __bfloat162float(__ldcg(h + lane)) : 0.f;
      const bool bad = !isfinite(v);
      const float s = tb.xs[tok];
      for (unsigned m = finite_row(s) ? __ballot_sync(0xffffffffu, bad) : 0u; m; m &= m - 1) {
        const int src = __ffs(m) - 1, row = t.erow + t.base + src;
        const float gate = dot_in_range(a.q[t.ma], a.sf[t.ma], row, t.K, x, s);
        const float up = dot_in_range(a.q[t.mb], a.sf[t.mb], row, t.K, x, s);
        if (lane == src) {
          const __nv_bfloat16 hx = __float2bfloat16_rn(swiglu(gate, up));
          h[lane] = hx;
          v = __bfloat162float(hx);
        }
      }
      if (bad) atomicMax(a.hmax + (t.sh ? a.T * a.k : 0) + t.row + i, __float_as_uint(fabsf(v)));
    }
}

// Output j of token tok, by one warp; v: what the products gave.
__device__ __noinline__ float output_in_range(const Args& a, const Tables& tb, int tok, int j, float v) {
  const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(a.h);
  float sum = 0.f;
  if (a.fs > 0) {
    const float s = tb.hs[MAX_T * MAX_K + tok];
    if (!finite_row(s)) return v;
    sum = tb.shw[tok] * dot_in_range(a.q[M_W2 + M_SHARED], a.sf[M_W2 + M_SHARED], j, a.fs,
                                     h + (size_t)a.T * a.k * a.f + (size_t)tok * a.fs, s);
  }
#pragma unroll 1
  for (int i = 0; i < tb.n_act; ++i) {
    const int e = tb.act[i];
#pragma unroll 1
    for (int r = tb.row0[e]; r < tb.row0[e + 1]; ++r) {
      if (tb.row_tok[r] != tok) continue;
      if (!finite_row(tb.hs[r])) return v;
      sum = fmaf(tb.row_w[r], dot_in_range(a.q[M_W2], a.sf[M_W2], e * a.d + j, a.f, h + (size_t)r * a.f, tb.hs[r]), sum);
    }
  }
  return sum;
}
// This CTA's outputs that are not finite, by the consumer warps (a token each).
__device__ __noinline__ void outputs_in_range(const Args& a, const Tables& tb) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Walk<Cfg<Mxfp4>, true> w(a, tb, false);
  for (int tok = warp; tok < a.T; tok += WARPS)
    for (int j0 = 8 * w.u; j0 < 8 * w.u1; j0 += 32) {
      __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + (size_t)tok * a.d + j0;
      const float v = j0 + lane < 8 * w.u1 ? __bfloat162float(__ldcg(y + lane)) : 0.f;
      for (unsigned m = __ballot_sync(0xffffffffu, !isfinite(v)); m; m &= m - 1) {
        const int src = __ffs(m) - 1;
        const float again = output_in_range(a, tb, tok, j0 + src, __shfl_sync(0xffffffffu, v, src));
        if (lane == src) y[lane] = __float2bfloat16_rn(again);
      }
    }
}

// One tile pass: all its stages, then the warps' partial sums through shared memory and the
// tile's results.  gate/up: h = silu(gate) * up to memory; down: weighted sums into yacc.
template <typename W, bool DOWN, int NT>
__device__ __forceinline__ void run_pass(const Args& a, Tables& tb, const Tile& t, Ring& r, const uint8_t* stages, float* red,
                                         float* yacc, int& buf) {
  using C = Cfg<W>;
  using XT = typename C::XT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Product<W, DOWN, NT> p;
  p.init(t, tb, lane, t.n < 32 ? (1u << t.n) - 1u : 0xffffffffu);
  for (int k0 = 0; k0 < t.K; k0 += t.seg) {
    wait(&tb.full[r.stage], r.phase, tb);
    p.stage(t, k0, stages + r.stage * stage_bytes<C>(), warp, lane);
    __syncwarp();
    if (lane == 0) mbar_arrive(&tb.empty[r.stage]);
    r.next(C::STAGES);
  }
  const int wk = p.QT == 4 ? warp : warp >> 2;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (8 * n >= t.n) break;
    float* rb = red + buf * red_floats<C>();
    // one buffer: the sums before these have been read (a meeting here and not after the reads
    // lets the warps that read nothing go on with the next tile: 1040 -> 1017 us for 24 tokens)
    if (C::RED == 1) worker_sync();
#pragma unroll
    for (int q = 0; q < p.QT; ++q) {
      float c[4];
      p.result(q, n, lane, c);
      float* o = rb + (wk * 8 + 2 * (lane & 3)) * RED_LD + 16 * (p.QT == 4 ? q : warp & 3) + (lane >> 2);
      o[0] = c[0];
      o[RED_LD] = c[1];
      o[8] = c[2];
      o[RED_LD + 8] = c[3];
    }
    worker_sync();
    if (DOWN) {
      // 64 rows by 8 tokens, one each
      const int i = 8 * n + (tid >> 6), s = tid & 63;
      if (i < t.n && slot_row<DOWN>(t, s) >= 0) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < C::WK; ++w) v += rb[(w * 8 + (tid >> 6)) * RED_LD + s];
        if (t.sub == 2)
#pragma unroll
          for (int w = 0; w < C::WK; ++w) v += rb[(w * 8 + (tid >> 6)) * RED_LD + s + 16];
        if (C::MX) v *= inverse_pow2(token_scale<DOWN>(t, tb, i));
        const int tok = t.sh ? t.row + i : tb.row_tok[t.row + i];
        yacc[tok * SLOTS + s] += v * (t.sh ? tb.shw[tok] : tb.row_w[t.row + i]);
      }
    } else if (tid < 256) {
      // 32 hidden units by 8 tokens: a warp per token
      const int i = 8 * n + warp, s = 16 * (lane >> 3) + (lane & 7);
      const int j = slot_row<DOWN>(t, s);
      float h = 0.f;
      if (i < t.n && j >= 0) {
        float gate = 0.f, up = 0.f;
#pragma unroll
        for (int w = 0; w < C::WK; ++w) {
          gate += rb[(w * 8 + warp) * RED_LD + s];
          up += rb[(w * 8 + warp) * RED_LD + s + 8];
        }
        if (C::MX) {
          const float inv = inverse_pow2(token_scale<DOWN>(t, tb, i));
          gate *= inv;
          up *= inv;
        }
        // the hidden row is rounded to x's type, as the rows of the other forms are: 2^-9 of a
        // value on average, beside the 2^-9 of the output's own rounding
        const XT hx = (XT)swiglu(gate, up);
        XT* hr = static_cast<XT*>(a.h) + (t.sh ? (size_t)a.T * a.k * a.f : 0);
        hr[(size_t)(t.row + i) * (t.sh ? a.fs : a.f) + j] = hx;
        h = fabsf((float)hx);
        if (C::MX && !isfinite(h)) {             // a sum that is not finite leaves no finite h
          tb.redo[0] = 1;
          h = 0.f;
        }
      }
      if (C::MX) {                               // the row's largest, for the down pass's fp16
        const unsigned m = __reduce_max_sync(0xffffffffu, __float_as_uint(h));
        if (lane == 0 && i < t.n) atomicMax(a.hmax + (t.sh ? a.T * a.k : 0) + t.row + i, m);
      }
    }
    if (C::RED == 2) buf ^= 1;
  }
}

template <typename W, bool DOWN>
__device__ __forceinline__ void run_tile(const Args& a, Tables& tb, const Tile& t, Ring& r, const uint8_t* stages,
                                         float* red, float* yacc, int& buf) {
  if (t.nt == 1) run_pass<W, DOWN, 1>(a, tb, t, r, stages, red, yacc, buf);
  else if (t.nt == 2) run_pass<W, DOWN, 2>(a, tb, t, r, stages, red, yacc, buf);
  else run_pass<W, DOWN, 4>(a, tb, t, r, stages, red, yacc, buf);
}

// Down with 8 tokens or fewer: all passes of a tile, columns by token, one meeting at the end.
// w: at the tile's first pass; t: its passes in turn.
template <typename W>
__device__ __forceinline__ void run_down_by_token(const Args& a, Tables& tb, Walk<Cfg<W>, true>& w, Ring& r,
                                                  const uint8_t* stages, float* red) {
  using C = Cfg<W>;
  using XT = typename C::XT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, T = a.T;
  XT* y = static_cast<XT*>(a.y);
  Product<W, true, 1> p;
  Tile t;
  while (w.next(t)) {
    // this lane's tokens: column g of the operand, columns 2 tq and 2 tq + 1 of the result
    uint32_t cols = 0;
    float w0 = 0.f, w1 = 0.f, s0 = 1.f, s1 = 1.f;
    int mine = -1;
    for (int i = 0; i < t.n; ++i) {
      const int tok = t.sh ? i : tb.row_tok[t.row + i];
      const float v = t.sh ? tb.shw[tok] : tb.row_w[t.row + i];
      // a product of the two could fall below fp32's normal numbers
      const float s = C::MX ? inverse_pow2(token_scale<true>(t, tb, i)) : 1.f;
      cols |= 1u << tok;
      if (tok == 2 * (lane & 3)) { w0 = v; s0 = s; }
      if (tok == 2 * (lane & 3) + 1) { w1 = v; s1 = s; }
      if (tok == (lane >> 2)) mine = i;
    }
    p.init(t, tb, lane, cols);
    if constexpr (C::MX) p.scale_of(t, tb, mine);
    for (int k0 = 0; k0 < t.K; k0 += t.seg) {
      wait(&tb.full[r.stage], r.phase, tb);
      p.stage(t, k0, stages + r.stage * stage_bytes<C>(), warp, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&tb.empty[r.stage]);
      r.next(C::STAGES);
    }
    if constexpr (C::MX) p.unscale(s0, s1);
    p.fold(w0, w1, (cols >> (2 * (lane & 3))) & 1u, (cols >> (2 * (lane & 3) + 1)) & 1u, lane);
    if (!t.last) continue;
    const int wk = p.QT == 4 ? warp : warp >> 2;
#pragma unroll
    for (int q = 0; q < p.QT; ++q) {
      float* o = red + (wk * 8 + 2 * (lane & 3)) * RED_LD + 16 * (p.QT == 4 ? q : warp & 3) + (lane >> 2);
      o[0] = p.sum[q][0];
      o[RED_LD] = p.sum[q][1];
      o[8] = p.sum[q][2];
      o[RED_LD + 8] = p.sum[q][3];
#pragma unroll
      for (int i = 0; i < 4; ++i) p.sum[q][i] = 0.f;
    }
    worker_sync();
    const int tok = tid >> 6, j = slot_row<true>(t, tid & 63);
    if (tok < T && j >= 0) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < C::WK; ++k) v += red[(k * 8 + tok) * RED_LD + (tid & 63)];
      if (t.sub == 2)
#pragma unroll
        for (int k = 0; k < C::WK; ++k) v += red[(k * 8 + tok) * RED_LD + (tid & 63) + 16];
      y[(size_t)tok * a.d + j] = (XT)v;
      if (C::MX && !isfinite(v)) tb.redo[1] = 1;
    }
    worker_sync();
  }
}

template <typename W>
__global__ void __launch_bounds__(THREADS, 1)
few_kernel(const __grid_constant__ Args a, const __grid_constant__ Maps maps) {
  using C = Cfg<W>;
  using XT = typename C::XT;
  using Gate = Walk<C, false>;
  using Down = Walk<C, true>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t stages = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (stages - smem_u32(smem_raw));
  float* red = reinterpret_cast<float*>(smem + C::STAGES * stage_bytes<C>());
  float* yacc = red + C::RED * red_floats<C>();
  Tables& tb = *reinterpret_cast<Tables*>(yacc + YACC);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = a.T;

  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&tb.full[s], 1 + 32 * X_WARPS);
      mbar_init(&tb.empty[s], WARPS);
    }
    tb.abort = 0;
    tb.n_act = 0;
    tb.redo[0] = tb.redo[1] = 0;
    fence_barrier_init();
  }
  __syncthreads();

  if (warp == W_WARP) {
    // ---------------------------------------------------------------- weights
    // read once: scales, hidden rows and sums stay in L2 beside the stream (MXFP4 with one token
    // 108 -> 101 us, bf16 149 -> 147)
    const uint64_t policy = l2_evict_first();
    Ring r{0, 0};
    int issued = 0;
    auto stream = [&](auto walk) {
      Tile t;
      while (walk.next(t)) {
        const int seg = t.seg / t.sub, v = seg != C::seg(1), box = 8 * C::wbytes(seg);
        for (int k0 = 0; k0 < t.K && !tb.abort; k0 += t.seg) {
          wait(&tb.empty[r.stage], r.phase ^ 1u, tb);
          if (lane == 0)
            issue_w<C, decltype(walk)::kDown>(maps.m[t.ma][v], maps.m[t.mb][v], t, k0, box,
                                              smem + r.stage * stage_bytes<C>(), &tb.full[r.stage], policy);
          __syncwarp();
          ++issued;
          r.next(C::STAGES);
        }
      }
    };
    if (a.fs > 0) stream(Gate(a, tb, true));
    __syncthreads();                       // the tables are there
    stream(Gate(a, tb, false));
    stream(Down(a, tb, false));
    // nothing may still be landing in shared memory when the CTA leaves
    for (int i = 0; i < min(issued, C::STAGES); ++i) {
      r.phase ^= r.stage == 0 ? 1u : 0u;
      r.stage = (r.stage + C::STAGES - 1) % C::STAGES;
      if (lane == 0) mbar_wait(&tb.full[r.stage], r.phase, tb.abort ? kWaitLimitCycles / 100 : kWaitLimitCycles);
    }
  } else if (warp == SELECT_WARP) {
    select_and_build(a, tb);
    __syncthreads();
  } else if (warp > W_WARP) {
    // ---------------------------------------------------------------- tokens
    if constexpr (C::MX) x_to_f16(a, tb, warp - X_WARP0, lane);
    Ring r{0, 0};
    auto stream = [&](auto walk) {
      Tile t;
      Gather<C, decltype(walk)::kDown> g;
      while (walk.next(t) && !tb.abort) {
        g.tile(a, tb, t, warp - X_WARP0, lane);
        for (int k0 = 0; k0 < t.K; k0 += t.seg) {
          wait(&tb.empty[r.stage], r.phase ^ 1u, tb);
          g.stage(a, tb, t, k0, stages + r.stage * stage_bytes<C>(), warp - X_WARP0, lane);
          cp_async_arrive_noinc(&tb.full[r.stage]);      // a thread's arrival once its copies have landed
          r.next(C::STAGES);
        }
      }
    };
    if (a.fs > 0) stream(Gate(a, tb, true));
    __syncthreads();
    stream(Gate(a, tb, false));
    if (lane == 0) grid_wait(a.bar + BAR_HIDDEN, gridDim.x, tb);     // the grid's hidden rows
    __syncwarp();
    stream(Down(a, tb, false));
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ---------------------------------------------------------------- products
    Ring r{0, 0};
    int buf = 0;
    Tile t;
    router_logits<XT>(a, red);
    worker_sync();
    if (tid == 0) grid_arrive(a.bar + BAR_LOGITS);
    if (C::MX) {
      if (tid == 0) grid_wait(a.bar + BAR_X, T, tb);
      worker_sync();
      if (tid < T) tb.xs[tid] = __ldcg(a.xscale + tid);
      worker_sync();
    }
    if (a.fs > 0)
      for (Gate w(a, tb, true); w.next(t);) run_tile<W, false>(a, tb, t, r, smem, red, yacc, buf);
    __syncthreads();                       // the tables are there
    for (Gate w(a, tb, false); w.next(t);) run_tile<W, false>(a, tb, t, r, smem, red, yacc, buf);
    // this CTA's hidden rows to the grid
    __threadfence();
    worker_sync();
    if (C::MX && tb.redo[0]) {
      if (a.fs > 0) hidden_in_range(a, tb, true);
      hidden_in_range(a, tb, false);
      __threadfence();
      worker_sync();
    }
    if (tid == 0) {
      grid_arrive(a.bar + BAR_HIDDEN);
      if (C::MX) grid_wait(a.bar + BAR_HIDDEN, gridDim.x, tb);
    }
    if (C::MX) {
      worker_sync();
      for (int i = tid; i < T * a.k; i += CONSUMERS) tb.hs[i] = row_scale(__ldcg(a.hmax + i));
      for (int i = tid; i < T; i += CONSUMERS) tb.hs[MAX_T * MAX_K + i] = row_scale(__ldcg(a.hmax + T * a.k + i));
    }
    for (int i = tid; i < T * SLOTS; i += CONSUMERS) yacc[i] = 0.f;
    worker_sync();

    XT* y = static_cast<XT*>(a.y);
    Down w(a, tb, false);
    if (w.empty()) {
      // nothing adds to any output
      for (size_t i = (size_t)blockIdx.x * CONSUMERS + tid; i < (size_t)T * a.d; i += (size_t)gridDim.x * CONSUMERS)
        y[i] = (XT)0.f;
    }
    if (by_token(a)) run_down_by_token<W>(a, tb, w, r, smem, red);
    while (w.next(t)) {
      run_tile<W, true>(a, tb, t, r, smem, red, yacc, buf);
      if (!t.last) continue;
      worker_sync();
      for (int i = tid; i < T * SLOTS; i += CONSUMERS) {
        const int j = slot_row<true>(t, i & (SLOTS - 1));
        if (j >= 0) y[(size_t)(i / SLOTS) * a.d + j] = (XT)yacc[i];
        if (C::MX && !isfinite(yacc[i])) tb.redo[1] = 1;
        yacc[i] = 0.f;
      }
      worker_sync();
    }
    if (C::MX && tb.redo[1]) outputs_in_range(a, tb);
  }
}

template <typename W>
cudaError_t launch(const Args& a, const void* const* w, size_t zero, cudaStream_t s) {
  using C = Cfg<W>;
  Maps maps{};
  for (int i = 0; i < (a.fs > 0 ? 6 : 3); ++i) {
    const bool down = i % 3 == M_W2, shared = i >= M_SHARED;
    const int width = shared ? a.fs : a.f, rows = down ? a.d : width, cols = down ? width : a.d;
    const uint64_t all = (uint64_t)(shared ? 1 : a.N) * rows;
    // the narrow boxes serve passes of 17 tokens and more (MXFP4: of 9)
    for (int v = 0; v < (a.T > (C::MX ? 8 : 16) ? 2 : 1); ++v)
      if (C::MX ? !make_map_u4_rows8(&maps.m[i][v][0], w[i], all, cols, C::seg(v ? 4 : 1) / 128)
                : !make_map_rows(&maps.m[i][v][0], w[i], C::EB == 4, all, cols, C::seg(v ? 4 : 1), 8) ||
                      !make_map_rows(&maps.m[i][v][1], w[i], C::EB == 4, all, cols, C::seg(v ? 4 : 1), 32))
        return cudaErrorInvalidValue;
  }
  const void* fn = (const void*)few_kernel<W>;
  const int smem = smem_bytes<C>();
  cudaError_t e = ensure_smem_attr(fn, smem);
  if (e != cudaSuccess) return e;
  e = cudaMemsetAsync(a.bar, 0, zero, s);
  if (e != cudaSuccess) return e;
  void* ptrs[] = {const_cast<Args*>(&a), &maps};
  return cudaLaunchCooperativeKernel(fn, dim3(sm_count()), dim3(THREADS), ptrs, smem, s);
}

}  // namespace few

size_t few_workspace_bytes(const moe_config_t& c, int fs) {
  const size_t eb = c.x_dtype == MOE_DTYPE_F32 ? 4 : 2;
  return few::zero_bytes(c) + 2 * few::shw_bytes(c) + few::x16_bytes(c) + few::logit_bytes(c) +
         few::align256(((size_t)c.T * c.top_k * c.d_ff + (size_t)c.T * fs) * eb);
}

cudaError_t launch_few(const moe_config_t& c, int64_t capacity, const void* x, const float* w_gate,
                       const float* logit_offset, const float* bias, bool mxfp4, const void* const* w,
                       const uint8_t* const* sf, int fs, int32_t* topk_idx, float* topk_w, void* y, void* ws,
                       cudaStream_t s) {
  few::Args a{};
  a.x = x;
  a.w_gate = w_gate;
  for (int i = 0; i < 6; ++i) {
    a.q[i] = mxfp4 ? static_cast<const uint8_t*>(w[i]) : nullptr;
    a.sf[i] = mxfp4 ? sf[i] : nullptr;
  }
  a.T = (int)c.T; a.d = c.d_model; a.f = c.d_ff; a.fs = fs; a.N = c.n_experts; a.k = c.top_k; a.sink = c.shared_sink;
  a.capacity = capacity;
  a.route = rt::RouteArgs{logit_offset, bias, c.T, c.n_experts, c.top_k, c.score_fn, c.renorm, c.n_groups,
                          c.topk_groups, c.group_score_topn, nullptr, nullptr, nullptr, nullptr, nullptr,
                          c.shared_sink, nullptr, nullptr};
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.y = y;
  uint8_t* p = static_cast<uint8_t*>(ws);
  a.bar = reinterpret_cast<unsigned*>(p);
  a.hmax = reinterpret_cast<unsigned*>(p + 256);
  const size_t zero = few::zero_bytes(c);
  p += zero;
  a.shw = reinterpret_cast<float*>(p);
  p += few::shw_bytes(c);
  a.xscale = reinterpret_cast<float*>(p);
  p += few::shw_bytes(c);
  a.x16 = p;
  p += few::x16_bytes(c);
  a.logits = reinterpret_cast<float*>(p);
  a.h = p + few::logit_bytes(c);
  if (mxfp4) return few::launch<few::Mxfp4>(a, w, zero, s);
  return c.x_dtype == MOE_DTYPE_F32 ? few::launch<float>(a, w, zero, s) : few::launch<__nv_bfloat16>(a, w, zero, s);
}

}  // namespace moe
