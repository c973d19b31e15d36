// A whole MoE layer for few tokens (1 .. 64), in one launch: router, top-k, routed and
// shared experts, weighted sum.
//
//   y_t = sum_j w_tj W2_e (silu(W1_e x_t) * (W3_e x_t)) + shared(x_t)
//
// Bound: the bytes of the weights of the experts that at least one token picks (and of the
// router and the shared expert); every weight is read once, from HBM.
//
// One cooperative launch, one CTA per SM, two barriers over the grid:
//   logits     each CTA takes whole experts of the router, all tokens; arrive at barrier 1
//   shared     the shared experts' gate/up rows, cut evenly over the grid: they do not
//              depend on the routing, so they stand between arriving and waiting
//   selection  every CTA selects for all tokens by itself (the same result everywhere,
//              without a third barrier) and builds the experts' token lists
//   gate/up    the met experts' hidden units, cut evenly over the grid
//   -- barrier 2 --
//   down       each CTA takes rows of W2 of all met experts, so a token's sum over its
//              experts stays inside one CTA: fixed order, no atomics, no second pass
//
// One warp streams the weights through a ring of shared-memory stages with TMA, 8 rows by 512
// bytes a copy (4 KB: at 512 bytes a copy, the engine's ~57 cycles for one would hold the
// stream to 2.5 TB/s), and runs ahead of the phases: the first down stages' weights are in
// flight while the CTA waits at barrier 2 for the hidden rows.  Three warps gather the same
// columns of the expert's tokens with cp.async.  Sixteen warps multiply with mma.sync
// m16n8k16: 16 weight
// rows by 8 tokens, which leaves nothing to gain from tcgen05 (its smallest tile is 128
// rows, and no tensor pipe is near its limit: at 8 tokens a weight is used 8 times, two
// orders below what the pipes need to be the bound).  The order of k inside a fragment is
// free as long as both operands use it, so a thread feeds the MMA with its own 16-byte
// loads and no shuffles.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace few {

constexpr int MAX_T = 64, MAX_N = 512, MAX_K = 16;
constexpr int WARPS = 16;                       // consumer warps
constexpr int X_WARPS = 3;                      // warps that gather tokens' columns
constexpr int CONSUMERS = 32 * WARPS, THREADS = CONSUMERS + 32 + 32 * X_WARPS;
constexpr int MAX_PASS = 32;                    // tokens of an expert per pass over its weights
constexpr int SLOTS = 64;                       // weight rows of a stage
constexpr int ROUTE_TILE = 16, ROUTE_COLS = 1024;   // router: experts and columns at a time
enum { W_F32 = 0, W_BF16 = 1, W_MXFP4 = 2 };

// The six expert stacks [experts * rows, cols]: W1, W3, W2 routed, then shared.
enum { M_W1 = 0, M_W3 = 1, M_W2 = 2, M_SHARED = 3 };
struct Maps {
  CUtensorMap m[6][2];     // boxes of 8 rows by a stage's columns: for 8 tokens, for 32
};

struct Args {
  const void* x;
  const float* w_gate;
  const uint8_t* sf[6];    // MXFP4: tile-atom scales of the stacks
  int T, d, f, fs, N, k, sink;
  int64_t capacity;
  rt::RouteArgs route;     // selection options (outputs set by the kernel)
  int32_t* topk_idx;
  float* topk_w;
  void* y;
  unsigned* bar;           // two barrier counters, zero at launch
  unsigned* hmax;          // MXFP4: [T k + T] largest |h| of each row as bits, zero at launch
  float* logits;           // [slices, T, N + sink] partial sums
  void* h;                 // [T k, f] routed, then [T, fs] shared; x's type
};

// Per weight type.  NT: 8-token columns of a pass (1, 2 or 4); seg(NT): columns of a stage.
// A stage holds 8 groups of 8 weight rows as TMA leaves them (bf16, fp32: row by row; MXFP4:
// by 64-byte column chunks, the chunk's 8 rows, 64-byte swizzle, so that the 16 bytes that
// a quad takes of each of 8 rows fall into different banks), then the tokens' rows (64 mod
// 128 bytes apart, for the same reason), then MXFP4's scales, 36 bytes a row.
// WK warps split a stage's columns, WARPS / WK its 16-row tiles.
template <int WT> struct Cfg;
template <> struct Cfg<W_BF16> {
  using XT = __nv_bfloat16;
  static constexpr int STAGES = 4, WK = 4, RED = 2;
  static __host__ __device__ constexpr int seg(int nt) { return nt == 4 ? 128 : 256; }
  static __host__ __device__ constexpr int wbytes(int c) { return 2 * c; }
};
template <> struct Cfg<W_F32> {
  using XT = float;
  static constexpr int STAGES = 4, WK = 4, RED = 2;
  static __host__ __device__ constexpr int seg(int nt) { return nt == 4 ? 64 : 128; }
  static __host__ __device__ constexpr int wbytes(int c) { return 4 * c; }
};
template <> struct Cfg<W_MXFP4> {
  using XT = __nv_bfloat16;
  static constexpr int STAGES = 3, WK = 16, RED = 1;
  static __host__ __device__ constexpr int seg(int nt) { return nt == 1 ? 1024 : 512; }
  static __host__ __device__ constexpr int wbytes(int c) { return c / 2; }
};
constexpr int SF_LD = 36;                       // scales of a row (MXFP4)

template <int WT> __host__ __device__ constexpr int wstride(int seg) { return Cfg<WT>::wbytes(seg); }
template <int WT> __host__ __device__ constexpr int xstride(int seg) { return (int)sizeof(typename Cfg<WT>::XT) * seg + 64; }
template <int WT> __host__ __device__ constexpr int stage_use(int nt) {
  return SLOTS * wstride<WT>(Cfg<WT>::seg(nt)) + 8 * nt * xstride<WT>(Cfg<WT>::seg(nt)) +
         (WT == W_MXFP4 ? SLOTS * SF_LD : 0);
}
template <int WT> __host__ __device__ constexpr int stage_bytes() {
  int m = stage_use<WT>(1) > stage_use<WT>(2) ? stage_use<WT>(1) : stage_use<WT>(2);
  m = m > stage_use<WT>(4) ? m : stage_use<WT>(4);
  return (m + 1023) / 1024 * 1024;
}

constexpr int RED_LD = SLOTS + 4;               // partial sums [token][row], padded: 32 banks
template <int WT> __host__ __device__ constexpr int red_floats() { return Cfg<WT>::WK * 8 * RED_LD; }

constexpr int RED_X_FLOATS = 8 * ROUTE_COLS;    // the router's tokens lie over the partial sums and the output tile

// What selection leaves for the rest of the kernel.
struct Tables {
  int16_t row0[MAX_N + 1];           // first row of each expert; rows of e: row0[e] .. row0[e + 1]
  int16_t act[MAX_N];                // met experts, ascending
  uint8_t row_tok[MAX_T * MAX_K];
  float row_w[MAX_T * MAX_K];
  float shw[MAX_T];
  float xs[MAX_T];                   // MXFP4: scale of each token's x
  float hs[MAX_T * MAX_K + MAX_T];   // MXFP4: scale of each hidden row
  uint64_t full[4], empty[4];
  int32_t n_act;
  volatile int32_t abort;
};
// Only while selecting; lies over the partial sums and the output tile.
struct Scratch {
  int32_t idx[MAX_T * MAX_K];
  float w[MAX_T * MAX_K];
  unsigned mask[MAX_N][2];           // tokens of each expert
  int2 sums[WARPS];
};
constexpr int YACC_FLOATS = MAX_T * SLOTS;
template <int WT> __host__ __device__ constexpr int smem_bytes() {
  return 1024 + Cfg<WT>::STAGES * stage_bytes<WT>() + (Cfg<WT>::RED * red_floats<WT>() + YACC_FLOATS) * 4 + (int)sizeof(Tables);
}
static_assert(smem_bytes<W_BF16>() <= 232448 && smem_bytes<W_F32>() <= 232448 && smem_bytes<W_MXFP4>() <= 232448,
              "shared memory per CTA");
static_assert(WARPS * 2 * (MAX_N + 8) * 4 <= 3 * 43008, "scores in the ring");
static_assert(RED_X_FLOATS <= 2 * red_floats<W_BF16>() + YACC_FLOATS && RED_X_FLOATS <= red_floats<W_MXFP4>() + YACC_FLOATS,
              "router tokens");
static_assert(sizeof(Scratch) <= (2 * red_floats<W_BF16>() + YACC_FLOATS) * 4, "selection scratch");

// ------------------------------------------------------------------ waits
// Every wait is bounded.  After one ran out the CTA goes on without waiting (its barriers
// stay matched, its results are lost) and the device status word says so.
__device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, Tables& tb) {
  if (mbar_try_wait(bar, parity)) return;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (tb.abort) return;
    if (clock64() - t0 > kWaitLimitCycles) {
      flag_timeout();
      tb.abort = 1;
    }
  }
}
// Arrive, then wait for the whole grid.
__device__ __forceinline__ void grid_arrive(unsigned* bar) {
  __threadfence();
  atomicAdd(bar, 1u);
}
__device__ __forceinline__ void grid_wait(unsigned* bar, Tables& tb) {
  const long long t0 = clock64();
  for (;;) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(bar) : "memory");
    if (v >= gridDim.x || tb.abort) return;
    if (clock64() - t0 > kWaitLimitCycles) {
      flag_timeout();
      tb.abort = 1;
    }
  }
}
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(CONSUMERS) : "memory"); }

// ------------------------------------------------------------------ router
// Logits in K slices: tiles of 16 experts (a warp each) by `slices` column ranges, spread over
// the grid, so that a CTA reads a slice of x and not all of it.  Eight tokens at a time, their
// columns in shared memory as fp32; partial sums to memory, added by the selection.
__host__ __device__ __forceinline__ int route_tiles(int ld) { return (ld + ROUTE_TILE - 1) / ROUTE_TILE; }
// At most 16 (the selection adds them one by one), at least 256 columns each, 144 jobs in all:
// one for every SM of the grid.
__host__ __device__ __forceinline__ int route_slices(int ld, int d) {
  int n = 144 / route_tiles(ld), most = (d + 255) / 256;
  n = n < most ? n : most;
  return n < 1 ? 1 : n > 16 ? 16 : n;
}
__device__ __forceinline__ void load4(const float* p, float* f) { unpack16(ldg_nc16(p), f, 0.f); }
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* f) {
  const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
  f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xffff0000u);
  f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xffff0000u);
}
template <typename XT>
__device__ __forceinline__ void router_logits(const Args& a, float4* xs) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ld = a.N + a.sink, tiles = route_tiles(ld), slices = route_slices(ld, a.d);
  const int quads = (a.d / 4 + slices - 1) / slices;
  const XT* x = static_cast<const XT*>(a.x);
  for (int job = blockIdx.x; job < tiles * slices; job += gridDim.x) {
    const int s = job / tiles, e = (job - s * tiles) * ROUTE_TILE + warp;
    const int q0 = s * quads, q1 = min(q0 + quads, a.d / 4);
    const float* wg = a.w_gate + (size_t)min(e, ld - 1) * a.d;
    for (int t0 = 0; t0 < a.T; t0 += 8) {
      const int n = min(8, a.T - t0);
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int c0 = q0; c0 < q1; c0 += ROUTE_COLS / 4) {
        const int nq = min(ROUTE_COLS / 4, q1 - c0);
        float4 w[ROUTE_COLS / 128];
#pragma unroll
        for (int u = 0; u < ROUTE_COLS / 128; ++u)
          w[u] = lane + 32 * u < nq ? __ldg(reinterpret_cast<const float4*>(wg) + c0 + lane + 32 * u)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = tid; i < n * (ROUTE_COLS / 4); i += CONSUMERS) {
          const int j = i / (ROUTE_COLS / 4), q = i % (ROUTE_COLS / 4);
          float v[4] = {0.f, 0.f, 0.f, 0.f};
          if (q < nq) load4(x + (size_t)(t0 + j) * a.d + 4 * (c0 + q), v);
          xs[i] = make_float4(v[0], v[1], v[2], v[3]);
        }
        consumer_sync();
        for (int j = 0; j < n; ++j) {
          float p = 0.f;
#pragma unroll
          for (int u = 0; u < ROUTE_COLS / 128; ++u) {
            const float4 v = xs[j * (ROUTE_COLS / 4) + lane + 32 * u];
            p = fmaf(w[u].x, v.x, p);
            p = fmaf(w[u].y, v.y, p);
            p = fmaf(w[u].z, v.z, p);
            p = fmaf(w[u].w, v.w, p);
          }
#pragma unroll
          for (int m = 0; m < 8; ++m) acc[m] += m == j ? p : 0.f;
        }
        consumer_sync();
      }
      float mine = 0.f;                       // lane j: token t0 + j
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = warp_sum(acc[j]);
        if (lane == j) mine = v;
      }
      if (lane < n && e < ld) a.logits[((size_t)s * a.T + t0 + lane) * ld + e] = mine;
    }
  }
}

// The next best of q[lo .. hi) after (key, index) in the order of falling key, then rising
// index; index 0x7fffffff when none is left.
__device__ __forceinline__ void next_best(const uint32_t* q, int lo, int hi, int lane, uint32_t& key, int& idx) {
  uint32_t bk = 0;
  int bi = 0x7fffffff;
  for (int e = lo + lane; e < hi; e += 32) {
    const uint32_t v = q[e];
    if ((v < key || (v == key && e > idx)) && v > bk) { bk = v; bi = e; }
  }
  key = __reduce_max_sync(0xffffffffu, bk);
  idx = (int)__reduce_min_sync(0xffffffffu, bk == key && bk > 0 ? (uint32_t)bi : 0x7fffffffu);
}

// Selection, a warp per token: moe_route's formulas, ties and order, in loops instead of
// registers (a few tokens meet this code once, cold: its size counts more than its steps).
// sv: the affinities, q: the selection scores as order-preserving keys (0: not eligible).
__device__ __noinline__ void select_token(const Args& a, Tables& tb, Scratch& sc, int t, float* sv, uint32_t* q) {
  const int lane = threadIdx.x & 31, N = a.N, k = a.k;
  const int ld = N + a.sink, slices = route_slices(ld, a.d);
  const rt::RouteArgs& r = a.route;
  float m = -INFINITY;
#pragma unroll 1
  for (int e = lane; e < ld; e += 32) {
    float z = 0.f;
#pragma unroll 4
    for (int s = 0; s < slices; ++s) z += __ldcg(a.logits + ((size_t)s * a.T + t) * ld + e);
    if (r.logit_offset && e < N) z += r.logit_offset[e];
    sv[e] = z;
    m = fmaxf(m, z);
  }
  m = warp_max(m);
  const bool soft = r.score_fn == MOE_SCORE_SOFTMAX;
  float se = 0.f;
  if (soft) {
#pragma unroll 1
    for (int e = lane; e < ld; e += 32) se += expf(sv[e] - m);
    se = warp_sum(se);
  }
#pragma unroll 1
  for (int e = lane; e < ld; e += 32) {
    const float z = sv[e];
    const float s = soft ? expf(z - m) / se : 1.f / (1.f + expf(-z));
    sv[e] = s;
    if (e < N) q[e] = f32_key(r.bias ? s + r.bias[e] : s);
  }
  __syncwarp();
  if (r.n_groups > 1) {
    const int size = N / r.n_groups;
    uint32_t mine = 0;                        // lane g: group g's score
#pragma unroll 1
    for (int g = 0; g < r.n_groups; ++g) {
      uint32_t key = 0xffffffffu;
      int idx = -1;
      float sum = 0.f;
#pragma unroll 1
      for (int i = 0; i < r.group_topn; ++i) {
        next_best(q, g * size, (g + 1) * size, lane, key, idx);
        sum += key_f32(key);
      }
      if (lane == g) mine = f32_key(sum);
    }
    uint32_t kept = 0;
#pragma unroll 1
    for (int i = 0; i < r.topk_groups; ++i) {
      const uint32_t v = lane < r.n_groups && !((kept >> lane) & 1u) ? mine : 0u;
      const uint32_t best = __reduce_max_sync(0xffffffffu, v);
      kept |= 1u << __reduce_min_sync(0xffffffffu, v == best && lane < r.n_groups && !((kept >> lane) & 1u) ? lane : 31);
    }
#pragma unroll 1
    for (int g = 0; g < r.n_groups; ++g)
      if (!((kept >> g) & 1u))
        for (int e = g * size + lane; e < (g + 1) * size; e += 32) q[e] = 0;
    __syncwarp();
  }
  uint32_t key = 0xffffffffu;
  int idx = -1, my = 0x7fffffff;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    next_best(q, 0, N, lane, key, idx);
    if (lane == j) my = idx;
  }
  const float s = lane < k && my < N ? sv[my] : 0.f;
  const float sh = a.sink ? sv[N] : 0.f;
  const float sum = warp_sum(s) + sh;
  if (lane < k) {
    sc.idx[t * k + lane] = my;
    sc.w[t * k + lane] = r.renorm ? s / sum : s;
  }
  if (lane == 0 && a.sink) tb.shw[t] = r.renorm ? sh / sum : sh;
}

// Experts' token masks, met experts in ascending order, rows (expert major, tokens
// ascending); a token past its expert's capacity gets no row.  A thread per expert.
static_assert(CONSUMERS >= MAX_N, "a thread per expert");
__device__ void build_tables(const Args& a, Tables& tb, Scratch& sc) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.T * a.k;
  if (tid < MAX_N) sc.mask[tid][0] = sc.mask[tid][1] = 0;
  consumer_sync();
  for (int s = tid; s < n; s += CONSUMERS) {
    const int e = sc.idx[s], t = s / a.k;
    if ((unsigned)e < (unsigned)a.N) atomicOr(&sc.mask[e][t >> 5], 1u << (t & 31));
    else flag_invalid_index();
  }
  consumer_sync();
  int c = tid < a.N ? __popc(sc.mask[tid][0]) + __popc(sc.mask[tid][1]) : 0;
  if (c > a.capacity) c = (int)a.capacity;
  int incl = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  const unsigned met = __ballot_sync(0xffffffffu, c > 0);
  if (lane == 31) sc.sums[warp] = make_int2(incl, __popc(met));
  consumer_sync();
  int rows = 0, act = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const int2 v = sc.sums[w];
    rows += w < warp ? v.x : 0;
    act += w < warp ? v.y : 0;
    all += v.y;
  }
  if (tid < a.N) tb.row0[tid + 1] = (int16_t)(rows + incl);
  if (c > 0) tb.act[act + __popc(met & ((1u << lane) - 1u))] = (int16_t)tid;
  if (tid == 0) {
    tb.row0[0] = 0;
    tb.n_act = all;
  }
  consumer_sync();
  for (int s = tid; s < n; s += CONSUMERS) {
    const int e = sc.idx[s], t = s / a.k;
    if ((unsigned)e >= (unsigned)a.N) continue;
    const unsigned below = t < 32 ? __popc(sc.mask[e][0] & ((1u << t) - 1u))
                                  : __popc(sc.mask[e][0]) + __popc(sc.mask[e][1] & ((1u << (t - 32)) - 1u));
    if ((int64_t)below < a.capacity) {
      tb.row_tok[tb.row0[e] + below] = (uint8_t)t;
      tb.row_w[tb.row0[e] + below] = sc.w[s];
    }
  }
}

// ------------------------------------------------------------------ schedule
// One pass over one tile of weight rows: at most 64 rows (gate/up: 32 hidden units, their
// gate and up rows) by one expert's tokens, 32 at most.  Producers and consumers walk the
// same sequence.  A unit is eight consecutive rows (a TMA box); a CTA's units are one
// contiguous range, so the grid's shares differ by one unit.
struct Tile {
  int ma, mb;         // stacks: gate and up, or down
  int erow;           // the stacks' rows before this expert's
  int K;              // columns
  int base;           // first row, within the expert
  int nu;             // units
  int n;              // tokens of this pass
  int row;            // first hidden row (routed: table row; shared: token), this pass
  int nt, seg;
  bool sh, last;      // last: the tile's last pass (down: of the last expert)
};

template <int WT, bool DOWN>
struct Walk {
  static constexpr bool kDown = DOWN;
  const Args* g;
  const Tables* tb;
  int u, u1, per;     // units: next, end; per expert (gate/up)
  int slot, slots, first;
  int done;           // tokens of earlier passes
  bool sh;

  // gate/up: shared or routed part; down: both, the shared expert first (slot -1)
  __device__ void init(const Args& a, const Tables& t, bool shared) {
    g = &a; tb = &t; sh = shared; done = 0;
    const int P = gridDim.x, b = blockIdx.x;
    per = (shared ? a.fs : a.f) / 8;
    const int64_t all = DOWN ? a.d / 8 : shared ? per : (int64_t)t.n_act * per;
    u = (int)(all * b / P);
    u1 = (int)(all * (b + 1) / P);
    first = DOWN && a.fs > 0 ? -1 : 0;
    slots = DOWN ? t.n_act : 0;
    slot = first;
    if (DOWN && slots + (first < 0) == 0) u = u1;      // no expert at all: no weights to read
  }
  __device__ bool next(Tile& t) {
    if (u >= u1) return false;
    int j = u, e = 0;
    bool shared = sh;
    if (DOWN) {
      shared = slot < 0;
      e = shared ? 0 : tb->act[slot];
    } else if (!sh) {
      const int s = u / per;
      j = u - s * per;
      e = tb->act[s];
    }
    t.sh = shared;
    t.nu = min(DOWN ? 8 : 4, u1 - u);
    if (!DOWN) t.nu = min(t.nu, per - j);
    t.base = 8 * j;
    const int f = shared ? g->fs : g->f;
    t.K = DOWN ? f : g->d;
    t.erow = e * (DOWN ? g->d : f);
    t.ma = (DOWN ? M_W2 : M_W1) + (shared ? M_SHARED : 0);
    t.mb = M_W3 + (shared ? M_SHARED : 0);
    const int n = shared ? g->T : tb->row0[e + 1] - tb->row0[e];
    t.n = min(n - done, MAX_PASS);
    t.row = (shared ? 0 : tb->row0[e]) + done;
    t.nt = t.n <= 8 ? 1 : t.n <= 16 ? 2 : 4;
    t.seg = Cfg<WT>::seg(t.nt);
    done += t.n;
    t.last = false;
    if (done < n) return true;
    done = 0;
    if (DOWN) {
      if (++slot < slots) return true;
      slot = first;
    }
    t.last = true;
    u += t.nu;
    return true;
  }
};

// Row (within the expert) of slot s (0 .. 63) of a stage, or -1.  Down: 64 rows in order;
// gate/up: 8 gate rows, then the same 8 units' up rows, four times.
template <bool DOWN>
__device__ __forceinline__ int slot_row(const Tile& t, int s) {
  const int r = DOWN ? s : 8 * (s >> 4) + (s & 7);
  return r < 8 * t.nu ? t.base + r : -1;
}

// Weights of the stage at column k0, by one thread: one box per group of 8 rows.  Columns
// past K arrive as zeros and count as bytes.
template <int WT, bool DOWN>
__device__ __forceinline__ void issue_w(const Maps& maps, const Tile& t, int k0, uint8_t* stage, uint64_t* bar) {
  const int box = 8 * wstride<WT>(t.seg), v = t.seg == Cfg<WT>::seg(1) ? 0 : 1;
  mbar_arrive_expect_tx(bar, (DOWN ? 1 : 2) * t.nu * box);
  for (int i = 0; i < t.nu; ++i)
#pragma unroll
    for (int h = 0; h < (DOWN ? 1 : 2); ++h) {
      const CUtensorMap* m = &maps.m[h ? t.mb : t.ma][v];
      uint8_t* dst = stage + (DOWN ? i : 2 * i + h) * box;
      const int row = t.erow + t.base + 8 * i;
      if (WT == W_MXFP4) tma_load_3d(m, dst, bar, 0, row, k0 / 128);
      else tma_load_2d(m, dst, bar, k0, row);
    }
}
__device__ __forceinline__ void cp_async4(uint32_t smem_dst, const void* gsrc) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_dst), "l"(gsrc) : "memory");
}
// The same columns of the pass's tokens (x gathered by token, or hidden rows) and, for MXFP4,
// the rows' scales; then one arrival per thread once its copies have landed.
template <int WT, bool DOWN>
__device__ __forceinline__ void issue_x(const Args& a, const Tables& tb, const Tile& t, int k0, uint32_t stage,
                                        uint64_t* bar, int xw, int lane) {
  using XT = typename Cfg<WT>::XT;
  const int cols = min(t.seg, t.K - k0);
  const int chunks = cols * (int)sizeof(XT) / 16;
  const uint32_t xs = stage + SLOTS * wstride<WT>(t.seg);
  for (int i = xw; i < t.n; i += X_WARPS) {
    const XT* src;
    if (DOWN) {
      src = static_cast<const XT*>(a.h) + (t.sh ? (size_t)a.T * a.k * a.f : 0) + (size_t)(t.row + i) * t.K;
    } else {
      const int tok = t.sh ? t.row + i : tb.row_tok[t.row + i];
      src = static_cast<const XT*>(a.x) + (size_t)tok * t.K;
    }
    const uint8_t* p = reinterpret_cast<const uint8_t*>(src + k0);
    for (int c = lane; c < chunks; c += 32) cp_async16(xs + i * xstride<WT>(t.seg) + 16 * c, p + 16 * c);
  }
  if (WT == W_MXFP4) {
    const uint32_t sd = xs + 8 * t.nt * xstride<WT>(t.seg);
    const int kb = lane & 7;                       // a lane's column block; four rows at a time
    if (kb < cols / 128)
      for (int s = 4 * xw + (lane >> 3); s < SLOTS; s += 4 * X_WARPS) {
        const int r = slot_row<DOWN>(t, s);
        if (r < 0) continue;
        const int row = t.erow + r;
        const uint8_t* sf = a.sf[(DOWN || !(s & 8)) ? t.ma : t.mb];
        cp_async4(sd + SF_LD * s + 4 * kb, sf + mx::atom_byte(row >> 7, t.K / 128, k0 / 128 + kb, row & 127, 0));
      }
  }
  cp_async_arrive_noinc(bar);
}

// ------------------------------------------------------------------ products
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds1(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
// D += A B, 16 x 8 x 16, fp32 accumulators: rows g and g + 8, columns 2t and 2t + 1 of lane 4g + t.
__device__ __forceinline__ void mma_bf16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Eight E2M1 codes of a word to four pairs of fp16 (exact), in order.
__device__ __forceinline__ void e2m1_f16(uint32_t w, uint32_t* o) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]) : "r"(w));
}
// Two bf16 to fp16, times a power of two.
__device__ __forceinline__ uint32_t scaled_f16(uint32_t v, float s) {
  const __half2 h = __floats2half2_rn(__uint_as_float(v << 16) * s, __uint_as_float(v & 0xffff0000u) * s);
  return *reinterpret_cast<const uint32_t*>(&h);
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

// One stage's products of this warp into acc[16-row tile][8-token column][4].
template <int WT, bool DOWN, int NT>
struct Product;

template <bool DOWN, int NT>
struct Product<W_BF16, DOWN, NT> {
  static constexpr int QT = 1;            // 16-row tiles of a warp
  float acc[1][NT][4];
  __device__ __forceinline__ void init(const Tile&, const Tables&, int) {
#pragma unroll
    for (int i = 0; i < NT * 4; ++i) acc[0][0][i] = 0.f;
  }
  __device__ __forceinline__ void stage(const Tile& t, int k0, uint32_t st, int warp, int lane) {
    constexpr int SEG = Cfg<W_BF16>::seg(NT), WS = wstride<W_BF16>(SEG), XS = xstride<W_BF16>(SEG);
    const int q = warp & 3, kq = warp >> 2, g = lane >> 2, tq = lane & 3;
    if ((DOWN ? 2 : 1) * q >= t.nu) return;
    const int cols = t.K - k0;
    const uint32_t wa = st + (16 * q + g) * WS, xa = st + SLOTS * WS + g * XS;
#pragma unroll
    for (int kk = 0; kk < SEG / 4; kk += 32) {
      const int c = kq * (SEG / 4) + kk + 8 * tq;
      const uint4 z = make_uint4(0, 0, 0, 0);
      const bool ok = c < cols;
      const uint4 a0 = ok ? lds16(wa + 2 * c) : z, a1 = ok ? lds16(wa + 8 * WS + 2 * c) : z;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 b = ok ? lds16(xa + n * 8 * XS + 2 * c) : z;
        mma_bf16(acc[0][n], a0.x, a1.x, a0.y, a1.y, b.x, b.y);
        mma_bf16(acc[0][n], a0.z, a1.z, a0.w, a1.w, b.z, b.w);
      }
    }
  }
  __device__ __forceinline__ void result(int, int n, int, float* c) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = acc[0][n][i];
  }
};

// fp32: no tensor form keeps its bits.  A lane multiplies its 4 columns of rows g and g + 8 by
// all 8 tokens; the quad's partial sums meet at the tile's end.
template <bool DOWN, int NT>
struct Product<W_F32, DOWN, NT> {
  static constexpr int QT = 1;
  float acc[2][NT][8];
  __device__ __forceinline__ void init(const Tile&, const Tables&, int) {
#pragma unroll
    for (int i = 0; i < 2 * NT * 8; ++i) acc[0][0][i] = 0.f;
  }
  __device__ __forceinline__ void stage(const Tile& t, int k0, uint32_t st, int warp, int lane) {
    constexpr int SEG = Cfg<W_F32>::seg(NT), WS = wstride<W_F32>(SEG), XS = xstride<W_F32>(SEG);
    const int q = warp & 3, kq = warp >> 2, g = lane >> 2, tq = lane & 3;
    if ((DOWN ? 2 : 1) * q >= t.nu) return;
    const int cols = t.K - k0;
    const uint32_t wa = st + (16 * q + g) * WS, xa = st + SLOTS * WS;
#pragma unroll
    for (int kk = 0; kk < SEG / 4; kk += 16) {
      const int c = kq * (SEG / 4) + kk + 4 * tq;
      if (c >= cols) continue;
      float w0[4], w1[4];
      unpack16(lds16(wa + 4 * c), w0, 0.f);
      unpack16(lds16(wa + 8 * WS + 4 * c), w1, 0.f);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float x[4];
          unpack16(lds16(xa + (8 * n + j) * XS + 4 * c), x, 0.f);
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
// sum of 32 columns, which the row's block scale multiplies in fp32.
template <bool DOWN, int NT>
struct Product<W_MXFP4, DOWN, NT> {
  static constexpr int QT = 4;
  float acc[4][NT][4];
  float ts[NT];                            // scale of token 8 n + g
  __device__ __forceinline__ void init(const Tile& t, const Tables& tb, int lane) {
#pragma unroll
    for (int i = 0; i < 4 * NT * 4; ++i) acc[0][0][i] = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) ts[n] = 8 * n + (lane >> 2) < t.n ? token_scale<DOWN>(t, tb, 8 * n + (lane >> 2)) : 0.f;
  }
  __device__ __forceinline__ void stage(const Tile& t, int k0, uint32_t st, int warp, int lane) {
    constexpr int SEG = Cfg<W_MXFP4>::seg(NT), WS = wstride<W_MXFP4>(SEG), XS = xstride<W_MXFP4>(SEG);
    const int g = lane >> 2, tq = lane & 3;
    const int c0 = warp * (SEG / WARPS);
    if (c0 >= t.K - k0) return;              // whole 128-column blocks: uniform over the warp
    const uint32_t wa = st + 64 * g + 4 * tq, xa = st + SLOTS * WS + g * XS + 16 * tq;
    const uint32_t sa = st + SLOTS * WS + 8 * NT * XS + SF_LD * g;
    const int swz = (g >> 1) & 3;
#pragma unroll
    for (int kk = 0; kk < SEG / WARPS; kk += 32) {
      const int c = c0 + kk;
      uint32_t b[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 v = lds16(xa + n * 8 * XS + 2 * c);
        b[n][0] = scaled_f16(v.x, ts[n]);
        b[n][1] = scaled_f16(v.y, ts[n]);
        b[n][2] = scaled_f16(v.z, ts[n]);
        b[n][3] = scaled_f16(v.w, ts[n]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t a0[4], a1[4];
        if ((DOWN ? 2 : 1) * q >= t.nu) break;
        // 16-byte unit (c / 32) % 4 of 64-byte chunk c / 128 of the group's rows
        const uint32_t wq = wa + 16 * q * WS + 512 * (c >> 7) + 16 * (((c >> 5) & 3) ^ swz);
        e2m1_f16(lds4(wq), a0);
        e2m1_f16(lds4(wq + 8 * WS), a1);
        const uint32_t sp = sa + 16 * SF_LD * q + (c >> 5);
        // byte 0 is 2^-127, a subnormal; 255 (NaN) becomes an infinity, which times the zero
        // codes of such a block is NaN
        const float s0 = __uint_as_float(max(lds1(sp) << 23, 0x00400000u));
        const float s1 = __uint_as_float(max(lds1(sp + 8 * SF_LD) << 23, 0x00400000u));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float p[4] = {0.f, 0.f, 0.f, 0.f};
          mma_f16(p, a0[0], a1[0], a0[1], a1[1], b[n][0], b[n][1]);
          mma_f16(p, a0[2], a1[2], a0[3], a1[3], b[n][2], b[n][3]);
          acc[q][n][0] = fmaf(p[0], s0, acc[q][n][0]);
          acc[q][n][1] = fmaf(p[1], s0, acc[q][n][1]);
          acc[q][n][2] = fmaf(p[2], s1, acc[q][n][2]);
          acc[q][n][3] = fmaf(p[3], s1, acc[q][n][3]);
        }
      }
    }
  }
  template <bool D>
  static __device__ __forceinline__ float token_scale(const Tile& t, const Tables& tb, int i) {
    if (D) return tb.hs[t.sh ? MAX_T * MAX_K + t.row + i : t.row + i];
    return tb.xs[t.sh ? t.row + i : tb.row_tok[t.row + i]];
  }
  __device__ __forceinline__ void result(int q, int n, int, float* c) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = acc[q][n][i];
  }
};

// A consumer's place in the ring.
struct Ring {
  uint32_t stage, phase;
};

// One tile pass: all its stages, then the warps' partial sums through shared memory and the
// tile's results.  gate/up: h = silu(gate) * up to memory; down: weighted sums into yacc.
template <int WT, bool DOWN, int NT>
__device__ __forceinline__ void run_pass(const Args& a, Tables& tb, const Tile& t, Ring& r, uint32_t stages, float* red,
                                         float* yacc, int& buf) {
  using C = Cfg<WT>;
  using XT = typename C::XT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Product<WT, DOWN, NT> p;
  p.init(t, tb, lane);
  for (int k0 = 0; k0 < t.K; k0 += C::seg(NT)) {
    wait(&tb.full[r.stage], r.phase, tb);
    p.stage(t, k0, stages + r.stage * stage_bytes<WT>(), warp, lane);
    __syncwarp();
    if (lane == 0) mbar_arrive(&tb.empty[r.stage]);
    if (++r.stage == C::STAGES) { r.stage = 0; r.phase ^= 1u; }
  }
  const int wk = WT == W_MXFP4 ? warp : warp >> 2;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (8 * n >= t.n) break;
    float* rb = red + buf * red_floats<WT>();
#pragma unroll
    for (int q = 0; q < p.QT; ++q) {
      float c[4];
      p.result(q, n, lane, c);
      float* o = rb + (wk * 8 + 2 * (lane & 3)) * RED_LD + 16 * (WT == W_MXFP4 ? q : warp & 3) + (lane >> 2);
      o[0] = c[0];
      o[RED_LD] = c[1];
      o[8] = c[2];
      o[RED_LD + 8] = c[3];
    }
    consumer_sync();
    if (DOWN) {
      // 64 rows by 8 tokens, one each
      const int i = 8 * n + (tid >> 6), s = tid & 63;
      if (i < t.n && slot_row<DOWN>(t, s) >= 0) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < C::WK; ++w) v += rb[(w * 8 + (tid >> 6)) * RED_LD + s];
        const int tok = t.sh ? t.row + i : tb.row_tok[t.row + i];
        if constexpr (WT == W_MXFP4) v *= inverse_pow2(Product<WT, DOWN, NT>::template token_scale<true>(t, tb, i));
        v *= t.sh ? tb.shw[tok] : tb.row_w[t.row + i];
        yacc[tok * SLOTS + s] += v;
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
        if constexpr (WT == W_MXFP4) {
          const float inv = inverse_pow2(Product<WT, DOWN, NT>::template token_scale<false>(t, tb, i));
          gate *= inv;
          up *= inv;
        }
        // the hidden row is rounded to x's type, as the rows of the other forms are: 2^-9 of a
        // value on average, beside the 2^-9 of the output's own rounding
        const XT hx = (XT)(gate / (1.f + expf(-gate)) * up);
        const int f = t.sh ? a.fs : a.f;
        XT* hr = static_cast<XT*>(a.h) + (t.sh ? (size_t)a.T * a.k * a.f : 0);
        hr[(size_t)(t.row + i) * f + j] = hx;
        h = fabsf((float)hx);
      }
      if (WT == W_MXFP4) {
        const unsigned m = __reduce_max_sync(0xffffffffu, __float_as_uint(h));
        if (lane == 0 && i < t.n) atomicMax(a.hmax + (t.sh ? a.T * a.k : 0) + t.row + i, m);
      }
    }
    if (C::RED == 2) buf ^= 1;
    else consumer_sync();
  }
}

template <int WT, bool DOWN>
__device__ __forceinline__ void run_tile(const Args& a, Tables& tb, const Tile& t, Ring& r, uint32_t stages, float* red,
                                         float* yacc, int& buf) {
  if (t.nt == 1) run_pass<WT, DOWN, 1>(a, tb, t, r, stages, red, yacc, buf);
  else if (t.nt == 2) run_pass<WT, DOWN, 2>(a, tb, t, r, stages, red, yacc, buf);
  else run_pass<WT, DOWN, 4>(a, tb, t, r, stages, red, yacc, buf);
}

template <int WT>
__global__ void __launch_bounds__(THREADS, 1) few_kernel(const __grid_constant__ Args a,
                                                               const __grid_constant__ Maps maps) {
  using C = Cfg<WT>;
  using XT = typename C::XT;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t stages = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (stages - smem_u32(smem_raw));
  float* red = reinterpret_cast<float*>(smem + C::STAGES * stage_bytes<WT>());
  float* yacc = red + C::RED * red_floats<WT>();
  Tables& tb = *reinterpret_cast<Tables*>(yacc + YACC_FLOATS);
  Scratch& sc = *reinterpret_cast<Scratch*>(red);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = a.T;

  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&tb.full[s], 1 + 32 * X_WARPS);
      mbar_init(&tb.empty[s], WARPS);
    }
    tb.abort = 0;
    tb.n_act = 0;
    fence_barrier_init();
  }
  __syncthreads();

  if (warp == WARPS) {
    // ---------------------------------------------------------------- weights
    Ring r{0, 0};
    int issued = 0;
    auto stream = [&](auto walk) {
      constexpr bool DOWN = decltype(walk)::kDown;
      Tile t;
      while (walk.next(t))
        for (int k0 = 0; k0 < t.K && !tb.abort; k0 += t.seg) {
          wait(&tb.empty[r.stage], r.phase ^ 1u, tb);
          if (lane == 0) issue_w<WT, DOWN>(maps, t, k0, smem + r.stage * stage_bytes<WT>(), &tb.full[r.stage]);
          __syncwarp();
          ++issued;
          if (++r.stage == C::STAGES) { r.stage = 0; r.phase ^= 1u; }
        }
    };
    Walk<WT, false> w;
    if (a.fs > 0) {
      w.init(a, tb, true);
      stream(w);
    }
    __syncthreads();                       // the tables are there
    w.init(a, tb, false);
    stream(w);
    Walk<WT, true> wd;
    wd.init(a, tb, false);
    stream(wd);
    // nothing may still be landing in shared memory when the CTA leaves
    for (int i = 0; i < min(issued, C::STAGES); ++i) {
      r.phase ^= r.stage == 0 ? 1u : 0u;
      r.stage = (r.stage + C::STAGES - 1) % C::STAGES;
      if (lane == 0) mbar_wait(&tb.full[r.stage], r.phase, tb.abort ? kWaitLimitCycles / 100 : kWaitLimitCycles);
    }
  } else if (warp > WARPS) {
    // ---------------------------------------------------------------- tokens
    Ring r{0, 0};
    auto stream = [&](auto walk) {
      constexpr bool DOWN = decltype(walk)::kDown;
      Tile t;
      while (walk.next(t))
        for (int k0 = 0; k0 < t.K && !tb.abort; k0 += t.seg) {
          wait(&tb.empty[r.stage], r.phase ^ 1u, tb);
          issue_x<WT, DOWN>(a, tb, t, k0, stages + r.stage * stage_bytes<WT>(), &tb.full[r.stage], warp - WARPS - 1, lane);
          if (++r.stage == C::STAGES) { r.stage = 0; r.phase ^= 1u; }
        }
    };
    Walk<WT, false> w;
    if (a.fs > 0) {
      w.init(a, tb, true);
      stream(w);
    }
    __syncthreads();
    w.init(a, tb, false);
    stream(w);
    if (lane == 0) grid_wait(a.bar + 1, tb);     // the grid's hidden rows
    __syncwarp();
    Walk<WT, true> wd;
    wd.init(a, tb, false);
    stream(wd);
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ---------------------------------------------------------------- consumers
    Ring r{0, 0};
    int buf = 0;
    Tile t;
    router_logits<XT>(a, reinterpret_cast<float4*>(red));
    consumer_sync();
    if (tid == 0) grid_arrive(a.bar);
    if (WT == W_MXFP4) {
      for (int tok = warp; tok < T; tok += WARPS) {
        uint32_t m = 0;
        const uint4* row = reinterpret_cast<const uint4*>(static_cast<const XT*>(a.x) + (size_t)tok * a.d);
        for (int c = lane; c < a.d / 8; c += 32) {
          float v[8];
          unpack16(ldg_nc16(row + c), v, __nv_bfloat16());
#pragma unroll
          for (int u = 0; u < 8; ++u) m = max(m, __float_as_uint(v[u]) & 0x7fffffffu);
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) tb.xs[tok] = row_scale(m);
      }
    }
    if (!a.sink)
      for (int i = tid; i < T; i += CONSUMERS) tb.shw[i] = 1.f;
    consumer_sync();
    if (a.fs > 0) {
      Walk<WT, false> w;
      w.init(a, tb, true);
      while (w.next(t)) run_tile<WT, false>(a, tb, t, r, stages, red, yacc, buf);
    }
    if (tid == 0) grid_wait(a.bar, tb);
    consumer_sync();

    // the ring is empty now: it holds the warps' scores
    {
      float* sv = reinterpret_cast<float*>(smem) + warp * 2 * (MAX_N + 8);
      for (int t0 = warp; t0 < T; t0 += WARPS)
        select_token(a, tb, sc, t0, sv, reinterpret_cast<uint32_t*>(sv + MAX_N + 8));
    }
    fence_proxy_async();                   // before TMA writes there again
    consumer_sync();
    if (blockIdx.x == 0)
      for (int s = tid; s < T * a.k; s += CONSUMERS) {
        a.topk_idx[s] = sc.idx[s];
        a.topk_w[s] = sc.w[s];
      }
    build_tables(a, tb, sc);
    __syncthreads();                       // to the producer

    {
      Walk<WT, false> w;
      w.init(a, tb, false);
      while (w.next(t)) run_tile<WT, false>(a, tb, t, r, stages, red, yacc, buf);
    }
    // this CTA's hidden rows to the grid
    __threadfence();
    consumer_sync();
    if (tid == 0) {
      grid_arrive(a.bar + 1);
      if (WT == W_MXFP4) grid_wait(a.bar + 1, tb);
    }
    if (WT == W_MXFP4) {
      consumer_sync();
      for (int i = tid; i < T * a.k; i += CONSUMERS) tb.hs[i] = row_scale(__ldcg(a.hmax + i));
      for (int i = tid; i < T; i += CONSUMERS) tb.hs[MAX_T * MAX_K + i] = row_scale(__ldcg(a.hmax + T * a.k + i));
    }
    for (int i = tid; i < T * SLOTS; i += CONSUMERS) yacc[i] = 0.f;
    consumer_sync();

    Walk<WT, true> w;
    w.init(a, tb, false);
    XT* y = static_cast<XT*>(a.y);
    if (w.slots + (w.first < 0) == 0) {
      // nothing adds to any output
      for (size_t i = (size_t)blockIdx.x * CONSUMERS + tid; i < (size_t)T * a.d; i += (size_t)gridDim.x * CONSUMERS)
        y[i] = (XT)0.f;
    }
    while (w.next(t)) {
      run_tile<WT, true>(a, tb, t, r, stages, red, yacc, buf);
      if (!t.last) continue;
      consumer_sync();
      for (int i = tid; i < T * SLOTS; i += CONSUMERS) {
        const int j = slot_row<true>(t, i & (SLOTS - 1));
        if (j >= 0) y[(size_t)(i / SLOTS) * a.d + j] = (XT)yacc[i];
        yacc[i] = 0.f;
      }
      consumer_sync();
    }
  }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

template <int WT>
cudaError_t launch(const Args& a, const Maps& maps, size_t zero, cudaStream_t s) {
  const void* fn = (const void*)few_kernel<WT>;
  const int smem = smem_bytes<WT>();
  cudaError_t e = ensure_smem_attr(fn, smem);
  if (e != cudaSuccess) return e;
  e = cudaMemsetAsync(a.bar, 0, zero, s);
  if (e != cudaSuccess) return e;
  void* ptrs[] = {const_cast<Args*>(&a), const_cast<Maps*>(&maps)};
  return cudaLaunchCooperativeKernel(fn, dim3(sm_count()), dim3(THREADS), ptrs, smem, s);
}

// Workspace, in this order: barrier counters and row maxima (zeroed by every call), logits,
// hidden rows.
size_t zero_bytes(const moe_config_t& c) { return align256(256 + (size_t)c.T * (c.top_k + 1) * 4); }
size_t logit_bytes(const moe_config_t& c) {
  const int ld = c.n_experts + c.shared_sink;
  return align256((size_t)route_slices(ld, c.d_model) * c.T * ld * 4);
}

}  // namespace few

size_t few_workspace_bytes(const moe_config_t& c, int fs) {
  const size_t eb = c.x_dtype == MOE_DTYPE_F32 ? 4 : 2;
  return few::zero_bytes(c) + few::logit_bytes(c) +
         few::align256(((size_t)c.T * c.top_k * c.d_ff + (size_t)c.T * fs) * eb);
}

cudaError_t launch_few(const moe_config_t& c, int64_t capacity, const void* x, const float* w_gate,
                       const float* logit_offset, const float* bias, bool mxfp4, const void* const* w,
                       const uint8_t* const* sf, int fs, int32_t* topk_idx, float* topk_w, void* y, void* ws,
                       cudaStream_t s) {
  few::Args a{};
  few::Maps maps{};
  a.x = x;
  a.w_gate = w_gate;
  a.T = (int)c.T; a.d = c.d_model; a.f = c.d_ff; a.fs = fs; a.N = c.n_experts; a.k = c.top_k; a.sink = c.shared_sink;
  const bool f32 = c.x_dtype == MOE_DTYPE_F32;
  const int seg[2] = {mxfp4 ? few::Cfg<few::W_MXFP4>::seg(1) : f32 ? few::Cfg<few::W_F32>::seg(1) : few::Cfg<few::W_BF16>::seg(1),
                      mxfp4 ? few::Cfg<few::W_MXFP4>::seg(4) : f32 ? few::Cfg<few::W_F32>::seg(4) : few::Cfg<few::W_BF16>::seg(4)};
  for (int i = 0; i < (fs > 0 ? 6 : 3); ++i) {
    const bool down = i % 3 == few::M_W2, shared = i >= few::M_SHARED;
    const int width = shared ? fs : a.f, rows = down ? a.d : width, cols = down ? width : a.d;
    const uint64_t all = (uint64_t)(shared ? 1 : a.N) * rows;
    for (int v = 0; v < (a.T > 8 ? 2 : 1); ++v)          // the narrow boxes serve 9 tokens and more
      if (!(mxfp4 ? make_map_u4_rows8(&maps.m[i][v], w[i], all, cols, seg[v] / 128)
                  : make_map_rows8(&maps.m[i][v], w[i], f32, all, cols, seg[v])))
        return cudaErrorInvalidValue;
    a.sf[i] = mxfp4 ? sf[i] : nullptr;
  }
  a.capacity = capacity;
  a.route = rt::RouteArgs{logit_offset, bias, c.T, c.n_experts, c.top_k, c.score_fn, c.renorm, c.n_groups,
                          c.topk_groups, c.group_score_topn, nullptr, nullptr, nullptr, nullptr, nullptr,
                          c.shared_sink, nullptr, nullptr};
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.y = y;
  uint8_t* p = static_cast<uint8_t*>(ws);
  const size_t zero = few::zero_bytes(c);
  a.bar = reinterpret_cast<unsigned*>(p);
  a.hmax = reinterpret_cast<unsigned*>(p + 256);
  a.logits = reinterpret_cast<float*>(p + zero);
  a.h = p + zero + few::logit_bytes(c);
  if (mxfp4) return few::launch<few::W_MXFP4>(a, maps, zero, s);
  if (f32) return few::launch<few::W_F32>(a, maps, zero, s);
  return few::launch<few::W_BF16>(a, maps, zero, s);
}

}  // namespace moe
