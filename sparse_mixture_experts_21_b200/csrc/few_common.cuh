// Parts of the few-token layer (few.cu) that do not depend on the weights' type:
// arguments, waits, router, selection, token tables, the schedule of weight tiles.
#pragma once

#include <stddef.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace few {

constexpr int MAX_T = 64, MAX_N = 512, MAX_K = 16;
constexpr int WORKERS = 16;                     // warps of the router's first part
constexpr int SLOTS = 64;                       // rows of a down tile
constexpr int ROUTE_TILE = 16, ROUTE_COLS = 1024;   // router: experts and columns at a time
constexpr int LOCAL_T = 2;                      // up to here every CTA selects for all tokens
enum { BAR_LOGITS = 0, BAR_PICKS = 16, BAR_HIDDEN = 32, BAR_X = 48 };

// The six expert stacks [experts * rows, cols]: W1, W3, W2 routed, then shared.
enum { M_W1 = 0, M_W3 = 1, M_W2 = 2, M_SHARED = 3 };

struct Args {
  const void* x;
  const float* w_gate;
  const uint8_t* q[6];     // MXFP4: codes of the stacks
  const uint8_t* sf[6];    // and their tile-atom scales
  int T, d, f, fs, N, k, sink;
  int64_t capacity;
  rt::RouteArgs route;     // selection options
  int32_t* topk_idx;
  float* topk_w;
  void* y;
  unsigned* bar;           // grid counters BAR_*, zero at launch
  unsigned* hmax;          // MXFP4: [T k + T] largest |h| of each hidden row as bits, zero at launch
  float* shw;              // [T] shared expert's weights (sink)
  float* logits;           // [slices, T, N + sink] partial sums
  void* x16;               // MXFP4: [T, d] x in fp16, times xscale [T]
  float* xscale;
  void* h;                 // [T k, f] routed, then [T, fs] shared; x's type
};

// The selecting warp's.
constexpr int PART = 1536;           // partial sums of logits at a time
struct Scratch {
  union {
    struct {
      float sv[MAX_N + 8];           // affinities of a token
      uint32_t q[MAX_N];             // its selection scores, as keys
    };
    float w[MAX_T * MAX_K];          // then all picks' weights
  };
  union {
    alignas(16) float part[PART];
    struct {
      int16_t e[MAX_T * MAX_K];      // then all picks
      unsigned mask[MAX_N][2];       // tokens of each expert
    };
  };
  float wl[LOCAL_T * MAX_K];         // picks of one or two tokens
  int16_t el[LOCAL_T * MAX_K];
};
static_assert(PART >= MAX_N + 4, "a slice at a time");
// What selection leaves for the rest of the kernel.
struct Tables {
  int16_t row0[MAX_N + 1];           // first row of each expert; rows of e: row0[e] .. row0[e + 1]
  int16_t act[MAX_N];                // met experts, ascending
  uint8_t row_tok[MAX_T * MAX_K];
  float row_w[MAX_T * MAX_K];
  float shw[MAX_T];
  float xs[MAX_T];                   // MXFP4: scale of each token's x
  uint32_t xmax[2];
  uint64_t full[4], empty[4];
  int32_t n_act;
  volatile int32_t abort;
  int32_t redo[2];                   // MXFP4: this CTA's hidden rows or outputs hold some that are not finite
  union {
    Scratch sc;                      // while selecting
    float hs[MAX_T * MAX_K + MAX_T]; // then, MXFP4: scale of each hidden row
  };
};

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
// Arrive at a grid counter; wait until it has its arrivals.
__device__ __forceinline__ void grid_arrive(unsigned* bar) {
  __threadfence();
  atomicAdd(bar, 1u);
}
__device__ __forceinline__ void grid_wait(unsigned* bar, unsigned target, Tables& tb) {
  const long long t0 = clock64();
  for (;;) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(bar) : "memory");
    if (v >= target || tb.abort) return;
    if (clock64() - t0 > kWaitLimitCycles) {
      flag_timeout();
      tb.abort = 1;
    }
  }
}
__device__ __forceinline__ void worker_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * WORKERS) : "memory"); }

// ------------------------------------------------------------------ router
// Logits in K slices: tiles of 16 experts (a warp each) by `slices` column ranges, spread over
// the grid, so that a CTA reads a slice of x and not all of it.  A warp holds its expert's
// slice in registers; eight tokens' columns at a time pass through shared memory as fp32, the
// next eight already on their way.  Partial sums to memory, added by the selection.
__host__ __device__ __forceinline__ int route_tiles(int ld) { return (ld + ROUTE_TILE - 1) / ROUTE_TILE; }
// One job for every SM of the grid (144 in all), slices of at least 256 columns and 16 at most
// (the selection adds them one by one), but none wider than the registers hold.
// With up to WHOLE_T tokens x is little to read and every CTA takes two experts' whole rows:
// no partial sums (their adding up would be the selection's longest step: 13 us of one warp
// for 256 experts in 9 slices, under the shared experts' stream).
constexpr int WHOLE_T = 4;
__host__ __device__ __forceinline__ int route_slices(int ld, int d, int T) {
  if (T <= WHOLE_T) return 1;
  int n = 144 / route_tiles(ld);
  const int most = (d + 255) / 256, least = (d + ROUTE_COLS - 1) / ROUTE_COLS;
  n = n < most ? n : most;
  n = n < 16 ? n : 16;
  return n > least ? n : least;
}
// Floats between the rows of the partial sums: a row is copied 16 bytes at a time.
__host__ __device__ __forceinline__ int route_ld(int ld) { return (ld + 3) & ~3; }
__device__ __forceinline__ void ldg_quad(const float* p, uint4& v) { v = ldg_nc16(p); }
__device__ __forceinline__ void ldg_quad(const __nv_bfloat16* p, uint2& v) {
  v = __ldg(reinterpret_cast<const uint2*>(p));
}
__device__ __forceinline__ float4 quad_f32(const uint4& v) {
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ float4 quad_f32(const uint2& v) {
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xffff0000u));
}
template <typename XT> struct Quad { using T = uint2; };
template <> struct Quad<float> { using T = uint4; };

// Whole rows: warps 0, 2, .. take expert blockIdx.x (+ 2 grid ..), the others the one a grid
// further, an eighth of the columns each; part: 64 floats of shared memory.
template <typename XT>
__device__ __forceinline__ void router_logits_whole(const Args& a, float* part) {
  constexpr int SL = WORKERS / 2;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, P = gridDim.x;
  const int ld = a.N + a.sink, quads = a.d / 4;
  const XT* x = static_cast<const XT*>(a.x);
  for (int e0 = blockIdx.x; e0 < ld; e0 += 2 * P) {
    const int e = e0 + (warp & 1) * P;
    const float4* wg = reinterpret_cast<const float4*>(a.w_gate + (size_t)min(e, ld - 1) * a.d);
    float acc[WHOLE_T] = {};
#pragma unroll 4
    for (int q = (warp >> 1) * 32 + lane; q < quads; q += 32 * SL) {
      const float4 w = __ldg(wg + q);
#pragma unroll
      for (int j = 0; j < WHOLE_T; ++j) {
        if (j >= a.T) break;
        typename Quad<XT>::T v;
        ldg_quad(x + (size_t)j * a.d + 4 * q, v);
        const float4 b = quad_f32(v);
        acc[j] = fmaf(w.x, b.x, fmaf(w.y, b.y, fmaf(w.z, b.z, fmaf(w.w, b.w, acc[j]))));
      }
    }
#pragma unroll
    for (int j = 0; j < WHOLE_T; ++j) {
      acc[j] = warp_sum(acc[j]);
      if (lane == 0) part[warp * WHOLE_T + j] = acc[j];
    }
    worker_sync();
    if (tid < 2 * WHOLE_T) {
      const int j = tid >> 1, i = tid & 1;
      float v = 0.f;
#pragma unroll
      for (int s = 0; s < SL; ++s) v += part[(2 * s + i) * WHOLE_T + j];
      if (j < a.T && e0 + i * P < ld) a.logits[(size_t)j * route_ld(ld) + e0 + i * P] = v;
    }
    worker_sync();
  }
}

// By the CTA's first 16 warps; part: 32 KB of shared memory.
template <typename XT>
__device__ __forceinline__ void router_logits(const Args& a, float* part) {
  if (a.T <= WHOLE_T) {
    router_logits_whole<XT>(a, part);
    return;
  }
  float4* xs = reinterpret_cast<float4*>(part);
  constexpr int QUADS = ROUTE_COLS / 4, PER = 8 * QUADS / (32 * WORKERS);   // a thread's share of eight tokens
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ld = a.N + a.sink, tiles = route_tiles(ld), slices = route_slices(ld, a.d, a.T);
  const int quads = (a.d / 4 + slices - 1) / slices;
  const XT* x = static_cast<const XT*>(a.x);
  for (int job = blockIdx.x; job < tiles * slices; job += gridDim.x) {
    const int s = job / tiles, e = (job - s * tiles) * ROUTE_TILE + warp;
    const int q0 = s * quads, nq = min(quads, a.d / 4 - q0);       // nq <= 0: an empty slice, sums of 0
    typename Quad<XT>::T v[PER];
    auto fetch = [&](int t0) {
#pragma unroll
      for (int u = 0; u < PER; ++u) {
        const int i = tid + 32 * WORKERS * u, t = t0 + i / QUADS, q = i % QUADS;
        if (t < a.T && q < nq) ldg_quad(x + (size_t)t * a.d + 4 * (q0 + q), v[u]);
        else v[u] = typename Quad<XT>::T{};
      }
    };
    fetch(0);
    const float4* wg = reinterpret_cast<const float4*>(a.w_gate + (size_t)min(e, ld - 1) * a.d) + q0;
    float4 w[QUADS / 32];
#pragma unroll
    for (int u = 0; u < QUADS / 32; ++u)
      w[u] = lane + 32 * u < nq ? __ldg(wg + lane + 32 * u) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int t0 = 0; t0 < a.T; t0 += 8) {
      const int n = min(8, a.T - t0);
#pragma unroll
      for (int u = 0; u < PER; ++u) xs[tid + 32 * WORKERS * u] = quad_f32(v[u]);
      worker_sync();
      fetch(t0 + 8);
      float mine = 0.f;                       // lane j: token t0 + j
#pragma unroll 2
      for (int j = 0; j < n; ++j) {
        float p = 0.f;
#pragma unroll
        for (int u = 0; u < QUADS / 32; ++u) {
          const float4 b = xs[j * QUADS + lane + 32 * u];
          p = fmaf(w[u].x, b.x, p);
          p = fmaf(w[u].y, b.y, p);
          p = fmaf(w[u].z, b.z, p);
          p = fmaf(w[u].w, b.w, p);
        }
        p = warp_sum(p);
        if (lane == j) mine = p;
      }
      if (lane < n && e < ld) a.logits[((size_t)s * a.T + t0 + lane) * route_ld(ld) + e] = mine;
      worker_sync();
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

// Selection for token t by one warp: moe_route's formulas, ties and order, in loops instead of
// registers (a few tokens meet this code once, cold: its size counts more than its steps).
// dry (N = 1, k = 1, t = 0): all of its steps on some word of x, and no results.
__device__ __noinline__ void select_token(const Args& a, Tables& tb, int t, int N, int k, bool dry) {
  Scratch& sc = tb.sc;
  float* sv = sc.sv;
  uint32_t* q = sc.q;
  const int lane = threadIdx.x & 31;
  const int ld = N + a.sink, slices = dry ? 1 : route_slices(ld, a.d, a.T);
  const rt::RouteArgs& r = a.route;
  // the slices' sums, through shared memory: one wait for as many as fit
  const int ldp = route_ld(ld), per = PART / ldp;
#pragma unroll 1
  for (int s0 = 0; s0 < slices; s0 += per) {
    const int n = min(per, slices - s0);
#pragma unroll 1
    for (int s = 0; s < n; ++s) {
      const float* src = dry ? static_cast<const float*>(a.x) : a.logits + ((size_t)(s0 + s) * a.T + t) * ldp;
#pragma unroll 1
      for (int c = 4 * lane; c < ldp; c += 128) cp_async16(smem_u32(sc.part + s * ldp + c), src + c);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
#pragma unroll 1
    for (int e = lane; e < ld; e += 32) {
      float z = s0 ? sv[e] : 0.f;
#pragma unroll 4
      for (int s = 0; s < n; ++s) z += sc.part[s * ldp + e];
      sv[e] = z;
    }
    __syncwarp();
  }
  float m = -INFINITY;
#pragma unroll 1
  for (int e = lane; e < ld; e += 32) {
    if (r.logit_offset && e < N) sv[e] += r.logit_offset[e];
    m = fmaxf(m, sv[e]);
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
    const int per = 32 / r.n_groups;
    if (r.group_topn <= 2 && per * r.n_groups == 32) {
      // the usual case, all groups at once: `per` lanes each keep a group's two best, then merge
      const int g = lane / per;
      uint32_t k1 = 0, k2 = 0;
#pragma unroll 1
      for (int e = g * size + lane % per; e < (g + 1) * size; e += per) {
        const uint32_t v = q[e];
        k2 = max(k2, min(k1, v));
        k1 = max(k1, v);
      }
#pragma unroll 1
      for (int o = 1; o < per; o <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(0xffffffffu, k1, o), o2 = __shfl_xor_sync(0xffffffffu, k2, o);
        k2 = max(max(k2, o2), min(k1, o1));
        k1 = max(k1, o1);
      }
      const uint32_t score = f32_key(r.group_topn == 1 ? 0.f + key_f32(k1) : key_f32(k1) + key_f32(k2));
      mine = __shfl_sync(0xffffffffu, score, (lane % r.n_groups) * per);
    } else {
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
    }
    uint32_t kept = 0;
#pragma unroll 1
    for (int i = 0; i < r.topk_groups; ++i) {
      const bool open = lane < r.n_groups && !((kept >> lane) & 1u);
      const uint32_t best = __reduce_max_sync(0xffffffffu, open ? mine : 0u);
      kept |= 1u << __reduce_min_sync(0xffffffffu, open && mine == best ? lane : 31);
    }
#pragma unroll 1
    for (int g = 0; g < r.n_groups; ++g)
      if (!((kept >> g) & 1u))
        for (int e = g * size + lane; e < (g + 1) * size; e += 32) q[e] = 0;
    __syncwarp();
  }
  // k picks: each lane holds the best of its experts (e = lane mod 32) not yet picked; the
  // winner looks for its next
  uint32_t bk = 0, key = 0xffffffffu;
  int bi = 0x7fffffff, idx = -1, my = 0x7fffffff;
  bool stale = true;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    if (stale) {
      bk = 0;
      bi = 0x7fffffff;
      for (int e = lane; e < N; e += 32) {
        const uint32_t v = q[e];
        if ((v < key || (v == key && e > idx)) && v > bk) { bk = v; bi = e; }
      }
    }
    key = __reduce_max_sync(0xffffffffu, bk);
    idx = (int)__reduce_min_sync(0xffffffffu, bk == key && bk > 0 ? (uint32_t)bi : 0x7fffffffu);
    stale = bi == idx;
    if (lane == j) my = idx;
  }
  const float s = lane < k && my < N ? sv[my] : 0.f;
  const float sh = a.sink ? sv[N] : 0.f;
  const float sum = warp_sum(s) + sh;
  const float w = r.renorm ? s / sum : s;
  if (dry) return;
  // the CTA that owns the token writes the outputs
  if (lane < k) {
    if (a.T <= LOCAL_T) {
      sc.el[t * k + lane] = (int16_t)my;
      sc.wl[t * k + lane] = w;
    }
    if (t % (int)gridDim.x == (int)blockIdx.x) {
      a.topk_idx[t * k + lane] = my;
      a.topk_w[t * k + lane] = w;
    }
  }
  if (lane == 0 && a.sink) {
    tb.shw[t] = r.renorm ? sh / sum : sh;
    if (t % (int)gridDim.x == (int)blockIdx.x) a.shw[t] = tb.shw[t];
  }
  __syncwarp();
}

// Experts' token masks, met experts in ascending order, rows (expert major, tokens
// ascending); a token past its expert's capacity gets no row.  By one warp.
// dry (N = 1, n = 1): as if one slot had picked expert 0.
__device__ __noinline__ void build_tables(const Args& a, Tables& tb, int N, int n, bool dry) {
  Scratch& sc = tb.sc;
  const int lane = threadIdx.x & 31;
  for (int e = lane; e < N; e += 32) sc.mask[e][0] = sc.mask[e][1] = 0;
  if (a.T <= LOCAL_T) {
    if (lane < n) {
      const int e = dry ? 0 : sc.el[lane];
      sc.e[lane] = (unsigned)e < (unsigned)N ? (int16_t)e : (int16_t)-1;
      sc.w[lane] = sc.wl[lane];
    }
  } else {                                    // the picks that the grid wrote
#pragma unroll 4
    for (int s = lane; s < n; s += 32) {
      const int e = dry ? 0 : __ldcg(a.topk_idx + s);
      const float w = dry ? 0.f : __ldcg(a.topk_w + s);
      sc.e[s] = (unsigned)e < (unsigned)N ? (int16_t)e : (int16_t)-1;
      sc.w[s] = w;
    }
    if (a.sink)
      for (int t = lane; t < a.T; t += 32) tb.shw[t] = __ldcg(a.shw + t);
  }
  if (!a.sink)
    for (int t = lane; t < a.T; t += 32) tb.shw[t] = 1.f;
  __syncwarp();
  for (int s = lane; s < n; s += 32) {
    const int e = sc.e[s], t = s / a.k;
    if ((unsigned)e < (unsigned)N) atomicOr(&sc.mask[e][t >> 5], 1u << (t & 31));
    else flag_invalid_index();
  }
  __syncwarp();
  int rows = 0, act = 0;
#pragma unroll 1
  for (int base = 0; base < N; base += 32) {
    const int e = base + lane;
    int c = e < N ? __popc(sc.mask[e][0]) + __popc(sc.mask[e][1]) : 0;
    if (c > a.capacity) c = (int)a.capacity;
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const unsigned met = __ballot_sync(0xffffffffu, c > 0);
    if (e < N) tb.row0[e + 1] = (int16_t)(rows + incl);
    if (c > 0) tb.act[act + __popc(met & ((1u << lane) - 1u))] = (int16_t)e;
    rows += __shfl_sync(0xffffffffu, incl, 31);
    act += __popc(met);
  }
  if (lane == 0) {
    tb.row0[0] = 0;
    tb.n_act = act;
  }
  __syncwarp();
  for (int s = lane; s < n; s += 32) {
    const int e = sc.e[s], t = s / a.k;
    if ((unsigned)e >= (unsigned)N) continue;
    const unsigned below = t < 32 ? __popc(sc.mask[e][0] & ((1u << t) - 1u))
                                  : __popc(sc.mask[e][0]) + __popc(sc.mask[e][1] & ((1u << (t - 32)) - 1u));
    if ((int64_t)below < a.capacity) {
      tb.row_tok[tb.row0[e] + below] = (uint8_t)t;
      tb.row_w[tb.row0[e] + below] = sc.w[s];
    }
  }
}

// The selecting warp's whole part.  One or two tokens: every CTA selects for all by itself.
// More: token t on CTA t, and all CTAs read the picks when they are there.
__device__ __forceinline__ void select_and_build(const Args& a, Tables& tb) {
  const int lane = threadIdx.x & 31;
  // The code comes from memory line by line, longer than its steps take: once through it while
  // the logits are under way (one token of 256 experts: the tables stand after 16 us instead of
  // 23, the layer takes 140 us in bf16 instead of 147, 94 in MXFP4 instead of 101).
  const bool local = a.T <= LOCAL_T;
  if (local || (int)blockIdx.x < a.T) select_token(a, tb, 0, 1, 1, true);
  build_tables(a, tb, 1, 1, true);
  __syncwarp();
  if (lane == 0) grid_wait(a.bar + BAR_LOGITS, gridDim.x, tb);
  __syncwarp();
  for (int t = local ? 0 : (int)blockIdx.x; t < a.T; t += local ? 1 : (int)gridDim.x)
    select_token(a, tb, t, a.N, a.k, false);
  if (!local) {
    if (lane == 0) {
      if ((int)blockIdx.x < a.T) grid_arrive(a.bar + BAR_PICKS);
      grid_wait(a.bar + BAR_PICKS, min(a.T, (int)gridDim.x), tb);
    }
    __syncwarp();
  }
  build_tables(a, tb, a.N, a.T * a.k, false);
}

// ------------------------------------------------------------------ schedule
// One pass over one tile of weight rows by some of one expert's tokens.  Producers and consumers walk the
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
  int nt, sub, seg;   // 8-token columns; column ranges of a stage, columns of a stage
  bool sh, last;      // last: the tile's last pass (down: of the last expert)
};

// C::seg(nt): columns of a stage; C::GATE_UNITS: units of a gate/up tile; C::PASS: tokens of an
// expert per pass over its weights; C::SPLIT: two column ranges a stage for narrow down tiles.
template <class C, bool DOWN>
struct Walk {
  static constexpr bool kDown = DOWN;
  const Args* g;
  const Tables* tb;
  int u, u1, per;     // units: next, end; per expert (gate/up)
  int slot, slots, first;
  int done;           // tokens of earlier passes
  bool sh;

  // gate/up: shared or routed part; down: both, the shared expert first (slot -1)
  __device__ Walk(const Args& a, const Tables& t, bool shared) {
    g = &a; tb = &t; sh = shared; done = 0;
    const int P = gridDim.x, b = blockIdx.x;
    per = (shared ? a.fs : a.f) / 8;
    const int64_t all = DOWN ? a.d / 8 : shared ? per : (int64_t)t.n_act * per;
    u = (int)(all * b / P);
    u1 = (int)(all * (b + 1) / P);
    first = DOWN && a.fs > 0 ? -1 : 0;
    slots = DOWN ? t.n_act : 0;
    slot = first;
    if (DOWN && empty()) u = u1;
  }
  __device__ bool empty() const { return slots + (first < 0) == 0; }     // down: no expert at all
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
    t.nu = min(DOWN ? SLOTS / 8 : C::GATE_UNITS, u1 - u);
    if (!DOWN) t.nu = min(t.nu, per - j);
    t.base = 8 * j;
    const int f = shared ? g->fs : g->f;
    t.K = DOWN ? f : g->d;
    t.erow = e * (DOWN ? g->d : f);
    t.ma = (DOWN ? M_W2 : M_W1) + (shared ? M_SHARED : 0);
    t.mb = M_W3 + (shared ? M_SHARED : 0);
    const int n = shared ? g->T : tb->row0[e + 1] - tb->row0[e];
    t.n = min(n - done, C::PASS);
    t.row = (shared ? 0 : tb->row0[e]) + done;
    t.nt = t.n <= 8 ? 1 : t.n <= 16 ? 2 : 4;
    // a narrow down tile takes two column ranges a stage, for warps and bytes in flight that a
    // wide one gets from its rows
    t.sub = DOWN && C::SPLIT && t.nt == 1 && t.nu <= 2 ? 2 : 1;
    t.seg = C::seg(t.nt) * t.sub;
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

// A place in the ring of stages.
struct Ring {
  uint32_t stage, phase;
  __device__ __forceinline__ void next(uint32_t stages) {
    if (++stage == stages) { stage = 0; phase ^= 1u; }
  }
};

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace, in this order: grid counters and hidden rows' maxima (zeroed by every call), shared
// weights, logits, hidden rows.
size_t zero_bytes(const moe_config_t& c) { return align256(256 + (size_t)c.T * (c.top_k + 1) * 4); }
size_t shw_bytes(const moe_config_t& c) { return align256((size_t)c.T * 4); }
size_t x16_bytes(const moe_config_t& c) { return align256((size_t)c.T * c.d_model * 2); }
size_t logit_bytes(const moe_config_t& c) {
  const int ld = c.n_experts + c.shared_sink;
  return align256((size_t)route_slices(ld, c.d_model, (int)c.T) * c.T * route_ld(ld) * 4);
}

}  // namespace few

}  // namespace moe
