// A whole MoE layer for few tokens (1 .. 64), in one launch: router, top-k, routed and
// shared experts, weighted sum.
//
//   y_t = sum_j w_tj W2_e (silu(W1_e x_t) * (W3_e x_t)) + shared(x_t)
//
// Bound: the bytes of the weights of the experts that at least one token picks (and of the
// router and the shared expert); every weight is read once, from HBM.
//
// One cooperative launch, one CTA per SM, two barriers over the grid:
//   logits     each CTA takes whole experts of the router, all tokens
//   -- barrier --
//   selection  every CTA selects for all tokens by itself (the same result everywhere,
//              without a third barrier) and builds the experts' token lists
//   gate/up    the hidden units of the shared and the met experts, cut evenly over the grid
//   -- barrier --
//   down       each CTA takes rows of W2 of all met experts, so a token's sum over its
//              experts stays inside one CTA: fixed order, no atomics, no second pass
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace few {

constexpr int MAX_T = 64, MAX_N = 512, MAX_K = 16;
constexpr int WARPS = 16, THREADS = 32 * WARPS;
enum { W_F32 = 0, W_BF16 = 1, W_MXFP4 = 2 };

struct Matrix {            // an expert stack: [experts * rows, cols]
  const void* w;           // values, or packed E2M1 codes
  const uint8_t* sf;       // MXFP4: tile-atom scales
};

struct Args {
  const void* x;
  const float* w_gate;
  Matrix w1, w3, w2, ws1, ws3, ws2;
  int T, d, f, fs, N, k, sink;
  int64_t capacity;
  rt::RouteArgs route;     // selection options (outputs set by the kernel)
  int32_t* topk_idx;
  float* topk_w;
  void* y;
  unsigned* bar;           // two barrier counters, zero at launch
  float* logits;           // [T, N + sink]
  void* h;                 // [T k, f] routed, then [T, fs] shared; x's type
};

template <int WT> struct Elem { using T = __nv_bfloat16; };
template <> struct Elem<W_F32> { using T = float; };

struct Tables {
  int32_t idx[MAX_T * MAX_K];
  float w[MAX_T * MAX_K];
  float lse[MAX_T], shw[MAX_T];
  unsigned mask[MAX_N][2];           // tokens of each expert
  int16_t row0[MAX_N];               // first row of each expert
  int16_t act[MAX_N];                // met experts, ascending
  int32_t n_act;
  uint8_t row_tok[MAX_T * MAX_K];
  float row_w[MAX_T * MAX_K];
  int32_t abort;
};

// Arrive, then wait for the whole grid (bounded: false after kWaitLimitCycles).
__device__ __forceinline__ void grid_arrive(unsigned* bar) {
  __threadfence();
  atomicAdd(bar, 1u);
}
__device__ __forceinline__ bool grid_poll(unsigned* bar) {
  const long long t0 = clock64();
  for (;;) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(bar) : "memory");
    if (v >= gridDim.x) return true;
    if (clock64() - t0 > kWaitLimitCycles) {
      flag_timeout();
      return false;
    }
  }
}

// Selection for all T tokens by the CTA's warps (kept out of line: it needs more registers
// than the rest of the kernel).
template <int NV>
__device__ __noinline__ void select_all(const float* logits, int ld, const rt::RouteArgs& a) {
  float pacc[NV];
  rt::select_tokens<NV, WARPS>(logits, ld, (int)a.T, 0, a, pacc);
}

// Experts' token masks, met experts in ascending order, rows (expert major, tokens
// ascending); a token past its expert's capacity gets no row.
__device__ void build_tables(const Args& a, Tables& tb) {
  const int tid = threadIdx.x, n = a.T * a.k;
  for (int e = tid; e < a.N; e += THREADS) tb.mask[e][0] = tb.mask[e][1] = 0;
  __syncthreads();
  for (int s = tid; s < n; s += THREADS) {
    const int e = tb.idx[s], t = s / a.k;
    if ((unsigned)e < (unsigned)a.N) atomicOr(&tb.mask[e][t >> 5], 1u << (t & 31));
    else flag_invalid_index();
  }
  __syncthreads();
  if (tid < 32) {
    int rows = 0, act = 0;
    for (int base = 0; base < a.N; base += 32) {
      const int e = base + tid;
      int c = e < a.N ? __popc(tb.mask[e][0]) + __popc(tb.mask[e][1]) : 0;
      if (c > a.capacity) c = (int)a.capacity;
      int incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (tid >= o) incl += v;
      }
      const unsigned met = __ballot_sync(0xffffffffu, c > 0);
      if (e < a.N) tb.row0[e] = (int16_t)(rows + incl - c);
      if (c > 0) tb.act[act + __popc(met & ((1u << tid) - 1u))] = (int16_t)e;
      rows += __shfl_sync(0xffffffffu, incl, 31);
      act += __popc(met);
    }
    if (tid == 0) tb.n_act = act;
  }
  __syncthreads();
  for (int s = tid; s < n; s += THREADS) {
    const int e = tb.idx[s], t = s / a.k;
    if ((unsigned)e >= (unsigned)a.N) continue;
    const unsigned below = t < 32 ? __popc(tb.mask[e][0] & ((1u << t) - 1u))
                                  : __popc(tb.mask[e][0]) + __popc(tb.mask[e][1] & ((1u << (t - 32)) - 1u));
    if ((int64_t)below < a.capacity) {
      tb.row_tok[tb.row0[e] + below] = (uint8_t)t;
      tb.row_w[tb.row0[e] + below] = tb.w[s];
    }
  }
  __syncthreads();
}
__device__ __forceinline__ int rows_of(const Args& a, const Tables& tb, int e) {
  const int c = __popc(tb.mask[e][0]) + __popc(tb.mask[e][1]);
  return c > a.capacity ? (int)a.capacity : c;
}

// Eight weights of a row (a global row of the stack) from column c.
template <int WT>
__device__ __forceinline__ void load_w(const Matrix& m, int64_t row, int cols, int c, float* f) {
  if constexpr (WT == W_MXFP4) {
    const uint32_t q = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(m.w) + (row * cols + c) / 2);
    const float s = mx4::e8m0_value(m.sf[mx::atom_byte(row >> 7, cols / 128, c >> 7, (int)(row & 127), (c >> 5) & 3)]);
#pragma unroll
    for (int u = 0; u < 8; ++u) f[u] = mx4::e2m1_value(q >> (4 * u)) * s;
  } else {
    mx4::load8(static_cast<const typename Elem<WT>::T*>(m.w) + row * cols + c, f);
  }
}
__device__ __forceinline__ void load_cg(const __nv_bfloat16* p, float* f) {
  unpack16(__ldcg(reinterpret_cast<const uint4*>(p)), f, __nv_bfloat16());
}
__device__ __forceinline__ void load_cg(const float* p, float* f) {
  unpack16(__ldcg(reinterpret_cast<const uint4*>(p)), f, 0.f);
  unpack16(__ldcg(reinterpret_cast<const uint4*>(p) + 1), f + 4, 0.f);
}

template <int WT>
__global__ void __launch_bounds__(THREADS, 1) few_kernel(const __grid_constant__ Args a) {
  using XT = typename Elem<WT>::T;
  extern __shared__ __align__(16) uint8_t smem[];
  Tables& tb = *reinterpret_cast<Tables*>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int P = gridDim.x, T = a.T, d = a.d;
  const XT* x = static_cast<const XT*>(a.x);
  XT* h = static_cast<XT*>(a.h);
  const int ld = a.N + a.sink;

  // logits: one warp per (expert, token)
  for (int i = blockIdx.x * WARPS + warp; i < ld * T; i += P * WARPS) {
    const int e = i % ld, t = i / ld;
    float acc = 0.f;
    for (int c = lane * 8; c < d; c += 256) {
      float xv[8], wv[8];
      mx4::load8(x + (int64_t)t * d + c, xv);
      mx4::load8(a.w_gate + (int64_t)e * d + c, wv);
#pragma unroll
      for (int u = 0; u < 8; ++u) acc = fmaf(xv[u], wv[u], acc);
    }
    acc = warp_sum(acc);
    if (lane == 0) a.logits[(int64_t)t * ld + e] = acc;
  }
  __syncthreads();
  if (tid == 0) {
    grid_arrive(a.bar);
    tb.abort = !grid_poll(a.bar);
  }
  __syncthreads();
  if (tb.abort) return;

  rt::RouteArgs ra = a.route;
  ra.topk_idx = tb.idx;
  ra.topk_w = tb.w;
  ra.lse = tb.lse;
  ra.shared_w = tb.shw;
  if (a.N <= 32) select_all<1>(a.logits, ld, ra);
  else if (a.N <= 64) select_all<2>(a.logits, ld, ra);
  else if (a.N <= 128) select_all<4>(a.logits, ld, ra);
  else if (a.N <= 256) select_all<8>(a.logits, ld, ra);
  else select_all<16>(a.logits, ld, ra);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int s = tid; s < T * a.k; s += THREADS) {
      a.topk_idx[s] = tb.idx[s];
      a.topk_w[s] = tb.w[s];
    }
  build_tables(a, tb);

  // gate/up: one warp per hidden unit
  const int64_t units = a.fs + (int64_t)tb.n_act * a.f;
  for (int64_t u = (int64_t)blockIdx.x * WARPS + warp; u < units; u += (int64_t)P * WARPS) {
    const bool sh = u < a.fs;
    const int slot = sh ? 0 : (int)((u - a.fs) / a.f);
    const int j = sh ? (int)u : (int)((u - a.fs) - (int64_t)slot * a.f);
    const int e = sh ? 0 : tb.act[slot];
    const int n = sh ? T : rows_of(a, tb, e), r0 = sh ? 0 : tb.row0[e];
    const int f = sh ? a.fs : a.f;
    const int64_t wrow = (int64_t)e * f + j;
    XT* hr = sh ? h + (int64_t)T * a.k * a.f : h;
    for (int i = 0; i < n; ++i) {
      const int t = sh ? i : tb.row_tok[r0 + i];
      float g = 0.f, up = 0.f;
      for (int c = lane * 8; c < d; c += 256) {
        float xv[8], wv[8];
        mx4::load8(x + (int64_t)t * d + c, xv);
        load_w<WT>(sh ? a.ws1 : a.w1, wrow, d, c, wv);
#pragma unroll
        for (int q = 0; q < 8; ++q) g = fmaf(xv[q], wv[q], g);
        load_w<WT>(sh ? a.ws3 : a.w3, wrow, d, c, wv);
#pragma unroll
        for (int q = 0; q < 8; ++q) up = fmaf(xv[q], wv[q], up);
      }
      g = warp_sum(g);
      up = warp_sum(up);
      if (lane == 0) hr[(int64_t)(r0 + i) * f + j] = (XT)(g / (1.f + expf(-g)) * up);
    }
  }
  __syncthreads();
  if (tid == 0) {
    grid_arrive(a.bar + 1);
    tb.abort = !grid_poll(a.bar + 1);
  }
  __syncthreads();
  if (tb.abort) return;

  // down: one warp per output column, tokens on lanes (t and t + 32)
  for (int j = blockIdx.x * WARPS + warp; j < d; j += P * WARPS) {
    float y0 = 0.f, y1 = 0.f;
    for (int s = a.fs > 0 ? -1 : 0; s < tb.n_act; ++s) {
      const bool sh = s < 0;
      const int e = sh ? 0 : tb.act[s];
      const int n = sh ? T : rows_of(a, tb, e), r0 = sh ? 0 : tb.row0[e];
      const int f = sh ? a.fs : a.f;
      const XT* hr = sh ? h + (int64_t)T * a.k * a.f : h;
      for (int i = 0; i < n; ++i) {
        const int t = sh ? i : tb.row_tok[r0 + i];
        float acc = 0.f;
        for (int c = lane * 8; c < f; c += 256) {
          float hv[8], wv[8];
          load_cg(hr + (int64_t)(r0 + i) * f + c, hv);
          load_w<WT>(sh ? a.ws2 : a.w2, (int64_t)e * d + j, f, c, wv);
#pragma unroll
          for (int q = 0; q < 8; ++q) acc = fmaf(hv[q], wv[q], acc);
        }
        acc = warp_sum(acc) * (sh ? (a.sink ? tb.shw[t] : 1.f) : tb.row_w[r0 + i]);
        if ((t & 31) == lane) {
          if (t < 32) y0 += acc;
          else y1 += acc;
        }
      }
    }
    XT* y = static_cast<XT*>(a.y);
    if (lane < T) y[(int64_t)lane * d + j] = (XT)y0;
    if (lane + 32 < T) y[(int64_t)(lane + 32) * d + j] = (XT)y1;
  }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

template <int WT>
cudaError_t launch(const Args& a, cudaStream_t s) {
  const void* fn = (const void*)few_kernel<WT>;
  const int smem = (int)sizeof(Tables);
  cudaError_t e = ensure_smem_attr(fn, smem);
  if (e != cudaSuccess) return e;
  e = cudaMemsetAsync(a.bar, 0, 256, s);
  if (e != cudaSuccess) return e;
  Args args = a;
  void* ptrs[] = {&args};
  return cudaLaunchCooperativeKernel(fn, dim3(sm_count()), dim3(THREADS), ptrs, smem, s);
}

}  // namespace few

// Workspace: 256 bytes of counters, the logits, the hidden rows.
size_t few_workspace_bytes(const moe_config_t& c, int fs) {
  const size_t eb = c.x_dtype == MOE_DTYPE_F32 ? 4 : 2;
  return 256 + few::align256((size_t)c.T * (c.n_experts + c.shared_sink) * 4) +
         few::align256(((size_t)c.T * c.top_k * c.d_ff + (size_t)c.T * fs) * eb);
}

cudaError_t launch_few(const moe_config_t& c, int64_t capacity, const void* x, const float* w_gate,
                       const float* logit_offset, const float* bias, bool mxfp4, const void* const* w,
                       const uint8_t* const* sf, int fs, int32_t* topk_idx, float* topk_w, void* y, void* ws,
                       cudaStream_t s) {
  few::Args a{};
  a.x = x;
  a.w_gate = w_gate;
  few::Matrix* m[6] = {&a.w1, &a.w3, &a.w2, &a.ws1, &a.ws3, &a.ws2};
  for (int i = 0; i < 6; ++i) *m[i] = {w[i], mxfp4 ? sf[i] : nullptr};
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
  a.logits = reinterpret_cast<float*>(p + 256);
  a.h = p + 256 + few::align256((size_t)c.T * (c.n_experts + c.shared_sink) * 4);
  if (mxfp4) return few::launch<few::W_MXFP4>(a, s);
  if (c.x_dtype == MOE_DTYPE_F32) return few::launch<few::W_F32>(a, s);
  return few::launch<few::W_BF16>(a, s);
}

}  // namespace moe
