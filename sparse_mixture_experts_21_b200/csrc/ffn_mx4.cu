// MXFP4 expert weights (OCP Microscaling: E2M1 codes, one E8M0 scale per 32 elements along
// the contraction dimension): quantisation, its inverse, and the grouped SwiGLU FFN of
// MXFP8 rows times MXFP4 weights.
//
// Quantisation.  A block of 32 with largest magnitude amax takes the scale byte
// b = max(0, expfield(amax) - 2), value 2^(b - 127): the largest E2M1 exponent is 2, so
// amax / scale lies in [4, 8) and what exceeds 6 saturates.  code = E2M1(x / scale), ties
// to even; the division by a power of two is exact, so the codes are a pure function of the
// input bits.  A block that holds an infinity or a NaN takes the byte 255 (the format's NaN
// scale) and zero codes, so it reads back as NaN instead of as a finite number.
// Scales are stored in ffn_mx.cu's tile atoms (the order the tensor cores take them in).
//
// Product.  Rows are MXFP8 (E4M3) rather than MXFP4: an E2M1 row loses ~10% of its norm
// where an E4M3 row loses 2-3%, and tcgen05.mma.kind::mxf8f6f4 takes E4M3 x E2M1 at its full
// rate, applying both operands' scales.  It wants 4-bit codes as 16-byte groups of 8 bytes
// of codes and 8 unused bytes; TMA expands the packed codes to that on the way into shared
// memory (16U4_ALIGN16B), so the weights cost half of MXFP8's bytes in HBM and L2 and the
// same shared memory, and no thread touches a code.
#include <cuda.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace mx4 {

// Eight fp32 values to a word of E2M1 codes (the first in bits 0..3), nearest even, saturating.
__device__ __forceinline__ uint32_t f32_e2m1(const float* f) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r) : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// Eight E2M1 codes of a word to four pairs of fp16 (exact), in order.  Read all four: with
// nvcc 12.9.86, where nothing reads the results of the upper bytes, those of the lower ones came
// out as zeros (tried: whole, masked and 2-byte words; a shifted word with all four read is right).
__device__ __forceinline__ void e2m1_f16(uint32_t w, uint32_t* o) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]) : "r"(w));
}

// 2^(b - 127); 255 is the format's NaN.
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return b == 255u ? __int_as_float(0x7fffffff) : b ? __uint_as_float(b << 23) : __uint_as_float(0x00400000u);
}

// Sixteen consecutive elements: their words, values, and largest magnitude as fp32 bits (so
// that a NaN or an infinity is the largest).
template <typename T> struct Words;
template <> struct Words<__nv_bfloat16> {
  uint4 v[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v[0] = ldg_nc16(p); v[1] = ldg_nc16(p + 8); }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a = __vmaxu2(a, __vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu));
      a = __vmaxu2(a, __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu));
    }
    return max(a << 16, a & 0xffff0000u);
  }
  __device__ __forceinline__ void values(int half, float* f) const { unpack16(v[half], f, __nv_bfloat16()); }
};
template <> struct Words<float> {
  uint4 v[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ldg_nc16(p + 4 * i);
  }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a = max(a, max(max(v[i].x & 0x7fffffffu, v[i].y & 0x7fffffffu), max(v[i].z & 0x7fffffffu, v[i].w & 0x7fffffffu)));
    return a;
  }
  __device__ __forceinline__ void values(int half, float* f) const {
    unpack16(v[2 * half], f, 0.f);
    unpack16(v[2 * half + 1], f + 4, 0.f);
  }
};

// Row and column block of block blk of a matrix's 128-column blocks, row major.  32 bits: the
// entry points take up to 2^32 blocks (256 GB of codes).
__device__ __forceinline__ void row_block(uint32_t blk, int nkb, uint32_t& r, int& kb) {
  r = blk / (uint32_t)nkb;
  kb = (int)(blk - r * (uint32_t)nkb);
}

// Memory-bound: 2 (or 4) bytes in and 0.53 out per element, one pass.  A thread owns 16
// consecutive elements, two threads a block of 32, 8 threads one row's 128-column block (so its
// four scale bytes leave as one 4-byte store), and takes VECS of them a step with the loads
// ahead of the work.  bf16, 32768 x 7168: 100 us, 5.9 TB/s; with 8 elements a thread the
// shuffles, the row's division and the scale cost 141 us.
constexpr int VECS = 2;
template <typename XT>
__global__ void __launch_bounds__(256)
quant_kernel(const XT* __restrict__ x, int64_t n16, int cols, uint2* __restrict__ q, uint8_t* __restrict__ sf) {
  const int nkb = cols / 128;
  const int64_t step = (int64_t)gridDim.x * 256 * VECS;
  for (int64_t i0 = (int64_t)blockIdx.x * 256 * VECS + threadIdx.x; i0 - threadIdx.x < n16; i0 += step) {
    Words<XT> w[VECS] = {};
#pragma unroll
    for (int v = 0; v < VECS; ++v)
      if (i0 + 256 * v < n16) w[v].load(x + 16 * (i0 + 256 * v));
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
      const int64_t i = i0 + 256 * v;       // n16 is a multiple of 8: i < n16 alike over a block
      uint32_t amax = w[v].amax();
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      const uint32_t ef = amax >> 23;
      const uint32_t b = ef == 255u ? 255u : ef > 2u ? ef - 2u : 0u;
      const float m = __uint_as_float((254u - min(b, 253u)) << 23);
      uint32_t c[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float f[8];
        w[v].values(h, f);
#pragma unroll
        for (int u = 0; u < 8; ++u) f[u] *= m;
        c[h] = b == 255u ? 0u : f32_e2m1(f);
      }
      // the block's four scale bytes in its first thread
      uint32_t s = b | __shfl_down_sync(0xffffffffu, b, 2) << 8;
      s |= __shfl_down_sync(0xffffffffu, s, 4) << 16;
      if (i < n16) {
        q[i] = make_uint2(c[0], c[1]);
        if ((threadIdx.x & 7) == 0) {
          uint32_t r;
          int kb;
          row_block((uint32_t)(i >> 3), nkb, r, kb);
          *reinterpret_cast<uint32_t*>(sf + mx::atom_byte(r >> 7, nkb, kb, (int)(r & 127), 0)) = s;
        }
      }
    }
  }
}

// Memory-bound.  A thread owns 8 consecutive elements (4 fp32), so a warp's stores are
// contiguous: 32768 x 7168 in 111 us to bf16, 197 us to fp32 (5.4 TB/s; 264 us with 8 fp32 a
// thread).  It reads all of a word's results either way, as e2m1_f16 wants.
template <typename YT>
__global__ void __launch_bounds__(256)
dequant_kernel(const uint32_t* __restrict__ q, const uint8_t* __restrict__ sf, int64_t n, int cols,
               YT* __restrict__ y) {
  constexpr int E = 16 / sizeof(YT), U = 4;
  const int nkb = cols / 128;
  const int64_t step = (int64_t)gridDim.x * 256 * U;
  for (int64_t i0 = (int64_t)blockIdx.x * 256 * U + threadIdx.x; i0 < n; i0 += step) {
    uint32_t w[U];
    uint8_t b[U];
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int64_t i = i0 + 256 * v;
      if (i >= n) break;
      w[v] = q[E == 8 ? i : i >> 1];
      uint32_t r;
      int kb;
      row_block((uint32_t)(i / (128 / E)), nkb, r, kb);
      b[v] = sf[mx::atom_byte(r >> 7, nkb, kb, (int)(r & 127), (int)(i / (32 / E) & 3))];
    }
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int64_t i = i0 + 256 * v;
      if (i >= n) break;
      const float s = e8m0_value(b[v]);
      uint32_t h[4];
      e2m1_f16(w[v], h);
      if (E == 4 && (i & 1)) {       // the word's upper four codes
        h[0] = h[2];
        h[1] = h[3];
      }
      float f[E];
#pragma unroll
      for (int u = 0; u < E / 2; ++u) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h[u]));
        f[2 * u] = p.x * s;
        f[2 * u + 1] = p.y * s;
      }
      stg16(y + E * i, pack16(f, YT()));
    }
  }
}

inline int quant_grid(int64_t threads) {
  const int64_t want = (threads + 255) / 256, cap = (int64_t)sm_count() * 16;
  return (int)(want < cap ? want : cap);
}

// ---------------------------------------------------------------- grouped GEMM
// The tiles, pipeline, barriers and epilogue of ffn_mx_kernel (128 rows by 256 B rows, one
// 128-wide K block a stage), with B's codes expanded from 4 bits by the TMA.
using namespace mx;

// bytes that complete on a stage's barrier: the TMA counts 4-bit codes as packed in memory
constexpr uint32_t kStageTx = A_BYTES + B_BYTES / 2 + SF_BYTES;
constexpr uint32_t kB_E2M1 = 5u << 10;       // instruction descriptor: B holds E2M1

// MODE 0: A = x codes [rows_cap, d] E4M3, B0/B1 = W1/W3 codes [G f, d] E2M1; writes h codes
//         [rows_cap, f] E4M3 and h scales.
// MODE 1: A = h codes [rows_cap, f], B0 = W2 codes [G d, f]; writes y bf16 [rows_cap, d].
template <int MODE>
__global__ void __launch_bounds__(THREADS, 1)
ffn_mx4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
              const __grid_constant__ CUtensorMap tmB1, const uint8_t* __restrict__ sfa,
              const uint8_t* __restrict__ sfb0, const uint8_t* __restrict__ sfb1,
              const int32_t* __restrict__ offsets, int G, int K, int n_out, int64_t rows_cap,
              uint8_t* __restrict__ out_q, uint8_t* __restrict__ out_sf, __nv_bfloat16* __restrict__ out,
              const __grid_constant__ CUtensorMap tmY) {
  constexpr int BN = MODE == 0 ? 128 : 256;      // output columns per tile
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  MxShared* sh = reinterpret_cast<MxShared*>(smem + (size_t)STAGES * STAGE_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles_n = (n_out + BN - 1) / BN;
  const int nkb = K / BK;
  const int64_t b_tiles = (int64_t)G * n_out / 128;      // 128-row tiles of B

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < STAGES; ++s) { mbar_init(&sh->full[s], 1); mbar_init(&sh->empty[s], 1); }
    mbar_init(&sh->tfull, 1);
    mbar_init(&sh->tempty, EPI_WARPS);
    mbar_init(&sh->mma_done, 1);
    sh->abort = 0;
    fence_barrier_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB0);
    if (MODE == 0) prefetch_tmap(&tmB1);
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == 2) {
    int carry = 0;
    for (int base = 0; base < G; base += 32) {
      const int g = base + lane;
      int mt = 0;
      if (g < G) {
        const int o0 = offsets[g], o1 = offsets[g + 1];
        sh->goff[g] = o0;
        mt = o1 > o0 ? (o1 - o0 + BM - 1) / BM : 0;
      }
      int incl = mt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (g < G) sh->tpre[g + 1] = carry + incl;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) { sh->tpre[0] = 0; sh->goff[G] = offsets[G]; }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = sh->tmem_base;
  const int total = sh->tpre[G] * tiles_n;

  if (warp == 0) {
    // ---------------- producer (one thread): codes by TMA, the stage's three scale atoms
    // by bulk copies, all completing on the stage's full barrier
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      int issued = 0;
      bool ok = true;
      for (int L = blockIdx.x; L < total && ok; L += gridDim.x) {
        const Tile t = decode(L, sh, G, tiles_n, BN);
        const int64_t brow = (int64_t)t.g * n_out + t.n0;
        const int64_t bt0 = brow / 128;
        // MODE 1: the second B atom is the next 128 rows (past the end: repeat the first;
        // those output columns are not stored)
        const int64_t bt1 = MODE == 0 ? bt0 : (bt0 + 1 < b_tiles ? bt0 + 1 : bt0);
        for (int kb = 0; kb < nkb; ++kb) {
          if (!waitmx(&sh->empty[stage], phase ^ 1u, sh)) { ok = false; break; }
          uint8_t* a = smem + (size_t)stage * STAGE_BYTES;
          uint8_t* b = a + A_BYTES;
          uint8_t* sfs = sh->sf[stage];
          mbar_arrive_expect_tx(&sh->full[stage], kStageTx);
          tma_load_2d(&tmA, a, &sh->full[stage], kb * BK, t.row0);
          if (MODE == 0) {
            tma_load_2d(&tmB0, b, &sh->full[stage], kb * BK, (int32_t)brow);
            tma_load_2d(&tmB1, b + B_BYTES / 2, &sh->full[stage], kb * BK, (int32_t)brow);
          } else {
            tma_load_2d(&tmB0, b, &sh->full[stage], kb * BK, (int32_t)brow);
          }
          bulk_load(sfs, sfa + ((int64_t)t.tile * nkb + kb) * 512, 512, &sh->full[stage]);
          bulk_load(sfs + 512, sfb0 + (bt0 * nkb + kb) * 512, 512, &sh->full[stage]);
          bulk_load(sfs + 1024, (MODE == 0 ? sfb1 : sfb0) + (bt1 * nkb + kb) * 512, 512, &sh->full[stage]);
          ++issued;
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {
        for (int i = 1; i <= min(issued, STAGES); ++i) {
          const int s = ((int)stage - i + 2 * STAGES) % STAGES;
          mbar_wait(&sh->full[s], ((int)stage - i < 0) ? (phase ^ 1u) : phase);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, tile_i = 0;
      bool ok = true;
      for (int L = blockIdx.x; L < total && ok; L += gridDim.x, ++tile_i) {
        if (!waitmx(&sh->tempty, (tile_i & 1u) ^ 1u, sh)) { ok = false; break; }
        for (int kb = 0; kb < nkb; ++kb) {
          if (!waitmx(&sh->full[stage], phase, sh)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + (size_t)stage * STAGE_BYTES);
          const uint32_t b_addr = a_addr + A_BYTES;
          const uint32_t sf_addr = smem_u32(sh->sf[stage]);
          const uint32_t sfa_t = tmem_base + kSfCol0 + stage * kSfColsPerStage;
          const uint32_t sfb_t = sfa_t + 8;
          tmem_cp_sf(sfa_t, sf_desc(sf_addr));
          tmem_cp_sf(sfb_t, sf_desc(sf_addr + 512));
          tmem_cp_sf(sfb_t + 4, sf_desc(sf_addr + 1024));
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            umma_mx(tmem_base, umma_desc_sw128(a_addr + kk * 32), umma_desc_sw128(b_addr + kk * 32),
                    idesc_mx(BM, 256, (uint32_t)kk) | kB_E2M1, sfa_t, sfb_t, (kb | kk) != 0 ? 1u : 0u);
          umma_commit(&sh->empty[stage]);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        umma_commit(&sh->tfull);
      }
      umma_commit(&sh->mma_done);
      mbar_wait(&sh->mma_done, 0);
    }
  } else {
    // ---------------- epilogue: TMEM lanes 32 q .. 32 q + 31; MODE 0: gate columns
    // c_lo .. c_lo + 63 and up columns 128 + c_lo ..; MODE 1: output columns c_lo .. + 127
    const int q = warp & 3;
    const int half = (warp - 2) >> 2;
    const int c_lo = MODE == 0 ? half * 64 : half * 128;
    // down pass: this warp's output staging box (1024-aligned, for the 64-byte swizzle)
    const uint32_t box = smem_u32(smem + (size_t)STAGES * STAGE_BYTES + kSharedPad) + (warp - 2) * OUT_BOX;
    bool box_busy = false;                    // a TMA store may still be reading the box
    uint32_t tile_i = 0;
    for (int L = blockIdx.x; L < total; L += gridDim.x, ++tile_i) {
      const Tile t = decode(L, sh, G, tiles_n, BN);
      if (!waitmx(&sh->tfull, tile_i & 1u, sh)) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16);
      uint32_t v[128];
#pragma unroll
      for (int c = 0; c < 128; c += 16) {
        const int col = MODE == 0 ? (c < 64 ? c_lo + c : 128 + c_lo + c - 64) : c_lo + c;
        tmem_ld16(tb + col, v + c);
      }
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->tempty);        // accumulator free for the next tile
      if (MODE == 1 && q * 32 + 32 <= t.rows && t.n0 + c_lo < n_out) {
        // all 32 rows of this warp are the group's: four 32 x 32 boxes through shared
        // memory (lane l writes row l's 64 bytes, 16-byte chunk c at slot c ^ ((l >> 1) & 3),
        // the 64-byte swizzle), fenced for the TMA engine, stored by lane 0; the store
        // clips columns past the output.  A group's last, partial tile stores row by row.
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          if (box_busy) {
            if (lane == 0) bulk_wait_read();
            __syncwarp();
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t* e = v + cc * 32 + c * 8;
            uint4 pk;
            pk.x = pack_bf16x2(__uint_as_float(e[0]), __uint_as_float(e[1]));
            pk.y = pack_bf16x2(__uint_as_float(e[2]), __uint_as_float(e[3]));
            pk.z = pack_bf16x2(__uint_as_float(e[4]), __uint_as_float(e[5]));
            pk.w = pack_bf16x2(__uint_as_float(e[6]), __uint_as_float(e[7]));
            sts16(box + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4), pk);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmY, box, t.n0 + c_lo + cc * 32, t.row0 + q * 32);
            bulk_commit();
          }
          box_busy = true;
        }
        continue;
      }
      const int r = q * 32 + lane;
      const int64_t grow = (int64_t)t.row0 + r;
      if (r >= t.rows || grow >= rows_cap) continue;
      if (MODE == 0) {
        // h = silu(gate) * up for 64 hidden units, then MXFP8 in two blocks of 32
        uint8_t* dq = out_q + grow * (int64_t)n_out + t.n0 + c_lo;
        uint32_t sfw = 0;
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
          float h[32];
          float amax = 0.f;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            h[j] = silu(__uint_as_float(v[32 * blk + j])) * __uint_as_float(v[64 + 32 * blk + j]);
            amax = fmaxf(amax, fabsf(h[j]));
          }
          const uint32_t b = e8m0_of(amax);
          const float m = inv_scale(b);
          sfw |= b << (8 * blk);
#pragma unroll
          for (int j0 = 0; j0 < 32; j0 += 16) {
            uint32_t w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              w[u] = (uint32_t)to_e4m3(h[j0 + 4 * u] * m) | ((uint32_t)to_e4m3(h[j0 + 4 * u + 1] * m) << 8) |
                     ((uint32_t)to_e4m3(h[j0 + 4 * u + 2] * m) << 16) |
                     ((uint32_t)to_e4m3(h[j0 + 4 * u + 3] * m) << 24);
            *reinterpret_cast<uint4*>(dq + 32 * blk + j0) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        // scales c_lo / 32 and + 1 of row r in the atom of (this tile, K block n0 / 128) of h
        *reinterpret_cast<uint16_t*>(out_sf + atom_byte(t.tile, n_out / 128, t.n0 / 128, r, c_lo / 32)) =
            (uint16_t)sfw;
      } else if (t.n0 + c_lo < n_out) {
        __nv_bfloat16* orow = out + grow * (int64_t)n_out + t.n0 + c_lo;
#pragma unroll
        for (int j = 0; j < 128; j += 8) {
          uint4 pk;
          pk.x = pack_bf16x2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
          pk.y = pack_bf16x2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
          pk.z = pack_bf16x2(__uint_as_float(v[j + 4]), __uint_as_float(v[j + 5]));
          pk.w = pack_bf16x2(__uint_as_float(v[j + 6]), __uint_as_float(v[j + 7]));
          stg16(orow + j, pk);
        }
      }
    }
    // every output box of this warp is in global memory before the kernel ends
    if (MODE == 1 && lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

template <int MODE>
cudaError_t launch_mx4(const CUtensorMap& a, const CUtensorMap& b0, const CUtensorMap& b1, const uint8_t* sfa,
                      const uint8_t* sfb0, const uint8_t* sfb1, const int32_t* offsets, int G, int K, int n_out,
                      int64_t rows_cap, uint8_t* out_q, uint8_t* out_sf, void* out, cudaStream_t s) {
  constexpr int BN = MODE == 0 ? 128 : 256;
  const cudaError_t e = ensure_smem_attr((const void*)ffn_mx4_kernel<MODE>, (int)kSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles_n = (n_out + BN - 1) / BN;
  const int64_t max_tiles = ((rows_cap + BM - 1) / BM + G) * tiles_n;
  const int grid = (int)(max_tiles < sm_count() ? max_tiles : sm_count());
  if (grid <= 0) return cudaSuccess;
  // the down pass's output map (the gate/up pass writes no bf16 rows and never reads it)
  CUtensorMap my{};
  if (MODE == 1 && !make_map_bf16_store32(&my, out, (uint64_t)rows_cap, (uint64_t)n_out))
    return cudaErrorInvalidValue;
  ffn_mx4_kernel<MODE><<<grid, THREADS, kSmem, s>>>(a, b0, b1, sfa, sfb0, sfb1, offsets, G, K, n_out, rows_cap,
                                                   out_q, out_sf, static_cast<__nv_bfloat16*>(out), my);
  return cudaGetLastError();
}

}  // namespace mx4

cudaError_t launch_mx4_quant(const void* x, bool f32, int64_t rows, int cols, uint8_t* q, uint8_t* sf,
                             cudaStream_t s) {
  const int64_t n = rows * (int64_t)cols / 16;
  if (n == 0) return cudaSuccess;
  const int grid = mx4::quant_grid((n + mx4::VECS - 1) / mx4::VECS);
  uint2* qw = reinterpret_cast<uint2*>(q);
  if (f32) mx4::quant_kernel<<<grid, 256, 0, s>>>(static_cast<const float*>(x), n, cols, qw, sf);
  else mx4::quant_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(x), n, cols, qw, sf);
  return cudaGetLastError();
}

cudaError_t launch_mx4_dequant(const uint8_t* q, const uint8_t* sf, int64_t rows, int cols, bool f32, void* y,
                               cudaStream_t s) {
  const int64_t n = rows * (int64_t)cols / (f32 ? 4 : 8);
  if (n == 0) return cudaSuccess;
  const int grid = mx4::quant_grid((n + 3) / 4);
  const uint32_t* qw = reinterpret_cast<const uint32_t*>(q);
  if (f32) mx4::dequant_kernel<<<grid, 256, 0, s>>>(qw, sf, n, cols, static_cast<float*>(y));
  else mx4::dequant_kernel<<<grid, 256, 0, s>>>(qw, sf, n, cols, static_cast<__nv_bfloat16*>(y));
  return cudaGetLastError();
}

cudaError_t launch_ffn_mx4(const uint8_t* xq, const uint8_t* xsf, int64_t rows_cap, const int32_t* offsets, int G,
                           const uint8_t* w1q, const uint8_t* w1sf, const uint8_t* w3q, const uint8_t* w3sf,
                           const uint8_t* w2q, const uint8_t* w2sf, int d, int f, uint8_t* hq, uint8_t* hsf,
                           void* y, cudaStream_t s) {
  if (rows_cap == 0 || G == 0) return cudaSuccess;
  if (G > mx::kMaxGroups) return cudaErrorInvalidValue;
  CUtensorMap mxm, m1, m3, mh, m2;
  if (!make_map_u8(&mxm, xq, rows_cap, d, 128) || !make_map_u4(&m1, w1q, (uint64_t)G * f, d, 128) ||
      !make_map_u4(&m3, w3q, (uint64_t)G * f, d, 128) || !make_map_u8(&mh, hq, rows_cap, f, 128) ||
      !make_map_u4(&m2, w2q, (uint64_t)G * d, f, 256))
    return cudaErrorInvalidValue;
  cudaError_t e = mx4::launch_mx4<0>(mxm, m1, m3, xsf, w1sf, w3sf, offsets, G, d, f, rows_cap, hq, hsf, nullptr, s);
  if (e != cudaSuccess) return e;
  return mx4::launch_mx4<1>(mh, m2, m2, hsf, w2sf, w2sf, offsets, G, f, d, rows_cap, nullptr, nullptr, y, s);
}

}  // namespace moe
