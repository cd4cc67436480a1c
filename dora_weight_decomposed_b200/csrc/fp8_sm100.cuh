// 8-bit block-scaled products on tcgen05:
//
//   out[t, n] = sum_kb xs[kb, t] ws[n / 128, kb] sum_{k in kb} xq[t, k] wq[n, k]
//
// The scales change every 128 values of K, so the tensor cores' accumulator
// holds one k-block at a time: the four MMAs of a k-block write a fresh
// accumulator in TMEM, and the epilogue warps fold it into fp32 sums in
// registers, one multiply-add per value with the row's scale times the
// tile's. Two accumulators let the MMAs of the next k-block run meanwhile.
#pragma once

#include "sm100_ptx.cuh"

namespace dora {

constexpr int kF8BM = 128;  // token rows per tile
constexpr int kF8BK = 128;  // K per block: one 128-byte swizzle row, one scale
constexpr int kF8Threads = 192;

struct Fp8Geom {
  const float* xs;   // [kb][T]
  const float* ws;   // the weight's scales: n block * ws_n + k block * ws_k
  void* out;         // [T x N]
  int T, N, nkb;
  int ws_n, ws_k;
  int out_fp32;
  int a_e5m2;
};

// 32 results of one row, columns n .. n + 31 (N is a multiple of 16).
__device__ __forceinline__ void fp8_store32(const Fp8Geom& g, int m, int n, const float* v) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (n + 16 * h >= g.N) return;
    const size_t at = (size_t)m * g.N + n + 16 * h;
    if (g.out_fp32) {
      float4* o = reinterpret_cast<float4*>((float*)g.out + at);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = make_float4(v[16 * h + 4 * i], v[16 * h + 4 * i + 1], v[16 * h + 4 * i + 2], v[16 * h + 4 * i + 3]);
    } else {
      uint4* o = reinterpret_cast<uint4*>((__nv_bfloat16*)g.out + at);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        __nv_bfloat162 p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = __floats2bfloat162_rn(v[16 * h + 8 * i + 2 * j], v[16 * h + 8 * i + 2 * j + 1]);
        o[i] = *reinterpret_cast<const uint4*>(p);
      }
    }
  }
}

// One 128 x 128 tile per CTA. B_MN: the weight's rows run along K (the input
// gradient reads W [d_out x d_in] with K = d_out), so its tile is MN-major.
template <bool B_MN>
struct Fp8Tile {
  static constexpr int TILE_BYTES = 128 * 128;
  static constexpr int STAGE_BYTES = 2 * TILE_BYTES;
  static constexpr int STAGES = 6;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 256 + 1024;
};

template <bool B_MN>
__global__ void __launch_bounds__(kF8Threads, 1)
    fp8_tile_kernel(const __grid_constant__ CUtensorMap tA, const __grid_constant__ CUtensorMap tB, const Fp8Geom g) {
  using Cfg = Fp8Tile<B_MN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::STAGES * Cfg::STAGE_BYTES);
  uint64_t* empty = full + Cfg::STAGES;
  uint64_t* accf = empty + Cfg::STAGES;  // [2] accumulator complete
  uint64_t* acce = accf + 2;             // [2] accumulator folded
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int n_tile = blockIdx.x, m_tile = blockIdx.y;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], 4);
    }
    fence_mbar_init();
    prefetch_tmap(&tA);
    prefetch_tmap(&tB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();
  pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
#pragma unroll 1
      for (int i = 0; i < g.nkb; ++i) {
        const int s = i % Cfg::STAGES;
        if (!mbar_wait(&empty[s], ((uint32_t)(i / Cfg::STAGES) & 1u) ^ 1u)) break;
        uint8_t* sa = smem + s * Cfg::STAGE_BYTES;
        mbar_arrive_expect_tx(&full[s], Cfg::STAGE_BYTES);
        tma_load_2d(sa, &tA, &full[s], i * kF8BK, m_tile * kF8BM);
        if (!B_MN)
          tma_load_2d(sa + Cfg::TILE_BYTES, &tB, &full[s], i * kF8BK, n_tile * 128);
        else
          tma_load_2d(sa + Cfg::TILE_BYTES, &tB, &full[s], n_tile * 128, i * kF8BK);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_fp8_f32(128, 128, g.a_e5m2 != 0, false, B_MN);
      constexpr uint32_t b_kstep = B_MN ? 32u * 128u : 32u;
#pragma unroll 1
      for (int i = 0; i < g.nkb; ++i) {
        const int s = i % Cfg::STAGES, b = i & 1;
        if (!mbar_wait(&acce[b], ((uint32_t)(i >> 1) & 1u) ^ 1u)) break;
        if (!mbar_wait(&full[s], (uint32_t)(i / Cfg::STAGES) & 1u)) break;
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + s * Cfg::STAGE_BYTES);
        const uint32_t sb = sa + Cfg::TILE_BYTES;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_fp8(tmem + b * 128u, sdesc_sw128(sa + kk * 32u, 16u, 1024u), sdesc_sw128(sb + kk * b_kstep, 16u, 1024u),
                   idesc, kk > 0 ? 1u : 0u);
        umma_commit(&empty[s]);
        umma_commit(&accf[b]);
      }
    }
  } else {
    const int q = warp & 3;
    const int m = m_tile * kF8BM + q * 32 + lane;
    const bool live = m < g.T;
    float acc[128];
#pragma unroll
    for (int j = 0; j < 128; ++j) acc[j] = 0.f;
#pragma unroll 1
    for (int i = 0; i < g.nkb; ++i) {
      const int b = i & 1;
      const float s = (live ? g.xs[(size_t)i * g.T + m] : 0.f) * g.ws[(size_t)n_tile * g.ws_n + (size_t)i * g.ws_k];
      if (!mbar_wait(&accf[b], (uint32_t)(i >> 1) & 1u)) break;
      tc_fence_after();
      const uint32_t ta = tmem + b * 128u + ((uint32_t)(q * 32) << 16);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float v[32];
        tmem_ld32(ta + c * 32u, v);
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[c * 32 + j] = fmaf(v[j], s, acc[c * 32 + j]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acce[b]);
    }
    if (live) {
#pragma unroll
      for (int c = 0; c < 4; ++c) fp8_store32(g, m, n_tile * 128 + c * 32, acc + c * 32);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

}  // namespace dora
