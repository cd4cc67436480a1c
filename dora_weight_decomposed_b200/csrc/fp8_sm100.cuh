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

// ------------------------------------------------------------------ CTA pairs
//
// The wide tile: a cluster of two CTAs computes 256 x 256 results with
// cta_group::2 MMAs, each CTA staging its 128 rows of the operand and half of
// the weight tile's 256, so that per k-block (512 clocks of MMA per SM) only 32 KB
// come in per SM. TMEM (512 columns) holds two accumulators of 256. Eight
// epilogue warps fold: warp w reads TMEM lanes 32 (w % 4) .. + 31 and
// half of the columns, 128 fp32 sums per thread, so that each scheduler issues
// about half as many instructions as a k-block of MMAs takes clocks. Tiles
// are walked persistently; the MMAs of the next tile start while this one is stored.
constexpr int kF8FoldWarps = 8;
constexpr int kF8PairThreads = 64 + 32 * kF8FoldWarps;
constexpr int kF8PairStages = 6;
constexpr int kF8StageBytes = 2 * 128 * 128;
constexpr int kF8PairSmem = kF8PairStages * kF8StageBytes + 256 + 1024;

// Tiles in groups of 8 rows of tiles, rows fastest: the tiles in flight share operands in L2.
__device__ __forceinline__ void fp8_tile_coords(int t, int m_tiles, int n_tiles, int& m, int& n) {
  const int per_group = 8 * n_tiles;
  const int first_m = t / per_group * 8;
  const int gm = min(8, m_tiles - first_m);
  const int rem = t % per_group;
  m = first_m + rem % gm;
  n = rem / gm;
}

// a.xy += v.xy * s (two fp32 multiply-adds in one instruction)
__device__ __forceinline__ void fma2(float2& a, uint32_t v0, uint32_t v1, float s) {
  asm("{\n\t.reg .b64 v, s, a;\n\t"
      "mov.b64 v, {%2, %3};\n\tmov.b64 s, {%4, %4};\n\tmov.b64 a, {%0, %1};\n\t"
      "fma.rn.f32x2 a, v, s, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a.x), "+f"(a.y)
      : "r"(v0), "r"(v1), "f"(s));
}

template <bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kF8PairThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap tA, const __grid_constant__ CUtensorMap tB, const Fp8Geom g) {
  constexpr int STAGES = kF8PairStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * kF8StageBytes);  // used in the leader
  uint64_t* empty = full + STAGES;
  uint64_t* accf = empty + STAGES;  // [2] accumulator complete
  uint64_t* acce = accf + 2;        // [2] accumulator folded by both CTAs, used in the leader
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce + 2);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int m_tiles = (g.T + 255) / 256, n_tiles = (g.N + 255) / 256;
  const int tiles = m_tiles * n_tiles;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], 2 * kF8FoldWarps);
    }
    fence_mbar_init();
    prefetch_tmap(&tA);
    prefetch_tmap(&tB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();
  pdl_wait();

  if (warp < 2) {
    if (warp == 0 && lane == 0) {
      int it = 0;
      bool ok = true;
#pragma unroll 1
      for (int t = pair; t < tiles && ok; t += npairs) {
        int tm, tn;
        fp8_tile_coords(t, m_tiles, n_tiles, tm, tn);
        const int m0 = tm * 256 + (int)rank * 128, n0 = tn * 256 + (int)rank * 128;
#pragma unroll 1
        for (int kb = 0; kb < g.nkb; ++kb, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait(&empty[s], ((uint32_t)(it / STAGES) & 1u) ^ 1u)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + s * kF8StageBytes;
          const uint32_t fb = mapa_shared(smem_u32(&full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kF8StageBytes);
          tma_load_2d_pair(sa, &tA, fb, kb * kF8BK, m0);
          if (!B_MN)
            tma_load_2d_pair(sa + 16384, &tB, fb, kb * kF8BK, n0);
          else
            tma_load_2d_pair(sa + 16384, &tB, fb, n0, kb * kF8BK);
        }
      }
      if (!ok && rank == 0) {  // a wait ran out: let the copies in flight land before the shared memory goes
        for (int j = max(0, it - STAGES); j < it; ++j)
          mbar_wait(&full[j % STAGES], (uint32_t)(j / STAGES) & 1u, kWaitLimitNs / 16);
      }
    } else if (warp == 1 && lane == 0 && rank == 0) {
      const uint32_t idesc = idesc_fp8_f32(256, 256, g.a_e5m2 != 0, false, B_MN);
      constexpr uint32_t b_kstep = B_MN ? 32u * 128u : 32u;
      int it = 0;
      bool ok = true;
#pragma unroll 1
      for (int t = pair; t < tiles && ok; t += npairs) {
#pragma unroll 1
        for (int kb = 0; kb < g.nkb; ++kb, ++it) {
          const int s = it % STAGES, b = it & 1;
          if (!mbar_wait(&acce[b], ((uint32_t)(it >> 1) & 1u) ^ 1u) || !mbar_wait(&full[s], (uint32_t)(it / STAGES) & 1u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + s * kF8StageBytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_fp8_pair(tmem + b * 256u, sdesc_sw128(sa + kk * 32u, 16u, 1024u),
                          sdesc_sw128(sa + 16384u + kk * b_kstep, 16u, 1024u), idesc, kk > 0 ? 1u : 0u);
          umma_commit_pair(&empty[s], 0x3);
          umma_commit_pair(&accf[b], 0x3);
        }
      }
    }
  } else {
    constexpr int COLS = 4 * 256 / kF8FoldWarps;  // columns per warp
    const int q = warp & 3, part = (warp - 2) >> 2;
    const uint32_t done = mapa_shared(smem_u32(acce), 0);
    int it = 0;
    bool ok = true;
#pragma unroll 1
    for (int t = pair; t < tiles && ok; t += npairs) {
      int tm, tn;
      fp8_tile_coords(t, m_tiles, n_tiles, tm, tn);
      const int mw = tm * 256 + (int)rank * 128 + q * 32;  // first row of the warp
      const int m = mw + lane;
      const int n0 = tn * 256 + part * COLS;
      const bool live = mw < g.T && n0 < g.N;  // of the warp
      const float* xs = g.xs + min(m, g.T - 1);
      const float* ws = g.ws + (live ? (size_t)(n0 >> 7) * g.ws_n : 0);
      float2 acc[COLS / 2];
#pragma unroll
      for (int j = 0; j < COLS / 2; ++j) acc[j] = make_float2(0.f, 0.f);
      // Scales are fetched two k-blocks ahead and multiplied where they are used, so that nothing waits for them.
      float x0 = xs[0], w0 = ws[0], x1 = 0.f, w1 = 0.f;
      if (g.nkb > 1) x1 = xs[(size_t)g.T], w1 = ws[g.ws_k];
#pragma unroll 1
      for (int kb = 0; kb < g.nkb; ++kb, ++it) {
        const int b = it & 1;
        const float s = x0 * w0;
        x0 = x1, w0 = w1;
        if (kb + 2 < g.nkb) x1 = xs[(size_t)(kb + 2) * g.T], w1 = ws[(size_t)(kb + 2) * g.ws_k];
        if (!mbar_wait(&accf[b], (uint32_t)(it >> 1) & 1u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (live) {
          const uint32_t ta = tmem + b * 256u + part * COLS + ((uint32_t)(q * 32) << 16);
          uint32_t v[16];
#pragma unroll
          for (int c = 0; c < COLS / 16; ++c) {
            tmem_ld16_async(ta + c * 16, v);
            tmem_ld_wait();
            if (c == COLS / 16 - 1) {  // the accumulator is read: the MMAs may have it
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster(done + 8 * b);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) fma2(acc[c * 8 + j], v[2 * j], v[2 * j + 1], s);
          }
        } else if (lane == 0) {
          mbar_arrive_cluster(done + 8 * b);
        }
      }
      if (ok && live && m < g.T) {
#pragma unroll
        for (int c = 0; c < COLS / 32; ++c) fp8_store32(g, m, n0 + c * 32, reinterpret_cast<const float*>(acc) + c * 32);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace dora
