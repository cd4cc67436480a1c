// 8-bit block-scaled products on tcgen05:
//
//   out[t, n] = sum_kb xs[kb, t] ws[n / 128, kb] sum_{k in kb} xq[t, k] wq[n, k]
//
// Scales that are powers of two (all that dora_fp8_quantize makes) are applied
// by the tensor cores, from exponent bytes in TMEM, and one accumulator holds
// the whole sum. Other scales change every 128 values of K, so an accumulator
// then holds one k-block at a time: the four MMAs of a k-block write a fresh
// one, and the epilogue warps fold it into fp32 sums in registers, one
// multiply-add per value with the row's scale times the tile's. Two
// accumulators let the MMAs of the next k-block run meanwhile.
#pragma once

#include <type_traits>

#include "sm100_ptx.cuh"

namespace dora {

// ------------------------------------------------------------------ block scales and codes

// max(a, |b|) that keeps a NaN.
__device__ __forceinline__ float absmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// The scale of a block and its inverse. Both are powers of two, read off the
// exponent of amax: amax = 1.f 2^x fits top = 1.75 2^k at e = x - k when
// 1.f <= 1.75, else at x - k + 1. Non-finite: scale = amax, inverse 0 (inf) or NaN.
struct BlockScale {
  float scale, inv;
};
template <bool E5M2>
__device__ __forceinline__ BlockScale block_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u >= 0x7f800000u) return {amax, 1.0f / amax};
  int e = (int)(u >> 23) - 127 - (E5M2 ? 15 : 8) + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, -126);
  return {__uint_as_float((uint32_t)(e + 127) << 23), __uint_as_float((uint32_t)(127 - e) << 23)};
}

// Two values to 8-bit codes, rounded to nearest even (the scale keeps them in range; NaN stays NaN).
template <bool E5M2>
__device__ __forceinline__ uint32_t to_fp8x2(float lo, float hi) {
  uint16_t r;
  if (E5M2)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool E5M2>
__device__ __forceinline__ uint2 to_fp8x8(const float* v, float inv) {
  uint2 r;
  r.x = to_fp8x2<E5M2>(v[0] * inv, v[1] * inv) | to_fp8x2<E5M2>(v[2] * inv, v[3] * inv) << 16;
  r.y = to_fp8x2<E5M2>(v[4] * inv, v[5] * inv) | to_fp8x2<E5M2>(v[6] * inv, v[7] * inv) << 16;
  return r;
}

// Eight consecutive values as they lie in memory (a bf16 thread holds half the registers that fp32 would take).
struct Raw8Bf16 {
  uint4 u;
  __device__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ void clear() { u = make_uint4(0u, 0u, 0u, 0u); }
  __device__ float absmax() const {  // NaN if one is
    uint32_t m;
    asm("{\n\t.reg .b32 a, b;\n\tmax.NaN.bf16x2 a, %1, %2;\n\tmax.NaN.bf16x2 b, %3, %4;\n\tmax.NaN.bf16x2 %0, a, b;\n\t}"
        : "=r"(m)
        : "r"(u.x & 0x7fff7fffu), "r"(u.y & 0x7fff7fffu), "r"(u.z & 0x7fff7fffu), "r"(u.w & 0x7fff7fffu));
    return absmax_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  __device__ void values(float* v) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
struct Raw8Float {
  float4 a, b;
  __device__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ float absmax() const {
    float v[8], m = 0.f;
    values(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = absmax_nan(m, v[i]);
    return m;
  }
  __device__ void values(float* v) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
template <class T>
struct Raw8 : Raw8Float {};
template <>
struct Raw8<__nv_bfloat16> : Raw8Bf16 {};

// ------------------------------------------------------------------ products

constexpr int kF8BK = 128;  // K per block: one 128-byte swizzle row, one scale
constexpr int kF8Threads = 192;

struct Fp8Geom {
  const void* x;     // bf16 or fp32 [T x K] where a kernel quantises it itself
  int K;
  const float* xs;   // [kb][T]
  const float* ws;   // the weight's scales: n block * ws_n + k block * ws_k
  void* out;         // [T x N]
  int T, N, nkb;
  int ws_n, ws_k;
  int out_fp32;
  int a_e5m2;
  // Whether every scale is a power of two: n_flags words, each nonzero if its part of them is (pair kernel). None: the
  // scales are applied in fp32.
  const int* flags;
  int n_flags;
  int xs_given;  // x's scales come from the caller and may be no powers of two
};

// A scale that the tensor cores can apply: a positive normal power of two; or a non-finite scale of x, which stands for
// NaN there. Its row's results are not finite either way: the quantiser's codes under such a scale make NaN, other codes
// under an infinite one would make infinities where the scale is applied in fp32.
__device__ __forceinline__ bool is_power(float s) {
  const uint32_t u = __float_as_uint(s);
  return (u & 0x807fffffu) == 0 && u != 0 && u < 0x7f800000u;
}
__device__ __forceinline__ bool is_power_or_bad(float s) { return is_power(s) || !(fabsf(s) < __uint_as_float(0x7f800000u)); }

constexpr int kF8MaxFlags = 64;
constexpr int kF8MaxBlocksFp32 = 32;  // k-blocks that the tensor cores add up for an fp32 result

// Eight 16-byte pieces of one row of a box (32 rows of 128 bytes, 128-byte swizzle), as a tiled store reads it.
__device__ __forceinline__ void fp8_stage_row(uint8_t* box, int lane, const uint4 (&p)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(box + lane * 128 + ((i ^ (lane & 7)) << 4)) = p[i];
}

// a.xy += v.xy * s.xy: two fp32 multiply-adds in one instruction (T = 512, K = 16384 on 16 pairs: 71 us, 84 us with
// two instructions).
__device__ __forceinline__ void fma2(float2& a, uint32_t v0, uint32_t v1, float s0, float s1) {
  asm("{\n\t.reg .b64 v, s, a;\n\t"
      "mov.b64 v, {%2, %3};\n\tmov.b64 s, {%4, %5};\n\tmov.b64 a, {%0, %1};\n\t"
      "fma.rn.f32x2 a, v, s, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a.x), "+f"(a.y)
      : "r"(v0), "r"(v1), "f"(s0), "f"(s1));
}

// ------------------------------------------------------------------ few tokens
//
// With few tokens the weight's bytes are the cost, so the operands change places: 128 rows of the weight are the
// MMA's M, NT tokens its N, and D holds the result transposed (lane = weight row, column = token). The K
// blocks of a tile are split over the CTAs of a cluster so that enough of the weight is in flight on every SM; two
// CTAs fit on one SM. Where the CTA's scales are powers of two the tensor cores apply them (see the CTA pairs below)
// and add up all of its k-blocks; else each k-block is folded into registers (T = 100 of 27648 x 5120: 32 against 55 us,
// T = 128 of 8192 x 8192: 21.5 against 29; T = 37 of 27648 x 5120, where the weight's bytes are 22 us: 28.5 against 29.6).
// The cluster then adds the splits
// through distributed shared memory in rank order, so the result does not depend on timing.
// W_MN: the weight's rows run along K (the input gradient, W [d_out x d_in] with K = d_out).
template <int NT>
struct Fp8Narrow {
  static constexpr int X_BYTES = NT * 128;
  static constexpr int STAGE_BYTES = 16384 + X_BYTES;
  static constexpr int STAGES = NT == 16 ? 6 : NT == 32 ? 5 : NT == 64 ? 4 : 3;
  static constexpr int SCALE_BYTES = 8 * NT * 4;  // token scales: two k-blocks per folding warp, or one per stage
  static_assert(STAGES <= 8, "scales");
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + SCALE_BYTES + 256 + 1024;
  // TMEM: two accumulators of k-blocks, or one for all of them and 8 columns of scales per stage.
  static constexpr uint32_t ACC_COLS = NT;
  static constexpr uint32_t USED = 2 * NT > NT + 8 * STAGES ? 2 * NT : NT + 8 * STAGES;
  static constexpr uint32_t TMEM_COLS = USED <= 64 ? 64 : USED <= 128 ? 128 : 256;
  static_assert(NT * 128 * 4 <= STAGES * STAGE_BYTES, "the splits' sums fit the ring");
  static_assert(SMEM_BYTES + 1024 <= 114 * 1024, "two CTAs per SM");
};

// The splits' sums of every CS-th token, starting with this CTA's own, added in rank order: a distributed shared
// memory read costs hundreds of clocks, so each thread has all CS of a float4 in flight.
template <int CS>
__device__ __forceinline__ void fp8_reduce_splits(const Fp8Geom& g, const float* sum, int rank, int t0, int live, int n0) {
  const int mine = (live - rank + CS - 1) / CS * 32;  // float4s of this CTA
#pragma unroll 2
  for (int i = threadIdx.x; i < mine; i += kF8Threads) {
    const int t = rank + i / 32 * CS, n = i % 32 * 4;
    float4 v[CS];
#pragma unroll
    for (int r = 0; r < CS; ++r)
      v[r] = *reinterpret_cast<const float4*>(CS == 1 ? sum + t * 128 + n : dsmem_ptr(sum + t * 128 + n, r));
    float4 a = v[0];
#pragma unroll
    for (int r = 1; r < CS; ++r) a.x += v[r].x, a.y += v[r].y, a.z += v[r].z, a.w += v[r].w;
    if (n0 + n >= g.N) continue;  // N is a multiple of 16
    const size_t at = (size_t)(t0 + t) * g.N + n0 + n;
    if (g.out_fp32) {
      *reinterpret_cast<float4*>((float*)g.out + at) = a;
    } else {
      __nv_bfloat162 p[2] = {__floats2bfloat162_rn(a.x, a.y), __floats2bfloat162_rn(a.z, a.w)};
      *reinterpret_cast<uint2*>((__nv_bfloat16*)g.out + at) = *reinterpret_cast<const uint2*>(p);
    }
  }
}

// XT: the type of x that the kernel quantises itself, or void where x comes in codes through tX. For up to 16 tokens
// and no more k-blocks per CTA than the ring has stages, the folding warps turn the CTA's blocks of x into codes while
// the weight is on its way, which saves a launch, its latency and the workspace. (Doing so inside a longer loop costs
// more than the launch: T = 1 of 27648 x 5120, 40 blocks per CTA, took 40 us so and 27 us with the launch.)
template <int NT, bool W_MN, class XT>
__global__ void __launch_bounds__(kF8Threads, 2)
    fp8_narrow_kernel(const __grid_constant__ CUtensorMap tW, const __grid_constant__ CUtensorMap tX, const Fp8Geom g,
                      int cs, int early_w) {
  using Cfg = Fp8Narrow<NT>;
  constexpr int STAGES = Cfg::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* scales = reinterpret_cast<float*>(smem + STAGES * Cfg::STAGE_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * Cfg::STAGE_BYTES + Cfg::SCALE_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* accf = empty + STAGES;  // [2] accumulator complete
  uint64_t* acce = accf + 2;        // [2] accumulator folded
  uint64_t* sff = acce + 2;         // [STAGES] a k-block's scales are in TMEM
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sff + STAGES);

  constexpr bool OWN_X = !std::is_same<XT, void>::value;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = blockIdx.x % cs;  // the cluster's CTAs are neighbours in x
  const int t_tiles = (g.T + NT - 1) / NT;  // the token tiles of a weight tile run side by side and share it in L2
  const int n0 = blockIdx.x / cs / t_tiles * 128, t0 = blockIdx.x / cs % t_tiles * NT;
  const int per = (g.nkb + cs - 1) / cs;
  const int kb0 = min(g.nkb, rank * per), nkb = min(g.nkb, kb0 + per) - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], OWN_X ? 5 : 1);  // the loads, and the four warps that write x
      mbar_init(&empty[s], 1);
      mbar_init(&sff[s], 4);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], 4);
    }
    fence_mbar_init();
    prefetch_tmap(&tW);
    if (!OWN_X) prefetch_tmap(&tX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();
  if (!early_w) pdl_wait();

  const float* ws = g.ws + (size_t)(n0 >> 7) * g.ws_n + (size_t)kb0 * g.ws_k;
  // The weight does not come from the preceding grid (the quantisation of x): its first stages are under way before
  // that grid is done.
  auto load_w = [&](int i) {
    uint8_t* sw = smem + i % STAGES * Cfg::STAGE_BYTES;
    mbar_arrive_expect_tx(&full[i % STAGES], OWN_X ? 16384 : Cfg::STAGE_BYTES);
    if (!W_MN)
      tma_load_2d(sw, &tW, &full[i % STAGES], (kb0 + i) * kF8BK, n0);
    else
      tma_load_2d(sw, &tW, &full[i % STAGES], n0, (kb0 + i) * kF8BK);
  };
  const int ahead = min(nkb, STAGES);
  if (warp == 0 && lane == 0)
    for (int i = 0; i < ahead; ++i) load_w(i);
  // The tensor cores apply the scales where every one is a power of two. A call that may quantise x itself folds
  // (T = 1 of 4096 x 4096: 7.2 us, and 7.8 if its scales are looked at first), with given codes too: the same sums.
  bool mx = !OWN_X && (NT > 16 || per > STAGES);
  if constexpr (!OWN_X) {
    mx = mx && (!g.out_fp32 || nkb <= kF8MaxBlocksFp32);
    if (warp >= 2) {  // this CTA's scales (those of an x quantised in the call are powers of two by their making)
      const int tid = threadIdx.x - 64;
      for (int i = tid; i < nkb; i += 128) mx = mx && is_power(ws[(size_t)i * g.ws_k]);
      if (g.xs_given) {
        for (int i = tid; i < nkb * NT; i += 128) {
          const int t = t0 + i % NT;
          mx = mx && (t >= g.T || is_power_or_bad(g.xs[(size_t)(kb0 + i / NT) * g.T + t]));
        }
      }
    }
    mx = __syncthreads_and(mx);
  }

  float2 acc[NT / 2];
#pragma unroll
  for (int t = 0; t < NT / 2; ++t) acc[t] = make_float2(0.f, 0.f);
  if (warp == 0) {
    if (lane == 0) {
      if (early_w) pdl_wait();
      int i = 0;
#pragma unroll 1
      for (; i < nkb; ++i) {
        const int s = i % STAGES;
        if (i >= ahead) {
          if (!mbar_wait(&empty[s], ((uint32_t)(i / STAGES) & 1u) ^ 1u)) break;
          load_w(i);
        }
        if (!OWN_X) tma_load_2d(smem + s * Cfg::STAGE_BYTES + 16384, &tX, &full[s], (kb0 + i) * kF8BK, t0);
      }
      if (i < nkb)  // a wait ran out: let the copies in flight land before the shared memory goes
        for (int j = max(0, i - STAGES); j < i; ++j) mbar_wait(&full[j % STAGES], (uint32_t)(j / STAGES) & 1u, kWaitLimitNs / 16);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = (mx ? idesc_mxfp8(128, NT, false, g.a_e5m2 != 0, false)
                                 : idesc_fp8_f32(128, NT, false, g.a_e5m2 != 0, false)) | (W_MN ? 1u << 15 : 0u);
      constexpr uint32_t w_kstep = W_MN ? 32u * 128u : 32u;
      if (mx) {
        bool ok = true;
#pragma unroll 1
        for (int i = 0; i < nkb; ++i) {
          const int s = i % STAGES;
          const uint32_t ph = (uint32_t)(i / STAGES) & 1u;
          if (!mbar_wait(&sff[s], ph) || !mbar_wait(&full[s], ph)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sw = smem_u32(smem + s * Cfg::STAGE_BYTES), sf = tmem + NT + 8u * s;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_mxfp8(tmem, sdesc_sw128(sw + kk * w_kstep, 16u, 1024u), sdesc_sw128(sw + 16384u + kk * 32u, 16u, 1024u), idesc,
                       sf, sf + 4u, i > 0 || kk > 0 ? 1u : 0u);
          umma_commit(&empty[s]);
        }
        if (ok) umma_commit(accf);
      }
#pragma unroll 1
      for (int i = mx ? nkb : 0; i < nkb; ++i) {
        const int s = i % STAGES, b = i & 1;
        if (!mbar_wait(&acce[b], ((uint32_t)(i >> 1) & 1u) ^ 1u)) break;
        if (!mbar_wait(&full[s], (uint32_t)(i / STAGES) & 1u)) break;
        tc_fence_after();
        const uint32_t sw = smem_u32(smem + s * Cfg::STAGE_BYTES);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_fp8(tmem + b * Cfg::ACC_COLS, sdesc_sw128(sw + kk * w_kstep, 16u, 1024u),
                   sdesc_sw128(sw + 16384u + kk * 32u, 16u, 1024u), idesc, kk > 0 ? 1u : 0u);
        umma_commit(&empty[s]);
        umma_commit(&accf[b]);
      }
    }
  } else {
    if (early_w) pdl_wait();
    const int q = warp & 3;
    // Scales of block i into TMEM: x's exponent bytes (xs[c]: of token 32 c + lane) and the weight's one.
    auto put_scales = [&](int i, const float (&xs)[4], float w) {
      const auto word = [](float s) { return (__float_as_uint(s) >> 23 & 0xffu) * 0x01010101u; };
      const uint32_t col = tmem + NT + 8u * (i % STAGES) + ((uint32_t)(q * 32) << 16), a = word(w);
      tc_fence_after();
      tmem_st4(col, a, a, a, a);
      tmem_st4(col + 4, word(xs[0]), word(xs[1]), word(xs[2]), word(xs[3]));
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sff[i % STAGES]);
    };
    // The whole sum, once the last block's MMAs are done.
    auto read_sum = [&]() {
      if (nkb == 0 || !mbar_wait(accf, 0)) return;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < NT / 16; ++c) {
        uint32_t v[16];
        tmem_ld16_async(tmem + c * 16 + ((uint32_t)(q * 32) << 16), v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[8 * c + j] = make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
      }
    };
    auto fold = [&](int b, const float* sc) {
      const uint32_t ta = tmem + b * Cfg::ACC_COLS + ((uint32_t)(q * 32) << 16);
#pragma unroll
      for (int c = 0; c < NT / 16; ++c) {
        uint32_t v[16];
        tmem_ld16_async(ta + c * 16, v);
        tmem_ld_wait();
        if (c == NT / 16 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acce[b]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 s4 = *reinterpret_cast<const float4*>(sc + 16 * c + 4 * j);
          fma2(acc[8 * c + 2 * j], v[4 * j], v[4 * j + 1], s4.x, s4.y);
          fma2(acc[8 * c + 2 * j + 1], v[4 * j + 2], v[4 * j + 3], s4.z, s4.w);
        }
      }
    };
    if constexpr (OWN_X) {
      // Eight threads of 16 values make one token's block. Rows behind the last token stay as they are: they only
      // reach columns of D that nobody reads.
      const int tid = threadIdx.x - 64, t = tid >> 3, c = (tid & 7) * 16;
      const XT* x = reinterpret_cast<const XT*>(g.x) + (size_t)min(t0 + t, g.T - 1) * g.K;
      Raw8<XT> raw[STAGES][2];
      float w[STAGES];
#pragma unroll
      for (int i = 0; i < STAGES; ++i) {
        const int k = (kb0 + i) * kF8BK + c;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (i < nkb && k < g.K)  // K is a multiple of 16
            raw[i][j].load(x + k + 8 * j);
          else
            raw[i][j].clear();
        }
        w[i] = i < nkb ? ws[(size_t)i * g.ws_k] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < STAGES; ++i) {
        if (i >= nkb) break;
        float amax = absmax_nan(raw[i][0].absmax(), raw[i][1].absmax());
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) amax = absmax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const BlockScale bs = g.a_e5m2 ? block_scale<true>(amax) : block_scale<false>(amax);
        if (t0 + t < g.T) {
          uint2 code[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float v[8];
            raw[i][j].values(v);
            code[j] = g.a_e5m2 ? to_fp8x8<true>(v, bs.inv) : to_fp8x8<false>(v, bs.inv);
          }
          uint8_t* row = smem + i * Cfg::STAGE_BYTES + 16384 + t * 128;
          *reinterpret_cast<uint4*>(row + (((tid & 7) ^ (t & 7)) << 4)) = make_uint4(code[0].x, code[0].y, code[1].x, code[1].y);
          if ((tid & 7) == 0) scales[i * NT + t] = bs.scale * w[i];
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[i]);
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");  // the four warps' scales
#pragma unroll 1
      for (int i = 0; i < nkb; ++i) {
        if (!mbar_wait(&accf[i & 1], (uint32_t)(i >> 1) & 1u)) break;
        tc_fence_after();
        fold(i & 1, scales + i * NT);
      }
    } else if (mx) {
      // Scales are fetched four k-blocks ahead, without a move that would wait for them.
      float v[4][4], wv[4];
      auto fetch = [&](int i, float (&x4)[4], float& w) {
        if (i >= nkb) return;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int t = t0 + 32 * c + lane;
          x4[c] = 32 * c < NT && t < g.T ? g.xs[(size_t)(kb0 + i) * g.T + t] : 0.f;
        }
        w = ws[(size_t)i * g.ws_k];
      };
      bool ok = true;
#pragma unroll
      for (int u = 0; u < 4; ++u) fetch(u, v[u], wv[u]);
#pragma unroll 1
      for (int i4 = 0; i4 < nkb && ok; i4 += 4) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = i4 + u;
          if (i >= nkb) break;
          if (!mbar_wait(&empty[i % STAGES], ((uint32_t)(i / STAGES) & 1u) ^ 1u)) {
            ok = false;
            break;
          }
          put_scales(i, v[u], wv[u]);
          fetch(i + 4, v[u], wv[u]);
        }
      }
      if (ok) read_sum();
    } else {
      constexpr int NS = (NT + 31) / 32;
      // Lane l fetches the scales of tokens l, l + 32, ... one k-block ahead; every lane reads them back from the warp's
      // own piece of shared memory, four at a time.
      float* mine = scales + q * 2 * NT;
      float xn[NS], wn = 0.f;
      auto fetch = [&](int i) {
        wn = ws[(size_t)i * g.ws_k];
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const int t = t0 + 32 * j + lane;
          xn[j] = t < g.T ? g.xs[(size_t)(kb0 + i) * g.T + t] : 0.f;
        }
      };
      if (nkb > 0) fetch(0);
#pragma unroll 1
      for (int i = 0; i < nkb; ++i) {
        const int b = i & 1;
#pragma unroll
        for (int j = 0; j < NS; ++j)
          if (NT >= 32 || lane < NT) mine[b * NT + 32 * j + lane] = xn[j] * wn;
        __syncwarp();
        if (i + 1 < nkb) fetch(i + 1);
        if (!mbar_wait(&accf[b], (uint32_t)(i >> 1) & 1u)) break;
        tc_fence_after();
        fold(b, mine + b * NT);
      }
    }
  }

  // Thread (warp q, lane) of the folding warps holds weight row n0 + 32 q + lane of every token. The sums go through
  // shared memory, [token][128] (the ring is idle: every load and MMA has been waited for), so that the splits can be
  // added and the results leave in whole rows.
  const int live = min(NT, g.T - t0);
  float* sum = reinterpret_cast<float*>(smem);
  __syncthreads();
  if (warp >= 2) {
    const int row = (warp & 3) * 32 + lane;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (t < live) sum[t * 128 + row] = (t & 1) ? acc[t / 2].y : acc[t / 2].x;
  }
  if (early_w) pdl_wait();
  if (cs == 1) {
    __syncthreads();
    fp8_reduce_splits<1>(g, sum, 0, t0, live, n0);
  } else {
    cluster_sync();
    switch (cs) {
      case 2: fp8_reduce_splits<2>(g, sum, rank, t0, live, n0); break;
      case 3: fp8_reduce_splits<3>(g, sum, rank, t0, live, n0); break;
      case 4: fp8_reduce_splits<4>(g, sum, rank, t0, live, n0); break;
      case 5: fp8_reduce_splits<5>(g, sum, rank, t0, live, n0); break;
      case 6: fp8_reduce_splits<6>(g, sum, rank, t0, live, n0); break;
      case 7: fp8_reduce_splits<7>(g, sum, rank, t0, live, n0); break;
      default: fp8_reduce_splits<8>(g, sum, rank, t0, live, n0);
    }
    cluster_sync();  // the peers have read this CTA's sums
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::TMEM_COLS);
  }
}

// ------------------------------------------------------------------ CTA pairs
//
// The wide tile: a cluster of two CTAs computes 256 x 256 results with
// cta_group::2 MMAs, each CTA staging its 128 rows of the operand and half of
// the weight tile's 256, so that per k-block (512 clocks of MMA per SM) only 32 KB
// come in per SM. TMEM (512 columns) holds two accumulators of 256. Eight
// epilogue warps fold: warp w reads TMEM lanes 32 (w % 4) .. + 31 and
// half of the columns, 128 fp32 sums per thread. Tiles are walked persistently; the MMAs of the next tile start while
// this one is stored.
//
// Folding and MMAs take about 750 and 700 clocks per k-block and meet at the two accumulators, so the sum of a
// k-block costs 955. When every scale is a power of two (as dora_fp8_quantize makes them; `flags` says so) the tensor
// cores apply the scales themselves (kind::mxf8f6f4): four warps write each k-block's scales into TMEM as exponent
// bytes, one accumulator holds the tile's whole sum, and the folding warps only store it. The same values come out of
// both up to fp32 additions. Those of the tensor cores lose about 1e-10 of a result per product (K = 2048: 1.5e-7 off
// in all, 0.7e-7 when folded; some 20000: 2.4e-6), nothing beside the rounding to bf16; fp32 results take this way up
// to K = 4096 only.
constexpr int kF8FoldWarps = 8;
constexpr int kF8PairThreads = 128 + 32 * kF8FoldWarps;
// The block launches with 384 x 168 registers, the most that 384 threads can have; the folding warps take 216 each and
// leave 72 to the others: 256 * 216 + 128 * 72 = 384 * 168. (With 168 for all, the sums spill.)
constexpr int kF8LaunchRegs = 168, kF8FoldRegs = 216, kF8OtherRegs = 72;
static_assert(32 * kF8FoldWarps * kF8FoldRegs + 128 * kF8OtherRegs <= kF8PairThreads * kF8LaunchRegs, "registers");
constexpr int kF8PairStages = 6;
constexpr int kF8StageBytes = 2 * 128 * 128;
constexpr int kF8OutBytes = 4096;  // one box of results per folding warp: 32 rows of 128 bytes
constexpr int kF8PairSmem = kF8PairStages * kF8StageBytes + kF8FoldWarps * kF8OutBytes + 256 + 1024;
static_assert(kF8PairSmem <= 227 * 1024, "shared memory");

// Tiles in groups of 16 rows of tiles, rows fastest: the tiles in flight share operands in L2, and neighbours the
// weight's. (T = 4096 of 8192 x 8192, run for a second: 256 us, 262 in groups of 8, 270 of 4, 276 of 2; groups of
// columns 259 to 276. T = 8192 of 27648 x 5120 1072 against 1095 us in groups of 8; T = 16384 of 4096 x 4096 loses by
// it, 273.5 against 270.)
constexpr int kF8TileGroup = 16;
__device__ __forceinline__ void fp8_tile_coords(int t, int m_tiles, int n_tiles, int& m, int& n) {
  const int per_group = kF8TileGroup * n_tiles;
  const int first_m = t / per_group * kF8TileGroup;
  const int gm = min(kF8TileGroup, m_tiles - first_m);
  const int rem = t % per_group;
  m = first_m + rem % gm;
  n = rem / gm;
}

template <bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kF8PairThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap tA, const __grid_constant__ CUtensorMap tB,
                    const __grid_constant__ CUtensorMap tOut, const Fp8Geom g) {
  constexpr int STAGES = kF8PairStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out_smem = smem + STAGES * kF8StageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(out_smem + kF8FoldWarps * kF8OutBytes);  // used in the leader
  uint64_t* empty = full + STAGES;
  uint64_t* accf = empty + STAGES;  // [2] accumulator complete
  uint64_t* acce = accf + 2;        // [2] accumulator folded by both CTAs, used in the leader
  uint64_t* sff = acce + 2;         // [STAGES] a k-block's scales are in TMEM of both CTAs, used in the leader
  uint64_t* sume = sff + STAGES;    // the tile's sum has been read by both CTAs, used in the leader
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sume + 1);

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
      mbar_init(&sff[s], 8);
    }
    mbar_init(sume, 8);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], 2 * kF8FoldWarps);
    }
    fence_mbar_init();
    prefetch_tmap(&tA);
    prefetch_tmap(&tB);
    prefetch_tmap(&tOut);
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
  bool mx = g.n_flags > 0;
  for (int f = lane; f < g.n_flags; f += 32) mx = mx && g.flags[f] != 0;
  mx = __all_sync(0xffffffffu, mx);
  constexpr uint32_t SCALE_COL = 256;  // of stage s: 4 columns of x's scales and 8 of the weight's at 256 + 16 s

  if (warp < 4) {
    setmaxnreg_dec<kF8OtherRegs>();
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
      const uint32_t idesc = mx ? idesc_mxfp8(256, 256, g.a_e5m2 != 0, false, B_MN)
                                : idesc_fp8_f32(256, 256, g.a_e5m2 != 0, false, B_MN);
      constexpr uint32_t b_kstep = B_MN ? 32u * 128u : 32u;
      int it = 0;
      bool ok = true;
      if (mx) {
        int j = 0;
#pragma unroll 1
        for (int t = pair; t < tiles && ok; t += npairs, ++j) {
          if (!mbar_wait(sume, ((uint32_t)j & 1u) ^ 1u)) break;
#pragma unroll 1
          for (int kb = 0; kb < g.nkb; ++kb, ++it) {
            const int s = it % STAGES;
            const uint32_t ph = (uint32_t)(it / STAGES) & 1u;
            if (!mbar_wait(&sff[s], ph) || !mbar_wait(&full[s], ph)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + s * kF8StageBytes), sf = tmem + SCALE_COL + 16u * s;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_mxfp8_pair(tmem, sdesc_sw128(sa + kk * 32u, 16u, 1024u),
                              sdesc_sw128(sa + 16384u + kk * b_kstep, 16u, 1024u), idesc, sf, sf + 4u,
                              kb > 0 || kk > 0 ? 1u : 0u);
            umma_commit_pair(&empty[s], 0x3);
          }
          if (ok) umma_commit_pair(&accf[0], 0x3);
        }
        ok = false;  // the loop below is the other kind's
      }
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
    setmaxnreg_inc<kF8FoldRegs>();
    const int q = warp & 3, part = (warp - 4) >> 2;
    // Results leave by tiled stores of 32 rows x 128 bytes from one box per warp, so that the next tile's folding
    // begins after a few hundred clocks (row-per-thread stores: 3.2 us a tile; what lies outside is dropped).
    // 128 columns of the warp's 32 rows, from row mw and column n0 on; thread = row.
    auto store128 = [&](const float2 (&acc)[64], uint8_t* box, int boxes, int mw, int n0) {
      auto send = [&](int c, int n, const uint4 (&p)[8]) {
        uint8_t* to = box + (boxes > 1 ? c & 1 : 0) * kF8OutBytes;
        if (lane == 0) {
          if (boxes > 1)
            bulk_wait_read<1>();
          else
            bulk_wait_read<0>();
        }
        __syncwarp();
        fp8_stage_row(to, lane, p);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (n < g.N) tma_store_2d(&tOut, to, n, mw);
          bulk_commit();
        }
      };
      if (g.out_fp32) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint4 p[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            p[i] = make_uint4(__float_as_uint(acc[16 * c + 2 * i].x), __float_as_uint(acc[16 * c + 2 * i].y),
                              __float_as_uint(acc[16 * c + 2 * i + 1].x), __float_as_uint(acc[16 * c + 2 * i + 1].y));
          send(c, n0 + 32 * c, p);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint4 p[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            __nv_bfloat162 h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = __float22bfloat162_rn(acc[32 * c + 4 * i + j]);
            p[i] = *reinterpret_cast<const uint4*>(h);
          }
          send(c, n0 + 64 * c, p);
        }
      }
    };
    if (mx && part == 0) {
      // Scales of each k-block into TMEM. A word holds the exponent byte of one row four times (the k-block's four MMAs
      // share it); row 32 c + l of the 128 rows lies in lane l of column c, in all four lane quarters: this warp
      // writes quarter q.
      const uint32_t filled = mapa_shared(smem_u32(sff), 0);
      const uint32_t to = tmem + SCALE_COL + ((uint32_t)(q * 32) << 16);
      const auto word = [](float s) { return (__float_as_uint(s) >> 23 & 0xffu) * 0x01010101u; };
      int it = 0;
      bool ok = true;
#pragma unroll 1
      for (int t = pair; t < tiles && ok; t += npairs) {
        int tm, tn;
        fp8_tile_coords(t, m_tiles, n_tiles, tm, tn);
        const int m0 = tm * 256 + (int)rank * 128, n0 = tn * 256;
        const float* xs[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) xs[c] = g.xs + min(m0 + 32 * c + lane, g.T - 1);
        const float* w0 = g.ws + (size_t)(n0 >> 7) * g.ws_n;
        const float* w1 = n0 + 128 < g.N ? w0 + g.ws_n : w0;
        float v[4][6];  // fetched four k-blocks ahead, without a move that would wait for them
        auto fetch = [&](int kb, float (&f)[6]) {
          if (kb >= g.nkb) return;
#pragma unroll
          for (int c = 0; c < 4; ++c) f[c] = xs[c][(size_t)kb * g.T];
          f[4] = w0[(size_t)kb * g.ws_k];
          f[5] = w1[(size_t)kb * g.ws_k];
        };
#pragma unroll
        for (int u = 0; u < 4; ++u) fetch(u, v[u]);
#pragma unroll 1
        for (int kb4 = 0; kb4 < g.nkb && ok; kb4 += 4) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int kb = kb4 + u;
            if (kb >= g.nkb) break;
            const int s = it % STAGES;
            if (!mbar_wait(&empty[s], ((uint32_t)(it / STAGES) & 1u) ^ 1u)) {
              ok = false;
              break;
            }
            const uint32_t col = to + 16u * s;
            const uint32_t a = word(v[u][4]), b = word(v[u][5]);
            tc_fence_after();
            tmem_st4(col, word(v[u][0]), word(v[u][1]), word(v[u][2]), word(v[u][3]));
            tmem_st4(col + 4, a, a, a, a);
            tmem_st4(col + 8, b, b, b, b);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(filled + 8 * s);
            fetch(kb + 4, v[u]);
            ++it;
          }
        }
      }
    } else if (mx) {
      // The tile's sum: two halves of 128 columns; the accumulator goes back once the second has been read.
      const uint32_t done = mapa_shared(smem_u32(sume), 0);
      uint8_t* box = out_smem + (warp - 8) * 2 * kF8OutBytes;
      int j = 0;
#pragma unroll 1
      for (int t = pair; t < tiles; t += npairs, ++j) {
        int tm, tn;
        fp8_tile_coords(t, m_tiles, n_tiles, tm, tn);
        const int mw = tm * 256 + (int)rank * 128 + q * 32;
        if (!mbar_wait(&accf[0], (uint32_t)j & 1u)) break;
        tc_fence_after();
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const int n0 = tn * 256 + half * 128;
          float2 acc[64];
          uint32_t v[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32_async(tmem + half * 128 + c * 32 + ((uint32_t)(q * 32) << 16), v[c]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 64; ++c) acc[c] = make_float2(__uint_as_float(v[c / 16][2 * (c % 16)]), __uint_as_float(v[c / 16][2 * (c % 16) + 1]));
          if (half == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(done);
          }
          if (mw < g.T && n0 < g.N) store128(acc, box, 2, mw, n0);
        }
      }
    } else {
    constexpr int COLS = 4 * 256 / kF8FoldWarps;  // columns per warp
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
      float2 acc[64];
      static_assert(COLS == 128, "columns per folding warp");
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
            for (int j = 0; j < 8; ++j) fma2(acc[c * 8 + j], v[2 * j], v[2 * j + 1], s, s);
          }
        } else if (lane == 0) {
          mbar_arrive_cluster(done + 8 * b);
        }
      }
      if (ok && live) store128(acc, out_smem + (warp - 4) * kF8OutBytes, 1, mw, n0);
    }
    }
    if (lane == 0) bulk_wait_all();
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
