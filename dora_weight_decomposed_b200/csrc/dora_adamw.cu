// The update of the trained tensors: the global gradient norm and the AdamW
// step, each over many tensors in one launch (or a few: the table of tensors
// travels in the kernel's parameters, so nothing has to be laid out in device
// memory and every call checks and reads the table it is given).
//
// Both stream their tensors once and are bound by HBM. A work item is a chunk
// of 2048 consecutive elements of one tensor, 8 per thread; a persistent grid
// walks the chunks of all tensors in turn. Measured at 100 M elements with bf16
// gradients: the norm 35 us (5.6 TB/s; 49 right behind an update, whose dirty
// lines leave L2 meanwhile), the 8-bit update with a master copy 288 us and the
// 32-bit one 522 us (5.6 and 5.4 TB/s). Without a master copy the 8-bit update is bound
// by its instructions instead (17 M elements 48.6 us, 3.7 TB/s).
#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include <cuda_bf16.h>

#include "dora_internal.h"
#include "host_launch.h"
#include "sm100_ptx.cuh"

namespace dora {
namespace {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kThreads = 256;
constexpr int kChunk = kThreads * 8;

// ------------------------------------------------------------------ tables

// The kernels' parameters hold up to about 32 KB of tensors; first[i] is tensor i's first chunk.
template <class Entry, int MAX>
struct Table {
  int n;
  int chunks;
  int first[MAX];
  Entry e[MAX];
};

template <class Entry, int MAX>
__device__ __forceinline__ int find_tensor(const Table<Entry, MAX>& t, int chunk) {
  int lo = 0, hi = t.n - 1;  // the last tensor whose first chunk is <= chunk
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

struct GradEntry {
  const void* g;
  int64_t n;
  int fp32;
  int vec;
};
constexpr int kMaxGrads = 1100;
template <int MAX>
using GradTable = Table<GradEntry, MAX>;
static_assert(sizeof(GradTable<kMaxGrads>) < 32000, "kernel parameters");
// Calls of few tensors pass a short table: a full one costs the host 3 us more per launch.
constexpr int kFew = 24;

struct AdamEntry {
  void* p;
  const void* g;
  void* avg;
  void* sq;
  float* savg;
  float* ssq;
  float* master;
  int64_t n;
  uint32_t index0;  // of pairs: (index0 + i) / 2 modulo 2^32
  float wd;
  // vec: 16-byte aligned; bulk: all of the tensor's arrays are
  uint8_t p_fp32 : 1, g_fp32 : 1, p_vec : 1, g_vec : 1, bulk : 1;
};
constexpr int kMaxAdam = 385;
template <int MAX>
using AdamTable = Table<AdamEntry, MAX>;
static_assert(sizeof(AdamTable<kMaxAdam>) < 32600, "kernel parameters");

// ------------------------------------------------------------------ two fp32 at a time

// The 8-bit step is bound by its instructions, so its arithmetic is done on pairs (one instruction for two, each
// rounded by itself).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 r, a, b;\n\t"
      "mov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 r, a, b;\n\t"
      "mov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 r, a, b, c;\n\tmov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
// a + b of two products as single additions: a packed addition would be merged with one of the packed products.
__device__ __forceinline__ float2 add_rounded(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// ------------------------------------------------------------------ loads and stores of 8 elements

// Elements i .. i + 7 as they lie in memory: bf16 in a, fp32 in a and b; zeros beyond the tensor.
struct Raw8 {
  uint4 a, b;
};

// vec: the base is 16-byte aligned.
__device__ __forceinline__ Raw8 load_raw(const void* base, int fp32, int vec, int64_t i, int64_t n) {
  Raw8 r;
  r.a = r.b = make_uint4(0u, 0u, 0u, 0u);
  if (vec && i + 8 <= n) {
    const uint4* p = reinterpret_cast<const uint4*>((const char*)base + i * (fp32 ? 4 : 2));
    r.a = p[0];
    if (fp32) r.b = p[1];
  } else if (i < n) {
    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (i + j >= n) continue;
      if (fp32)
        w[j] = ((const uint32_t*)base)[i + j];
      else
        w[j / 2] |= (uint32_t)((const uint16_t*)base)[i + j] << (16 * (j & 1));
    }
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
    r.b = make_uint4(w[4], w[5], w[6], w[7]);
  }
  return r;
}

__device__ __forceinline__ void values(const Raw8& r, int fp32, float2 (&v)[4]) {
  if (fp32) {
    v[0] = make_float2(__uint_as_float(r.a.x), __uint_as_float(r.a.y));
    v[1] = make_float2(__uint_as_float(r.a.z), __uint_as_float(r.a.w));
    v[2] = make_float2(__uint_as_float(r.b.x), __uint_as_float(r.b.y));
    v[3] = make_float2(__uint_as_float(r.b.z), __uint_as_float(r.b.w));
  } else {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
  }
}

template <bool WHOLE = false>
__device__ __forceinline__ void store8(void* base, int fp32, int vec, int64_t i, int64_t n, const float2 (&v)[4]) {
  if constexpr (!WHOLE) {
    if (!vec || i + 8 > n) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (i + j >= n) return;
        const float x = (j & 1) ? v[j / 2].y : v[j / 2].x;
        if (fp32)
          ((float*)base)[i + j] = x;
        else
          ((__nv_bfloat16*)base)[i + j] = __float2bfloat16_rn(x);
      }
      return;
    }
  }
  if (fp32) {
    float4* p = reinterpret_cast<float4*>((float*)base + i);
    p[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    p[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  } else {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = __float22bfloat162_rn(v[j]);
    *reinterpret_cast<uint4*>((__nv_bfloat16*)base + i) = *reinterpret_cast<const uint4*>(h);
  }
}

// 8 e4m3 codes (zeros beyond n).
__device__ __forceinline__ uint2 load_codes(const uint8_t* base, int64_t i, int64_t n) {
  uint2 u = make_uint2(0u, 0u);
  if (i + 8 <= n) {
    u = *reinterpret_cast<const uint2*>(base + i);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) (j < 4 ? u.x : u.y) |= (uint32_t)base[i + j] << (8 * (j & 3));
  }
  return u;
}

__device__ __forceinline__ void code_values(uint2 u, float2 (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint16_t two = (uint16_t)((j < 2 ? u.x : u.y) >> (16 * (j & 1)));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    v[j] = __half22float2(*reinterpret_cast<const __half2*>(&h));
  }
}

template <bool WHOLE>
__device__ __forceinline__ void store_codes(uint8_t* base, int64_t i, int64_t n, uint2 u) {
  if constexpr (!WHOLE) {
    if (i + 8 > n) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j < n) base[i + j] = (uint8_t)((j < 4 ? u.x : u.y) >> (8 * (j & 3)));
      return;
    }
  }
  *reinterpret_cast<uint2*>(base + i) = u;
}

// The chunks [first, last) of one CTA: contiguous, so that the tensor they lie in is found once and then followed.
struct Range {
  int first, last;
};
__device__ __forceinline__ Range cta_range(int chunks) {
  const int per = chunks / (int)gridDim.x, more = chunks % (int)gridDim.x, b = blockIdx.x;
  const int first = b * per + min(b, more);
  return {first, first + per + (b < more ? 1 : 0)};
}

// ------------------------------------------------------------------ gradient norm

constexpr int kNormBlocksPerSM = 5;
constexpr int kNormBlocksMax = 1024;

// Sum of eight squares, in fp32 where it holds them.
__device__ __forceinline__ double squares(const Raw8& raw, int fp32) {
  float2 v[4];
  values(raw, fp32, v);
  float2 s = mul2(v[0], v[0]);
#pragma unroll
  for (int j = 1; j < 4; ++j) s = fma2(v[j], v[j], s);
  const float a = s.x + s.y;
  if (a > 1e-30f && a < 1e38f) return (double)a;
  double d = 0.0;  // squares beyond the range of fp32 (or zeros, or not finite)
#pragma unroll
  for (int j = 0; j < 4; ++j) d += (double)v[j].x * v[j].x + (double)v[j].y * v[j].y;
  return d;
}

// Sum of squares of this CTA's chunks: 8 values in fp32, everything above in double.
template <int MAX>
__global__ void __launch_bounds__(kThreads) grad_norm_partial_kernel(const __grid_constant__ GradTable<MAX> t,
                                                                     double* __restrict__ part) {
  __shared__ double red[kThreads / 32];
  pdl_wait();
  pdl_trigger();  // only now: the update that follows reads the parameters and moments ahead of this grid's end
  double sum = 0.0;
  const Range range = cta_range(t.chunks);
  for (int c = range.first, k = find_tensor(t, range.first); c < range.last; ++k) {
    // This CTA's chunks of tensor k, four loads in flight per thread.
    const GradEntry& e = t.e[k];
    const int end = min(range.last, k + 1 < t.n ? t.first[k + 1] : t.chunks);
    int64_t i = (int64_t)(c - t.first[k]) * kChunk + threadIdx.x * 8;
    for (; c < end; c += 4, i += 4 * kChunk) {
      Raw8 raw[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) raw[j] = load_raw(e.g, e.fp32, e.vec, i + j * kChunk, c + j < end ? e.n : 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum += squares(raw[j], e.fp32);
    }
    c = end;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) s += red[w];
    part[blockIdx.x] = s;
  }
}

// sqrt of the sum of the partial sums (the whole block takes part; every block gets the same value), and the scale. A
// norm that fp32 holds as infinite counts as not finite: the scale agrees with the norm that the caller reads.
struct NormScale {
  double norm;
  float scale;
};
__device__ __forceinline__ NormScale norm_and_scale(const double* part, int n, float max_norm) {
  __shared__ double red[kThreads / 32];
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) sum += part[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += red[w];
  s = sqrt(s);
  const double c = (double)max_norm / (s + 1e-6);
  return {s, !isfinite((float)s) ? __uint_as_float(0x7fffffffu) : (float)(c < 1.0 ? c : 1.0)};
}

__global__ void __launch_bounds__(kThreads) grad_norm_final_kernel(const double* __restrict__ part, int n, float max_norm,
                                                                   float* __restrict__ norm, float* __restrict__ scale) {
  pdl_trigger();
  pdl_wait();
  const NormScale r = norm_and_scale(part, n, max_norm);
  if (threadIdx.x == 0) {
    *norm = (float)r.norm;
    *scale = r.scale;
  }
}

// ------------------------------------------------------------------ AdamW

struct AdamArgs {
  float b1, omb1, b2, omb2;  // betas and one minus them (rounded from double)
  float ln_b1, ln_b2;
  float eps;
  uint32_t seed;
  // Clipping within the step: the partial sums of grad_norm_partial_kernel, which every CTA adds up for itself in the
  // same order (a few KB from L2, where a kernel of its own between the two would cost its launch).
  const double* part;
  int parts;
  float max_norm;
  float* norm;
};

// Integer hash: two rounds of xor-shift and an odd multiplier (the leading
// bits of the fractions of sqrt(2) and sqrt(3), made odd).
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x6A09E667u;
  x = (x ^ (x >> 15)) * 0xBB67AE85u;
  return x ^ (x >> 16);
}

// 0 <= y <= 448 as an e4m3 code, floor(y / step + u / 65536) with step the code spacing at y, in the top byte of the
// result (its top bit clear). From 2^-6 up the spacing is 2^-3 of the binade, so the code is the top bits of the fp32
// pattern (exponent offset 120) after u is added below them. Under 2^-6 it is 2^-9 throughout, and adding 2^-6 brings
// the same bits into the same place (offset 121). Doubling y moves the first offset to 121 too, and the larger of
// the two (t) is the one that holds. u: 16 bits.
__device__ __forceinline__ uint32_t stochastic_code(float t, uint32_t u) {
  return (__float_as_uint(t) + (u << 4)) * 16u - (121u << 27);
}

// The scale of a block of 16 lanes x 8 moments (all of the warp's lanes take part); not finite if one of them is not.
__device__ __forceinline__ float moment_scale(const float2 (&v)[4]) {
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(amax) : "f"(fabsf(v[j].x)));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(amax) : "f"(fabsf(v[j].y)));
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const float b = __shfl_xor_sync(0xffffffffu, amax, o);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(amax) : "f"(b));
  }
  float s = amax * (1.0f / 448.0f);
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(s) : "f"(1.17549435e-38f));
  return s;
}

// a / b rounded to nearest from the rounded reciprocal of b (Markstein's quotient step); minus_b = -b.
__device__ __forceinline__ float2 quotient(float2 a, float minus_b, float inv_b) {
  const float2 q = mul2(a, both(inv_b));
  return fma2(fma2(q, both(minus_b), a), both(inv_b), q);
}

// sqrt(v) = v rsqrt(v) with one Newton step on the residual v - s^2, to the last place for v >= kRootLeast. Zero for
// v = 0, NaN for inf, and below sqrt(kRootLeast) for the v between, where the estimate is held back: see root_small.
constexpr float kRootLeast = 1e-37f;
__device__ __forceinline__ float2 root(float2 v) {
  float2 y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(fmaxf(v.x, kRootLeast)));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(fmaxf(v.y, kRootLeast)));
  const float2 s = mul2(v, y);
  return fma2(fma2(mul2(s, both(-1.0f)), s, v), mul2(y, both(0.5f)), s);
}

// r with the roots of the v under kRootLeast, subnormal ones among them: those are scaled by 2^64, their roots by 2^-32.
__device__ __forceinline__ float2 root_small(float2 v, float2 r) {
  const float2 s = mul2(root(mul2(v, both(18446744073709551616.0f))), both(2.3283064365386963e-10f));
  return make_float2(v.x < kRootLeast ? s.x : r.x, v.y < kRootLeast ? s.y : r.y);
}

__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// 1 / b for a normal b: the approximation with one Newton step.
__device__ __forceinline__ float inverse(float b) {
  const float r = reciprocal(b);
  return fmaf(fmaf(-b, r, 1.0f), r, r);
}

// The four top bytes, first in the lowest place.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

struct StepScalars {
  float gs, lr, lr1, rbc2;
  uint32_t key;
};

// Eight elements as they lie in memory.
template <int BITS>
struct Elements {
  Raw8 g, p, m, v;  // m, v: 32 bits
  uint2 cm, cv;     // 8 bits
  float sm, sr;
};

// Elements i .. i + 7 of tensor e, of any alignment.
template <int BITS>
__device__ __forceinline__ void load_elements(const AdamEntry& e, int64_t i, Elements<BITS>& x) {
  const int64_t n = e.n;
  x.g = load_raw(e.g, e.g_fp32, e.g_vec, i, n);
  x.p = e.master ? load_raw(e.master, 1, 1, i, n) : load_raw(e.p, e.p_fp32, e.p_vec, i, n);
  if (BITS == 32) {
    x.m = load_raw(e.avg, 1, 1, i, n);
    x.v = load_raw(e.sq, 1, 1, i, n);
  } else {
    x.cm = load_codes((const uint8_t*)e.avg, i, n);
    x.cv = load_codes((const uint8_t*)e.sq, i, n);
    x.sm = i < n ? e.savg[i >> 7] : 0.f;
    x.sr = i < n ? e.ssq[i >> 7] : 0.f;
  }
}

// Elements i .. i + 7 of tensor e into L2 (32 bits; held in registers over the wait they would spill).
__device__ __forceinline__ void prefetch_elements(const AdamEntry& e, int64_t i) {
  if (i >= e.n) return;
  const auto fetch = [](const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); };
  fetch((const char*)e.g + i * (e.g_fp32 ? 4 : 2));
  fetch(e.master ? (const char*)(e.master + i) : (const char*)e.p + i * (e.p_fp32 ? 4 : 2));
  fetch((const float*)e.avg + i);
  fetch((const float*)e.sq + i);
}

// The update of elements i .. i + 7 of tensor e by one thread; the warp's lanes hold consecutive ones. WHOLE: the
// elements lie in a whole chunk of an aligned tensor.
template <int BITS, bool WHOLE>
__device__ __forceinline__ void update(const AdamEntry& e, const AdamArgs& a, const StepScalars& c, int64_t i,
                                       const Elements<BITS>& x) {
  const int64_t n = e.n;
  float2 g[4], p[4], m[4], v[4], r[4];
  values(x.g, e.g_fp32, g);
  values(x.p, e.master || e.p_fp32, p);
  float sm = x.sm, sr = x.sr;
  if (BITS == 32) {
    values(x.m, 1, m);
    values(x.v, 1, v);
  } else {
    code_values(x.cm, m);
    code_values(x.cv, v);
  }
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (BITS == 8) {
      m[j] = mul2(m[j], both(sm));
      v[j] = mul2(v[j], both(sr));
      v[j] = mul2(v[j], v[j]);
    }
    // Each product and sum rounded by itself: the moments' stored codes then depend on the formula alone.
    g[j] = mul2(g[j], both(c.gs));
    m[j] = add_rounded(mul2(m[j], both(a.b1)), mul2(g[j], both(a.omb1)));
    v[j] = add_rounded(mul2(v[j], both(a.b2)), mul2(mul2(g[j], g[j]), both(a.omb2)));
    r[j] = root(v[j]);
    if (BITS == 32) top = fmaxf(top, fmaxf(v[j].x, v[j].y));
  }
  float least = fminf(fminf(r[0].x, r[0].y), fminf(r[1].x, r[1].y));
  least = fminf(least, fminf(fminf(r[2].x, r[2].y), fminf(r[3].x, r[3].y)));
  const bool some_zero = !(least > 0.f);
  if (least < 3.2e-19f) {  // sqrt(kRootLeast) and its rounding: rare but for zero moments
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = root_small(v[j], r[j]);
  }
  if (BITS == 8) {
    sm = moment_scale(m);
    sr = moment_scale(r);
  }
  // An infinite v (the square of a gradient above 1e19) has made its root NaN: the exact one instead.
  if (BITS == 32 ? !(top < 3e38f) : __any_sync(0xffffffffu, !(sr < 3e38f))) {
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = make_float2(sqrtf(v[j].x), sqrtf(v[j].y));
    if (BITS == 8) sr = moment_scale(r);
  }
  const float2 keep = both(1.0f - c.lr * e.wd);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 den = fma2(r[j], both(c.rbc2), both(a.eps));
    p[j] = fma2(mul2(m[j], both(-c.lr1)), make_float2(reciprocal(den.x), reciprocal(den.y)), mul2(p[j], keep));
  }
  if (e.master) store8<WHOLE>(e.master, 1, 1, i, n, p);
  store8<WHOLE>(e.p, e.p_fp32, e.p_vec, i, n, p);
  if (BITS == 32) {
    store8<WHOLE>(e.avg, 1, 1, i, n, m);
    store8<WHOLE>(e.sq, 1, 1, i, n, v);
    return;
  }
  uint2 cm = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu), cr = cm;  // NaN codes
  if (sm < 1e37f && sr < 1e37f) {
    const float im = inverse(sm), ir = inverse(sr);
    uint32_t zm[8], zr[8];
    const uint32_t pair0 = e.index0 + (uint32_t)(i >> 1);
    // sqrt(v) > 0 is held as code 1 at least: t = 2^-6 (1 + 1 / 8).
    constexpr float kOne = 0.017578125f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t h = mix((pair0 + j) ^ c.key);
      const uint32_t u0 = h & 0xffffu, u1 = h >> 16;
      const float2 ym = quotient(m[j], -sm, im), yr = quotient(r[j], -sr, ir);
      const float2 am = make_float2(fabsf(ym.x), fabsf(ym.y));
      const float2 tm = add2(am, am), lm = add2(am, both(0.015625f)), tr = add2(yr, yr), lr = add2(yr, both(0.015625f));
      zm[2 * j] = stochastic_code(fmaxf(tm.x, lm.x), u0) | (__float_as_uint(ym.x) & 0x80000000u);
      zm[2 * j + 1] = stochastic_code(fmaxf(tm.y, lm.y), u1) | (__float_as_uint(ym.y) & 0x80000000u);
      zr[2 * j] = stochastic_code(fmaxf(fmaxf(tr.x, lr.x), kOne), u0);
      zr[2 * j + 1] = stochastic_code(fmaxf(fmaxf(tr.y, lr.y), kOne), u1);
    }
    if (some_zero) {  // a zero moment (padding, a row without gradient) stays zero
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!(r[j].x > 0.f)) zr[2 * j] = 0;
        if (!(r[j].y > 0.f)) zr[2 * j + 1] = 0;
      }
    }
    cm = make_uint2(top_bytes(zm[0], zm[1], zm[2], zm[3]), top_bytes(zm[4], zm[5], zm[6], zm[7]));
    cr = make_uint2(top_bytes(zr[0], zr[1], zr[2], zr[3]), top_bytes(zr[4], zr[5], zr[6], zr[7]));
  }
  store_codes<WHOLE>((uint8_t*)e.avg, i, n, cm);
  store_codes<WHOLE>((uint8_t*)e.sq, i, n, cr);
  if ((threadIdx.x & 15) == 0 && (WHOLE || i < n)) {
    e.savg[i >> 7] = sm;
    e.ssq[i >> 7] = sr;
  }
}

// The 8-bit step issues about 70 instructions per element, so its loads are taken off the threads: whole chunks of
// aligned tensors come by bulk copies, the next one under way while this one is computed. Other chunks (a tensor's
// last, odd alignments) are read directly. (25 M values: 80 us with all loads direct.) Odd alignments include scales
// that start off a 16-byte border, as those of all tensors behind one whose number of blocks is no multiple of 4 may
// (32 layers of 4104 x 4104, r = 64, a quarter of the values aligned: 55 us, 47.6 at 4096 x 4096).
struct __align__(128) Stage8 {
  uint8_t g[kChunk * 4];
  uint8_t p[kChunk * 4];
  uint8_t cm[kChunk];
  uint8_t cv[kChunk];
  float sm[kChunk / 128];
  float sr[kChunk / 128];
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

struct Stages {
  Stage8 stage[2];
  uint64_t full[2];
};

__device__ __forceinline__ bool is_whole(const AdamEntry& e, int64_t i0) { return e.bulk && i0 + kChunk <= e.n; }

// Chunk c of tensor e, which starts at chunk e_first, into stage b (one thread): bulk copies, or an empty phase.
__device__ __forceinline__ void issue_chunk(Stages& s, int b, const AdamEntry& e, int e_first, int c) {
  const int64_t i0 = (int64_t)(c - e_first) * kChunk;
  Stage8& to = s.stage[b];
  uint64_t* bar = &s.full[b];
  if (!is_whole(e, i0)) {
    mbar_arrive(bar);
    return;
  }
  const uint32_t gb = e.g_fp32 ? 4 : 2, pb = e.master || e.p_fp32 ? 4 : 2;
  const char* p = e.master ? (const char*)e.master : (const char*)e.p;
  mbar_arrive_expect_tx(bar, kChunk * (gb + pb + 2) + 2 * kChunk / 128 * 4);
  bulk_load(to.g, (const char*)e.g + i0 * gb, kChunk * gb, bar);
  bulk_load(to.p, p + i0 * pb, kChunk * pb, bar);
  bulk_load(to.cm, (const char*)e.avg + i0, kChunk, bar);
  bulk_load(to.cv, (const char*)e.sq + i0, kChunk, bar);
  bulk_load(to.sm, e.savg + (i0 >> 7), kChunk / 128 * 4, bar);
  bulk_load(to.sr, e.ssq + (i0 >> 7), kChunk / 128 * 4, bar);
}

// The CTA's chunks, the first of which (of tensor k) has been issued.
template <int MAX>
__device__ __forceinline__ void update_range_staged(Stages& s, const AdamTable<MAX>& t, const AdamArgs& a,
                                                    const StepScalars& sc, const Range range, int k) {
  int kn = k;
  bool ok = true;
#pragma unroll 1
  for (int c = range.first; c < range.last; ++c) {
    const int it = c - range.first;
    if (c + 1 < range.last) {
      while (kn + 1 < t.n && t.first[kn + 1] <= c + 1) ++kn;
      if (threadIdx.x == 0) issue_chunk(s, (it + 1) & 1, t.e[kn], t.first[kn], c + 1);
    }
    ok = __all_sync(0xffffffffu, ok && mbar_wait(&s.full[it & 1], (uint32_t)(it >> 1) & 1u));
    if (ok) {  // a wait that ran out leaves the rest of the warp's elements as they are
      const AdamEntry& e = t.e[k];
      const int64_t i0 = (int64_t)(c - t.first[k]) * kChunk, i = i0 + threadIdx.x * 8;
      Elements<8> x;
      if (is_whole(e, i0)) {
        const Stage8& st = s.stage[it & 1];
        const uint4* g = reinterpret_cast<const uint4*>(st.g) + threadIdx.x * (e.g_fp32 ? 2 : 1);
        const uint4* p = reinterpret_cast<const uint4*>(st.p) + threadIdx.x * (e.master || e.p_fp32 ? 2 : 1);
        x.g.a = g[0];
        x.p.a = p[0];
        if (e.g_fp32) x.g.b = g[1];
        if (e.master || e.p_fp32) x.p.b = p[1];
        x.cm = reinterpret_cast<const uint2*>(st.cm)[threadIdx.x];
        x.cv = reinterpret_cast<const uint2*>(st.cv)[threadIdx.x];
        x.sm = st.sm[threadIdx.x >> 4];
        x.sr = st.sr[threadIdx.x >> 4];
        update<8, true>(e, a, sc, i, x);
      } else {
        load_elements<8>(e, i, x);
        update<8, false>(e, a, sc, i, x);
      }
    }
    k = kn;
    __syncthreads();  // the stage has been read
  }
  if (!ok && threadIdx.x == 0) {  // let the last copies land before the shared memory goes
    const int last = range.last - 1 - range.first;
    mbar_wait(&s.full[last & 1], (uint32_t)(last >> 1) & 1u, kWaitLimitNs / 16);
  }
}

// early: the grid before this one is the gradient norm's, which starts only when all work before it is done and writes
// its partial sums alone. So the first chunk is read while that grid runs.
template <int BITS, int MAX>
__global__ void __launch_bounds__(kThreads, 4) adamw_kernel(const __grid_constant__ AdamTable<MAX> t, const AdamArgs a,
                                                            dora_adamw_control_t* __restrict__ control,
                                                            const float* __restrict__ grad_scale, int early, int last) {
  pdl_trigger();
  if (!early) pdl_wait();
  const Range range = cta_range(t.chunks);
  const bool any = range.first < range.last;
  const int k0 = any ? find_tensor(t, range.first) : 0;
  const int64_t i0 = any ? (int64_t)(range.first - t.first[k0]) * kChunk + threadIdx.x * 8 : 0;
  __shared__ typename std::conditional<BITS == 8, Stages, int>::type stages;
  if constexpr (BITS == 8) {
    if (threadIdx.x == 0) {
      mbar_init(&stages.full[0], 1);
      mbar_init(&stages.full[1], 1);
      fence_mbar_init();
      if (any) issue_chunk(stages, 0, t.e[k0], t.first[k0], range.first);
    }
    __syncthreads();
  } else if (early && any) {
    prefetch_elements(t.e[k0], i0);
  }
  const int64_t step = control->step + 1;
  StepScalars sc;
  sc.lr = control->lr;
  sc.gs = grad_scale ? *grad_scale : 1.0f;
  if (early) pdl_wait();
  if (a.part) {
    const NormScale r = norm_and_scale(a.part, a.parts, a.max_norm);
    sc.gs = r.scale;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)r.norm;
  }
  const bool run = isfinite(sc.gs);
  if (run && any) {
    const float bc1 = -expm1f((float)step * a.ln_b1), bc2 = -expm1f((float)step * a.ln_b2);
    sc.lr1 = sc.lr / bc1;
    sc.rbc2 = 1.0f / sqrtf(bc2);
    sc.key = mix(a.seed + (uint32_t)step * 0x9E3779B9u);
    if constexpr (BITS == 8) {
      update_range_staged(stages, t, a, sc, range, k0);
    } else {
      for (int c = range.first, k = k0; c < range.last; ++k) {
        const AdamEntry& e = t.e[k];
        const int end = min(range.last, k + 1 < t.n ? t.first[k + 1] : t.chunks);
        int64_t i = (int64_t)(c - t.first[k]) * kChunk + threadIdx.x * 8;
#pragma unroll 1
        for (; c < end; ++c, i += kChunk) {
          Elements<BITS> x;
          load_elements<BITS>(e, i, x);
          update<BITS, false>(e, a, sc, i, x);
        }
      }
    }
  }
  if constexpr (BITS == 8) {
    if (!run && any && threadIdx.x == 0) mbar_wait(&stages.full[0], 0);  // a skipped step's copies have landed
  }
  // The last CTA of the call's last launch counts the step: by then every CTA has read the count.
  if (last) {
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      if (atomicAdd(&control->counter, 1u) == gridDim.x - 1) {
        control->counter = 0;
        if (run) control->step = step;
      }
    }
  }
}

// After the stream is synchronised: the kernels' timeout flags, cleared.
cudaError_t read_and_clear_status(unsigned int* out) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_status, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_device_status, &zero, sizeof(zero));
  }
  *out = v;
  return e;
}
const bool status_added = add_status_reader(read_and_clear_status);

bool is_wide(dora_dtype_t t) { return t == DORA_BF16 || t == DORA_FP32; }
size_t width(dora_dtype_t t) { return t == DORA_FP32 ? 4 : 2; }
bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

std::string nth(const char* what, int i) { return std::string("tensor ") + std::to_string(i) + ": " + what; }

// check_ptr of tensor i; the message is made only for a pointer that is refused.
bool check_nth(const void* p, const char* name, int i, size_t align) {
  return (p && reinterpret_cast<uintptr_t>(p) % align == 0) || check_ptr(p, nth(name, i).c_str(), align);
}

constexpr int64_t kMaxNumel = int64_t(1) << 40;

// One launch over the tensors from i on, as many as the table holds.
template <int MAX, class Grads>
cudaError_t launch_norm(const Grads& grads, int n_tensors, int most, double* part, int& parts, int& i,
                        cudaStream_t st);

// The partial sums of all tensors (grads(i) is the i-th), `parts` of them.
template <class Grads>
cudaError_t norm_partials(const Grads& grads, int n_tensors, double* part, int& parts, cudaStream_t st) {
  const int most = std::min(kNormBlocksMax, device_sm_count() * kNormBlocksPerSM);
  cudaError_t e = cudaSuccess;
  parts = 0;
  for (int i = 0; i < n_tensors && e == cudaSuccess;)
    e = n_tensors <= kFew ? launch_norm<kFew>(grads, n_tensors, most, part, parts, i, st)
                          : launch_norm<kMaxGrads>(grads, n_tensors, most, part, parts, i, st);
  return e;
}

template <int MAX, class Grads>
cudaError_t launch_norm(const Grads& grads, int n_tensors, int most, double* part, int& parts, int& i,
                        cudaStream_t st) {
  GradTable<MAX> t;
  t.n = t.chunks = 0;
  for (; i < n_tensors && t.n < MAX; ++i) {
    const dora_grad_t g = grads(i);
    if (g.numel == 0) continue;
    t.first[t.n] = t.chunks;
    t.e[t.n++] = {g.grad, g.numel, g.dtype == DORA_FP32, aligned16(g.grad)};
    t.chunks += (int)cdiv(g.numel, kChunk);
  }
  if (t.n == 0) return cudaSuccess;
  const int blocks = std::min(t.chunks, most);
  double* to = part + parts;
  parts += blocks;
  ProfRange pr("grad_norm_partial", st);
  return launch_pdl(grad_norm_partial_kernel<MAX>, dim3((unsigned)blocks), dim3(kThreads), 0, st, t, to);
}

template <int BITS, int MAX>
cudaError_t launch_adamw(const AdamArgs& a, const dora_adamw_tensor_t* tensors, int n_tensors, int& i,
                         dora_adamw_control_t* control, const float* grad_scale, cudaStream_t st) {
  const bool early = i == 0 && a.parts > 0;
  AdamTable<MAX> t;
  t.n = t.chunks = 0;
  for (; i < n_tensors && t.n < MAX; ++i) {
    const dora_adamw_tensor_t& x = tensors[i];
    if (x.numel == 0) continue;
    t.first[t.n] = t.chunks;
    const bool p_vec = aligned16(x.param), g_vec = aligned16(x.grad);
    const bool bulk = p_vec && g_vec && aligned16(x.scale_avg) && aligned16(x.scale_sq);
    t.e[t.n++] = {x.param, x.grad, x.exp_avg, x.exp_avg_sq, x.scale_avg, x.scale_sq, x.master, x.numel,
                  (uint32_t)(x.index0 >> 1), x.weight_decay, x.param_dtype == DORA_FP32, x.grad_dtype == DORA_FP32,
                  p_vec, g_vec, bulk};
    t.chunks += (int)cdiv(x.numel, kChunk);
  }
  const int blocks = std::max(1, std::min(t.chunks, device_sm_count() * 4));
  ProfRange pr(BITS == 8 ? "adamw8" : "adamw32", st);
  return launch_pdl(adamw_kernel<BITS, MAX>, dim3((unsigned)blocks), dim3(kThreads), 0, st, t, a, control, grad_scale,
                    early ? 1 : 0, i == n_tensors ? 1 : 0);
}

}  // namespace
}  // namespace dora

using namespace dora;

template <class Grads>
static dora_status_t check_grads(const Grads& grads, int n_tensors, float max_norm, const void* ws, size_t ws_bytes) {
  if (!(max_norm > 0.f)) return set_error("max_norm must be > 0"), DORA_EINVAL;
  int64_t total = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const dora_grad_t g = grads(i);
    if (g.numel < 0 || g.numel > kMaxNumel) return set_error(nth("numel out of range", i)), DORA_EINVAL;
    if (!is_wide(g.dtype)) return set_error(nth("dtype is not DORA_BF16 or DORA_FP32", i)), DORA_EINVAL;
    if (g.numel > 0 && !check_nth(g.grad, "grad", i, width(g.dtype))) return DORA_EINVAL;
    total += cdiv(g.numel, kChunk);
  }
  if (total > INT32_MAX) return set_error("too many elements for one call"), DORA_EINVAL;
  return check_ws_bytes(dora_grad_norm_workspace_size(n_tensors), ws, ws_bytes);
}

// norm: clip by the global norm of the tensors' gradients, written there; else grad_scale (or 1).
static dora_status_t adamw(const dora_adamw_desc_t* desc, const dora_adamw_tensor_t* tensors, int n_tensors,
                           dora_adamw_control_t* control, const float* grad_scale, float max_norm, float* norm, void* ws,
                           size_t ws_bytes, dora_stream_t stream) {
  if (!desc) return set_error("desc is NULL"), DORA_EINVAL;
  if (!(desc->beta1 >= 0.0 && desc->beta1 < 1.0 && desc->beta2 >= 0.0 && desc->beta2 < 1.0))
    return set_error("beta1 and beta2 must be in [0, 1)"), DORA_EINVAL;
  if (!(desc->eps >= 0.f) || !std::isfinite(desc->eps)) return set_error("eps must be finite and >= 0"), DORA_EINVAL;
  if (desc->state_bits != 32 && desc->state_bits != 8) return set_error("state_bits must be 32 or 8"), DORA_EINVAL;
  if (n_tensors < 0 || (n_tensors > 0 && !tensors)) return set_error("tensors is NULL or n_tensors negative"), DORA_EINVAL;
  if (!check_ptr(control, "control", 8) || !check_opt_ptr(grad_scale, "grad_scale", 4)) return DORA_EINVAL;
  const bool eight = desc->state_bits == 8;
  int64_t total = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const dora_adamw_tensor_t& x = tensors[i];
    if (x.numel < 0 || x.numel > kMaxNumel) return set_error(nth("numel out of range", i)), DORA_EINVAL;
    if (!is_wide(x.param_dtype) || !is_wide(x.grad_dtype))
      return set_error(nth("dtype is not DORA_BF16 or DORA_FP32", i)), DORA_EINVAL;
    if (!std::isfinite(x.weight_decay)) return set_error(nth("weight_decay is not finite", i)), DORA_EINVAL;
    if (x.index0 < 0 || x.index0 % 8) return set_error(nth("index0 is not a multiple of 8", i)), DORA_EINVAL;
    total += cdiv(x.numel, kChunk);
    if (x.numel == 0) continue;
    if (!check_nth(x.param, "param", i, width(x.param_dtype)) || !check_nth(x.grad, "grad", i, width(x.grad_dtype)) ||
        !check_nth(x.exp_avg, "exp_avg", i, 16) || !check_nth(x.exp_avg_sq, "exp_avg_sq", i, 16) ||
        (x.master && !check_nth(x.master, "master", i, 16)) ||
        (eight && (!check_nth(x.scale_avg, "scale_avg", i, 4) || !check_nth(x.scale_sq, "scale_sq", i, 4))))
      return DORA_EINVAL;
  }
  if (total > INT32_MAX) return set_error("too many elements for one call"), DORA_EINVAL;
  const auto nth_grad = [=](int i) { return dora_grad_t{tensors[i].grad, tensors[i].numel, tensors[i].grad_dtype}; };
  dora_status_t s;
  if (norm && (s = check_grads(nth_grad, n_tensors, max_norm, ws, ws_bytes)) != DORA_OK) return s;
  if ((s = check_sm100("dora_adamw needs an sm_100 (B200) device")) != DORA_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  double* part = norm ? reinterpret_cast<double*>(ws) : nullptr;
  int parts = 0;
  if (norm) {
    const cudaError_t e = norm_partials(nth_grad, n_tensors, part, parts, st);
    if (e != cudaSuccess) return cuda_status(e, "dora_adamw_clipped");
  }
  const AdamArgs a{(float)desc->beta1,          (float)(1.0 - desc->beta1),   (float)desc->beta2,
                   (float)(1.0 - desc->beta2),  (float)std::log(desc->beta1), (float)std::log(desc->beta2),
                   desc->eps,                   desc->seed,                   part,
                   parts,                       max_norm,                     norm};
  const bool few = n_tensors <= kFew;
  cudaError_t e;
  int i = 0;
  do {
    e = eight ? (few ? launch_adamw<8, kFew>(a, tensors, n_tensors, i, control, grad_scale, st)
                     : launch_adamw<8, kMaxAdam>(a, tensors, n_tensors, i, control, grad_scale, st))
              : (few ? launch_adamw<32, kFew>(a, tensors, n_tensors, i, control, grad_scale, st)
                     : launch_adamw<32, kMaxAdam>(a, tensors, n_tensors, i, control, grad_scale, st));
  } while (i < n_tensors && e == cudaSuccess);
  return cuda_status(e, "dora_adamw");
}

extern "C" {

size_t dora_grad_norm_workspace_size(int n_tensors) {
  if (n_tensors < 0) return 0;
  return (size_t)std::max<int64_t>(1, cdiv(n_tensors, kMaxGrads)) * kNormBlocksMax * sizeof(double);
}

dora_status_t dora_grad_norm(const dora_grad_t* grads, int n_tensors, float max_norm, float* norm, float* scale,
                             void* ws, size_t ws_bytes, dora_stream_t stream) {
  if (!check_ptr(norm, "norm", 4) || !check_ptr(scale, "scale", 4)) return DORA_EINVAL;
  if (n_tensors < 0 || (n_tensors > 0 && !grads)) return set_error("grads is NULL or n_tensors negative"), DORA_EINVAL;
  const auto nth_grad = [=](int i) { return grads[i]; };
  dora_status_t s = check_grads(nth_grad, n_tensors, max_norm, ws, ws_bytes);
  if (s != DORA_OK) return s;
  if ((s = check_sm100("dora_grad_norm needs an sm_100 (B200) device")) != DORA_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  double* part = reinterpret_cast<double*>(ws);
  int parts = 0;
  cudaError_t e = norm_partials(nth_grad, n_tensors, part, parts, st);
  if (e == cudaSuccess) {
    ProfRange pr("grad_norm_final", st);
    e = launch_pdl(grad_norm_final_kernel, dim3(1), dim3(kThreads), 0, st, (const double*)part, parts, max_norm, norm,
                   scale);
  }
  return cuda_status(e, "dora_grad_norm");
}

dora_status_t dora_adamw(const dora_adamw_desc_t* desc, const dora_adamw_tensor_t* tensors, int n_tensors,
                         dora_adamw_control_t* control, const float* grad_scale, dora_stream_t stream) {
  return adamw(desc, tensors, n_tensors, control, grad_scale, 1.f, nullptr, nullptr, 0, stream);
}

dora_status_t dora_adamw_clipped(const dora_adamw_desc_t* desc, const dora_adamw_tensor_t* tensors, int n_tensors,
                                 dora_adamw_control_t* control, float max_norm, float* norm, void* ws, size_t ws_bytes,
                                 dora_stream_t stream) {
  if (!check_ptr(norm, "norm", 4)) return DORA_EINVAL;
  return adamw(desc, tensors, n_tensors, control, nullptr, max_norm, norm, ws, ws_bytes, stream);
}

}  // extern "C"
