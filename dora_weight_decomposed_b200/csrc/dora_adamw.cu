// The update of the trained tensors: the global gradient norm and the AdamW
// step, each over many tensors in one launch (or a few: the table of tensors
// travels in the kernel's parameters, so nothing has to be laid out in device
// memory and every call checks and reads the table it is given).
//
// Both stream their tensors once and are bound by HBM. A work item is a chunk
// of 2048 consecutive elements of one tensor, 8 per thread; a persistent grid
// walks the chunks of all tensors in turn.
#include <algorithm>
#include <cmath>
#include <string>

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
using GradTable = Table<GradEntry, kMaxGrads>;
static_assert(sizeof(GradTable) < 32000, "kernel parameters");

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
  int p_fp32, g_fp32, p_vec, g_vec;
};
constexpr int kMaxAdam = 340;
using AdamTable = Table<AdamEntry, kMaxAdam>;
static_assert(sizeof(AdamTable) < 32600, "kernel parameters");

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

__device__ __forceinline__ void values(const Raw8& r, int fp32, float* v) {
  if (fp32) {
    v[0] = __uint_as_float(r.a.x), v[1] = __uint_as_float(r.a.y), v[2] = __uint_as_float(r.a.z);
    v[3] = __uint_as_float(r.a.w), v[4] = __uint_as_float(r.b.x), v[5] = __uint_as_float(r.b.y);
    v[6] = __uint_as_float(r.b.z), v[7] = __uint_as_float(r.b.w);
  } else {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ void store8(void* base, int fp32, int vec, int64_t i, int64_t n, const float* v) {
  if (vec && i + 8 <= n) {
    if (fp32) {
      float4* p = reinterpret_cast<float4*>((float*)base + i);
      p[0] = make_float4(v[0], v[1], v[2], v[3]);
      p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      __nv_bfloat162 h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      *reinterpret_cast<uint4*>((__nv_bfloat16*)base + i) = *reinterpret_cast<const uint4*>(h);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (i + j >= n) return;
    if (fp32)
      ((float*)base)[i + j] = v[j];
    else
      ((__nv_bfloat16*)base)[i + j] = __float2bfloat16_rn(v[j]);
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

__device__ __forceinline__ void code_values(uint2 u, float* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint16_t two = (uint16_t)((j < 2 ? u.x : u.y) >> (16 * (j & 1)));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
}

__device__ __forceinline__ void store_codes(uint8_t* base, int64_t i, int64_t n, uint2 u) {
  if (i + 8 <= n) {
    *reinterpret_cast<uint2*>(base + i) = u;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) base[i + j] = (uint8_t)((j < 4 ? u.x : u.y) >> (8 * (j & 3)));
  }
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

constexpr int kNormBlocksPerSM = 4;
constexpr int kNormBlocksMax = 1024;

// Sum of squares of this CTA's chunks: 8 values in fp32, everything above in double.
__global__ void __launch_bounds__(kThreads) grad_norm_partial_kernel(const __grid_constant__ GradTable t,
                                                                     double* __restrict__ part) {
  __shared__ double red[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  double sum = 0.0;
  const Range range = cta_range(t.chunks);
  int k = find_tensor(t, range.first);
#pragma unroll 4
  for (int c = range.first; c < range.last; ++c) {
    while (k + 1 < t.n && t.first[k + 1] <= c) ++k;
    const GradEntry& e = t.e[k];
    const int64_t i = (int64_t)(c - t.first[k]) * kChunk + threadIdx.x * 8;
    if (i >= e.n) continue;
    float v[8];
    values(load_raw(e.g, e.fp32, e.vec, i, e.n), e.fp32, v);
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(v[j], v[j], s);
    if (s > 1e-30f && s < 1e38f) {
      sum += (double)s;
    } else {  // squares that fp32 cannot hold (or zeros, or not finite)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += (double)v[j] * (double)v[j];
    }
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

__global__ void __launch_bounds__(kThreads) grad_norm_final_kernel(const double* __restrict__ part, int n, float max_norm,
                                                                   float* __restrict__ norm, float* __restrict__ scale) {
  __shared__ double red[kThreads / 32];
  pdl_trigger();
  pdl_wait();
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) sum += part[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) s += red[w];
    s = sqrt(s);
    *norm = (float)s;
    const double c = (double)max_norm / (s + 1e-6);
    *scale = !isfinite(s) ? __uint_as_float(0x7fffffffu) : (float)(c < 1.0 ? c : 1.0);
  }
}

// ------------------------------------------------------------------ AdamW

struct AdamArgs {
  float b1, omb1, b2, omb2;  // betas and one minus them (rounded from double)
  float ln_b1, ln_b2;
  float eps;
  uint32_t seed;
};

// Integer hash: two rounds of xor-shift and an odd multiplier (the leading
// bits of the fractions of sqrt(2) and sqrt(3), made odd).
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x6A09E667u;
  x = (x ^ (x >> 15)) * 0xBB67AE85u;
  return x ^ (x >> 16);
}

// |y| <= 448 as an e4m3 code: floor(|y| / step + u / 65536), step being the code spacing at |y|. From 2^-6 up the
// spacing is 2^-3 of the binade, so the code is the top bits of the fp32 pattern (exponent offset 120) after u is
// added below them. Under 2^-6 it is 2^-9 throughout, and adding 2^-6 brings the same bits into the same place
// (offset 121). Each of the two is the larger one where it holds.
__device__ __forceinline__ uint32_t stochastic_code(float y, uint32_t u16) {
  const float a = fabsf(y);
  const int t = max(__float_as_int(a) - (120 << 23), __float_as_int(a + 0.015625f) - (121 << 23));
  return (uint32_t)(t + (int)u16) >> 20;  // u16 = 16 u
}

// The scale of a block of 16 lanes x 8 moments (all of the warp's lanes take part); not finite if one of them is not.
__device__ __forceinline__ float moment_scale(const float* v) {
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) asm("max.NaN.f32 %0, %0, %1;" : "+f"(amax) : "f"(fabsf(v[j])));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const float b = __shfl_xor_sync(0xffffffffu, amax, o);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(amax) : "f"(b));
  }
  float s = amax * (1.0f / 448.0f);
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(s) : "f"(1.17549435e-38f));
  return s;
}

// a / b rounded to nearest from the rounded reciprocal of b (Markstein's quotient step).
__device__ __forceinline__ float quotient(float a, float b, float inv_b) {
  const float q = a * inv_b;
  return fmaf(fmaf(-q, b, a), inv_b, q);
}

// What a thread reads of a chunk: its eight elements of everything.
template <int BITS>
struct Elements {
  Raw8 g, p, m, v;  // m, v: 32 bits
  uint2 cm, cv;     // 8 bits
  float sm, sv;
  int k;
  int64_t i;
};

template <int BITS>
__device__ __forceinline__ void fetch(const AdamTable& t, int c, int k, Elements<BITS>& x) {
  while (k + 1 < t.n && t.first[k + 1] <= c) ++k;
  const AdamEntry& e = t.e[k];
  const int64_t i = (int64_t)(c - t.first[k]) * kChunk + threadIdx.x * 8;
  x.k = k;
  x.i = i;
  x.g = load_raw(e.g, e.g_fp32, e.g_vec, i, e.n);
  x.p = e.master ? load_raw(e.master, 1, 1, i, e.n) : load_raw(e.p, e.p_fp32, e.p_vec, i, e.n);
  if (BITS == 32) {
    x.m = load_raw(e.avg, 1, 1, i, e.n);
    x.v = load_raw(e.sq, 1, 1, i, e.n);
  } else {
    x.cm = load_codes((const uint8_t*)e.avg, i, e.n);
    x.cv = load_codes((const uint8_t*)e.sq, i, e.n);
    x.sm = i < e.n ? e.savg[i >> 7] : 0.f;
    x.sv = i < e.n ? e.ssq[i >> 7] : 0.f;
  }
}

template <int BITS>
__device__ __forceinline__ void update(const AdamTable& t, const AdamArgs& a, const Elements<BITS>& x, float gs, float lr,
                                       float lr1, float rbc2, uint32_t key) {
  const AdamEntry& e = t.e[x.k];
  const int64_t i = x.i, n = e.n;
  float g[8], p[8], m[8], v[8], r[8];
  values(x.g, e.g_fp32, g);
  values(x.p, e.master || e.p_fp32, p);
  if (BITS == 32) {
    values(x.m, 1, m);
    values(x.v, 1, v);
  } else {
    code_values(x.cm, m);
    code_values(x.cv, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] *= x.sm;
      v[j] *= x.sv;
      v[j] *= v[j];
    }
  }
  const float keep = 1.0f - lr * e.wd;
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    // Each product and sum rounded by itself: the moments' stored codes then depend on the formula alone.
    const float gj = __fmul_rn(g[j], gs);
    m[j] = __fadd_rn(__fmul_rn(m[j], a.b1), __fmul_rn(gj, a.omb1));
    v[j] = __fadd_rn(__fmul_rn(v[j], a.b2), __fmul_rn(__fmul_rn(gj, gj), a.omb2));
    top = fmaxf(top, v[j]);
  }
  if (top < 1e37f) {
    // sqrt(v) = v rsqrt(v) with one Newton step on the residual v - s^2 (to the last place); zero for v = 0.
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float y;
      asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(fmaxf(v[j], 1e-37f)));
      const float s = v[j] * y;
      r[j] = fmaf(fmaf(-s, s, v[j]), 0.5f * y, s);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = sqrtf(v[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) p[j] = p[j] * keep - __fdividef(m[j] * lr1, fmaf(r[j], rbc2, a.eps));
  if (e.master) store8(e.master, 1, 1, i, n, p);
  store8(e.p, e.p_fp32, e.p_vec, i, n, p);
  if (BITS == 32) {
    store8(e.avg, 1, 1, i, n, m);
    store8(e.sq, 1, 1, i, n, v);
    return;
  }
  const float sm = moment_scale(m), sr = moment_scale(r);
  uint2 cm = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu), cr = cm;  // NaN codes
  if (sm < 1e38f && sr < 1e38f) {
    const float im = 1.0f / sm, ir = 1.0f / sr;
    uint32_t wm[2] = {0, 0}, wr[2] = {0, 0};
    const uint32_t pair0 = e.index0 + (uint32_t)(i >> 1);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const uint32_t h = mix((pair0 + j / 2) ^ key);
      const uint32_t u[2] = {h << 4 & 0xffff0u, h >> 12 & 0xffff0u};
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const float ym = quotient(m[j + d], sm, im), yr = quotient(r[j + d], sr, ir);
        const uint32_t km = stochastic_code(ym, u[d]) | (__float_as_uint(ym) >> 24 & 0x80u);
        const uint32_t kr = max(stochastic_code(yr, u[d]), r[j + d] > 0.f ? 1u : 0u);
        wm[j / 4] |= km << (8 * (j % 4 + d));
        wr[j / 4] |= kr << (8 * (j % 4 + d));
      }
    }
    cm = make_uint2(wm[0], wm[1]);
    cr = make_uint2(wr[0], wr[1]);
  }
  store_codes((uint8_t*)e.avg, i, n, cm);
  store_codes((uint8_t*)e.sq, i, n, cr);
  if ((threadIdx.x & 15) == 0 && i < n) {
    e.savg[i >> 7] = sm;
    e.ssq[i >> 7] = sr;
  }
}

template <int BITS>
__global__ void __launch_bounds__(kThreads, 3) adamw_kernel(const __grid_constant__ AdamTable t, const AdamArgs a,
                                                            dora_adamw_control_t* __restrict__ control,
                                                            const float* __restrict__ grad_scale, int last) {
  pdl_trigger();
  pdl_wait();
  const int64_t step = control->step + 1;
  const float lr = control->lr;
  const float gs = grad_scale ? *grad_scale : 1.0f;
  const bool run = isfinite(gs);
  const Range range = cta_range(t.chunks);
  if (run && range.first < range.last) {
    // The next chunk's loads are under way while this one is computed.
    Elements<BITS> now, next;
    fetch<BITS>(t, range.first, find_tensor(t, range.first), now);
    const float bc1 = -expm1f((float)step * a.ln_b1), bc2 = -expm1f((float)step * a.ln_b2);
    const float lr1 = lr / bc1, rbc2 = 1.0f / sqrtf(bc2);
    const uint32_t key = mix(a.seed + (uint32_t)step * 0x9E3779B9u);
#pragma unroll 1
    for (int c = range.first; c < range.last; ++c) {
      if (c + 1 < range.last) fetch<BITS>(t, c + 1, now.k, next);
      update<BITS>(t, a, now, gs, lr, lr1, rbc2, key);
      now = next;
    }
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

bool is_wide(dora_dtype_t t) { return t == DORA_BF16 || t == DORA_FP32; }
size_t width(dora_dtype_t t) { return t == DORA_FP32 ? 4 : 2; }
bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

std::string nth(const char* what, int i) { return std::string("tensor ") + std::to_string(i) + ": " + what; }

constexpr int64_t kMaxNumel = int64_t(1) << 40;

}  // namespace
}  // namespace dora

using namespace dora;

extern "C" {

size_t dora_grad_norm_workspace_size(int n_tensors) {
  if (n_tensors < 0) return 0;
  return (size_t)std::max<int64_t>(1, cdiv(n_tensors, kMaxGrads)) * kNormBlocksMax * sizeof(double);
}

dora_status_t dora_grad_norm(const dora_grad_t* grads, int n_tensors, float max_norm, float* norm, float* scale,
                             void* ws, size_t ws_bytes, dora_stream_t stream) {
  if (n_tensors < 0 || (n_tensors > 0 && !grads)) return set_error("grads is NULL or n_tensors negative"), DORA_EINVAL;
  if (!(max_norm > 0.f)) return set_error("max_norm must be > 0"), DORA_EINVAL;
  if (!check_ptr(norm, "norm", 4) || !check_ptr(scale, "scale", 4)) return DORA_EINVAL;
  int64_t total = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const dora_grad_t& g = grads[i];
    if (g.numel < 0 || g.numel > kMaxNumel) return set_error(nth("numel out of range", i)), DORA_EINVAL;
    if (!is_wide(g.dtype)) return set_error(nth("dtype is not DORA_BF16 or DORA_FP32", i)), DORA_EINVAL;
    if (g.numel > 0 && !check_ptr(g.grad, nth("grad", i).c_str(), width(g.dtype))) return DORA_EINVAL;
    total += cdiv(g.numel, kChunk);
  }
  if (total > INT32_MAX) return set_error("too many elements for one call"), DORA_EINVAL;
  dora_status_t s = check_ws_bytes(dora_grad_norm_workspace_size(n_tensors), ws, ws_bytes);
  if (s != DORA_OK) return s;
  if ((s = check_sm100("dora_grad_norm needs an sm_100 (B200) device")) != DORA_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  double* part = reinterpret_cast<double*>(ws);
  const int most = std::min(kNormBlocksMax, device_sm_count() * kNormBlocksPerSM);
  int parts = 0;
  cudaError_t e = cudaSuccess;
  GradTable t;
  for (int i = 0; i < n_tensors && e == cudaSuccess;) {
    t.n = t.chunks = 0;
    for (; i < n_tensors && t.n < kMaxGrads; ++i) {
      const dora_grad_t& g = grads[i];
      if (g.numel == 0) continue;
      t.first[t.n] = t.chunks;
      t.e[t.n++] = {g.grad, g.numel, g.dtype == DORA_FP32, aligned16(g.grad)};
      t.chunks += (int)cdiv(g.numel, kChunk);
    }
    if (t.n == 0) break;
    const int blocks = std::min(t.chunks, most);
    {
      ProfRange pr("grad_norm_partial", st);
      e = launch_pdl(grad_norm_partial_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, st, t, part + parts);
    }
    parts += blocks;
  }
  if (e == cudaSuccess) {
    ProfRange pr("grad_norm_final", st);
    e = launch_pdl(grad_norm_final_kernel, dim3(1), dim3(kThreads), 0, st, (const double*)part, parts, max_norm, norm,
                   scale);
  }
  return cuda_status(e, "dora_grad_norm");
}

dora_status_t dora_adamw(const dora_adamw_desc_t* desc, const dora_adamw_tensor_t* tensors, int n_tensors,
                         dora_adamw_control_t* control, const float* grad_scale, dora_stream_t stream) {
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
    if (!check_ptr(x.param, nth("param", i).c_str(), width(x.param_dtype)) ||
        !check_ptr(x.grad, nth("grad", i).c_str(), width(x.grad_dtype)) ||
        !check_ptr(x.exp_avg, nth("exp_avg", i).c_str(), 16) ||
        !check_ptr(x.exp_avg_sq, nth("exp_avg_sq", i).c_str(), 16) ||
        !check_opt_ptr(x.master, nth("master", i).c_str(), 16) ||
        (eight && (!check_ptr(x.scale_avg, nth("scale_avg", i).c_str(), 4) ||
                   !check_ptr(x.scale_sq, nth("scale_sq", i).c_str(), 4))))
      return DORA_EINVAL;
  }
  if (total > INT32_MAX) return set_error("too many elements for one call"), DORA_EINVAL;
  const dora_status_t s = check_sm100("dora_adamw needs an sm_100 (B200) device");
  if (s != DORA_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const AdamArgs a{(float)desc->beta1,          (float)(1.0 - desc->beta1),   (float)desc->beta2,
                   (float)(1.0 - desc->beta2),  (float)std::log(desc->beta1), (float)std::log(desc->beta2),
                   desc->eps,                   desc->seed};
  const int most = device_sm_count() * 3;
  cudaError_t e = cudaSuccess;
  AdamTable t;
  int i = 0;
  do {
    t.n = t.chunks = 0;
    for (; i < n_tensors && t.n < kMaxAdam; ++i) {
      const dora_adamw_tensor_t& x = tensors[i];
      if (x.numel == 0) continue;
      t.first[t.n] = t.chunks;
      t.e[t.n++] = {x.param, x.grad, x.exp_avg, x.exp_avg_sq, x.scale_avg, x.scale_sq, x.master, x.numel,
                    (uint32_t)(x.index0 >> 1), x.weight_decay, x.param_dtype == DORA_FP32, x.grad_dtype == DORA_FP32,
                    aligned16(x.param), aligned16(x.grad)};
      t.chunks += (int)cdiv(x.numel, kChunk);
    }
    const int blocks = std::max(1, std::min(t.chunks, most));
    const int last = i == n_tensors;
    ProfRange pr(eight ? "adamw8" : "adamw32", st);
    e = launch_pdl(eight ? adamw_kernel<8> : adamw_kernel<32>, dim3((unsigned)blocks), dim3(kThreads), 0, st, t, a,
                   control, grad_scale, last);
  } while (i < n_tensors && e == cudaSuccess);
  return cuda_status(e, "dora_adamw");
}

}  // extern "C"
