// Linear layers held in 8-bit floats: block quantisation, and the products
// y = x W^T and dx = dy W with one fp32 scale per block of 128 (the kernels of
// fp8_sm100.cuh).
#include <algorithm>
#include <string>

#include "dora_internal.h"
#include "fp8_sm100.cuh"
#include "host_launch.h"

namespace dora {
namespace {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// ------------------------------------------------------------------ quantisation

// 1 x 128 blocks. It lets the next grid start only once all work before it is done, so that a product which
// follows it may read the weight at once. A warp takes 2 R rows of one column block, 16 lanes of 8 values per block and all R of its loads
// in flight; the CTA's eight warps take neighbouring column blocks. Bound by HBM.
// ws, flag: in front of a product, one more CTA (the last in x) says whether all n_ws scales of the weight are powers
// of two. For a large weight that CTA is the last to end: 512 tokens with the scales of 27648 x 5120 take 20.7 us (10.3
// without), of 16384 x 53248 108 us (21). R: loads per thread; 2 R rows per warp.
template <class T, bool E5M2, int R>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 5 : 3) fp8_quantize_rows_kernel(const T* __restrict__ x, int rows, int cols, int nkb,
                                                                uint8_t* __restrict__ q, float* __restrict__ scale,
                                                                const float* __restrict__ ws, int n_ws, int* flag) {
  pdl_wait();
  pdl_trigger();
  if (flag && blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y > 0) return;
    bool all = true;
#pragma unroll 4
    for (int i = threadIdx.x; i < n_ws; i += 256) all = all && is_power(ws[i]);
    all = __syncthreads_and(all);
    if (threadIdx.x == 0) *flag = all ? 1 : 0;
    return;
  }
  const int kb = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (kb >= nkb) return;
  const int sub = threadIdx.x & 15, h = (threadIdx.x >> 4) & 1;
  const int c = kb * 128 + sub * 8, r0 = blockIdx.x * (2 * R) + h;
  const size_t at = (size_t)r0 * cols + c;
  Raw8<T> raw[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (c < cols && r0 + 2 * i < rows)
      raw[i].load(x + at + (size_t)(2 * i) * cols);
    else
      raw[i].clear();
  }
  float mine = 0.f;  // lane `sub` keeps the scale of its half's row `sub`, so that 2 R rows' scales are stored together
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float amax = raw[i].absmax();
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = absmax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const BlockScale s = block_scale<E5M2>(amax);
    if (sub == i) mine = s.scale;
    float v[8];
    raw[i].values(v);
    if (c < cols && r0 + 2 * i < rows)
      *reinterpret_cast<uint2*>(q + at + (size_t)(2 * i) * cols) = to_fp8x8<E5M2>(v, s.inv);
  }
  if (sub < R && r0 + 2 * sub < rows) scale[(size_t)kb * rows + r0 + 2 * sub] = mine;
}

// 128 x 128 blocks: one CTA each, 16 lanes per row, 8 rows per thread held in registers between the maximum and the
// codes, so that the matrix is read once. Bound by HBM (27648 x 5120 bf16: 74 us, 5.8 TB/s).
template <class T, bool E5M2>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 5 : 3) fp8_quantize_tiles_kernel(const T* __restrict__ x, int rows, int cols, int nkb,
                                                                 uint8_t* __restrict__ q, float* __restrict__ scale) {
  __shared__ float red[8];
  pdl_trigger();
  pdl_wait();
  const int tr = blockIdx.x / nkb, tc = blockIdx.x % nkb;
  const int c = tc * 128 + (threadIdx.x & 15) * 8, r0 = tr * 128 + (threadIdx.x >> 4);
  const size_t at = (size_t)r0 * cols + c;
  Raw8<T> raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (c < cols && r0 + 16 * i < rows)
      raw[i].load(x + at + (size_t)(16 * i) * cols);
    else
      raw[i].clear();
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = absmax_nan(amax, raw[i].absmax());
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = absmax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) amax = absmax_nan(amax, red[w]);
  const BlockScale s = block_scale<E5M2>(amax);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    raw[i].values(v);
    if (c < cols && r0 + 16 * i < rows)
      *reinterpret_cast<uint2*>(q + at + (size_t)(16 * i) * cols) = to_fp8x8<E5M2>(v, s.inv);
  }
  if (threadIdx.x == 0) scale[blockIdx.x] = s.scale;
}

// One flag per CTA: whether its part of x's scales (a non-finite one counts, see is_power_or_bad) and of the weight's
// are powers of two. For a product whose operand comes in codes.
__global__ void __launch_bounds__(256) fp8_check_scales_kernel(const float* __restrict__ xs, long long n_xs,
                                                               const float* __restrict__ ws, int n_ws, int* flags) {
  pdl_wait();
  pdl_trigger();
  bool all = true;
  const long long step = (long long)gridDim.x * 256;
#pragma unroll 4
  for (long long i = blockIdx.x * 256 + threadIdx.x; i < n_xs; i += step) all = all && is_power_or_bad(xs[i]);
#pragma unroll 4
  for (long long i = blockIdx.x * 256 + threadIdx.x; i < n_ws; i += step) all = all && is_power(ws[i]);
  all = __syncthreads_and(all);
  if (threadIdx.x == 0) flags[blockIdx.x] = all ? 1 : 0;
}

// The weight's scales that a product wants looked at on the way (none for the quantiser alone).
struct WeightCheck {
  const float* ws = nullptr;
  int n = 0;
  int* flag = nullptr;
};

template <class T, bool E5M2>
cudaError_t quantize_t(int64_t rows, int64_t cols, bool tiles, const void* x, void* q, float* scale, const WeightCheck& wc,
                       cudaStream_t st) {
  const int nkb = (int)cdiv(cols, 128);
  ProfRange pr(tiles ? "fp8_quantize_tiles" : "fp8_quantize_rows", st);
  if (tiles)
    return launch_pdl(fp8_quantize_tiles_kernel<T, E5M2>, dim3((unsigned)(cdiv(rows, 128) * nkb)), dim3(256), 0, st,
                      (const T*)x, (int)rows, (int)cols, nkb, (uint8_t*)q, scale);
  // Eight loads per thread while that makes a CTA for every SM (4096 x 8192: 18.7 us, 31 us with one load), else one:
  // small operands are bound by the length of a thread's work.
  const bool few = cdiv(rows, 16) * cdiv(nkb, 8) < device_sm_count();
  const int64_t groups = cdiv(rows, few ? 2 : 16) + (wc.flag ? 1 : 0);
  return launch_pdl(few ? fp8_quantize_rows_kernel<T, E5M2, 1> : fp8_quantize_rows_kernel<T, E5M2, 8>,
                    dim3((unsigned)groups, (unsigned)cdiv(nkb, 8)), dim3(256), 0, st, (const T*)x, (int)rows, (int)cols, nkb,
                    (uint8_t*)q, scale, wc.ws, wc.n, wc.flag);
}

cudaError_t quantize(int64_t rows, int64_t cols, dora_dtype_t in, dora_dtype_t fp8, bool tiles, const void* x, void* q,
                     float* scale, const WeightCheck& wc, cudaStream_t st) {
  if (in == DORA_BF16)
    return fp8 == DORA_E5M2 ? quantize_t<__nv_bfloat16, true>(rows, cols, tiles, x, q, scale, wc, st)
                            : quantize_t<__nv_bfloat16, false>(rows, cols, tiles, x, q, scale, wc, st);
  return fp8 == DORA_E5M2 ? quantize_t<float, true>(rows, cols, tiles, x, q, scale, wc, st)
                          : quantize_t<float, false>(rows, cols, tiles, x, q, scale, wc, st);
}

// ------------------------------------------------------------------ products

// Row-major matrix [rows x cols] of elements of `size` bytes in boxes of box_rows x 128 bytes, 128-byte swizzle, zeros
// out of bounds.
cudaError_t make_map_2d(CUtensorMap* map, const void* ptr, int64_t rows, int64_t cols, int size, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)cols * size};
  cuuint32_t box[2] = {128u / size, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1u, 1u};
  const CUtensorMapDataType type = size == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : size == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  const CUresult r = enc(map, type, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The current device, for what is asked once per device (63: none, or any behind it), and its SMs.
int this_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 63;
  }
  return std::min(dev, 63);
}
int sm_count(int dev) {
  static std::atomic<int> known[64];
  int n = known[dev].load();
  if (n == 0) known[dev].store(n = device_sm_count());
  return n;
}

template <int NT, bool W_MN, class XT>
cudaError_t narrow_smem() {
  static std::atomic<unsigned long long> set{0};
  return set_smem_once(set, fp8_narrow_kernel<NT, W_MN, XT>, Fp8Narrow<NT>::SMEM_BYTES);
}

// Clusters of cs CTAs, one CTA per SM, that the current device holds at once (a cluster has to fit in one GPC): the
// answer of the occupancy query, which counts one CTA per SM for the narrow kernels. The query knows the kernel by its
// shared-memory limit, so that is raised first (before, it says 0). 0: no answer.
template <int NT, bool W_MN>
int clusters_alone(int cs, int sms) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cs * 1024u);
  cfg.blockDim = dim3(kF8Threads);
  cfg.dynamicSmemBytes = Fp8Narrow<NT>::SMEM_BYTES;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (narrow_smem<NT, W_MN, void>() != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, fp8_narrow_kernel<NT, W_MN, void>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return std::min(n, std::max(1, sms / cs));
}

// The same with the two CTAs per SM that run there (shared memory, registers and TMEM leave room for two): twice as
// many. Seen in the times: 48 tiles in one wave with 5 splits and in two with 6, 96 tiles with 2 and 3. The small CTAs of
// 16 tokens also fit as one cluster on every (cs + 1) / 2 SMs: 32 tiles with 8 splits in one wave, which at 128 tokens
// (256 x 2048 x 2048) took 12.2 us, and 9.5 with 6. Asked for once per device; where there is no answer (no device),
// 7/8 of the SMs are assumed, for that call alone.
struct NarrowSlots {
  bool known = false;
  int n[9] = {};
};
template <int NT, bool W_MN>
NarrowSlots narrow_slots(int dev) {
  static std::mutex mu;
  static NarrowSlots of[64];
  std::lock_guard<std::mutex> lk(mu);
  if (of[dev].known) return of[dev];
  const int sms = sm_count(dev);
  NarrowSlots s;
  s.known = true;
  int alone[9];
  for (int cs = 1; cs <= 8; ++cs) {
    alone[cs] = clusters_alone<NT, W_MN>(cs, sms);
    if (alone[cs] < 1) {
      s.known = false;
      alone[cs] = std::max(1, sms / cs * 7 / 8);
    }
  }
  for (int cs = 1; cs <= 8; ++cs) s.n[cs] = std::max(2 * alone[cs], NT == 16 ? alone[(cs + 1) / 2] : 0);
  if (s.known) of[dev] = s;
  return s;
}

// CTAs per tile of the narrow kernel (K splits, one cluster) and the call's estimated time in microseconds: waves of
// clusters, in each 0.43 us per k-block where a CTA has its SM and 0.6 where two share it, which is what the operands'
// way in allows, 1 us to fill and, with splits, 2 us and 2 more at 128 tokens to add them; and 4 for the launch and the
// store. Measured around the chosen count: T = 1 of 4096 x 4096 7.2 us with 8 splits, 7.8 with 7; T = 37 of
// 27648 x 5120 27.8 with 1, 33.6 with 2; its backward call, 40 tiles of 216 k-blocks, 28.9 with 5, 28.7 with 6 and 42
// with 7 (two waves); T = 100 of 8192 x 8192 21.4 with 3, 20.6 with 4 and 28.9 with 5.
struct NarrowChoice {
  int cs = 1;
  double us = 1e300;
};
template <int NT, bool W_MN>
NarrowChoice narrow_choice(int dev, int64_t tiles, int64_t nkb, int64_t least = 1) {
  NarrowChoice best;
  const int sms = sm_count(dev);
  const NarrowSlots slots = narrow_slots<NT, W_MN>(dev);
  for (int cs = (int)least; cs <= 8 && cs <= nkb; ++cs) {
    const double block = tiles * cs > sms ? 0.6 : 0.43, add = cs > 1 ? 2.0 + NT / 64.0 : 0.0;
    const int64_t waves = cdiv(tiles, slots.n[cs]);
    const double us = (double)waves * ((double)cdiv(nkb, cs) * block + add + 1.0) + 4.0;
    if (us < best.us - 1e-9) {
      best.us = us;
      best.cs = cs;
    }
  }
  return best;
}

// The least number of splits that leaves a CTA no more k-blocks than the ring's stages, so that the kernel can quantise x
// itself, or 0 where the device's 2 CTAs per SM do not allow as many. Not by what clusters fit: those differ from one
// device to the next, and a workspace asked for on one of them has to do on another.
int64_t few_blocks_splits(int dev, int64_t T, int64_t N, int64_t nkb) {
  const int64_t most = std::clamp<int64_t>(2 * sm_count(dev) / cdiv(N, 128), 1, 8), least = cdiv(nkb, Fp8Narrow<16>::STAGES);
  return T <= 16 && least <= most ? least : 0;
}

// The pair kernel's time: waves of 256 x 256 tiles, 0.44 us per k-block, up to 0.56 with every pair busy, plus 6.
double pair_us(int dev, int64_t T, int64_t N, int64_t nkb) {
  const int64_t pairs = std::max(1, sm_count(dev) / 2), tiles = cdiv(T, 256) * cdiv(N, 256);
  return (double)cdiv(tiles, pairs) * (double)nkb * (0.44 + 0.12 * (double)std::min(tiles, pairs) / (double)pairs) + 6.0;
}

template <int NT, bool W_MN, class XT>
cudaError_t launch_narrow(const CUtensorMap& tw, const CUtensorMap& tx, const Fp8Geom& g, bool early_w, cudaStream_t st) {
  const cudaError_t e = narrow_smem<NT, W_MN, XT>();
  if (e != cudaSuccess) return e;
  const int64_t tiles = cdiv(g.N, 128), t_tiles = cdiv(g.T, NT);
  // (The same splits for an x that comes in codes as for one that is quantised here: the same sums.)
  const int dev = this_device();
  const int cs = narrow_choice<NT, W_MN>(dev, tiles * t_tiles, g.nkb, std::max<int64_t>(1, few_blocks_splits(dev, g.T, g.N, g.nkb))).cs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * t_tiles * cs));
  cfg.blockDim = dim3(kF8Threads);
  cfg.dynamicSmemBytes = Fp8Narrow<NT>::SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = profiling_on() ? 0 : 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cs;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  ProfRange pr(W_MN ? "fp8_backward" : "fp8_forward", st);
  return cudaLaunchKernelEx(&cfg, fp8_narrow_kernel<NT, W_MN, XT>, tw, tx, g, cs, early_w ? 1 : 0);
}

template <bool W_MN>
cudaError_t launch_narrow_nt(int nt, const CUtensorMap& tw, const CUtensorMap& tx, const Fp8Geom& g, bool early_w,
                             cudaStream_t st) {
  switch (nt) {
    case 16: return launch_narrow<16, W_MN, void>(tw, tx, g, early_w, st);
    case 32: return launch_narrow<32, W_MN, void>(tw, tx, g, early_w, st);
    case 64: return launch_narrow<64, W_MN, void>(tw, tx, g, early_w, st);
    default: return launch_narrow<128, W_MN, void>(tw, tx, g, early_w, st);
  }
}

template <bool B_MN>
cudaError_t launch_pairs(const CUtensorMap& ta, const CUtensorMap& tb, const Fp8Geom& g, cudaStream_t st) {
  CUtensorMap tout;
  cudaError_t e = make_map_2d(&tout, g.out, g.T, g.N, g.out_fp32 ? 4 : 2, 32);
  if (e != cudaSuccess) return e;
  auto kern = fp8_pair_kernel<B_MN>;
  static std::atomic<unsigned long long> smem_set{0};
  e = set_smem_once(smem_set, kern, kF8PairSmem);
  if (e != cudaSuccess) return e;
  // The register moves in the kernel count on this many registers per thread at launch.
  static const int regs = [&] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, kern) == cudaSuccess ? a.numRegs : 0;
  }();
  if (regs < kF8LaunchRegs) return cudaErrorInvalidKernelImage;
  const int64_t pairs = std::min<int64_t>(cdiv(g.T, 256) * cdiv(g.N, 256), std::max(1, sm_count(this_device()) / 2));
  ProfRange pr(B_MN ? "fp8_backward_pairs" : "fp8_forward_pairs", st);
  return launch_pdl(kern, dim3((unsigned)(2 * pairs)), dim3(kF8PairThreads), kF8PairSmem, st, ta, tb, tout, g);
}

// What a call keeps in its workspace (the quantised operand and its scales), unless the kernel quantises it itself.
struct Fp8Plan {
  bool own_x = false, narrow = true, flags = false;
  size_t off_q = 0, off_s = 0, off_flags = 0, total = 0;
};

bool is_fp8(dora_dtype_t t) { return t == DORA_E4M3 || t == DORA_E5M2; }
bool is_wide(dora_dtype_t t) { return t == DORA_BF16 || t == DORA_FP32; }

Fp8Plan fp8_plan(const dora_fp8_desc_t& d, int64_t T, int op) {
  Fp8Plan p;
  const bool back = op == DORA_FP8_OP_BACKWARD;
  const int64_t K = back ? d.d_out : d.d_in, N = back ? d.d_in : d.d_out, nkb = cdiv(K, 128);
  if (T == 0) return p;
  const int dev = this_device();
  // Tiles of up to 128 tokens with K split over clusters, or 256 x 256 tiles on CTA pairs: the latter need many
  // tiles (T = 512: 1024 x 8192 20 us narrow and 34 us on pairs, 4096 x 4096 18.4 and 21.1, 8192 x 8192 43.3 and 42.1,
  // 6144 x 2048 15.9 and 15.0). Where both need two waves the estimates are too near to tell: T = 256 of 27648 x 5120 is
  // given to pairs (50.8 us against 54 estimated), which took 58 us, and 51 narrow.
  if (T > 128) {
    const int64_t tiles = cdiv(N, 128) * cdiv(T, 128);
    const double us = back ? narrow_choice<128, true>(dev, tiles, nkb).us : narrow_choice<128, false>(dev, tiles, nkb).us;
    p.narrow = us < pair_us(dev, T, N, nkb);
  }
  p.flags = !p.narrow && (d.out_dtype == DORA_BF16 || nkb <= kF8MaxBlocksFp32);
  if (T > 128) p.total = kF8MaxFlags * sizeof(int);  // the choice may differ between devices, the workspace may not
  if (is_fp8(d.in_dtype)) return p;
  p.own_x = few_blocks_splits(dev, T, N, nkb) > 0;
  if (p.own_x) return p;
  p.off_q = p.total;
  p.off_s = p.off_q + align256((size_t)T * K);
  p.total = p.off_s + align256((size_t)T * nkb * 4);
  return p;
}

bool check_fp8_desc(const dora_fp8_desc_t* d) {
  if (!d) return set_error("desc is NULL"), false;
  if (d->d_out < 1 || d->d_in < 1) return set_error("d_out and d_in must be >= 1"), false;
  if (d->d_out > kMaxDim || d->d_in > kMaxDim) return set_error("d_out or d_in too large"), false;
  if (cdiv(d->d_out, 128) * cdiv(d->d_in, 128) > INT32_MAX) return set_error("weight too large"), false;
  if (d->d_out % 16 || d->d_in % 16) return set_error("8-bit layers need d_out and d_in to be multiples of 16"), false;
  if (!is_fp8(d->in_dtype) && !is_wide(d->in_dtype)) return set_error("desc->in_dtype is not a dora_dtype_t"), false;
  if (!is_fp8(d->in_dtype) && !is_fp8(d->fp8_dtype))
    return set_error("desc->fp8_dtype is not DORA_E4M3 or DORA_E5M2"), false;
  if (!is_wide(d->out_dtype)) return set_error("desc->out_dtype is not DORA_BF16 or DORA_FP32"), false;
  return true;
}

dora_status_t product(bool backward, const dora_fp8_desc_t* desc, int64_t T, const void* x, const float* x_scale,
                      const void* W, const float* w_scale, void* out, void* ws, size_t ws_bytes, cudaStream_t st) {
  if (!check_fp8_desc(desc) || !check_T(T)) return DORA_EINVAL;
  const bool given = is_fp8(desc->in_dtype);
  if (!check_ptr(W, "W", 16) || !check_ptr(w_scale, "w_scale", 4)) return DORA_EINVAL;
  if (given ? (T > 0 && !check_ptr(x_scale, backward ? "dy_scale" : "x_scale", 4)) : x_scale != nullptr) {
    if (!given) set_error(backward ? "dy_scale must be NULL for a bf16 or fp32 dy" : "x_scale must be NULL for a bf16 or fp32 x");
    return DORA_EINVAL;
  }
  if (T > 0 && (!check_ptr(x, backward ? "dy" : "x", 16) || !check_ptr(out, backward ? "dx" : "y", 16)))
    return DORA_EINVAL;
  const int op = backward ? DORA_FP8_OP_BACKWARD : DORA_FP8_OP_FORWARD;
  const Fp8Plan p = fp8_plan(*desc, T, op);
  dora_status_t s = check_ws_bytes(p.total, ws, ws_bytes);
  if (s != DORA_OK) return s;
  if ((s = check_sm100("the 8-bit products need an sm_100 (B200) device")) != DORA_OK) return s;
  if (T == 0) return DORA_OK;
  const char* where = backward ? "dora_fp8_backward" : "dora_fp8_forward";
  const int64_t K = backward ? desc->d_out : desc->d_in, N = backward ? desc->d_in : desc->d_out;
  const dora_dtype_t type = given ? desc->in_dtype : desc->fp8_dtype;
  const void* xq = x;
  const int n_ws = (int)(cdiv(desc->d_out, 128) * cdiv(desc->d_in, 128));
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  int* flags = p.flags ? reinterpret_cast<int*>(w + p.off_flags) : nullptr;
  int n_flags = 1;
  if (!given && !p.own_x) {
    const cudaError_t e = quantize(T, K, desc->in_dtype, type, false, x, w + p.off_q, reinterpret_cast<float*>(w + p.off_s),
                                   WeightCheck{w_scale, n_ws, flags}, st);
    if (e != cudaSuccess) return cuda_status(e, where);
    xq = w + p.off_q;
    x_scale = reinterpret_cast<const float*>(w + p.off_s);
  } else if (flags) {
    const long long n_xs = (long long)T * cdiv(K, 128);
    n_flags = (int)std::min<long long>(kF8MaxFlags, cdiv(n_xs, 1024));
    ProfRange pr("fp8_check_scales", st);
    const cudaError_t e = launch_pdl(fp8_check_scales_kernel, dim3((unsigned)n_flags), dim3(256), 0, st, x_scale, n_xs, w_scale,
                                     n_ws, flags);
    if (e != cudaSuccess) return cuda_status(e, where);
  }
  const int nkw = (int)cdiv(desc->d_in, 128);  // columns of w_scale
  Fp8Geom g{x, (int)K, x_scale, w_scale, out, (int)T, (int)N, (int)cdiv(K, 128), backward ? 1 : nkw, backward ? nkw : 1,
            desc->out_dtype == DORA_FP32, type == DORA_E5M2, flags, flags ? n_flags : 0, given};
  CUtensorMap tx, tw;
  cudaError_t e = make_map_2d(&tw, W, desc->d_out, desc->d_in, 1, 128);
  if (e != cudaSuccess) return cuda_status(e, where);
  if (p.own_x) {
    if (desc->in_dtype == DORA_BF16)
      e = backward ? launch_narrow<16, true, __nv_bfloat16>(tw, tw, g, false, st)
                   : launch_narrow<16, false, __nv_bfloat16>(tw, tw, g, false, st);
    else
      e = backward ? launch_narrow<16, true, float>(tw, tw, g, false, st)
                   : launch_narrow<16, false, float>(tw, tw, g, false, st);
    return cuda_status(e, where);
  }
  const int nt = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128;
  const bool narrow = p.narrow;
  e = make_map_2d(&tx, xq, T, K, 1, narrow ? nt : 128);
  if (e == cudaSuccess) {
    if (narrow)
      e = backward ? launch_narrow_nt<true>(nt, tw, tx, g, !given, st) : launch_narrow_nt<false>(nt, tw, tx, g, !given, st);
    else
      e = backward ? launch_pairs<true>(tx, tw, g, st) : launch_pairs<false>(tx, tw, g, st);
  }
  return cuda_status(e, where);
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

}  // namespace
}  // namespace dora

using namespace dora;

extern "C" {

dora_status_t dora_fp8_quantize(int64_t rows, int64_t cols, dora_dtype_t in_dtype, dora_dtype_t fp8_dtype,
                                dora_fp8_block_t block, const void* x, void* q, float* scale, dora_stream_t stream) {
  if (rows < 0 || cols < 1 || rows > kMaxDim || cols > kMaxDim) return set_error("rows or cols out of range"), DORA_EINVAL;
  if (cols % 16) return set_error("cols must be a multiple of 16"), DORA_EINVAL;
  if (!is_wide(in_dtype)) return set_error("in_dtype is not DORA_BF16 or DORA_FP32"), DORA_EINVAL;
  if (!is_fp8(fp8_dtype)) return set_error("fp8_dtype is not DORA_E4M3 or DORA_E5M2"), DORA_EINVAL;
  if (block != DORA_FP8_ROWS && block != DORA_FP8_TILES) return set_error("block is not a dora_fp8_block_t"), DORA_EINVAL;
  if (cdiv(rows, 128) * cdiv(cols, 128) > INT32_MAX) return set_error("matrix too large"), DORA_EINVAL;
  if (rows == 0) return DORA_OK;
  if (!check_ptr(x, "x", 16) || !check_ptr(q, "q", 16) || !check_ptr(scale, "scale", 4)) return DORA_EINVAL;
  const dora_status_t s = check_sm100("the 8-bit calls need an sm_100 (B200) device");
  if (s != DORA_OK) return s;
  return cuda_status(quantize(rows, cols, in_dtype, fp8_dtype, block == DORA_FP8_TILES, x, q, scale, WeightCheck{},
                              reinterpret_cast<cudaStream_t>(stream)),
                     "dora_fp8_quantize");
}

size_t dora_fp8_workspace_size(const dora_fp8_desc_t* desc, int64_t T, int op) {
  if (!check_fp8_desc(desc) || !check_T(T) || op < DORA_FP8_OP_FORWARD || op > DORA_FP8_OP_BACKWARD) return 0;
  return fp8_plan(*desc, T, op).total;
}

dora_status_t dora_fp8_forward(const dora_fp8_desc_t* desc, int64_t T, const void* x, const float* x_scale,
                               const void* W, const float* w_scale, void* y, void* ws, size_t ws_bytes,
                               dora_stream_t stream) {
  return product(false, desc, T, x, x_scale, W, w_scale, y, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

dora_status_t dora_fp8_backward(const dora_fp8_desc_t* desc, int64_t T, const void* dy, const float* dy_scale,
                                const void* W, const float* w_scale, void* dx, void* ws, size_t ws_bytes,
                                dora_stream_t stream) {
  return product(true, desc, T, dy, dy_scale, W, w_scale, dx, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
