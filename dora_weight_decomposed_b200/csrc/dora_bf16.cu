// bf16 path of the DoRA layer: tcgen05/TMA GEMMs with the DoRA arithmetic in
// their epilogues, plus bandwidth-bound SIMT kernels for the compose backward
// and the small reductions.
//
//   dora_norm     Gram G = A A^T (split-K partials -> (s/2) G as bf16 hi + lo), then
//                 one GEMM on CTA pairs  acc = [W0 | B | B] [A | Gs_hi | Gs_lo]^T  whose
//                 epilogue forms sum_k W0_ik^2 (read from the W0 tiles in shared
//                 memory once the MMAs consumed them) + 2 s B_i . acc_i  per row and
//                 K split; the last split of each row block sums the splits and
//                 takes C, g, g - 1.
//                 2 s B_i . acc_i = 2 s B_i (W0 A^T)_i + s^2 B_i G B_i^T: the cross
//                 and Gram terms of the factored norm (Scaling DoRA abstract).
//   dora_forward  su = s x A^T, then  pre = [x | su] [W0 | B]^T  with the
//                 compose y = pre + gm1 * pre  in the epilogue (one rounding).
//   dora_backward dz = g * dy and the dm column sums in one streaming pass;
//                 du = s dz B, dB = dz^T su, dA = du^T x, dx = [dz | du] [W0 ; A].
//   dora_backward_full  the above, then the eq. (A.1) corrections of dB and dA.
//   dora_merge    W' = diag(g) (W0 + s B A) (merge_sm100.cuh).
#include <algorithm>
#include <atomic>
#include <mutex>
#include <string>
#include <utility>

#include "dora_internal.h"
#include "host_launch.h"
#include "gemm_sm100.cuh"
#include "gram_sm100.cuh"
#include "grouped_sm100.cuh"
#include "merge_sm100.cuh"

namespace dora {

static inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ============================================================== tensor maps

// Row-major bf16 matrix [rows x cols], leading dimension ld elements.
struct Mat {
  const void* ptr = nullptr;
  int64_t rows = 0, cols = 0, ld = 0;
};

// Tiles of box_outer rows x 64 columns, 128-byte swizzle, zeros out of bounds.
static thread_local std::string t_detail;

static bool make_map(CUtensorMap* map, const Mat& m, int box_outer, const char* what) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) {
    t_detail = "cuTensorMapEncodeTiled unavailable";
    return false;
  }
  if (m.rows <= 0 || m.cols <= 0) {
    t_detail = std::string(what) + ": empty matrix";
    return false;
  }
  cuuint64_t dims[2] = {(cuuint64_t)m.cols, (cuuint64_t)m.rows};
  cuuint64_t strides[1] = {(cuuint64_t)m.ld * 2};
  cuuint32_t box[2] = {64u, (cuuint32_t)box_outer};
  cuuint32_t estr[2] = {1u, 1u};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(m.ptr), dims, strides, box,
                         estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    t_detail = std::string(what) + ": tensor map encode failed (CUresult " + std::to_string((int)r) + ", " +
               std::to_string(m.rows) + "x" + std::to_string(m.cols) + " ld " + std::to_string(m.ld) + " box " +
               std::to_string(box_outer) + ")";
    return false;
  }
  return true;
}

static dora_status_t gemm_status(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return DORA_OK;
  set_error(std::string(where) + ": " + cudaGetErrorString(e) + (t_detail.empty() ? "" : " [" + t_detail + "]"));
  return DORA_ECUDA;
}

// fp32 [d2][d1][d0] array (d0 contiguous) for tiled 3-D stores of box {b0, b1, 1}, 128-byte swizzle.
static bool make_map_f32_3d(CUtensorMap* map, void* base, int64_t d0, int64_t d1, int64_t d2, int b0, int b1) {
  EncodeTiledFn enc = encode_fn();
  if (!enc || d0 <= 0 || d1 <= 0 || d2 <= 0) {
    t_detail = "fp32 store map: bad extent or no encoder";
    return false;
  }
  cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
  cuuint64_t strides[2] = {(cuuint64_t)d0 * 4, (cuuint64_t)(d0 * d1) * 4};
  cuuint32_t box[3] = {(cuuint32_t)b0, (cuuint32_t)b1, 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    t_detail = "fp32 store map encode failed (CUresult " + std::to_string((int)r) + ")";
    return false;
  }
  return true;
}

// ============================================================== GEMM launch

struct GemmArgs {
  Mat a0, a1, b0, b1;  // K-source 0 and (if K1 > 0) 1 of each operand
  int64_t K0 = 0, K1 = 0;
  int M = 0, N = 0;
  Split split;
  int a1_kwrap = 0;  // see GemmGeom::a1_kwrap
  int defer_wait_src1 = 0;  // see GemmGeom::defer_wait_src1 (CTA-pair kernels)
  int wait_then_trigger = 0;  // see GemmGeom::wait_then_trigger
  const char* name = "gemm";
};

template <class Cfg, class Epi>
static cudaError_t launch_gemm(const GemmArgs& g, const typename Epi::Params& ep, cudaStream_t st) {
  CUtensorMap ta0, ta1, tb0, tb1;
  const int a_box = Cfg::A_MN ? 64 : kBM;
  const int b_box = Cfg::B_MN ? 64 : Cfg::B_BOX;
  t_detail.clear();
  if (!make_map(&ta0, g.a0, a_box, "A source 0") || !make_map(&tb0, g.b0, b_box, "B source 0"))
    return cudaErrorInvalidValue;
  const int kb0 = (int)ceil_div(g.K0, kBK);
  const int kb1 = g.K1 > 0 ? (int)ceil_div(g.K1, kBK) : 0;
  if (kb1 > 0) {
    if (!make_map(&ta1, g.a1, a_box, "A source 1") || !make_map(&tb1, g.b1, b_box, "B source 1"))
      return cudaErrorInvalidValue;
  } else {
    ta1 = ta0;
    tb1 = tb0;
  }
  GemmGeom geom{g.M, g.N, kb0, kb1, g.split.kb_per_split, g.a1_kwrap};
  dim3 grid((unsigned)ceil_div(g.N, Cfg::BN), (unsigned)ceil_div(g.M, kBM), (unsigned)g.split.splits);
  auto kern = gemm_sm100_kernel<Cfg, Epi>;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t e = set_smem_once(smem_set, kern, Cfg::SMEM_BYTES);
  if (e != cudaSuccess) {
    t_detail = "shared-memory attribute (" + std::to_string(Cfg::SMEM_BYTES) + " bytes)";
    return e;
  }
  {
    ProfRange pr(g.name, st);
    e = launch_pdl(kern, grid, dim3(kGemmThreads), Cfg::SMEM_BYTES, st, ta0, ta1, tb0, tb1, geom, ep);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess)
    t_detail = "launch grid (" + std::to_string(grid.x) + "," + std::to_string(grid.y) + "," +
               std::to_string(grid.z) + ") smem " + std::to_string(Cfg::SMEM_BYTES);
  return e;
}

// Persistent launch: one CTA per SM (at most one per tile), no K split.
// CTA-pair persistent launch: clusters of two CTAs, one pair per two SMs.
template <class Cfg, class Epi>
static cudaError_t launch_gemm_pair(const GemmArgs& g, const typename Epi::Params& ep, int sms, cudaStream_t st) {
  CUtensorMap ta0, ta1, tb0, tb1;
  const int a_box = Cfg::A_MN ? 64 : kBM;
  const int b_box = Cfg::B_MN ? 64 : Cfg::B_BOX;
  t_detail.clear();
  if (!make_map(&ta0, g.a0, a_box, "A source 0") || !make_map(&tb0, g.b0, b_box, "B source 0"))
    return cudaErrorInvalidValue;
  const int kb0 = (int)ceil_div(g.K0, kBK);
  const int kb1 = g.K1 > 0 ? (int)ceil_div(g.K1, kBK) : 0;
  if (kb1 > 0) {
    if (!make_map(&ta1, g.a1, a_box, "A source 1") || !make_map(&tb1, g.b1, b_box, "B source 1"))
      return cudaErrorInvalidValue;
  } else {
    ta1 = ta0;
    tb1 = tb0;
  }
  const int kps = g.split.kb_per_split > 0 ? g.split.kb_per_split : kb0 + kb1;
  GemmGeom geom{g.M, g.N, kb0, kb1, kps, g.a1_kwrap, g.defer_wait_src1, g.wait_then_trigger};
  const long long splits = ceil_div(std::max(kb0 + kb1, 1), kps);
  const long long items = ceil_div(g.N, Cfg::BN) * ceil_div(g.M, 2 * kBM) * splits;
  const long long pairs = std::max<long long>(1, std::min<long long>(items, sms / 2));
  auto kern = gemm_sm100_pair_kernel<Cfg, Epi>;
  constexpr int smem_bytes = PairLayout<Cfg, Epi>::SMEM_BYTES;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t e = set_smem_once(smem_set, kern, smem_bytes);
  if (e != cudaSuccess) {
    t_detail = "shared-memory attribute (" + std::to_string(smem_bytes) + " bytes)";
    return e;
  }
  {
    ProfRange pr(g.name, st);
    e = launch_pdl(kern, dim3((unsigned)(2 * pairs)), dim3(kGemmThreads), smem_bytes, st, ta0, ta1, tb0, tb1,
                   geom, ep);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) t_detail = "pair launch, " + std::to_string(pairs) + " clusters of 2";
  return e;
}

template <bool A_MN, bool B_MN, class Epi>
static cudaError_t gemm_bn(int bn, const GemmArgs& g, const typename Epi::Params& ep, cudaStream_t st) {
  if constexpr (!B_MN) {
    if (bn == 16) return launch_gemm<GemmCfg<16, A_MN, B_MN>, Epi>(g, ep, st);
    if (bn == 32) return launch_gemm<GemmCfg<32, A_MN, B_MN>, Epi>(g, ep, st);
  }
  if (bn == 64) return launch_gemm<GemmCfg<64, A_MN, B_MN>, Epi>(g, ep, st);
  if (bn == 128) return launch_gemm<GemmCfg<128, A_MN, B_MN>, Epi>(g, ep, st);
  if (bn == 192) return launch_gemm<GemmCfg<192, A_MN, B_MN>, Epi>(g, ep, st);
  if (bn == 256) return launch_gemm<GemmCfg<256, A_MN, B_MN>, Epi>(g, ep, st);
  if (bn == 384) return launch_gemm<GemmCfg<384, A_MN, B_MN>, Epi>(g, ep, st);
  if (bn == 512) return launch_gemm<GemmCfg<512, A_MN, B_MN>, Epi>(g, ep, st);
  return cudaErrorInvalidValue;
}

// ============================================================== DoRA epilogues

__device__ __forceinline__ void unpack_bf16x8(const uint4& w, float* f) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __bfloat1622float2(h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

// Factored-norm epilogue. For each row i of W0 and each K split z:
//   part[z][i] = sum_{k in split, k < d_in} W0_ik^2 + 2 s sum_n B_in acc_in
// with acc = [W0 | B | B] [A | (s/2) G_hi | (s/2) G_lo]^T over the split's k-blocks.
struct EpiNorm {
  struct Params {
    const __nv_bfloat16* B;  // [d_out x r]
    int r;
    float two_s;
    float* part;             // [splits][d_out]
    int d_out;
    unsigned int* counters;  // one per 128-row tile, zero before the launch
    const float* m;          // magnitude [d_out]
    float* C;                // outputs [d_out]
    float* g;
    float* gm1;
  };
  struct RowState {
    float ss = 0.f;
  };
  // C = sqrt(max(0, sum of squares)), g = m / C, g - 1 = (m - C) / C.
  __device__ static void finish(const Params& p, int m, float sq) {
    const float c = sqrtf(fmaxf(sq, 0.f));
    const float mi = p.m[m];
    p.C[m] = c;
    p.g[m] = mi / c;
    p.gm1[m] = (mi - c) / c;
  }
  static constexpr bool kReadsA = true;
  static constexpr bool kRefillA1 = true;
  // row_ptr: this thread's 128-byte row of the swizzled W0 tile. The swizzle
  // permutes the row's eight 16-byte chunks by (row mod 8), which a sum of
  // squares does not see; reading chunk j ^ (row mod 8) at step j keeps the
  // 32 lanes of a warp on distinct banks.
  __device__ static void on_a_stage(const Params&, RowState& st, const uint8_t* row_ptr, bool src1) {
    if (src1) return;
    const uint4* p = reinterpret_cast<const uint4*>(row_ptr);
    const int t = (int)(smem_u32(row_ptr) >> 7) & 7;
    float acc = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float f[8];
      unpack_bf16x8(p[j ^ t], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc = fmaf(f[i], f[i], acc);
    }
    st.ss += acc;
  }
  // The tile's B rows [128 x r] (the A source-1 operand) were prefetched by the
  // producer into the ring stages the last k-blocks released, in 64-column
  // slabs of the same swizzled layout (EpiCtx refill fields); each row is
  // dotted with its accumulator row, 128 columns of TMEM in flight at a time.
  __host__ __device__ static int refill_slabs(const Params& p) { return (p.r + 63) / 64; }
  template <int BN>
  __device__ static void run(const Params& p, RowState& st, const EpiCtx& c, const GemmGeom& g) {
    static_assert(BN % 32 == 0, "whole 32-column chunks");
    const bool row_ok = c.m < g.M;
    mbar_wait(c.aux_bar, 0);
    const int t = c.row & 7;
    // This thread's row in each 64-column slab of the prefetched B rows.
    constexpr int kSlabs = (BN + 63) / 64;
    const int sps = c.stage_stride / 16384;
    const uint8_t* slab_row[kSlabs];
#pragma unroll
    for (int sl = 0; sl < kSlabs; ++sl)
      slab_row[sl] = c.stage_smem + ((c.refill_first + sl / sps) % c.ring_stages) * c.stage_stride +
                     (sl % sps) * 16384 + c.row * 128;
    float dot8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};  // eight independent FMA chains
#pragma unroll
    for (int col0 = 0; col0 < BN; col0 += 128) {
      constexpr int kMaxChunks = BN < 128 ? BN / 32 : 4;
      uint32_t v[kMaxChunks][32];
      const int nch = min(kMaxChunks, (BN - col0) / 32);
      if (c.has_acc) {
#pragma unroll
        for (int q = 0; q < kMaxChunks; ++q)
          if (q < nch) tmem_ld32_async(c.taddr + (uint32_t)(col0 + 32 * q), v[q]);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int q = 0; q < kMaxChunks; ++q)
#pragma unroll
          for (int i = 0; i < 32; ++i) v[q][i] = 0u;
      }
#pragma unroll
      for (int q = 0; q < kMaxChunks; ++q) {
        if (q >= nch) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = col0 + 32 * q + 8 * j;
          if (n < p.r) {
            const int slab = n >> 6, chunk = (n & 63) >> 3;
            const uint4 w = *reinterpret_cast<const uint4*>(slab_row[slab] + ((chunk ^ t) << 4));
            float b[8];
            unpack_bf16x8(w, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot8[i] = fmaf(b[i], __uint_as_float(v[q][8 * j + i]), dot8[i]);
          }
        }
      }
    }
    const float dot = ((dot8[0] + dot8[1]) + (dot8[2] + dot8[3])) + ((dot8[4] + dot8[5]) + (dot8[6] + dot8[7]));
    const float part = fmaf(p.two_s, dot, st.ss);
    if (c.splits == 1) {
      if (row_ok) finish(p, c.m, part);
      return;
    }
    if (row_ok) p.part[(long long)c.split * p.d_out + c.m] = part;
    if (!split_arrive_last(c, p.counters) || !row_ok) return;
    float sq = 0.f;
    for (int z = 0; z < c.splits; ++z) sq += __ldcg(p.part + (long long)z * p.d_out + c.m);
    finish(p, c.m, sq);
  }
};


// Near-unity compose: y = pre + gm1[n] * pre (fp32, rounded once), pre optional.
struct EpiCompose {
  struct Params {
    __nv_bfloat16* y;
    __nv_bfloat16* pre;  // may be null
    const float* gm1;
    long long ldo;
  };
  using RowState = NoRowState;
  static constexpr bool kReadsA = false;
  static constexpr bool kRefillA1 = false;
  static constexpr int kStageOutBytes = 0;
  __device__ static void on_a_stage(const Params&, RowState&, const uint8_t*, bool) {}
  template <int BN>
  __device__ static void run(const Params& p, RowState&, const EpiCtx& c, const GemmGeom& g) {
    const bool row_ok = c.m < g.M;
    for_each_acc_chunk<BN>(c, [&](int col, float* v) {
      if (!row_ok) return;
      const int n = c.n0 + col;
      __nv_bfloat16* yrow = p.y + (long long)c.m * p.ldo + n;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (col + 8 * j < BN && n + 8 * j < g.N) {
          const float4 ga = __ldg(reinterpret_cast<const float4*>(p.gm1 + n + 8 * j));
          const float4 gb = __ldg(reinterpret_cast<const float4*>(p.gm1 + n + 8 * j + 4));
          const float gm[8] = {ga.x, ga.y, ga.z, ga.w, gb.x, gb.y, gb.z, gb.w};
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = fmaf(gm[i], v[8 * j + i], v[8 * j + i]);
          // y is not read again inside the layer step; pre is, by the compose backward.
          store_bf16x8_cs(yrow + 8 * j, o);
          if (p.pre) store_bf16x8(p.pre + (long long)c.m * p.ldo + n + 8 * j, v + 8 * j);
        }
      }
    });
  }
};

// out[m][n] = out[m][n] + alpha acc[m][n]: the old bf16 value is read and the
// sum rounded once. Each thread reads exactly the elements it writes.
struct EpiAxpyBF16 {
  struct Params {
    __nv_bfloat16* out;
    long long ldo;
    float alpha;
  };
  using RowState = NoRowState;
  static constexpr bool kReadsA = false;
  static constexpr bool kRefillA1 = false;
  static constexpr int kStageOutBytes = 0;
  __device__ static void on_a_stage(const Params&, RowState&, const uint8_t*, bool) {}
  template <int BN>
  __device__ static void run(const Params& p, RowState&, const EpiCtx& c, const GemmGeom& g) {
    const bool row_ok = c.m < g.M;
    // for_each_acc_chunk is warp-collective: rows past M skip only the memory work.
    for_each_acc_chunk<BN>(c, [&](int col, float* v) {
      if (!row_ok) return;
      const int n = c.n0 + col;
      __nv_bfloat16* dst = p.out + (long long)c.m * p.ldo + n;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (col + 8 * j < BN && n + 8 * j < g.N) {
          float o[8];
          unpack_bf16x8(*reinterpret_cast<const uint4*>(dst + 8 * j), o);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = fmaf(p.alpha, v[8 * j + i], o[i]);
          store_bf16x8(dst + 8 * j, o);
        }
      }
    });
  }
};

// Non-persistent CTA-pair launch: one 256 x BN tile and one K split per pair
// (grid 2 x tiles, 1, splits).
template <class Cfg, class Epi>
static cudaError_t launch_gemm_pair_split(const GemmArgs& g, const typename Epi::Params& ep, cudaStream_t st) {
  CUtensorMap ta0, ta1, tb0, tb1;
  const int a_box = Cfg::A_MN ? 64 : kBM;
  const int b_box = Cfg::B_MN ? 64 : Cfg::B_BOX;
  t_detail.clear();
  if (!make_map(&ta0, g.a0, a_box, "A source 0") || !make_map(&tb0, g.b0, b_box, "B source 0"))
    return cudaErrorInvalidValue;
  const int kb0 = (int)ceil_div(g.K0, kBK);
  const int kb1 = g.K1 > 0 ? (int)ceil_div(g.K1, kBK) : 0;
  if (kb1 > 0) {
    if (!make_map(&ta1, g.a1, a_box, "A source 1") || !make_map(&tb1, g.b1, b_box, "B source 1"))
      return cudaErrorInvalidValue;
  } else {
    ta1 = ta0;
    tb1 = tb0;
  }
  const int kps = g.split.kb_per_split > 0 ? g.split.kb_per_split : kb0 + kb1;
  GemmGeom geom{g.M, g.N, kb0, kb1, kps, g.a1_kwrap, g.defer_wait_src1};
  const long long splits = ceil_div(std::max(kb0 + kb1, 1), kps);
  const long long tiles = ceil_div(g.N, Cfg::BN) * ceil_div(g.M, 2 * kBM);
  auto kern = gemm_sm100_pair_split_kernel<Cfg, Epi>;
  constexpr int smem_bytes = PairSplitLayout<Cfg, Epi>::SMEM_BYTES;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t e = set_smem_once(smem_set, kern, smem_bytes);
  if (e != cudaSuccess) {
    t_detail = "shared-memory attribute (" + std::to_string(smem_bytes) + " bytes)";
    return e;
  }
  {
    ProfRange pr(g.name, st);
    e = launch_pdl(kern, dim3((unsigned)(2 * tiles), 1, (unsigned)splits), dim3(kGemmThreads), smem_bytes, st, ta0,
                   ta1, tb0, tb1, geom, ep);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) t_detail = "pair split launch, " + std::to_string(tiles) + " tiles x " +
                                   std::to_string(splits) + " splits";
  return e;
}

// The factored norm GEMM on CTA pairs: 256 rows x the whole rank per tile.
static cudaError_t norm_gemm(int bn, const GemmArgs& g, const EpiNorm::Params& ep, cudaStream_t st) {
  switch (bn) {
    case 64: return launch_gemm_pair_split<PairCfg<64, false, false>, EpiNorm>(g, ep, st);
    case 128: return launch_gemm_pair_split<PairCfg<128, false, false>, EpiNorm>(g, ep, st);
    case 256: return launch_gemm_pair_split<PairCfg<256, false, false>, EpiNorm>(g, ep, st);
    case 384: return launch_gemm_pair_split<PairCfg<384, false, false>, EpiNorm>(g, ep, st);
    case 512: return launch_gemm_pair_split<PairCfg<512, false, false>, EpiNorm>(g, ep, st);
  }
  t_detail = "no norm tile of width " + std::to_string(bn);
  return cudaErrorInvalidValue;
}

// ============================================================== SIMT kernels

// out = alpha * sum_z part[z] (split order fixed), bf16; out[n][m] if transpose.
__global__ void reduce_splits_bf16_kernel(const float* __restrict__ part, int splits, long long split_stride,
                                          int M, int N, float alpha, __nv_bfloat16* __restrict__ out,
                                          long long ldo, int transpose) {
  pdl_trigger();
  pdl_wait();
  const int ng = N / 4;
  const long long total = (long long)M * ng;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total;
       i += (long long)gridDim.x * blockDim.x) {
    int m, n;
    if (!transpose) {
      m = (int)(i / ng);
      n = (int)(i % ng) * 4;
    } else {
      n = (int)(i / M) * 4;
      m = (int)(i % M);
    }
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int z = 0; z < splits; ++z) {
      const float4 v = *reinterpret_cast<const float4*>(part + z * split_stride + (long long)m * N + n);
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    const float o[4] = {alpha * a.x, alpha * a.y, alpha * a.z, alpha * a.w};
    if (!transpose) {
      __nv_bfloat162 h[2] = {__floats2bfloat162_rn(o[0], o[1]), __floats2bfloat162_rn(o[2], o[3])};
      *reinterpret_cast<uint2*>(out + (long long)m * ldo + n) = *reinterpret_cast<const uint2*>(h);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) out[(long long)(n + j) * ldo + m] = __float2bfloat16_rn(o[j]);
    }
  }
}

// Compose backward, one streaming pass over [T x d_out]:
//   dz[t][i] = g_i * dy[t][i]   (bf16)
//   part[rb][i] = sum over the row block's t of dy[t][i] * pre[t][i]
// Block: 256 threads, 64 columns x rows_per_block rows (a multiple of 32; the
// plan sizes the row blocks so that the whole grid is resident at once). Lane
// = (row offset 0..3, 8-column vector 0..7), so each warp access covers 4 full
// 128-byte rows; the per-column sums are combined over the 4 row lanes with
// shuffles, then over the 8 warps in shared memory. The last row block of a
// column strip to finish (counter per strip, zero before the launch) sums the
// strip's partials in row-block order: dm_i = sum / C_i.
__global__ void __launch_bounds__(256) compose_bwd_bf16_kernel(const __nv_bfloat16* __restrict__ dy,
                                                               const __nv_bfloat16* __restrict__ pre,
                                                               const float* __restrict__ g,
                                                               const float* __restrict__ C,
                                                               __nv_bfloat16* __restrict__ dz,
                                                               float* __restrict__ part,
                                                               unsigned int* __restrict__ counters,
                                                               float* __restrict__ dm, int T, int d_out,
                                                               int rows_per_block) {
  pdl_trigger();
  pdl_wait();
  __shared__ float red[8][64];
  __shared__ unsigned int last_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cv = lane & 7, ro = lane >> 3;
  const int col = blockIdx.x * 64 + cv * 8;
  const bool col_ok = col < d_out;
  const int t0 = blockIdx.y * rows_per_block;
  const int t1 = min(T, t0 + rows_per_block);
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
  if (col_ok) {
    const float4 ga = __ldg(reinterpret_cast<const float4*>(g + col));
    const float4 gb = __ldg(reinterpret_cast<const float4*>(g + col + 4));
    const float gv[8] = {ga.x, ga.y, ga.z, ga.w, gb.x, gb.y, gb.z, gb.w};
#pragma unroll 4
    for (int t = t0 + warp * 4 + ro; t < t1; t += 32) {
      const size_t off = (size_t)t * d_out + col;
      const uint4 a = __ldcs(reinterpret_cast<const uint4*>(dy + off));
      const uint4 b = __ldcs(reinterpret_cast<const uint4*>(pre + off));
      float fa[8], fb[8], z[8];
      unpack_bf16x8(a, fa);
      unpack_bf16x8(b, fb);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc[j] = fmaf(fa[j], fb[j], acc[j]);
        z[j] = gv[j] * fa[j];
      }
      store_bf16x8(dz + off, z);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], 8);
    acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], 16);
  }
  if (ro == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) red[warp][cv * 8 + j] = acc[j];
  }
  __syncthreads();
  const int c = blockIdx.x * 64 + (int)threadIdx.x;
  if (threadIdx.x < 64) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += red[w][threadIdx.x];
    if (c < d_out) part[(size_t)blockIdx.y * d_out + c] = s;
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last_flag = (atomicAdd(&counters[blockIdx.x], 1u) == gridDim.y - 1) ? 1u : 0u;
  __syncthreads();
  if (last_flag && threadIdx.x < 64 && c < d_out) {
    __threadfence();
    float s = 0.f;
    for (unsigned int rb = 0; rb < gridDim.y; ++rb) s += __ldcg(part + (size_t)rb * d_out + c);
    dm[c] = s / C[c];
  }
}

// Full gradient, per row n: kappa_n = g_n dm_n / C_n and Bk[n] = bf16(kappa_n B[n]).
// One thread per 8 columns of a row; the row's first thread also stores kappa_n.
__global__ void full_kappa_kernel(const float* __restrict__ g, const float* __restrict__ dm,
                                  const float* __restrict__ C, const __nv_bfloat16* __restrict__ B, int d_out, int r,
                                  float* __restrict__ kappa, __nv_bfloat16* __restrict__ Bk) {
  pdl_trigger();
  pdl_wait();
  const int q = r / 8;
  const long long total = (long long)d_out * q;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total;
       i += (long long)gridDim.x * blockDim.x) {
    const int n = (int)(i / q), c = (int)(i % q) * 8;
    const float k = g[n] * dm[n] / C[n];
    if (c == 0) kappa[n] = k;
    float b[8];
    unpack_bf16x8(*reinterpret_cast<const uint4*>(B + (long long)n * r + c), b);
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] *= k;
    store_bf16x8(Bk + (long long)n * r + c, b);
  }
}

// Full gradient, dB[n][c] -= s kappa_n Q[n][c] with Q = sum_z part[z] (split
// order fixed); the old bf16 dB is read and the result rounded once.
__global__ void full_dB_kernel(const float* __restrict__ part, int splits, long long split_stride, int d_out, int r,
                               const float* __restrict__ kappa, float s, __nv_bfloat16* __restrict__ dB) {
  pdl_trigger();
  pdl_wait();
  const int q = r / 4;
  const long long total = (long long)d_out * q;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total;
       i += (long long)gridDim.x * blockDim.x) {
    const int n = (int)(i / q), c = (int)(i % q) * 4;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int z = 0; z < splits; ++z) {
      const float4 v = *reinterpret_cast<const float4*>(part + z * split_stride + (long long)n * r + c);
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    const float f = -s * kappa[n];
    __nv_bfloat162* d2 = reinterpret_cast<__nv_bfloat162*>(dB + (long long)n * r + c);
    const float2 o0 = __bfloat1622float2(d2[0]), o1 = __bfloat1622float2(d2[1]);
    d2[0] = __floats2bfloat162_rn(fmaf(f, a.x, o0.x), fmaf(f, a.y, o0.y));
    d2[1] = __floats2bfloat162_rn(fmaf(f, a.z, o1.x), fmaf(f, a.w, o1.y));
  }
}

static cudaError_t reduce_splits(const float* part, const Split& sp, long long split_stride, int M, int N,
                                 float alpha, __nv_bfloat16* out, long long ldo, bool transpose, const char* name,
                                 cudaStream_t st) {
  const long long total = (long long)M * (N / 4);
  const int threads = 256;
  const long long blocks = std::min<long long>(ceil_div(total, threads), 148LL * 16);
  ProfRange pr(name, st);
  cudaError_t e = launch_pdl(reduce_splits_bf16_kernel, dim3((unsigned)std::max<long long>(blocks, 1)),
                             dim3(threads), 0, st, part, sp.splits, split_stride, M, N, alpha, out, ldo,
                             transpose ? 1 : 0);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

// CTA-pair dispatch on the tile width.
template <bool A_MN, bool B_MN, class Epi>
static cudaError_t pair_gemm_bn(int bn, const GemmArgs& g, const typename Epi::Params& ep, int sms, cudaStream_t st) {
  if constexpr (!B_MN) {
    if (bn == 64) return launch_gemm_pair<PairCfg<64, A_MN, B_MN>, Epi>(g, ep, sms, st);
  }
  if (bn == 128) return launch_gemm_pair<PairCfg<128, A_MN, B_MN>, Epi>(g, ep, sms, st);
  if (bn == 256) return launch_gemm_pair<PairCfg<256, A_MN, B_MN>, Epi>(g, ep, sms, st);
  if (bn == 384) return launch_gemm_pair<PairCfg<384, A_MN, B_MN>, Epi>(g, ep, sms, st);
  if (bn == 512) return launch_gemm_pair<PairCfg<512, A_MN, B_MN>, Epi>(g, ep, sms, st);
  t_detail = "no pair tile of width " + std::to_string(bn);
  return cudaErrorInvalidValue;
}

// Narrow GEMM (N = r) with an alpha-scaled bf16 result: direct store when the
// K loop is not split, else fp32 partials summed in split order by
// reduce_splits. On single CTAs the threads store the partials; on CTA pairs
// the epilogue warps stage them for TMA stores.
template <bool A_MN, bool B_MN>
static cudaError_t narrow_gemm_1cta(int bn, const GemmArgs& g, float alpha, __nv_bfloat16* out, long long ldo,
                                    bool transpose, float* part, const char* reduce_name, cudaStream_t st) {
  if (g.split.splits == 1) {
    EpiStoreBF16::Params p{out, ldo, alpha, transpose ? 1 : 0};
    return gemm_bn<A_MN, B_MN, EpiStoreBF16>(bn, g, p, st);
  }
  const long long sstride = (long long)g.M * g.N;
  EpiPartialF32::Params p{part, g.N, sstride};
  cudaError_t e = gemm_bn<A_MN, B_MN, EpiPartialF32>(bn, g, p, st);
  if (e != cudaSuccess) return e;
  return reduce_splits(part, g.split, sstride, g.M, g.N, alpha, out, ldo, transpose, reduce_name, st);
}

// GEMM on CTA-pair clusters (gemm_sm100_pair_cluster_kernel): the K splits of
// each 256-row tile reduced inside its cluster; output per ClusterOut.
template <class Cfg, int CS>
static cudaError_t launch_pair_cluster(const GemmArgs& g, const ClusterOut& o, cudaStream_t st) {
  CUtensorMap ta0, ta1, tb0, tb1;
  const int a_box = Cfg::A_MN ? 64 : kBM;
  const int b_box = Cfg::B_MN ? 64 : Cfg::B_BOX;
  t_detail.clear();
  if (!make_map(&ta0, g.a0, a_box, "A source 0") || !make_map(&tb0, g.b0, b_box, "B source 0"))
    return cudaErrorInvalidValue;
  const int kb0 = (int)ceil_div(g.K0, kBK);
  const int kb1 = g.K1 > 0 ? (int)ceil_div(g.K1, kBK) : 0;
  if (kb1 > 0) {
    if (!make_map(&ta1, g.a1, a_box, "A source 1") || !make_map(&tb1, g.b1, b_box, "B source 1"))
      return cudaErrorInvalidValue;
  } else {
    ta1 = ta0;
    tb1 = tb0;
  }
  const int kb = std::max(kb0 + kb1, 1);
  GemmGeom geom{g.M, g.N, kb0, kb1, (int)ceil_div(kb, CS), 0, g.defer_wait_src1, g.wait_then_trigger};
  const long long tiles = ceil_div(g.N, Cfg::BN) * ceil_div(g.M, 2 * kBM);
  auto kern = gemm_sm100_pair_cluster_kernel<Cfg, CS>;
  constexpr int smem_bytes = PairClusterLayout<Cfg>::SMEM_BYTES;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t e = set_smem_once(smem_set, kern, smem_bytes);
  if (e == cudaSuccess && CS > 4) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) {
    t_detail = "shared-memory or cluster-size attribute (" + std::to_string(smem_bytes) + " bytes)";
    return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * CS * tiles));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem_bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  // Under the kernel profiler each launch is timed on its own: no early start.
  attr[0].val.programmaticStreamSerializationAllowed = profiling_on() ? 0 : 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2 * CS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  {
    ProfRange pr(g.name, st);
    e = cudaLaunchKernelEx(&cfg, kern, ta0, ta1, tb0, tb1, geom, o);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess)
    t_detail = "pair cluster launch, " + std::to_string(tiles) + " tiles x " + std::to_string(CS) + " pairs";
  return e;
}

template <int BN, bool A_MN, bool B_MN>
static cudaError_t pair_cluster_cs(int cs, const GemmArgs& g, const ClusterOut& o, cudaStream_t st) {
  using Cfg = PairCfg<BN, A_MN, B_MN>;
  if (cs == 1) return launch_pair_cluster<Cfg, 1>(g, o, st);
  if (cs == 2) return launch_pair_cluster<Cfg, 2>(g, o, st);
  if (cs == 3) return launch_pair_cluster<Cfg, 3>(g, o, st);
  if (cs == 4) return launch_pair_cluster<Cfg, 4>(g, o, st);
  if constexpr (BN <= 128) {
    if (cs == 8) return launch_pair_cluster<Cfg, 8>(g, o, st);
  }
  t_detail = "no cluster of " + std::to_string(cs) + " pairs";
  return cudaErrorInvalidValue;
}

// How many clusters of cs CTA pairs (each CTA one SM: ~200 KB of shared memory)
// the current device holds at once: a cluster must fit in one GPC, so this is
// below SMs / (2 cs) for the larger clusters (e.g. 15 clusters of 8 CTAs on a
// 148-SM B200). Queried once per device and cluster size; 0 if the query fails.
int max_active_pair_clusters(int cs) {
  static std::atomic<int> cache[64][9];
  if (cs < 1 || (cs > 4 && cs != 8)) return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  const int hit = cache[dev][cs].load();
  if (hit != 0) return hit > 0 ? hit : 0;
  using Cfg = PairCfg<384, false, false>;
  constexpr int smem_bytes = PairClusterLayout<Cfg>::SMEM_BYTES;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * cs * 64));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem_bytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  cudaError_t e = cudaSuccess;
  switch (cs) {
    case 1: {
      static std::atomic<unsigned long long> set{0};
      auto k = gemm_sm100_pair_cluster_kernel<Cfg, 1>;
      e = set_smem_once(set, k, smem_bytes);
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, k, &cfg);
      break;
    }
    case 2: {
      static std::atomic<unsigned long long> set{0};
      auto k = gemm_sm100_pair_cluster_kernel<Cfg, 2>;
      e = set_smem_once(set, k, smem_bytes);
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, k, &cfg);
      break;
    }
    case 3: {
      static std::atomic<unsigned long long> set{0};
      auto k = gemm_sm100_pair_cluster_kernel<Cfg, 3>;
      e = set_smem_once(set, k, smem_bytes);
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, k, &cfg);
      break;
    }
    case 4: {
      static std::atomic<unsigned long long> set{0};
      auto k = gemm_sm100_pair_cluster_kernel<Cfg, 4>;
      e = set_smem_once(set, k, smem_bytes);
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, k, &cfg);
      break;
    }
    default: {
      // 16-CTA clusters (non-portable), used with tiles up to 128 columns wide only.
      using Cfg8 = PairCfg<128, false, false>;
      constexpr int smem8 = PairClusterLayout<Cfg8>::SMEM_BYTES;
      cfg.dynamicSmemBytes = smem8;
      static std::atomic<unsigned long long> set{0};
      auto k = gemm_sm100_pair_cluster_kernel<Cfg8, 8>;
      e = set_smem_once(set, k, smem8);
      if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, k, &cfg);
      break;
    }
  }
  if (e != cudaSuccess || n <= 0) {
    cudaGetLastError();
    cache[dev][cs].store(-1);
    return 0;
  }
  cache[dev][cs].store(n);
  return n;
}

// Narrow GEMM (N = r): out = alpha * A B^T in bf16 on pair clusters.
template <bool A_MN, bool B_MN>
static cudaError_t narrow_cluster(int bn, int cs, const GemmArgs& g, float alpha, __nv_bfloat16* out, long long ldo,
                                  bool transpose, cudaStream_t st) {
  const ClusterOut o{out, nullptr, nullptr, ldo, alpha, transpose ? 1 : 0, 0};
  if constexpr (!B_MN) {
    if (bn == 64) return pair_cluster_cs<64, A_MN, B_MN>(cs, g, o, st);
    if (bn == 192) return pair_cluster_cs<192, A_MN, B_MN>(cs, g, o, st);
  }
  if (bn == 128) return pair_cluster_cs<128, A_MN, B_MN>(cs, g, o, st);
  if (bn == 256) return pair_cluster_cs<256, A_MN, B_MN>(cs, g, o, st);
  if (bn == 384) return pair_cluster_cs<384, A_MN, B_MN>(cs, g, o, st);
  if (bn == 512) return pair_cluster_cs<512, A_MN, B_MN>(cs, g, o, st);
  t_detail = "no pair cluster tile of width " + std::to_string(bn);
  return cudaErrorInvalidValue;
}

// ============================================================== grouped launches

// One or two GEMMs with the same K sources and tile shape in one persistent
// launch (gemm_sm100_pair_grouped_kernel): whole tiles, at most `pairs` CTA pairs.
template <class Cfg>
static cudaError_t launch_grouped(const GemmArgs* gs, const ClusterOut* os, int nprob, int pairs, const char* name,
                                  cudaStream_t st, bool early = true) {
  GroupMaps maps{};
  GroupGeom geom{};
  const int a_box = Cfg::A_MN ? 64 : kBM;
  const int b_box = Cfg::B_MN ? 64 : Cfg::B_BOX;
  t_detail.clear();
  int tiles = 0;
  for (int j = 0; j < nprob; ++j) {
    const GemmArgs& g = gs[j];
    const int kb0 = (int)ceil_div(g.K0, kBK);
    const int kb1 = g.K1 > 0 ? (int)ceil_div(g.K1, kBK) : 0;
    if ((j > 0 && (kb0 != geom.kb0 || kb1 != geom.kb1)) || os[j].compose) {
      t_detail = "grouped problems need the same K and a plain output";
      return cudaErrorInvalidValue;
    }
    geom.kb0 = kb0;
    geom.kb1 = kb1;
    if (!make_map(&maps.a0[j], g.a0, a_box, "A source 0") || !make_map(&maps.b0[j], g.b0, b_box, "B source 0"))
      return cudaErrorInvalidValue;
    if (kb1 > 0) {
      if (!make_map(&maps.a1[j], g.a1, a_box, "A source 1") || !make_map(&maps.b1[j], g.b1, b_box, "B source 1"))
        return cudaErrorInvalidValue;
    } else {
      maps.a1[j] = maps.a0[j];
      maps.b1[j] = maps.b0[j];
    }
    GroupProblem& pr = geom.pr[j];
    pr.M = g.M;
    pr.N = g.N;
    pr.n_tiles = (int)ceil_div(g.N, Cfg::BN);
    pr.tile_base = tiles;
    pr.o = os[j];
    tiles += (int)(ceil_div(g.M, 2 * kBM) * pr.n_tiles);
  }
  for (int j = nprob; j < 2; ++j) {
    maps.a0[j] = maps.a0[0];
    maps.a1[j] = maps.a1[0];
    maps.b0[j] = maps.b0[0];
    maps.b1[j] = maps.b1[0];
    geom.pr[j] = geom.pr[0];
    geom.pr[j].tile_base = tiles;
  }
  geom.tiles = tiles;
  geom.nprob = nprob;
  const int P = std::max(1, std::min(pairs, tiles));
  auto kern = gemm_sm100_pair_grouped_kernel<Cfg>;
  constexpr int smem_bytes = GroupLayout<Cfg>::SMEM_BYTES;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t e = set_smem_once(smem_set, kern, smem_bytes);
  if (e != cudaSuccess) {
    t_detail = "grouped shared-memory attribute (" + std::to_string(smem_bytes) + " bytes)";
    return e;
  }
  {
    ProfRange pr(name, st);
    e = launch_pdl_if(early, kern, dim3((unsigned)(2 * P)), dim3(kGemmThreads), (size_t)smem_bytes, st, maps, geom);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) t_detail = "grouped launch, " + std::to_string(tiles) + " tiles on " + std::to_string(P) + " pairs";
  return e;
}

template <bool A_MN, bool B_MN>
static cudaError_t grouped_bn(int bn, const GemmArgs* gs, const ClusterOut* os, int nprob, int pairs,
                              const char* name, cudaStream_t st, bool early = true) {
  if constexpr (!B_MN) {
    if (bn == 64) return launch_grouped<PairCfg<64, A_MN, B_MN>>(gs, os, nprob, pairs, name, st, early);
  }
  if (bn == 128) return launch_grouped<PairCfg<128, A_MN, B_MN>>(gs, os, nprob, pairs, name, st, early);
  if (bn == 256) return launch_grouped<PairCfg<256, A_MN, B_MN>>(gs, os, nprob, pairs, name, st, early);
  if (bn == 384) return launch_grouped<PairCfg<384, A_MN, B_MN>>(gs, os, nprob, pairs, name, st, early);
  if (bn == 512) return launch_grouped<PairCfg<512, A_MN, B_MN>>(gs, os, nprob, pairs, name, st, early);
  t_detail = "no grouped tile of width " + std::to_string(bn);
  return cudaErrorInvalidValue;
}

// ============================================================== operations

// Gs = scale * A A^T as bf16 hi and lo halves [r x 2 rp] for a K-extension of a
// later GEMM, in one cluster launch (gram_sm100.cuh). zero_words (may be null)
// are zeroed by the kernel before the next kernel is allowed to start.
// spare_sms: SMs the next kernel leaves free; when the Gram's tiles fit there
// with two or more CTAs each, it takes as many CTAs per tile as fit (it then
// runs beside the next kernel), else eight.
template <int CS>
static cudaError_t launch_gram_cs(const CUtensorMap& ta, const GramParams& gp0, int tiles, cudaStream_t st) {
  GramParams gp = gp0;
  gp.kps = (int)ceil_div(gp.kb_total, CS);
  auto kern = gram_cluster_kernel<CS>;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t e = set_smem_once(smem_set, kern, kGramSmemBytes);
  if (e != cudaSuccess) {
    t_detail = "Gram shared-memory attribute";
    return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CS, (unsigned)tiles);
  cfg.blockDim = dim3(192);
  cfg.dynamicSmemBytes = kGramSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  // Under the kernel profiler each launch is timed on its own: no early start.
  attr[0].val.programmaticStreamSerializationAllowed = profiling_on() ? 0 : 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  {
    ProfRange pr("gram_gemm", st);
    e = cudaLaunchKernelEx(&cfg, kern, ta, gp);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess)
    t_detail = "Gram cluster launch, " + std::to_string(tiles) + " tiles x " + std::to_string(CS) + " CTAs";
  return e;
}

static cudaError_t launch_gram(const dora_desc_t& d, const void* A, float scale, __nv_bfloat16* gs,
                               unsigned int* zero_words, int zero_count, int spare_sms, cudaStream_t st) {
  const int r = (int)d.r, d_in = (int)d.d_in;
  CUtensorMap ta;
  t_detail.clear();
  if (!make_map(&ta, Mat{A, r, d_in, d_in}, kGramTile, "A (Gram)")) return cudaErrorInvalidValue;
  GramParams gp;
  gp.r = r;
  gp.rp = (int)ceil_div(r, kBK) * kBK;
  gp.nt = (int)ceil_div(r, kGramTile);
  gp.kb_total = (int)ceil_div(d_in, kBK);
  gp.kps = 0;
  gp.scale = scale;
  gp.gs2 = gs;
  gp.zero_words = zero_words;
  gp.zero_count = zero_count;
  const int tiles = gp.nt * (gp.nt + 1) / 2;
  int cs = 8;
  if (2 * tiles <= spare_sms) cs = 8 * tiles <= spare_sms ? 8 : 4 * tiles <= spare_sms ? 4 : 2;
  switch (cs) {
    case 2: return launch_gram_cs<2>(ta, gp, tiles, st);
    case 4: return launch_gram_cs<4>(ta, gp, tiles, st);
    default: return launch_gram_cs<8>(ta, gp, tiles, st);
  }
}

dora_status_t bf16_norm(const dora_desc_t& d, const Plan& p, const void* W0, const void* A, const void* B,
                        const float* m, float* C, float* g, float* gm1, uint8_t* ws, cudaStream_t st) {
  const int r = (int)d.r, d_in = (int)d.d_in, d_out = (int)d.d_out;
  __nv_bfloat16* gs = reinterpret_cast<__nv_bfloat16*>(ws + p.off_gs);
  float* norm_part = reinterpret_cast<float*>(ws + p.off_norm_part);
  unsigned int* ctr = reinterpret_cast<unsigned int*>(ws + p.off_ctr);

  // (s/2) G as bf16 hi and lo halves; the same kernel zeroes the norm's split counters.
  const int rp = (int)ceil_div(r, kBK) * kBK;
  // SMs the norm GEMM leaves free (one CTA pair per tile and K split, at most one per SM pair).
  const long long norm_pairs = ceil_div(d_out, 2 * kBM) * p.norm.splits;
  const int spare = p.sms - 2 * (int)std::min<long long>(norm_pairs, p.sms / 2);
  cudaError_t e = launch_gram(d, A, 0.5f * d.s, gs, ctr, (int)(p.zero_bytes / 4), spare, st);
  if (e != cudaSuccess) return gemm_status(e, "dora_norm: Gram");

  // acc = [W0 | B | B] [A | Gs_hi | Gs_lo]^T with the factored-norm epilogue,
  // finished (C, g, g - 1) by the last split of each row tile.
  GemmArgs na;
  na.a0 = Mat{W0, d_out, d_in, d_in};
  na.a1 = Mat{B, d_out, r, r};
  na.b0 = Mat{A, r, d_in, d_in};
  na.b1 = Mat{gs, r, 2 * rp, 2 * rp};
  na.K0 = d_in;
  na.K1 = 2 * rp;
  na.a1_kwrap = rp;
  na.M = d_out;
  na.N = r;
  na.split = p.norm;
  na.defer_wait_src1 = 1;  // only Gs comes from the Gram kernel: stream W0 while it runs
  na.name = "norm_gemm";
  EpiNorm::Params np{reinterpret_cast<const __nv_bfloat16*>(B), r, 2.0f * d.s, norm_part, d_out, ctr, m, C, g,
                     gm1};
  e = norm_gemm(p.norm_bn, na, np, st);
  return gemm_status(e, "dora_norm: factored norm GEMM");
}

dora_status_t bf16_forward(const dora_desc_t& d, const Plan& p, int64_t T, const void* x, const void* W0,
                           const void* A, const void* B, const float* gm1, void* y, void* su_save,
                           void* pre_save, uint8_t* ws, cudaStream_t st) {
  if (T == 0) return DORA_OK;
  const int r = (int)d.r, d_in = (int)d.d_in, d_out = (int)d.d_out, Ti = (int)T;
  __nv_bfloat16* su = su_save ? reinterpret_cast<__nv_bfloat16*>(su_save)
                              : reinterpret_cast<__nv_bfloat16*>(ws + p.off_su);

  // su = s x A^T
  GemmArgs ua;
  ua.a0 = Mat{x, Ti, d_in, d_in};
  ua.b0 = Mat{A, r, d_in, d_in};
  ua.K0 = d_in;
  ua.M = Ti;
  ua.N = r;
  ua.name = "u_gemm";
  // Under fwd_defer the base GEMM below starts its x W0 main loop beside this one and waits
  // for it only before loading su: this grid then waits for its own predecessor first.
  ua.wait_then_trigger = p.fwd_defer;
  cudaError_t e = narrow_cluster<false, false>(p.u_bn, p.u_cs, ua, d.s, su, r, false, st);
  if (e != cudaSuccess) return gemm_status(e, "dora_forward: LoRA down projection");

  // pre = [x | su] [W0 | B]^T, y = pre + gm1 * pre
  GemmArgs ba;
  ba.a0 = Mat{x, Ti, d_in, d_in};
  ba.a1 = Mat{su, Ti, r, r};
  ba.b0 = Mat{W0, d_out, d_in, d_in};
  ba.b1 = Mat{B, d_out, r, r};
  ba.K0 = d_in;
  ba.K1 = r;
  ba.M = Ti;
  ba.N = d_out;
  ba.split.splits = 1;
  ba.name = "fwd_compose_gemm";
  ba.defer_wait_src1 = p.fwd_defer;
  ba.split.kb_per_split = (int)(ceil_div(d_in, kBK) + ceil_div(r, kBK));
  if (p.fwd_cs >= 1) {
    // Few tiles (small token batches): clusters of pairs split K and compose in the reduction.
    const ClusterOut o{reinterpret_cast<__nv_bfloat16*>(y), reinterpret_cast<__nv_bfloat16*>(pre_save), gm1, d_out,
                       1.0f, 0, 1};
    e = pair_cluster_cs<256, false, false>(p.fwd_cs, ba, o, st);
    return gemm_status(e, "dora_forward: base GEMM with compose");
  }
  EpiCompose::Params cp{reinterpret_cast<__nv_bfloat16*>(y), reinterpret_cast<__nv_bfloat16*>(pre_save), gm1,
                        d_out};
  e = launch_gemm_pair<PairCfg<256, false, false>, EpiCompose>(ba, cp, 2 * p.fwd_pairs, st);
  return gemm_status(e, "dora_forward: base GEMM with compose");
}

template <class Cfg>
static cudaError_t launch_merge(const CUtensorMap& ta, const CUtensorMap& tb, const MergeGeom& geom, long long pairs,
                                cudaStream_t st) {
  auto kern = merge_pair_kernel<Cfg>;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t e = set_smem_once(smem_set, kern, Cfg::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  ProfRange pr("merge_gemm", st);
  return launch_pdl(kern, dim3((unsigned)(2 * pairs)), dim3(Cfg::THREADS), (size_t)Cfg::SMEM_BYTES, st, ta, tb, geom);
}

dora_status_t bf16_merge(const dora_desc_t& d, const Plan& p, const void* W0, const void* A, const void* B,
                         const float* g, void* W_out, uint8_t*, cudaStream_t st) {
  // B A with A-operand = rows of B [d_out x r] (K = r contiguous) and
  // B-operand = A [r x d_in] read MN-major; W0 is streamed by the epilogue.
  CUtensorMap ta, tb;
  t_detail.clear();
  if (!make_map(&ta, Mat{B, d.d_out, d.r, d.r}, kBM, "B") || !make_map(&tb, Mat{A, d.r, d.d_in, d.d_in}, 64, "A"))
    return gemm_status(cudaErrorInvalidValue, "dora_merge");
  const int kb = (int)ceil_div(d.r, kBK);
  const MergeGeom geom{(int)d.d_out, (int)d.d_in, kb, g, d.s, reinterpret_cast<const __nv_bfloat16*>(W0),
                       reinterpret_cast<__nv_bfloat16*>(W_out)};
  const long long items = ceil_div(d.d_out, 2 * kBM) * ceil_div(d.d_in, 256);
  cudaError_t e = launch_merge<MergeLaunchCfg>(ta, tb, geom, merge_pairs(items, p.sms), st);
  if (e == cudaSuccess) e = cudaGetLastError();
  return gemm_status(e, "dora_merge");
}

// dB = dz^T su and dA^T = x^T du (stored transposed into dA [r x d_in]): both operands
// token-major, K = T. One grouped launch of whole tiles on `pairs` SM pairs, or two
// cluster split-K launches when their tiles are too few for the SM pairs.
static dora_status_t backward_dBA(const Plan& p, int Ti, int d_out, int d_in, int r, const __nv_bfloat16* dz,
                                  const void* su, const void* x, const __nv_bfloat16* du, void* dA, void* dB,
                                  int pairs, cudaStream_t st, bool early = true) {
  if (p.dBA_grouped) {
    GemmArgs a[2];
    a[0].a0 = Mat{dz, Ti, d_out, d_out};
    a[0].b0 = Mat{su, Ti, r, r};
    a[0].K0 = Ti;
    a[0].M = d_out;
    a[0].N = r;
    a[1].a0 = Mat{x, Ti, d_in, d_in};
    a[1].b0 = Mat{du, Ti, r, r};
    a[1].K0 = Ti;
    a[1].M = d_in;
    a[1].N = r;
    const ClusterOut o[2] = {{reinterpret_cast<__nv_bfloat16*>(dB), nullptr, nullptr, r, 1.0f, 0, 0},
                             {reinterpret_cast<__nv_bfloat16*>(dA), nullptr, nullptr, d_in, 1.0f, 1, 0}};
    cudaError_t e = grouped_bn<true, true>(p.dB_bn, a, o, 2, pairs, "dBA_gemm", st, early);
    if (e != cudaSuccess) return gemm_status(e, "dora_backward: dB and dA");
  } else {
    // dB = dz^T su  (both token-major: K = T)
    {
      GemmArgs a;
      a.a0 = Mat{dz, Ti, d_out, d_out};
      a.b0 = Mat{su, Ti, r, r};
      a.K0 = Ti;
      a.M = d_out;
      a.N = r;
      a.name = "dB_gemm";
      cudaError_t e = narrow_cluster<true, true>(p.dB_bn, p.dB_cs, a, 1.0f, reinterpret_cast<__nv_bfloat16*>(dB), r,
                                                 false, st);
      if (e != cudaSuccess) return gemm_status(e, "dora_backward: dB");
    }
    // dA^T = x^T du, stored transposed into dA [r x d_in]
    {
      GemmArgs a;
      a.a0 = Mat{x, Ti, d_in, d_in};
      a.b0 = Mat{du, Ti, r, r};
      a.K0 = Ti;
      a.M = d_in;
      a.N = r;
      a.name = "dA_gemm";
      cudaError_t e = narrow_cluster<true, true>(p.dA_bn, p.dA_cs, a, 1.0f, reinterpret_cast<__nv_bfloat16*>(dA), d_in,
                                                 true, st);
      if (e != cudaSuccess) return gemm_status(e, "dora_backward: dA");
    }
  }
  return DORA_OK;
}

// dx = [dz | du] [W0 ; A]  (W0 and A read MN-major: K rows, N = d_in contiguous); the
// persistent kernel on at most sms / 2 pairs; with defer, dx directly follows the du launch
// and waits for it only before its du k-block (du having waited for its own predecessor).
static dora_status_t backward_dx(const Plan& p, int Ti, int d_out, int d_in, int r, const __nv_bfloat16* dz,
                                 const __nv_bfloat16* du, const void* W0, const void* A, void* dx, int sms,
                                 bool defer, cudaStream_t st) {
  {
    GemmArgs a;
    a.a0 = Mat{dz, Ti, d_out, d_out};
    a.a1 = Mat{du, Ti, r, r};
    a.b0 = Mat{W0, d_out, d_in, d_in};
    a.b1 = Mat{A, r, d_in, d_in};
    a.K0 = d_out;
    a.K1 = r;
    a.M = Ti;
    a.N = d_in;
    a.split.splits = 1;
    a.name = "dx_gemm";
    a.defer_wait_src1 = defer ? 1 : 0;
    a.split.kb_per_split = (int)(ceil_div(d_out, kBK) + ceil_div(r, kBK));
    cudaError_t e;
    if (p.dx_cs >= 1) {
      const ClusterOut o{reinterpret_cast<__nv_bfloat16*>(dx), nullptr, nullptr, d_in, 1.0f, 0, 0};
      e = pair_cluster_cs<256, false, true>(p.dx_cs, a, o, st);
    } else {
      EpiStoreBF16::Params sp{reinterpret_cast<__nv_bfloat16*>(dx), d_in, 1.0f, 0};
      e = launch_gemm_pair<PairCfg<256, false, true>, EpiStoreBF16>(a, sp, sms, st);
    }
    if (e != cudaSuccess) return gemm_status(e, "dora_backward: dx");
  }
  return DORA_OK;
}

// The backward's second stream, with its fork and join events: one set per thread and
// device, created on first use outside a stream capture (creating them inside one is not
// allowed in every capture mode) and kept for the life of the thread.
struct SideStream {
  cudaStream_t s = nullptr;
  cudaEvent_t fork = nullptr, join = nullptr;
};

static SideStream* side_stream(cudaStream_t st) {
  constexpr int kMaxDevices = 64;
  thread_local SideStream per_device[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    (void)cudaGetLastError();
    return nullptr;
  }
  SideStream& ss = per_device[dev];
  if (ss.s != nullptr) return &ss;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(st, &cap) != cudaSuccess || cap != cudaStreamCaptureStatusNone) {
    (void)cudaGetLastError();
    return nullptr;
  }
  cudaStream_t s = nullptr;
  cudaEvent_t f = nullptr, j = nullptr;
  if (cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking) != cudaSuccess ||
      cudaEventCreateWithFlags(&f, cudaEventDisableTiming) != cudaSuccess ||
      cudaEventCreateWithFlags(&j, cudaEventDisableTiming) != cudaSuccess) {
    (void)cudaGetLastError();
    if (j) cudaEventDestroy(j);
    if (f) cudaEventDestroy(f);
    if (s) cudaStreamDestroy(s);
    return nullptr;
  }
  ss.s = s;
  ss.fork = f;
  ss.join = j;
  return &ss;
}

dora_status_t bf16_backward(const dora_desc_t& d, const Plan& p, int64_t T, const void* dy, const void* x,
                            const void* W0, const void* A, const void* B, const float* C, const float* g,
                            const void* su, const void* pre, float* dm, void* dA, void* dB, void* dx,
                            uint8_t* ws, cudaStream_t st) {
  const int r = (int)d.r, d_in = (int)d.d_in, d_out = (int)d.d_out, Ti = (int)T;
  if (T == 0) {
    cudaError_t e = cudaMemsetAsync(dm, 0, sizeof(float) * d_out, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(dA, 0, 2 * (size_t)r * d_in, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(dB, 0, 2 * (size_t)d_out * r, st);
    return cuda_status(e, "dora_backward: empty batch");
  }
  __nv_bfloat16* dz = reinterpret_cast<__nv_bfloat16*>(ws + p.off_dz);
  float* dm_part = reinterpret_cast<float*>(ws + p.off_dm_part);
  __nv_bfloat16* du = reinterpret_cast<__nv_bfloat16*>(ws + p.off_du);

  unsigned int* ctr = reinterpret_cast<unsigned int*>(ws + p.off_ctr);
  {
    cudaError_t e = cudaMemsetAsync(ws + p.off_ctr, 0, p.zero_bytes, st);
    if (e != cudaSuccess) return cuda_status(e, "dora_backward: clearing counters");
  }
  // dz = g * dy, dm = sum_t dy * pre / C
  {
    const unsigned col_tiles = (unsigned)ceil_div(d_out, 64);
    dim3 grid(col_tiles, (unsigned)p.dm_rowblocks);
    {
      ProfRange pr("compose_bwd", st);
      cudaError_t e = launch_pdl(compose_bwd_bf16_kernel, grid, dim3(256), 0, st,
                                 reinterpret_cast<const __nv_bfloat16*>(dy), reinterpret_cast<const __nv_bfloat16*>(pre),
                                 g, C, dz, dm_part, ctr, dm, Ti, d_out, p.dm_rows);
      if (e != cudaSuccess) return cuda_status(e, "dora_backward: compose backward");
    }
  }
  // du = s dz B  (B read MN-major: K = d_out rows, N = r contiguous), into `out` on `ss`
  auto launch_du = [&](__nv_bfloat16* out, bool wait_then_trigger, cudaStream_t ss) {
    GemmArgs a;
    a.a0 = Mat{dz, Ti, d_out, d_out};
    a.b0 = Mat{B, d_out, r, r};
    a.K0 = d_out;
    a.M = Ti;
    a.N = r;
    a.name = "du_gemm";
    a.wait_then_trigger = wait_then_trigger ? 1 : 0;
    return gemm_status(narrow_cluster<false, true>(p.du_bn, p.du_cs, a, d.s, out, r, false, ss), "dora_backward: du");
  };
  auto fork = [&](SideStream* ss) {
    cudaError_t e = cudaEventRecord(ss->fork, st);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(ss->s, ss->fork, 0);
    return cuda_status(e, "dora_backward: forking onto the second stream");
  };
  auto join = [&](SideStream* ss) {
    cudaError_t e = cudaEventRecord(ss->join, ss->s);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(st, ss->join, 0);
    return cuda_status(e, "dora_backward: joining the second stream");
  };
  // dx and dB/dA both follow du and nothing else. Under the plan's fork dx and the grouped
  // dB/dA launch run at once, on two streams, each on its own share of the SM pairs; the
  // caller's stream waits for both before this call returns. (Serial when the kernel
  // profiler times each launch on its own.)
  SideStream* side = (p.bwd_fork && dx && !profiling_on()) ? side_stream(st) : nullptr;
  if (side && p.dx_defer) {
    // dx also starts beside du: du, then dx on the caller's stream with nothing between
    // them (du waits for compose before letting dx launch; dx waits for du only before its
    // du k-block). dB/dA, forked right after compose, take their own copy of du from the
    // same kernel (the same bits) on the second stream, so that no event sits between du
    // and dx.
    __nv_bfloat16* du2 = reinterpret_cast<__nv_bfloat16*>(ws + p.off_du2);
    dora_status_t status = fork(side);
    if (status != DORA_OK) return status;
    status = launch_du(du2, false, side->s);
    // (dB/dA launch only once their du copy is complete: launched early they would hold
    // their pairs while du runs, and dx could not start all its tiles beside du.)
    const dora_status_t dBA_status =
        status != DORA_OK ? status
                          : backward_dBA(p, Ti, d_out, d_in, r, dz, su, x, du2, dA, dB, p.dBA_pairs, side->s, false);
    status = launch_du(du, true, st);
    const dora_status_t dx_status =
        status != DORA_OK ? status : backward_dx(p, Ti, d_out, d_in, r, dz, du, W0, A, dx, 2 * p.dx_pairs, true, st);
    status = join(side);
    if (status != DORA_OK) return status;
    return dBA_status != DORA_OK ? dBA_status : dx_status;
  }
  {
    const dora_status_t status = launch_du(du, false, st);
    if (status != DORA_OK) return status;
  }
  if (!side) {
    const dora_status_t status = backward_dBA(p, Ti, d_out, d_in, r, dz, su, x, du, dA, dB, p.sms / 2, st);
    if (status != DORA_OK || !dx) return status;
    return backward_dx(p, Ti, d_out, d_in, r, dz, du, W0, A, dx, p.sms, false, st);
  }
  {
    const dora_status_t status = fork(side);
    if (status != DORA_OK) return status;
  }
  const dora_status_t dBA_status = backward_dBA(p, Ti, d_out, d_in, r, dz, su, x, du, dA, dB, p.dBA_pairs, st);
  const dora_status_t dx_status = backward_dx(p, Ti, d_out, d_in, r, dz, du, W0, A, dx, 2 * p.dx_pairs, false, side->s);
  {
    const dora_status_t status = join(side);
    if (status != DORA_OK) return status;
  }
  return dBA_status != DORA_OK ? dBA_status : dx_status;
}

// Full (non-detached) gradient: the detached backward, then per row the
// A.1 projection term, kappa_n = g_n dm_n / C_n:
//   dB -= s diag(kappa) Q,       Q = W0 A^T + s B G  ([W0 | B | B] [A | sG_hi | sG_lo]^T)
//   dA -= s [(kappa B)^T W0 + H A],   H = s B^T diag(kappa) B
dora_status_t bf16_backward_full(const dora_desc_t& d, const Plan& p, int64_t T, const void* dy, const void* x,
                                 const void* W0, const void* A, const void* B, const float* C, const float* g,
                                 const void* su, const void* pre, float* dm, void* dA, void* dB, void* dx,
                                 uint8_t* ws, cudaStream_t st) {
  dora_status_t status = bf16_backward(d, p, T, dy, x, W0, A, B, C, g, su, pre, dm, dA, dB, dx, ws, st);
  if (status != DORA_OK || T == 0) return status;  // no tokens: dm = 0, so kappa = 0
  const int r = (int)d.r, d_in = (int)d.d_in, d_out = (int)d.d_out;
  const int rp = (int)ceil_div(r, kBK) * kBK;
  float* kappa = reinterpret_cast<float*>(ws + p.off_kappa);
  __nv_bfloat16* Bk = reinterpret_cast<__nv_bfloat16*>(ws + p.off_bk);
  __nv_bfloat16* gs = reinterpret_cast<__nv_bfloat16*>(ws + p.off_gs);
  __nv_bfloat16* H = reinterpret_cast<__nv_bfloat16*>(ws + p.off_h);
  float* qpart = reinterpret_cast<float*>(ws + p.off_q_part);
  cudaError_t e;
  {
    const long long total = (long long)d_out * (r / 8);
    ProfRange pr("full_kappa", st);
    e = launch_pdl(full_kappa_kernel, dim3((unsigned)std::min<long long>(ceil_div(total, 256), 2048)), dim3(256), 0,
                   st, g, (const float*)dm, C, reinterpret_cast<const __nv_bfloat16*>(B), d_out, r, kappa, Bk);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_status(e, "dora_backward_full: kappa");
  }
  // s G as bf16 hi + lo, then Q = W0 A^T + s B G into fp32 split partials.
  e = launch_gram(d, A, d.s, gs, nullptr, 0, 0, st);
  if (e != cudaSuccess) return gemm_status(e, "dora_backward_full: Gram");
  {
    GemmArgs a;
    a.a0 = Mat{W0, d_out, d_in, d_in};
    a.a1 = Mat{B, d_out, r, r};
    a.b0 = Mat{A, r, d_in, d_in};
    a.b1 = Mat{gs, r, 2 * rp, 2 * rp};
    a.K0 = d_in;
    a.K1 = 2 * rp;
    a.a1_kwrap = rp;
    a.M = d_out;
    a.N = r;
    a.split = p.q;
    a.name = "full_q_gemm";
    EpiPartialTMA::Params pp;
    if (!make_map_f32_3d(&pp.map, qpart, r, d_out, p.q.splits, 32, 32))
      return gemm_status(cudaErrorInvalidValue, "dora_backward_full: Q");
    e = pair_gemm_bn<false, false, EpiPartialTMA>(p.q_bn, a, pp, p.sms, st);
    if (e != cudaSuccess) return gemm_status(e, "dora_backward_full: Q");
    const long long total = (long long)d_out * (r / 4);
    ProfRange pr("full_dB", st);
    e = launch_pdl(full_dB_kernel, dim3((unsigned)std::min<long long>(ceil_div(total, 256), 148LL * 16)), dim3(256),
                   0, st, (const float*)qpart, p.q.splits, (long long)d_out * r, d_out, r, (const float*)kappa, d.s,
                   reinterpret_cast<__nv_bfloat16*>(dB));
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_status(e, "dora_backward_full: dB correction");
  }
  // H = s (kappa B)^T B  (both operands read MN-major from their [d_out x r] storage; K = d_out)
  {
    GemmArgs a;
    a.a0 = Mat{Bk, d_out, r, r};
    a.b0 = Mat{B, d_out, r, r};
    a.K0 = d_out;
    a.M = r;
    a.N = r;
    a.split = p.h;
    a.name = "full_h_gemm";
    e = narrow_gemm_1cta<true, true>(p.h_bn, a, d.s, H, r, false, reinterpret_cast<float*>(ws + p.off_h_part),
                                     "full_h_reduce", st);
    if (e != cudaSuccess) return gemm_status(e, "dora_backward_full: H");
  }
  // dA += -s [(kappa B)^T | H] [W0 ; A]  (M = r; A operands MN-major: kappa B as stored, H symmetric)
  {
    GemmArgs a;
    a.a0 = Mat{Bk, d_out, r, r};
    a.a1 = Mat{H, r, r, r};
    a.b0 = Mat{W0, d_out, d_in, d_in};
    a.b1 = Mat{A, r, d_in, d_in};
    a.K0 = d_out;
    a.K1 = r;
    a.M = r;
    a.N = d_in;
    a.split.splits = 1;
    a.split.kb_per_split = (int)(ceil_div(d_out, kBK) + ceil_div(r, kBK));
    a.name = "full_dA_gemm";
    EpiAxpyBF16::Params ap{reinterpret_cast<__nv_bfloat16*>(dA), d_in, -d.s};
    e = launch_gemm_pair<PairCfg<256, true, true>, EpiAxpyBF16>(a, ap, p.sms, st);
    if (e != cudaSuccess) return gemm_status(e, "dora_backward_full: dA correction");
  }
  return DORA_OK;
}

}  // namespace dora

namespace dora {

// Failure-detection self-test: one thread waits, through the same bounded
// wait every kernel uses, on an mbarrier that nothing ever completes. The wait
// runs out after limit_ns, records the timeout in this library's device status
// word and the kernel returns; nothing faults, traps or hangs.
__global__ void selftest_wait_timeout_kernel(uint64_t limit_ns, unsigned int* waited_out) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    fence_mbar_init();
    const bool done = mbar_wait(&bar, 0, limit_ns);
    *waited_out = done ? 0u : 1u;
  }
}

dora_status_t selftest_timeout(uint32_t limit_us, unsigned int* scratch, cudaStream_t st) {
  selftest_wait_timeout_kernel<<<1, 32, 0, st>>>((uint64_t)limit_us * 1000ull, scratch);
  return cuda_status(cudaGetLastError(), "dora_selftest_timeout");
}

cudaError_t read_and_clear_device_status(cudaStream_t st, unsigned int* out) {
  cudaError_t e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return e;
  unsigned int v = 0;
  e = cudaMemcpyFromSymbol(&v, g_device_status, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_device_status, &zero, sizeof(zero));
  }
  *out = v;
  return e;
}

}  // namespace dora
