// Host side of tlg_gemm_mxfp4: argument checks, the tile choice and the launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "tlg.h"
#include "tlg_mx_host.cuh"
#include "tlg_mxgemm_kernel.cuh"
#include "tlg_variants.cuh"

namespace tlg {

namespace {

constexpr uint64_t kWaitLimitNs = 1000000000ull;  // 1 s per pipeline wait

// --------------------------------------------------------------------------- launches

struct MxMaps {
  CUtensorMap a = {}, b = {}, sa = {}, sb = {}, c = {};
};

template <int CG, int BN, int STAGES, int OUT, bool EPI>
struct MxVariant {
  using Plan = MxPlan<CG, BN, STAGES>;
  static constexpr auto kKernel = mxgemm_kernel<CG, BN, STAGES, OUT, EPI>;

  static void fill(cudaLaunchConfig_t *cfg, cudaLaunchAttribute *attr, int ctas, cudaStream_t s) {
    *cfg = {};
    cfg->gridDim = dim3(static_cast<unsigned>(ctas));
    cfg->blockDim = dim3(kMxThreads);
    cfg->dynamicSmemBytes = Plan::kDynamicBytes;
    cfg->stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg->attrs = attr;
    cfg->numAttrs = CG > 1 ? 2 : 1;
  }

  static tlg_status units(int dev, int sms, int *out) {
    static LaunchState state[kMaxDevices];
    static std::mutex mutex;
    std::lock_guard<std::mutex> lock(mutex);
    LaunchState &st = state[dev];
    if (!st.ready) {
      if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan::kDynamicBytes) !=
          cudaSuccess) {
        cudaGetLastError();
        return TLG_ERR_CUDA;
      }
      int n = sms;
      if (CG > 1) {
        cudaLaunchConfig_t cfg;
        cudaLaunchAttribute attr[2];
        fill(&cfg, attr, CG * (sms / CG), nullptr);
        if (cudaOccupancyMaxActiveClusters(&n, kKernel, &cfg) != cudaSuccess || n < 1) {
          cudaGetLastError();
          return TLG_ERR_CUDA;
        }
      }
      st.units = n;
      st.ready = true;
    }
    *out = st.units;
    return TLG_OK;
  }

  static tlg_status launch(int units, const MxMaps &m, const MxGemmParams &p, cudaStream_t s) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    fill(&cfg, attr, units * CG, s);
    if (cudaLaunchKernelEx(&cfg, kKernel, m.a, m.b, m.sa, m.sb, m.c, p) != cudaSuccess) {
      cudaGetLastError();
      return TLG_ERR_CUDA;
    }
    return TLG_OK;
  }
};

struct MxFns {
  tlg_status (*units)(int, int, int *);
  tlg_status (*launch)(int, const MxMaps &, const MxGemmParams &, cudaStream_t);
};

template <int CG, int BN, int STAGES, int OUT, bool EPI>
constexpr MxFns fns() {
  return {MxVariant<CG, BN, STAGES, OUT, EPI>::units, MxVariant<CG, BN, STAGES, OUT, EPI>::launch};
}

// The kernel for few rows of A: `clusters` clusters of ks CTAs.
template <int BN, int OUT>
tlg_status launch_tokens(int dev, int clusters, int ks, const MxMaps &m, const MxGemmParams &p, cudaStream_t s) {
  using Plan = MxTokenPlan<BN>;
  constexpr auto kernel = mxgemm_tokens_kernel<BN, OUT>;
  static bool ready[kMaxDevices];
  static std::mutex mutex;
  {
    std::lock_guard<std::mutex> lock(mutex);
    if (!ready[dev]) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan::kDynamicBytes) !=
          cudaSuccess) {
        cudaGetLastError();
        return TLG_ERR_CUDA;
      }
      ready[dev] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters) * static_cast<unsigned>(ks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Plan::kDynamicBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ks);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, m.a, m.b, m.sa, m.sb, p, ks) != cudaSuccess) {
    cudaGetLastError();
    return TLG_ERR_CUDA;
  }
  return TLG_OK;
}

template <int BN>
tlg_status launch_tokens_typed(int out, int dev, int clusters, int ks, const MxMaps &m, const MxGemmParams &p,
                               cudaStream_t s) {
  if (out == TLG_TYPE_F32) return launch_tokens<BN, kTypeF32>(dev, clusters, ks, m, p, s);
  if (out == TLG_TYPE_F16) return launch_tokens<BN, kTypeF16>(dev, clusters, ks, m, p, s);
  return launch_tokens<BN, kTypeBF16>(dev, clusters, ks, m, p, s);
}

// Measured on a B200, in us; [0] the plain product, [1] with bias, GELU and residual.
struct MxTileCost {
  double kb;        // a k-block of 256
  double tile[2];   // beside its k-blocks
  double least[2];  // a tile of few k-blocks: the epilogue's pace
};

struct MxTile {
  int cta_group, block_n, stages;
  MxTileCost cost;
  MxFns fns[3][2];  // [tlg_type][epilogue]
};

#define TLG_MX_TILE(CG, BN, ST, ...)                                                                   \
  {                                                                                                    \
    CG, BN, ST, __VA_ARGS__, {                                                                         \
      {fns<CG, BN, ST, kTypeF32, false>(), fns<CG, BN, ST, kTypeF32, true>()},                         \
          {fns<CG, BN, ST, kTypeF16, false>(), fns<CG, BN, ST, kTypeF16, true>()},                     \
          {fns<CG, BN, ST, kTypeBF16, false>(), fns<CG, BN, ST, kTypeBF16, true>()},                   \
    }                                                                                                  \
  }

// Tiles the library is built with: 128 * cta_group rows by block_n columns.  The costs are
// fitted to 4096^3 (16 k-blocks a tile) and 16384 x 4096 x 1024 (4), fp16 C, back to back: plain
// 37.5 / 27.4 / 27.4 us and 47 / 40 / 38 us with the 128, 192 and 256 wide tiles, with the full
// epilogue 41 / 33 / 32 and 75 / 75 / 76.  They serve every type of C; with fp32, which stores twice the
// bytes, they are not fitted.
const MxTile kTiles[] = {
    TLG_MX_TILE(1, 64, 6, {0.273, {0.4, 0.8}, {1.3, 2.0}}),
    TLG_MX_TILE(1, 128, 5, {0.305, {0.5, 1.0}, {1.65, 2.7}}),
    TLG_MX_TILE(2, 192, 5, {0.313, {0.5, 1.7}, {2.0, 4.0}}),
    TLG_MX_TILE(2, 256, 5, {0.385, {0.7, 1.9}, {2.7, 5.35}}),
};

// --------------------------------------------------------------------------- tile choice

struct MxChoice {
  const MxTile *tile;  // nullptr: the kernel for few rows of A
  int units;
  int tokens;          // its columns (tokens), 0 otherwise
  tlg_config cfg;
};

// Columns of the tokens kernel that hold M rows of A, 0 when there are too many.
int token_columns(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : 0; }

// CTAs sharing the K range: doubled while there is an SM for each and a k-block too, or two CTAs
// to an SM and 16 k-blocks for each (one token, 4096 x 4096 weights: 3.6 us with 4, 4.8 with 2,
// 4.7 with 8, whose 256 CTAs share SMs; 16384 x 4096: 6.6 with 1, 6.7 with 2; 8192 x 28672:
// 21.4 with 4, 24.1 with 2).
int token_split(int64_t N, int num_kb, int sms) {
  const int64_t tiles = (N + 127) / 128;
  int ks = 1;
  while (ks < 8 && ((tiles * ks * 2 <= sms && ks * 2 <= num_kb) ||
                    (tiles * ks * 2 <= 2 * int64_t(sms) && ks * 2 * 16 <= num_kb)))
    ks *= 2;
  return ks;
}

tlg_status choose(int dev, int sms, int64_t M, int64_t N, int64_t K, int type, bool epi, const tlg_config *req,
                  MxChoice *out) {
  tlg_config r = {};
  if (req != nullptr) r = *req;
  if (r.raster_group < 0 || r.raster_group > 64 || r.max_ctas < 0 || r.stages < 0 || r.block_n < 0 ||
      r.cta_group < 0 || (r.overlap_prev != 0 && r.overlap_prev != 1) || (r.split_k != 0 && r.split_k != 1) ||
      r.k_split < 0 || r.k_split > 8)
    return TLG_ERR_UNSUPPORTED;
  const int num_kb = static_cast<int>((K + kMxBK - 1) / kMxBK);
  out->tokens = 0;
  // Few rows of A.  A request for a cta_group, stages or max_ctas alone asks for tiles; beside the
  // kernel's block_n they have to be what it runs with, as in its own answer.
  const bool named = r.block_n != 0 && r.block_n == token_columns(M);
  if (named ? r.cta_group <= 1 && (r.stages == 0 || r.stages == MxTokenPlan<16>::kStages)
            : token_columns(M) != 0 && r.block_n == 0 && r.cta_group == 0 && r.stages == 0 && r.max_ctas == 0) {
    const int ks = r.k_split != 0 ? r.k_split : token_split(N, num_kb, sms);
    if ((ks & (ks - 1)) != 0 || ks > num_kb) return TLG_ERR_UNSUPPORTED;
    out->tile = nullptr;
    out->tokens = token_columns(M);
    out->units = static_cast<int>((N + 127) / 128);
    if (r.max_ctas != 0 && r.max_ctas < out->units * ks) return TLG_ERR_UNSUPPORTED;
    out->cfg = {out->tokens, MxTokenPlan<16>::kStages, 1, 1, out->units * ks, 1, 1, ks};
    return TLG_OK;
  }
  if (r.k_split > 1) return TLG_ERR_UNSUPPORTED;
  double best = 0;
  out->tile = nullptr;
  for (const MxTile &t : kTiles) {
    if ((r.cta_group != 0 && r.cta_group != t.cta_group) || (r.block_n != 0 && r.block_n != t.block_n) ||
        (r.stages != 0 && r.stages != t.stages))
      continue;
    int units = 0;
    const tlg_status us = t.fns[type][epi].units(dev, sms, &units);
    if (us != TLG_OK) return us;
    if (r.max_ctas > 0) units = std::max(1, std::min(units, r.max_ctas / t.cta_group));
    const int64_t tm = 128 * t.cta_group;
    const int64_t tiles = ((M + tm - 1) / tm) * ((N + t.block_n - 1) / t.block_n);
    units = static_cast<int>(std::min<int64_t>(units, tiles));
    // the busiest unit's tiles, one after the other
    const double tile_us = std::max(num_kb * t.cost.kb + t.cost.tile[epi], t.cost.least[epi]);
    const double cost = static_cast<double>((tiles + units - 1) / units) * tile_us;
    if (out->tile == nullptr || cost < best * 0.999) {
      best = cost;
      out->tile = &t;
      out->units = units;
    }
  }
  if (out->tile == nullptr) return TLG_ERR_UNSUPPORTED;
  tlg_config &c = out->cfg;
  c.block_n = out->tile->block_n;
  c.stages = out->tile->stages;
  c.cta_group = out->tile->cta_group;
  // Tile rows walked together: 32 for the 256 wide tile (8192^3 under the power cap: 220 us against
  // 226 with 8; 87 MB of DRAM reads against 150), 8 for the others, which do not care.
  c.raster_group = r.raster_group != 0 ? r.raster_group : (c.block_n == 256 ? 32 : 8);
  c.max_ctas = out->units * c.cta_group;
  c.split_k = 1;
  c.overlap_prev = 1;
  c.k_split = 1;
  return TLG_OK;
}

// Whether the epilogue is more than the plain product's.
bool has_work(const tlg_fused_epilogue *e) {
  return e != nullptr && (e->bias != nullptr || e->activation != TLG_ACT_NONE || e->residual != nullptr);
}

tlg_status check_sizes(int64_t M, int64_t N, int64_t K, int out) {
  if (!valid_type(out) || M < 0 || N < 0 || K < 0) return TLG_ERR_INVALID_ARG;
  if (M > kMaxExtent || N > kMaxExtent || K > kMaxExtent) return TLG_ERR_UNSUPPORTED;
  if (((M + 127) / 128) * ((N + 63) / 64) > kMaxExtent) return TLG_ERR_UNSUPPORTED;
  return TLG_OK;
}

}  // namespace

TLG_DEFINE_ERROR_WORD_READER(error_word_mxgemm)

}  // namespace tlg

using namespace tlg;

extern "C" {

tlg_status tlg_gemm_mxfp4(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, const void *SA, const void *B,
                          int64_t ldb, const void *SB, const tlg_fused_epilogue *epilogue, void *C, int64_t ldc,
                          tlg_type out, const tlg_config *config, void *stream) {
  tlg_status st = check_sizes(M, N, K, out);
  if (st != TLG_OK) return st;
  tlg_fused_epilogue e = {};
  if (epilogue != nullptr) e = *epilogue;
  if (!valid_activation(e.activation)) return TLG_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return TLG_OK;
  const int64_t osz = type_bytes(out);
  Range rc, rr, ra, rsa, rb, rsb;
  st = check_matrix(C, M, N, ldc, osz, &rc);
  if (st != TLG_OK) return st;
  if (K > 0) {
    st = check_mx(TLG_MX_E2M1, M, K, A, lda, SA, &ra, &rsa);
    if (st != TLG_OK) return st;
    st = check_mx(TLG_MX_E2M1, N, K, B, ldb, SB, &rb, &rsb);
    if (st != TLG_OK) return st;
    if (meets(rc, ra) || meets(rc, rsa) || meets(rc, rb) || meets(rc, rsb)) return TLG_ERR_INVALID_ARG;
  }
  if (e.bias != nullptr) {
    if (reinterpret_cast<uintptr_t>(e.bias) % 2 != 0) return TLG_ERR_ALIGNMENT;
    const uintptr_t b0 = reinterpret_cast<uintptr_t>(e.bias);
    if (meets(rc, Range{b0, b0 + static_cast<uintptr_t>(2 * N)})) return TLG_ERR_INVALID_ARG;
  }
  if (e.residual != nullptr) {
    st = check_matrix(e.residual, M, N, e.ldr, osz, &rr);
    if (st != TLG_OK) return st;
    if (meets(rc, rr) && !(e.residual == C && e.ldr == ldc)) return TLG_ERR_INVALID_ARG;
  }
  int dev = 0;
  DeviceInfo info;
  st = current_device(&dev, &info);
  if (st != TLG_OK) return st;
  for (const void *q : {static_cast<const void *>(C), K > 0 ? A : nullptr, K > 0 ? SA : nullptr, K > 0 ? B : nullptr,
                        K > 0 ? SB : nullptr, e.bias, e.residual})
    if (q != nullptr && !device_accessible(q, dev)) return TLG_ERR_INVALID_ARG;

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool epi = has_work(&e);
  MxGemmParams p = {};
  p.C = C;
  p.ldc = ldc;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.num_kb = static_cast<int>((K + kMxBK - 1) / kMxBK);
  p.n_aligned = (N * osz) % 16 == 0 ? 1 : 0;
  p.c_plain = (!aligned16(C) || (ldc * osz) % 16 != 0) ? 1 : 0;
  p.limit_ns = kWaitLimitNs;
  p.bias = e.bias;
  p.act = e.activation;
  p.R = e.residual;
  p.ldr = e.ldr;
  p.r_vec = (e.residual != nullptr && aligned16(e.residual) && (e.ldr * osz) % 16 == 0) ? 1 : 0;
  p.r_words = (reinterpret_cast<uintptr_t>(e.residual) % 4 == 0 && (e.ldr * osz) % 4 == 0) ? 1 : 0;
  if (K == 0) {
    const int64_t total = M * N;
    const int blocks = static_cast<int>(std::min<int64_t>((total + 255) / 256, 4096));
    if (out == TLG_TYPE_F32)
      mx_fill_empty_k_kernel<kTypeF32><<<blocks, 256, 0, s>>>(p);
    else if (out == TLG_TYPE_F16)
      mx_fill_empty_k_kernel<kTypeF16><<<blocks, 256, 0, s>>>(p);
    else
      mx_fill_empty_k_kernel<kTypeBF16><<<blocks, 256, 0, s>>>(p);
    if (cudaPeekAtLastError() != cudaSuccess) {
      cudaGetLastError();
      return TLG_ERR_CUDA;
    }
    return TLG_OK;
  }

  MxChoice c;
  st = choose(dev, info.sm_count, M, N, K, out, epi, config, &c);
  if (st != TLG_OK) return st;
  p.raster_group = c.cfg.raster_group;
  // Boxes (inner x outer): A 128 bytes (256 k) x 128 rows, B 128 bytes x the CTA's rows, scales
  // two tiles (256 words) x the 128-row groups a tile meets, C 64 bytes x 32 rows.
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8, u32 = CU_TENSOR_MAP_DATA_TYPE_UINT32;
  const uint64_t kbytes = static_cast<uint64_t>(row_bytes(TLG_MX_E2M1, K));
  if (M == 1) lda = static_cast<int64_t>(kbytes);  // the stride of a single row may be anything
  if (N == 1) ldb = static_cast<int64_t>(kbytes);
  const uint64_t tx = static_cast<uint64_t>(scale_tiles_x(K));
  // Rows of A and B in a box, and the 128-row scale groups of B a tile meets.
  const uint32_t a_rows = c.tokens != 0 ? static_cast<uint32_t>(c.tokens) : 128u;
  const uint32_t b_rows = c.tokens != 0 ? 128u : static_cast<uint32_t>(c.cfg.block_n / c.cfg.cta_group);
  const uint32_t b_groups = c.tokens == 0 && c.cfg.block_n > 128 ? 2u : 1u;
  MxMaps m;
  if (!encode_2d(&m.a, u8, A, kbytes, static_cast<uint64_t>(M), static_cast<uint64_t>(lda), 128, a_rows) ||
      !encode_2d(&m.b, u8, B, kbytes, static_cast<uint64_t>(N), static_cast<uint64_t>(ldb), 128, b_rows) ||
      !encode_2d(&m.sa, u32, SA, tx * 128, static_cast<uint64_t>((M + 127) / 128), tx * 512, 256, 1,
                 CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !encode_2d(&m.sb, u32, SB, tx * 128, static_cast<uint64_t>((N + 127) / 128), tx * 512, 256, b_groups,
                 CU_TENSOR_MAP_SWIZZLE_NONE))
    return TLG_ERR_CUDA;
  if (c.tokens != 0) {
    const int ks = c.cfg.k_split;
    return c.tokens == 16 ? launch_tokens_typed<16>(out, dev, c.units, ks, m, p, s)
                          : launch_tokens_typed<32>(out, dev, c.units, ks, m, p, s);
  }
  const CUtensorMapDataType ct = out == TLG_TYPE_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                 : out == TLG_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  auto stride = [&](int64_t ld) { return static_cast<uint64_t>(M == 1 ? (N * osz + 15) / 16 * 16 : ld * osz); };
  if (!p.c_plain && !encode_2d(&m.c, ct, C, static_cast<uint64_t>(N), static_cast<uint64_t>(M), stride(ldc),
                               static_cast<uint32_t>(64 / osz), 32, CU_TENSOR_MAP_SWIZZLE_64B))
    return TLG_ERR_CUDA;
  return c.tile->fns[out][epi].launch(c.units, m, p, s);
}

tlg_status tlg_choose_config_mxfp4_fused(int64_t M, int64_t N, int64_t K, const tlg_fused_epilogue *epilogue,
                                         tlg_type out, tlg_config *config) {
  if (config == nullptr) return TLG_ERR_INVALID_ARG;
  tlg_status st = check_sizes(M, N, K, out);
  if (st != TLG_OK) return st;
  if (epilogue != nullptr && !valid_activation(epilogue->activation)) return TLG_ERR_INVALID_ARG;
  int dev = 0;
  DeviceInfo info;
  st = current_device(&dev, &info);
  if (st != TLG_OK) return st;
  MxChoice c;
  const tlg_config req = *config;
  st = choose(dev, info.sm_count, std::max<int64_t>(M, 1), std::max<int64_t>(N, 1), std::max<int64_t>(K, 1), out,
              has_work(epilogue), &req, &c);
  if (st == TLG_OK) *config = c.cfg;
  return st;
}

tlg_status tlg_choose_config_mxfp4(int64_t M, int64_t N, int64_t K, tlg_type out, tlg_config *config) {
  return tlg_choose_config_mxfp4_fused(M, N, K, nullptr, out, config);
}

}  // extern "C"
