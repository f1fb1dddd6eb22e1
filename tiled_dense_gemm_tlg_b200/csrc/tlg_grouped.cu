// Host side of the products grouped by expert: argument checks, the choice of tile and the launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "tlg.h"
#include "tlg_grouped_kernel.cuh"
#include "tlg_mx_host.cuh"
#include "tlg_variants.cuh"

namespace tlg {

namespace {

constexpr uint64_t kWaitLimitNs = 1000000000ull;  // 1 s per pipeline wait
// What the next launches are given; tests make waits run out with less.
std::atomic<uint64_t> wait_limit_ns{kWaitLimitNs}, wait_limit_kb_ns{kWaitPerKBlockNs};
constexpr int64_t kMostTiles = int64_t(1) << 30;
constexpr int64_t kMaxStackStride = int64_t(1) << 38;

struct GroupedMaps {
  CUtensorMap w = {}, x = {}, x128 = {};
};

template <int KIND, int CG, int BN, int STAGES, int TYPE, int OUT, bool LSU, bool KSPLIT = false>
struct GroupedVariant {
  using Plan = GroupedPlan<CG, BN, STAGES>;
  static constexpr auto kKernel = grouped_kernel<KIND, CG, BN, STAGES, TYPE, OUT, LSU, KSPLIT>;

  static void fill(cudaLaunchConfig_t *cfg, cudaLaunchAttribute *attr, int ctas, int cluster, cudaStream_t s) {
    *cfg = {};
    cfg->gridDim = dim3(static_cast<unsigned>(ctas));
    cfg->blockDim = dim3(GroupedRoles<OUT, BN, LSU>::kThreads);
    cfg->dynamicSmemBytes = Plan::kDynamicBytes;
    cfg->stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg->attrs = attr;
    cfg->numAttrs = cluster > 1 ? 2 : 1;
  }

  // ks: CTAs that share a tile (KSPLIT).
  static tlg_status launch(int dev, int sms, int64_t most_tiles, const GroupedMaps &m, const GroupedParams &p,
                           cudaStream_t s, int ks = 1) {
    static LaunchState state[kMaxDevices];
    static std::mutex mutex;
    int units;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    {
      std::lock_guard<std::mutex> lock(mutex);
      LaunchState &st = state[dev];
      if (!st.ready) {
        if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan::kDynamicBytes) !=
            cudaSuccess) {
          cudaGetLastError();
          return TLG_ERR_CUDA;
        }
        st.units = sms * Plan::kCtasPerSm;
        if (CG > 1) {
          fill(&cfg, attr, CG * (sms / CG), CG, nullptr);
          if (cudaOccupancyMaxActiveClusters(&st.units, kKernel, &cfg) != cudaSuccess || st.units < 1) {
            cudaGetLastError();
            return TLG_ERR_CUDA;
          }
        }
        st.ready = true;
      }
      units = st.units;
    }
    if (KSPLIT)
      fill(&cfg, attr, ks * static_cast<int>(most_tiles), ks, s);
    else
      fill(&cfg, attr, CG * static_cast<int>(std::min<int64_t>(units, most_tiles)), CG, s);
    if (cudaLaunchKernelEx(&cfg, kKernel, m.w, m.x, m.x128, p) != cudaSuccess) {
      cudaGetLastError();
      return TLG_ERR_CUDA;
    }
    return TLG_OK;
  }
};

template <typename F>
tlg_status with_types(int type, int out, F f) {
  using F16 = std::integral_constant<int, kTypeF16>;
  using BF16 = std::integral_constant<int, kTypeBF16>;
  using F32 = std::integral_constant<int, kTypeF32>;
  if (type == TLG_TYPE_F16) return out == TLG_TYPE_F32 ? f(F16(), F32()) : f(F16(), F16());
  return out == TLG_TYPE_F32 ? f(BF16(), F32()) : f(BF16(), BF16());
}

tlg_status check_call(int64_t rows, int64_t N, int64_t K, int64_t groups, int type, int op, int out) {
  if (rows < 0 || N < 0 || K < 0 || groups < 0 || (op != TLG_OP_N && op != TLG_OP_T)) return TLG_ERR_INVALID_ARG;
  if (type != TLG_TYPE_F16 && type != TLG_TYPE_BF16) return TLG_ERR_INVALID_ARG;
  if (out != TLG_TYPE_F32 && out != type) return TLG_ERR_INVALID_ARG;
  if (rows > kMaxExtent || N > kMaxExtent || K > kMaxExtent || groups > kGroupedMax) return TLG_ERR_UNSUPPORTED;
  return TLG_OK;
}

// groups matrices of rows x cols, `stride` elements apart.
tlg_status check_stack(const void *p, int64_t groups, int64_t rows, int64_t cols, int64_t ld, int64_t stride,
                       int64_t esz, Range *r) {
  const tlg_status st = check_matrix(p, rows, cols, ld, esz, r);
  if (st != TLG_OK) return st;
  if (groups > 1) {
    if (stride < 0) return TLG_ERR_INVALID_ARG;
    if (stride > kMaxStackStride) return TLG_ERR_UNSUPPORTED;
    r->hi += static_cast<uintptr_t>((groups - 1) * stride * esz);
  }
  return TLG_OK;
}

tlg_status check_offsets(const int32_t *offsets, int64_t groups, Range *r) {
  if (offsets == nullptr) return TLG_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(offsets) % 4 != 0) return TLG_ERR_ALIGNMENT;
  r->lo = reinterpret_cast<uintptr_t>(offsets);
  r->hi = r->lo + static_cast<uintptr_t>(groups + 1) * 4;
  return TLG_OK;
}

// The stride of a single row may be anything; TMA wants a multiple of 16 bytes.
int64_t tma_ld(int64_t rows, int64_t cols, int64_t ld) { return rows > 1 ? ld : (cols + 7) / 8 * 8; }

bool tma_ok(const void *p, int64_t ld) { return aligned16(p) && ld % 8 == 0; }

}  // namespace

TLG_DEFINE_ERROR_WORD_READER(error_word_grouped)

}  // namespace tlg

using namespace tlg;

extern "C" {

// Not part of the interface, for tests: the limit of the pipeline waits of the grouped products launched from here on,
// and what a k-block adds to it.  A limit of 0 restores both.
void tlg_internal_grouped_wait_limit(uint64_t limit_ns, uint64_t per_k_block_ns) {
  wait_limit_ns = limit_ns != 0 ? limit_ns : kWaitLimitNs;
  wait_limit_kb_ns = limit_ns != 0 ? per_k_block_ns : kWaitPerKBlockNs;
}

tlg_status tlg_gemm_grouped(int64_t rows, int64_t N, int64_t K, int32_t groups, const int32_t *offsets, tlg_type type,
                            const void *A, int64_t lda, tlg_op op_b, const void *B, int64_t ldb, int64_t stride_b,
                            tlg_activation activation, void *C, int64_t ldc, tlg_type out, void *stream) {
  tlg_status st = check_call(rows, N, K, groups, type, op_b, out);
  if (st != TLG_OK) return st;
  if (!valid_activation(activation)) return TLG_ERR_INVALID_ARG;
  if (rows == 0 || N == 0 || groups == 0) return TLG_OK;
  const bool t = op_b == TLG_OP_T;
  const int64_t b_rows = t ? N : K, b_cols = t ? K : N;
  Range ra = {0, 0}, rb = {0, 0}, rc, ro;
  st = check_matrix(C, rows, N, ldc, type_bytes(out), &rc);
  if (st != TLG_OK) return st;
  st = check_offsets(offsets, groups, &ro);
  if (st != TLG_OK) return st;
  if (K > 0) {
    st = check_matrix(A, rows, K, lda, 2, &ra);
    if (st != TLG_OK) return st;
    st = check_stack(B, groups, b_rows, b_cols, ldb, stride_b, 2, &rb);
    if (st != TLG_OK) return st;
  }
  if (meets(rc, ro) || (K > 0 && (meets(rc, ra) || meets(rc, rb)))) return TLG_ERR_INVALID_ARG;
  int dev = 0;
  DeviceInfo info;
  st = current_device(&dev, &info);
  if (st != TLG_OK) return st;
  for (const void *q : {static_cast<const void *>(C), static_cast<const void *>(offsets), K > 0 ? A : nullptr, K > 0 ? B : nullptr})
    if (q != nullptr && !device_accessible(q, dev)) return TLG_ERR_INVALID_ARG;
  GroupedParams p = {};
  p.offsets = offsets;
  p.groups = groups;
  p.rows = static_cast<int>(rows);
  p.lanes = static_cast<int>(N);
  p.inner = static_cast<int>(K);
  p.C = C;
  p.ldc = ldc;
  p.raster = 8;
  p.act = activation;
  p.shared_w = groups == 1 || stride_b == 0;
  p.limit_ns = wait_limit_ns;
  p.limit_kb_ns = wait_limit_kb_ns;
  p.W = static_cast<const uint16_t *>(B);
  p.X = static_cast<const uint16_t *>(A);
  p.ldw = ldb;
  p.ldx = lda;
  p.stride_w = p.shared_w ? 0 : stride_b;
  // At most this many tiles of `bn` rows by `bl` columns.
  auto most = [&](int64_t bn, int64_t bl) { return (rows / bn + std::min<int64_t>(groups, rows)) * ((N + bl - 1) / bl); };
  if (most(64, 128) > kMostTiles) return TLG_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  GroupedMaps m;
  const int64_t tlda = tma_ld(rows, K, lda), tldb = tma_ld(b_rows, b_cols, ldb);
  // Tiles of 128 lanes by up to 64 rows, two CTAs to an SM, up to 16 rows a group on average, then pairs with 256 x 256.
  // 8 groups of 4096 x 4096, bf16, small tiles against pairs: 16 rows a group 46.4 us against 49.3, 20 rows 46.7 against
  // 49.6.  As long as no group takes a second small tile the pairs are 5 % slower; where one does, the small tiles read
  // its weights again: 32 rows a group on average, most of them in one group, 57.0 us against 52.9, 48 rows spread
  // unevenly 61.7 against 50.9.  The sizes are on the device, so the average has to decide, and 16 is on the side that
  // loses little.  Where the small tiles are few, clusters share their K.
  const bool few = most(64, 128) * 2 <= 2 * int64_t(info.sm_count) && K >= 2 * 4 * kBK;
  const bool wide = !few && rows > int64_t(groups) * 16;
  const bool tma = K > 0 && tma_ok(A, tlda) && tma_ok(B, tldb) && p.stride_w % 8 == 0;
  if (tma) {
    const CUtensorMapDataType ty =
        type == TLG_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t mats = p.shared_w ? 1 : static_cast<uint64_t>(groups);
    const uint64_t mat_bytes = static_cast<uint64_t>(p.shared_w ? tldb : stride_b) * 2;
    if (!encode_3d(&m.w, ty, B, static_cast<uint64_t>(b_cols), static_cast<uint64_t>(b_rows), mats,
                   static_cast<uint64_t>(tldb) * 2, mat_bytes, 64, t ? 128 : 64) ||
        !encode_2d(&m.x, ty, A, static_cast<uint64_t>(K), static_cast<uint64_t>(rows), static_cast<uint64_t>(tlda) * 2, 64, wide ? 32 : 16) ||
        !encode_2d(&m.x128, ty, A, static_cast<uint64_t>(K), static_cast<uint64_t>(rows), static_cast<uint64_t>(tlda) * 2, 64, 128))
      return TLG_ERR_CUDA;
  }
  return with_types(type, out, [&](auto TY, auto OU) {
    constexpr int kTy = decltype(TY)::value, kOu = decltype(OU)::value;
    auto run = [&](auto kind) {
      constexpr int kKind = decltype(kind)::value;
      if (!tma)
        return GroupedVariant<kKind, 1, 128, 6, kTy, kOu, true>::launch(dev, info.sm_count, most(128, 128), m, p, s);
      if (wide)
        return GroupedVariant<kKind, 2, 256, 6, kTy, kOu, false>::launch(dev, info.sm_count, most(256, 256), m, p, s);
      // With few tiles each CTA's ring, 64 KB in flight, sets the pace (64 tiles of K = 4096: 23 us, 15.8 with
      // four CTAs to a tile; its bytes take 10): more CTAs to a tile while two to an SM suffice and each has
      // a ring's worth of k-blocks.
      int ks = 1;
      while (ks < 8 && most(64, 128) * ks * 2 <= 2 * int64_t(info.sm_count) && K >= int64_t(ks) * 2 * 4 * kBK) ks *= 2;
      if (ks > 1)
        return GroupedVariant<kKind, 1, 64, 4, kTy, kOu, false, true>::launch(dev, info.sm_count, most(64, 128), m, p, s, ks);
      return GroupedVariant<kKind, 1, 64, 4, kTy, kOu, false>::launch(dev, info.sm_count, most(64, 128), m, p, s);
    };
    return t ? run(std::integral_constant<int, kGroupedT>()) : run(std::integral_constant<int, kGroupedN>());
  });
}

tlg_status tlg_gemm_grouped_dw(int64_t rows, int64_t N, int64_t K, int32_t groups, const int32_t *offsets,
                               tlg_type type, const void *A, int64_t lda, const void *dC, int64_t lddc, tlg_op op_b,
                               void *dB, int64_t lddb, int64_t stride_db, tlg_type out, void *stream) {
  tlg_status st = check_call(rows, N, K, groups, type, op_b, out);
  if (st != TLG_OK) return st;
  if (N == 0 || K == 0 || groups == 0) return TLG_OK;
  const bool t = op_b == TLG_OP_T;
  const int64_t b_rows = t ? N : K, b_cols = t ? K : N;
  Range ra = {0, 0}, rd = {0, 0}, rb, ro;
  st = check_stack(dB, groups, b_rows, b_cols, lddb, stride_db, type_bytes(out), &rb);
  if (st != TLG_OK) return st;
  if (groups > 1 && stride_db < (b_rows - 1) * lddb + b_cols) return TLG_ERR_INVALID_ARG;  // they would overlap
  st = check_offsets(offsets, groups, &ro);
  if (st != TLG_OK) return st;
  if (rows > 0) {
    st = check_matrix(A, rows, K, lda, 2, &ra);
    if (st != TLG_OK) return st;
    st = check_matrix(dC, rows, N, lddc, 2, &rd);
    if (st != TLG_OK) return st;
  }
  if (meets(rb, ro) || (rows > 0 && (meets(rb, ra) || meets(rb, rd)))) return TLG_ERR_INVALID_ARG;
  int dev = 0;
  DeviceInfo info;
  st = current_device(&dev, &info);
  if (st != TLG_OK) return st;
  for (const void *q : {static_cast<const void *>(dB), static_cast<const void *>(offsets), rows > 0 ? A : nullptr, rows > 0 ? dC : nullptr})
    if (q != nullptr && !device_accessible(q, dev)) return TLG_ERR_INVALID_ARG;
  // dB_g (K x N) = A_g^T . dC_g with the columns of dC on the lanes; its transpose with those of A.
  const void *W = t ? A : dC, *X = t ? dC : A;
  const int64_t ldw = t ? lda : lddc, ldx = t ? lddc : lda;
  GroupedParams p = {};
  p.offsets = offsets;
  p.groups = groups;
  p.rows = static_cast<int>(rows);
  p.lanes = static_cast<int>(b_cols);
  p.inner = static_cast<int>(b_rows);
  p.C = dB;
  p.ldc = lddb;
  p.stride_c = stride_db;
  p.raster = 8;
  p.limit_ns = wait_limit_ns;
  p.limit_kb_ns = wait_limit_kb_ns;
  p.W = static_cast<const uint16_t *>(W);
  p.X = static_cast<const uint16_t *>(X);
  p.ldw = ldw;
  p.ldx = ldx;
  auto most = [&](int64_t bn, int64_t bl) {
    return int64_t(groups) * ((b_rows + bn - 1) / bn) * ((b_cols + bl - 1) / bl);
  };
  if (most(128, 128) > kMostTiles) return TLG_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  GroupedMaps m;
  const int64_t tldw = tma_ld(rows, b_cols, ldw), tldx = tma_ld(rows, b_rows, ldx);
  const bool tma = rows > 0 && tma_ok(W, tldw) && tma_ok(X, tldx);
  if (tma) {
    const CUtensorMapDataType ty =
        type == TLG_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if (!encode_2d(&m.w, ty, W, static_cast<uint64_t>(b_cols), static_cast<uint64_t>(rows), static_cast<uint64_t>(tldw) * 2, 64, 64) ||
        !encode_2d(&m.x, ty, X, static_cast<uint64_t>(b_rows), static_cast<uint64_t>(rows), static_cast<uint64_t>(tldx) * 2, 64, 64))
      return TLG_ERR_CUDA;
  }
  return with_types(type, out, [&](auto TY, auto OU) {
    constexpr int kTy = decltype(TY)::value, kOu = decltype(OU)::value;
    if (!tma)
      return GroupedVariant<kGroupedDw, 1, 128, 6, kTy, kOu, true>::launch(dev, info.sm_count, most(128, 128), m, p, s);
    return GroupedVariant<kGroupedDw, 2, 256, 6, kTy, kOu, false>::launch(dev, info.sm_count, most(256, 256), m, p, s);
  });
}

}  // extern "C"
