// Persistent, warp-specialised product of E2M1 (4-bit) MX matrices for sm_100a:
// C = act(A . B^T + bias) + residual, A M x K and B N x K, both with K contiguous and one E8M0
// scale per 32 k.  The tensor core applies the scales itself (tcgen05.mma.kind::mxf4 with
// block scaling): each product a * b * 2^(ea + eb) is exact and the sum is kept in fp32.
//
// The roles are the fp16 kernel's (tlg_gemm_kernel.cuh): a TMA producer warp, an MMA warp and
// epilogue warps (sixteen here) over a ring of operand slots and two TMEM accumulators.  What
// differs:
//
//  - A k-block is 256 elements, 128 bytes a row (one 128-byte swizzle row of 4-bit elements),
//    and four MMAs of 64 k.
//  - Beside the operand tiles a slot holds their scales: 1 KB per 128 rows (two scale tiles of
//    128 rows x 4 blocks).  The MMA lane copies them to TMEM (tcgen05.cp, which spreads a
//    tile's 512 bytes over 32 lanes x 4 columns and repeats them for the four lane groups)
//    right before the MMAs that use them.
//  - Every ring slot has TMEM columns of its own for its scales, so the wait for the slot's
//    bytes, which the producer only requested once the slot's earlier MMAs were done, also
//    covers overwriting the scales those MMAs read.
//
//  - The epilogue of a tile has to fit beside a main loop four times as short, and one warp
//    alone waits most of the time (for TMEM, shared memory, the special-function unit).  So
//    sixteen warps, four to a quarter of the rows, take 32 columns each time, little enough
//    for 96 registers, and copy the residual of a piece to shared memory while they compute its
//    activation.  With bias, GELU and residual, back to back: 4096^3 32 us, 16384 x 4096 x 1024
//    74; with eight warps, 64 columns and the residual read where it is added it was 3 and 24 us
//    more, with all pieces of a tile unrolled 1.5 and 14 more (code that did not stay in the
//    instruction cache).  Tried and dropped: ordinary stores from the box in place of TMA
//    stores, eight columns at a time in a rolled loop (17 and 28 us more at 16384 x 4096 x 1024).
//  - The 256-column accumulators overlap: TMEM holds two of 256 columns 128 apart and the
//    scales of five slots.  The epilogue drains the shared 128 columns first and hands them
//    back; the next tile's MMAs, into the other accumulator, start then.
//
// Tiles are 128 * CG rows by BN columns.  A tile's columns start at a multiple of 64, its
// scales at a multiple of 128 rows of B: for a start in the second half of a scale tile the
// MMA's scale address skips the two columns (of 32 rows of B each) before it.
#pragma once

#include "tlg_mx_device.cuh"

namespace tlg {

constexpr int kMxBK = 256;  // elements of a k-block
constexpr uint32_t kSfTileBytes = 512;  // 128 rows x 4 blocks

__device__ __forceinline__ uint64_t smem_desc_plain(uint32_t saddr) {
  // No swizzle; 8-row core matrices of 16-byte rows, 128 bytes apart.
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>(128u >> 4) << 16 |
         static_cast<uint64_t>(128u >> 4) << 32 | static_cast<uint64_t>(1u) << 46;
}

// Copies one scale tile (512 bytes of shared memory) to four TMEM columns.  With CG == 2 each
// CTA of the pair copies from its own shared memory to its own TMEM.
template <int CG>
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// D[tmem] (+)= (A x scales) . (B x scales) over 64 k; E2M1 operands, a scale per 32 k.
template <int CG>
__device__ __forceinline__ void mma_mxf4_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of tcgen05.mma.kind::mxf4 with block scaling, both operands K-major:
//   bits 4-5 which bytes of a TMEM scale word B uses (0: blocks 0 and 1; 2: blocks 2 and 3),
//   7-9 A format (1 = E2M1), 10-11 B format, 17-22 N >> 3, bit 23 scale format (1 = E8M0),
//   27-28 M >> 7, 29-30 as bits 4-5, for A.
__host__ __device__ constexpr uint32_t make_idesc_mxf4(int m, int n, int sf) {
  return (static_cast<uint32_t>(sf) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (1u << 23) | (static_cast<uint32_t>(m >> 7) << 27) | (static_cast<uint32_t>(sf) << 29);
}

struct MxGemmParams {
  void *C;
  int64_t ldc;
  int M, N;
  int num_kb;        // k-blocks of 256
  int raster_group;  // tile rows walked together
  int n_aligned;     // N * sizeof(out) is a multiple of 16: every box may go through TMA
  int c_plain;       // C cannot be written by TMA
  uint64_t limit_ns;
  const void *bias;  // 16-bit: bf16 for a bf16 C, else fp16
  int act;
  const void *R;     // residual in C's type, or nullptr; may be C itself (same ldc)
  int64_t ldr;
  int r_vec;         // R's base and row stride are 16-byte aligned
  int r_words;       // and 4-byte aligned
};

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

constexpr int kMxEpiWarps = 16;  // four to a quarter of the tile's rows, taking its 32-column pieces in turn
constexpr uint32_t kMxBoxBytes = 32 * 64;  // an epilogue warp's box: 32 rows x 64 bytes
constexpr int kMxThreads = 32 * (2 + kMxEpiWarps);

template <int CG, int BN, int STAGES>
struct MxPlan {
  static constexpr int kBNc = BN / CG;                 // B rows held by one CTA
  static constexpr int kGroups = BN <= 128 ? 1 : 2;    // 128-row groups of B's scales a tile meets
  static constexpr uint32_t kABytes = kBM * 128;
  static constexpr uint32_t kBBytes = kBNc * 128;
  static constexpr uint32_t kSfaBytes = 2 * kSfTileBytes;
  static constexpr uint32_t kSfbBytes = kGroups * 2 * kSfTileBytes;
  static constexpr uint32_t kStageBytes = kABytes + kBBytes + kSfaBytes + kSfbBytes;
  static constexpr uint32_t kBOffset = STAGES * kABytes;
  static constexpr uint32_t kSfOffset = kBOffset + STAGES * kBBytes;
  static constexpr uint32_t kOutOffset = kSfOffset + STAGES * (kSfaBytes + kSfbBytes);
  static constexpr uint32_t kBiasOffset = kOutOffset + kMxEpiWarps * kMxBoxBytes;
  static constexpr uint32_t kBarOffset = kBiasOffset + kMxEpiWarps * 128;  // each warp's 32 columns of bias in fp32
  static constexpr uint32_t kNumBars = 2 * STAGES + 4 + 1;
  static constexpr uint32_t kMiscOffset = kBarOffset + kNumBars * 8;
  static constexpr uint32_t kDynamicBytes = kMiscOffset + 16 + 1024;
  static constexpr int kSfCols = 8 + 8 * kGroups;      // TMEM columns of one slot's scales
  static constexpr bool kOverlap = BN == 256;          // the two accumulators share columns
  static constexpr int kAccStride = kOverlap ? 128 : BN;
  static constexpr int kAccBars = kOverlap ? 1 : 2;
  static constexpr int kSf0 = kAccStride + BN;
  static constexpr uint32_t kTmemCols = kSf0 + STAGES * kSfCols <= 256 ? 256 : 512;
  static_assert(kSf0 + STAGES * kSfCols <= 512, "accumulators and scales must fit in TMEM");
  static_assert(kBBytes % 1024 == 0, "operand tiles are 1024-byte aligned");
  static_assert(BN % 64 == 0 && BN <= 256, "tile columns start in the first or second half of a scale tile");
  static_assert(kDynamicBytes <= 232448, "shared memory per CTA exceeded");
};

template <int OUT>
__device__ __forceinline__ float load_elem(const void *p, int64_t i) {
  if constexpr (OUT == kTypeF32) {
    return static_cast<const float *>(p)[i];
  } else if constexpr (OUT == kTypeF16) {
    return __half2float(static_cast<const __half *>(p)[i]);
  } else {
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
  }
}

template <int OUT>
__device__ __forceinline__ void store_elem(void *p, int64_t i, float v) {
  if constexpr (OUT == kTypeF32)
    static_cast<float *>(p)[i] = v;
  else if constexpr (OUT == kTypeF16)
    static_cast<__half *>(p)[i] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// Type of the bias beside a C of type OUT.
template <int OUT>
constexpr int kBiasType = OUT == kTypeBF16 ? kTypeBF16 : kTypeF16;

// A bias element as loaded; converted where it is used, so that the load is not waited for before.
template <int OUT>
__device__ __forceinline__ float bias_value(uint16_t bits) {
  if constexpr (OUT == kTypeBF16)
    return __uint_as_float(static_cast<uint32_t>(bits) << 16);
  else
    return __half2float(__ushort_as_half(bits));
}

// The residual of a warp's 32 rows goes through its output box, 64 bytes of a row at a time, copied
// there asynchronously while bias and activation are computed.  Tried and dropped: loaded to
// registers a piece ahead (tcgen05.wait::ld waits for ordinary loads in flight too, and the
// registers spill: fp32 C at 16384 x 4096 x 1024 156 us against 141), the tile's residual
// prefetched to L2 by the producer (4096^3 from DRAM with bias and GELU: 39.3 us against 38.2).
// R may be C: the warp reads these elements before it stores them.
//
// Byte `byte` of row r of a box: 16-byte piece c of a row sits at (c ^ (r / 2 % 4)) * 16, so that
// eight lanes on eight rows, or on two whole rows, meet all banks.
__device__ __forceinline__ uint32_t box_at(uint32_t box, int r, int byte) {
  return box + static_cast<uint32_t>(r * 64 + (((byte / 16) ^ ((r >> 1) & 3)) * 16) + byte % 16);
}

// Starts the copy in pieces of BYTES, neighbouring lanes on neighbouring pieces; zeros beyond R.
template <int OUT, int BYTES>
__device__ __forceinline__ void mx_copy_box(const MxGemmParams &p, int row0, int col0, int lane, uint32_t box) {
  constexpr int kLanes = 64 / BYTES;  // to a row
  const int byte = lane % kLanes * BYTES;
  // Counted in elements first: a row of R may hold more than 2^31 bytes.
  const int cols = min(p.N - col0, 64 / kTypeBytes<OUT>);
  const int left = max(0, min(BYTES, cols * kTypeBytes<OUT> - byte));
  const char *q = static_cast<const char *>(p.R) + (static_cast<int64_t>(row0) * p.ldr + col0) * kTypeBytes<OUT> + byte;
#pragma unroll 4
  for (int r = lane / kLanes; r < 32; r += 32 / kLanes) {
    const int size = row0 + r < p.M ? left : 0;
    const void *from = size > 0 ? q + r * p.ldr * kTypeBytes<OUT> : p.R;
    if constexpr (BYTES == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(box_at(box, r, byte)), "l"(from), "r"(size)
                   : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(box_at(box, r, byte)), "l"(from), "r"(size)
                   : "memory");
  }
}

// box: read by all lanes before this.
template <int OUT>
__device__ __forceinline__ void mx_fetch_residual(const MxGemmParams &p, int row0, int col0, int lane, uint32_t box) {
  if (p.r_vec) {
    mx_copy_box<OUT, 16>(p, row0, col0, lane, box);
  } else if (kTypeBytes<OUT> == 4 || p.r_words) {
    mx_copy_box<OUT, 4>(p, row0, col0, lane, box);
  } else {  // 16-bit elements at odd places: too small for an asynchronous copy
    constexpr int kBatch = 4;
    const bool in = col0 + lane < p.N;
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += kBatch) {
      const uint16_t *q = static_cast<const uint16_t *>(p.R) + static_cast<int64_t>(row0 + r0) * p.ldr + col0 + lane;
      uint16_t y[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) y[i] = in && row0 + r0 + i < p.M ? q[i * p.ldr] : uint16_t(0);
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(box_at(box, r0 + i, lane * 2)), "h"(y[i]) : "memory");
    }
  }
}

// Adds what mx_fetch_residual brought to the piece's columns [16 h, ..) (fp32) or to all 32.
template <int OUT>
__device__ __forceinline__ void mx_add_residual(int h, int lane, uint32_t box, float (&v)[32]) {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint4 y = ld_shared_v4(box_at(box, lane, c * 16));
    const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (OUT == kTypeF32) {
        v[16 * h + 4 * c + k] += __uint_as_float(w[k]);
      } else if constexpr (OUT == kTypeF16) {
        add_half2_to(v[8 * c + 2 * k], v[8 * c + 2 * k + 1], w[k]);
      } else {
        float lo, hi;
        unpack2<OUT>(w[k], lo, hi);
        f2_add_to(v[8 * c + 2 * k], v[8 * c + 2 * k + 1], lo, hi);
      }
    }
  }
}

// Writes one 64-byte row piece of a 32-row box.
__device__ __forceinline__ void st_box_row_64(uint32_t box, int r, const uint32_t *w) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box_at(box, r, c * 16)),
                 "r"(w[4 * c]), "r"(w[4 * c + 1]), "r"(w[4 * c + 2]), "r"(w[4 * c + 3])
                 : "memory");
}

// Writes a warp's box (32 rows x 64 bytes, C's rows row0 .. and columns col0 ..) to a C that TMA
// cannot store, element by element, neighbouring lanes on neighbouring columns.
template <int OUT>
__device__ __forceinline__ void mx_store_box(const MxGemmParams &p, int row0, int col0, int lane, uint32_t box) {
  constexpr int B = kTypeBytes<OUT>;
  constexpr int kCols = 64 / B;  // of the box
  const int cc = lane % kCols;
#pragma unroll 4
  for (int r = lane / kCols; r < 32; r += 32 / kCols) {
    const uint32_t at = box_at(box, r, cc * B);
    if (row0 + r < p.M && col0 + cc < p.N) {
      const int64_t to = static_cast<int64_t>(row0 + r) * p.ldc + col0 + cc;
      if constexpr (B == 4) {
        uint32_t y;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(y) : "r"(at) : "memory");
        static_cast<uint32_t *>(p.C)[to] = y;
      } else {
        uint16_t y;
        asm volatile("ld.shared.b16 %0, [%1];" : "=h"(y) : "r"(at) : "memory");
        static_cast<uint16_t *>(p.C)[to] = y;
      }
    }
  }
}

// Tells the pair's MMA warp that this warp has read its TMEM columns (tcgen05.wait::ld, then
// tcgen05.fence::before_thread_sync, come before it).  Nothing in memory is handed over, so the
// arrival is relaxed: a release at cluster scope waits for the warp's earlier memory traffic, up
// to 3000 cycles a tile under load (16384 x 4096 x 1024 with 256 x 192 tiles).
__device__ __forceinline__ void mbar_arrive_drained(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

template <int CG, int BN, int STAGES, int OUT, bool EPI>
__global__ void __launch_bounds__(kMxThreads, 1)
    mxgemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                  const __grid_constant__ CUtensorMap tmC, const MxGemmParams p) {
  using Plan = MxPlan<CG, BN, STAGES>;
  constexpr int kTileM = kBM * CG;
  constexpr int G = Plan::kGroups;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t s0 = smem_u32(smem);
  auto a_slot = [&](int s) { return s0 + s * Plan::kABytes; };
  auto b_slot = [&](int s) { return s0 + Plan::kBOffset + s * Plan::kBBytes; };
  auto sfa_slot = [&](int s) { return s0 + Plan::kSfOffset + s * (Plan::kSfaBytes + Plan::kSfbBytes); };
  const uint32_t bar0 = s0 + Plan::kBarOffset;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);
  uint32_t *misc = reinterpret_cast<uint32_t *>(smem + Plan::kMiscOffset);
  volatile uint32_t *abort_flag = misc + 1;

  // Shuffled from lane 0: the same in every lane, and known to be.
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = (CG == 2) ? __shfl_sync(0xffffffffu, cluster_ctarank(), 0) : 0u;
  const bool leader = rank == 0;
  const int unit = CG == 2 ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int num_units = CG == 2 ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);
  const int num_m = (p.M + kTileM - 1) / kTileM;
  const int num_n = (p.N + BN - 1) / BN;
  const int tiles = num_m * num_n;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), kMxEpiWarps * CG);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
    if (!p.c_plain) tma_prefetch_desc(&tmC);
  }
  if (warp == 1) {
    tmem_alloc<CG>(smem_u32(misc), Plan::kTmemCols);
    tmem_relinquish<CG>();
  }
  tc_fence_before_sync();
  __syncwarp();
  if constexpr (CG == 2)
    cluster_sync_all();
  else
    __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(misc);
  grid_dependency_wait();  // global memory is touched only after this
  grid_launch_dependents();

  if (warp == 0) {
    // ---------------------------------------------------------------- producer (every CTA)
    int stage = 0;
    uint32_t phase = 0;
    uint32_t issued_mask = 0, issued_parity = 0;
    bool ok = true;
    for (int t = unit; t < tiles && ok; t += num_units) {
      int mb, nb;
      tile_coords(t, num_m, num_n, p.raster_group, mb, nb);
      const int a_row = mb * kTileM + static_cast<int>(rank) * kBM;
      const int b_row = nb * BN + static_cast<int>(rank) * Plan::kBNc;
      for (int kb = 0; kb < p.num_kb; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait_spin(empty_bar(stage), phase ^ 1u, abort_flag, p.limit_ns,
                                                    kRoleProducer, &g_device_error, 4096));
        if (!ok) break;
        if (elect_one()) {
          uint32_t bar;
          if constexpr (CG == 1) {
            bar = full_bar(stage);
            mbar_arrive_expect_tx(bar, Plan::kStageBytes);
          } else {
            if (leader) mbar_arrive_expect_tx(full_bar(stage), 2 * Plan::kStageBytes);
            bar = mapa_shared(full_bar(stage), 0);
          }
          auto load = [&](uint32_t dst, const CUtensorMap *tm, int32_t x, int32_t y) {
            if constexpr (CG == 1)
              tma_load_2d(dst, tm, bar, x, y);
            else
              tma_load_2d_pair(dst, tm, bar, x, y);
          };
          load(a_slot(stage), &tmA, kb * 128, a_row);
          load(b_slot(stage), &tmB, kb * 128, b_row);
          load(sfa_slot(stage), &tmSA, kb * 256, a_row / 128);  // 256 words: two scale tiles
          load(sfa_slot(stage) + Plan::kSfaBytes, &tmSB, kb * 256, nb * BN / 128);
        }
        __syncwarp();
        issued_mask |= 1u << stage;
        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (ok) {
      // Wait until every slot has been released: no commit-arrive is still on its way.
      for (int i = 0; i < STAGES && ok; ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.limit_ns, kRoleProducer,
                                               &g_device_error));
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && leader) {
      // Let the copies already issued land before shared memory goes away.
      for (int s = 0; s < STAGES; ++s)
        if (issued_mask & (1u << s))
          mbar_wait(full_bar(s), (issued_parity >> s) & 1u, nullptr, p.limit_ns, kRoleProducer, &g_device_error);
    }
  } else if (warp == 1 && leader) {
    // ---------------------------------------------------------------- MMA issuer (leader CTA)
    constexpr uint32_t idesc[2] = {make_idesc_mxf4(kTileM, BN, 0), make_idesc_mxf4(kTileM, BN, 2)};
    int stage = 0;
    uint32_t phase = 0;
    int acc = 0;
    uint32_t j = 0;  // tiles done
    bool ok = true;
    for (int t = unit; t < tiles && ok; t += num_units, ++j) {
      int mb, nb;
      tile_coords(t, num_m, num_n, p.raster_group, mb, nb);
      const uint32_t skip = static_cast<uint32_t>((nb * BN) % 128 / 32);
      // Two accumulators apart: each waits for its own last drain.  Overlapping ones: tile j
      // waits for the shared columns of tile j - 1, and so for everything before them.
      ok = __all_sync(0xffffffffu, mbar_wait(tempty_bar(j % Plan::kAccBars), ((j / Plan::kAccBars) & 1u) ^ 1u,
                                             abort_flag, p.limit_ns, kRoleMma, &g_device_error));
      if (!ok) break;
      tc_fence_after_sync();
      const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * Plan::kAccStride);
      for (int kb = 0; kb < p.num_kb; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait_spin(full_bar(stage), phase, abort_flag, p.limit_ns, kRoleMma,
                                                    &g_device_error, 4096));
        if (!ok) break;
        tc_fence_after_sync();
        if (elect_one()) {
          const uint32_t sfa = tmem_base + static_cast<uint32_t>(Plan::kSf0 + stage * Plan::kSfCols);
          const uint32_t sfb = sfa + 8;
          const uint64_t sf_desc = smem_desc_plain(sfa_slot(stage));
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // the two scale tiles (128 k each)
            tmem_copy_scales<CG>(sfa + 4 * h, sf_desc + h * (kSfTileBytes / 16));
#pragma unroll
            for (int g = 0; g < G; ++g)
              tmem_copy_scales<CG>(sfb + 4 * (h * G + g),
                                   sf_desc + (Plan::kSfaBytes + (g * 2 + h) * kSfTileBytes) / 16);
          }
          const uint64_t ad = smem_desc_sw128(a_slot(stage), 16, 1024);
          const uint64_t bd = smem_desc_sw128(b_slot(stage), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 64 k: 32 bytes along the swizzled row
            mma_mxf4_ss<CG>(d_tmem, ad + kk * 2, bd + kk * 2, idesc[kk & 1], sfa + 4 * (kk >> 1),
                            sfb + 4 * G * (kk >> 1) + skip, (kb > 0 || kk > 0) ? 1u : 0u);
          mma_commit<CG>(empty_bar(stage));
        }
        __syncwarp();
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (elect_one()) mma_commit<CG>(tfull_bar(j % Plan::kAccBars));
      __syncwarp();
      acc ^= 1;
    }
    if (!ok) {
      if (elect_one()) mma_commit_local<CG>(drain_bar);
      __syncwarp();
      mbar_wait(drain_bar, 0, nullptr, p.limit_ns, kRoleMma, &g_device_error);
    }
  } else if (warp >= 2) {
    // ---------------------------------------------------------------- epilogue (every CTA)
    // Warp w drains TMEM lanes 32*(w%4) .. +31, 32 columns at a time, by way of a 2 KB box.  The
    // four warps of a quarter take its pieces in turn; where there are two or six pieces, the pair
    // of warps with a piece more changes from tile to tile.
    const int quarter = warp & 3;
    const int ew = warp - 2;
    const int side = ew >> 2;
    constexpr int kPieces = BN / 32;
    static_assert(kPieces % 2 == 0, "pieces go to pairs of warps");
    auto first_piece = [&](uint32_t tile) { return kPieces % 4 != 0 && (tile & 1u) != 0 ? side ^ 2 : side; };
    const uint32_t box = s0 + Plan::kOutOffset + static_cast<uint32_t>(ew) * kMxBoxBytes;
    const uint32_t release_bar0 = (CG == 2) ? mapa_shared(tempty_bar(0), 0) : tempty_bar(0);
    constexpr int kBoxCols = 64 / kTypeBytes<OUT>;  // 32 columns of a 16-bit type, 16 of fp32
    uint32_t j = 0;
    const uint64_t tile_limit_ns = p.limit_ns + static_cast<uint64_t>(p.num_kb) * kWaitPerKBlockNs;
    // First row of this warp and first column of tile t; the tile column of piece i.
    int row0 = 0, col_t = 0;
    auto place = [&](int t) {
      int mb, nb;
      tile_coords(t, num_m, num_n, p.raster_group, mb, nb);
      row0 = mb * kTileM + static_cast<int>(rank) * kBM + quarter * 32;
      col_t = nb * BN;
    };
    auto piece_col = [&](int i, uint32_t tile) {
      // Overlapping accumulators: the shared columns (the upper half of accumulator 0, the lower
      // of accumulator 1) first.
      return 32 * (Plan::kOverlap && (tile & 1u) == 0 ? (i + 4) % 8 : i);
    };
    // The bias of this warp's next piece is loaded while it works on this one.
    uint16_t ahead = 0;
    auto load_bias = [&](int col) {
      if (p.bias != nullptr && col + lane < p.N) ahead = static_cast<const uint16_t *>(p.bias)[col + lane];
    };
    const uint32_t sbias = s0 + Plan::kBiasOffset + static_cast<uint32_t>(ew) * 128u;
    if (unit < tiles) place(unit);
    if (EPI && unit < tiles && side < kPieces) load_bias(col_t + piece_col(side, 0));
    for (int t = unit; t < tiles; t += num_units, ++j) {
      // On a timeout the warp stops reading tiles.
      bool ok = *abort_flag == 0u;
      if (ok && !mbar_wait(tfull_bar(j % Plan::kAccBars), (j / Plan::kAccBars) & 1u, abort_flag, tile_limit_ns,
                           kRoleEpilogue, &g_device_error))
        ok = false;
      ok = __all_sync(0xffffffffu, ok);
      const int tile_row0 = row0, tile_col = col_t;
      if (t + num_units < tiles) place(t + num_units);  // where the next bias comes from
      if (!ok) continue;
      tc_fence_after_sync();
      auto release = [&]() {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2)
            mbar_arrive_drained(release_bar0 + 8u * (j % Plan::kAccBars));
          else
            mbar_arrive(release_bar0 + 8u * (j % Plan::kAccBars));
        }
      };
      const int first = first_piece(j), next = first_piece(j + 1);
      auto load_ahead = [&](int i) {  // for the piece after piece i of this tile
        const bool here = i + 4 < kPieces;
        if (EPI && (here || (t + num_units < tiles && next < kPieces)))
          load_bias(here ? tile_col + piece_col(i + 4, j) : col_t + piece_col(next, j + 1));
      };
      if (first >= kPieces) {
        release();
        load_ahead(kPieces);
      }
#pragma unroll 1
      for (int i = first; i < kPieces; i += 4) {
        const int tc = piece_col(i, j);
        const int col0 = tile_col + tc;
        const uint32_t acc = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                             static_cast<uint32_t>((j & 1u) * Plan::kAccStride + tc);
        const bool releases = Plan::kOverlap ? i < 4 : i + 4 >= kPieces;
        const bool inside = tile_row0 < p.M && col0 < p.N;
        auto box_free = [&]() {  // its last store has read it, and so has every lane
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
        };
        float v[32];
        {
          uint32_t r[32];
          __syncwarp();
          tmem_load_32cols(acc, r);
          if (releases) release();
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c] = __uint_as_float(r[c]);
        }
        if constexpr (EPI) {
          if (inside) {
            if (p.R != nullptr) {
              box_free();
              mx_fetch_residual<OUT>(p, tile_row0, col0, lane, box);
            }
            if (p.bias != nullptr) {
              st_shared_u32(sbias + static_cast<uint32_t>(lane * 4), __float_as_uint(bias_value<OUT>(ahead)));
              __syncwarp();
              add_bias_smem_32(sbias, 0, v);
            }
            activate_lane<OUT, 32>(p.act, v);
            if (p.R != nullptr) {
              mx_add_residual<OUT>(0, lane, box, v);
              if constexpr (OUT == kTypeF32) {
                __syncwarp();
                mx_fetch_residual<OUT>(p, tile_row0, col0 + 16, lane, box);
                mx_add_residual<OUT>(1, lane, box, v);
              }
            }
            __syncwarp();  // every lane has read the bias
          }
          load_ahead(i);
        }
        if (!inside) continue;
#pragma unroll
        for (int h = 0; h < 32 / kBoxCols; ++h) {
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            if constexpr (OUT == kTypeF32)
              w[c] = __float_as_uint(v[16 * h + c]);
            else
              w[c] = pack2<OUT>(v[2 * c], v[2 * c + 1]);
          }
          box_free();
          st_box_row_64(box, lane, w);
          const int c0 = col0 + h * kBoxCols;
          if (p.c_plain || (!p.n_aligned && c0 + kBoxCols > p.N)) {
            __syncwarp();
            mx_store_box<OUT>(p, tile_row0, c0, lane, box);
          } else {
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0 && c0 < p.N) {
              tma_store_2d(&tmC, box, c0, tile_row0);
              bulk_commit_group();
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();  // every store of this warp has completed
    __syncwarp();
  }

  tc_fence_before_sync();
  __syncwarp();
  if constexpr (CG == 2)
    cluster_sync_all();
  else
    __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc<CG>(tmem_base, Plan::kTmemCols);
  }
}

// ------------------------------------------------------------------ few rows of A (tokens)

// The same product for M <= BN <= 32 rows of A, where reading B (the weights) once is all the
// work: the roles are swapped, 128 rows of B being the MMA's M and the rows of A its N, so a
// single token costs 16 columns of an MMA and not a 128-row tile.  A cluster of KS CTAs (its size)
// shares the K range of every 128 rows of B, so that few rows of B still keep most SMs
// loading; each CTA adds the KS fp32 partial sums of its 128 / KS rows in slice order, received
// through distributed shared memory, and writes them.  Measured back to back in a graph, one
// token: 4096 x 4096 weights 3.6 us with KS = 4 (6.4 with KS = 1, 7.0 with 128-row tiles),
// 16384 x 4096 6.7 us with KS = 1 (11 with 128-row tiles; its bytes take 5.5 us).  At 64 rows of
// A and 16384 x 4096 weights, tiles enough for every SM, the 128-row tiles win (6.6 against 8.7 us).
template <int BN>
struct MxTokenPlan {
  static constexpr int kStages = 4;
  static constexpr uint32_t kWBytes = kBM * 128;
  static constexpr uint32_t kTBytes = BN * 128;
  static constexpr uint32_t kSfBytes = 4 * kSfTileBytes;  // two scale tiles of each operand
  static constexpr uint32_t kStageBytes = kWBytes + kTBytes + kSfBytes;
  static constexpr uint32_t kTOffset = kStages * kWBytes;
  static constexpr uint32_t kSfOffset = kTOffset + kStages * kTBytes;
  static constexpr uint32_t kRecvOffset = kSfOffset + kStages * kSfBytes;
  // Partial sums [slice][row of this CTA][token], fp32; the pad keeps 16-byte accesses of
  // neighbouring rows in different banks.
  static constexpr int kRecvRow = BN + 4;
  static constexpr uint32_t kRecvBytes = kBM * kRecvRow * 4;
  static constexpr uint32_t kBarOffset = kRecvOffset + kRecvBytes;
  static constexpr uint32_t kNumBars = 2 * kStages + 2;
  static constexpr uint32_t kMiscOffset = kBarOffset + kNumBars * 8;
  static constexpr uint32_t kDynamicBytes = kMiscOffset + 16 + 1024;
  static constexpr int kSf0 = 32;  // after the accumulator
  static constexpr uint32_t kTmemCols = 128;
  static_assert(BN <= kSf0 && kSf0 + 16 * kStages <= kTmemCols, "accumulator and scales must fit");
  static_assert(kDynamicBytes <= 232448, "shared memory per CTA exceeded");
};

// The two halves of a cluster barrier (see cluster_sync_all).
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// tmT: the tokens (A), tmW: the weights (B), tmST / tmSW their scales.  The grid is
// ceil(N / 128) clusters of KS CTAs.
template <int BN, int OUT>
__global__ void __launch_bounds__(kThreads, 1)
    mxgemm_tokens_kernel(const __grid_constant__ CUtensorMap tmT, const __grid_constant__ CUtensorMap tmW,
                         const __grid_constant__ CUtensorMap tmST, const __grid_constant__ CUtensorMap tmSW,
                         const MxGemmParams p, const int ks) {
  using Plan = MxTokenPlan<BN>;
  constexpr int ST = Plan::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t s0 = smem_u32(smem);
  auto w_slot = [&](int s) { return s0 + s * Plan::kWBytes; };
  auto t_slot = [&](int s) { return s0 + Plan::kTOffset + s * Plan::kTBytes; };
  auto sf_slot = [&](int s) { return s0 + Plan::kSfOffset + s * Plan::kSfBytes; };
  const uint32_t bar0 = s0 + Plan::kBarOffset;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (ST + s); };
  const uint32_t done_bar = bar0 + 8u * (2 * ST);
  const uint32_t drain_bar = bar0 + 8u * (2 * ST + 1);
  uint32_t *misc = reinterpret_cast<uint32_t *>(smem + Plan::kMiscOffset);
  volatile uint32_t *abort_flag = misc + 1;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const int slice = ks > 1 ? static_cast<int>(__shfl_sync(0xffffffffu, cluster_ctarank(), 0)) : 0;
  const int tile = static_cast<int>(blockIdx.x) / ks;
  const int kb0 = static_cast<int>(static_cast<int64_t>(slice) * p.num_kb / ks);
  const int kb1 = static_cast<int>(static_cast<int64_t>(slice + 1) * p.num_kb / ks);

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(done_bar, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&tmT);
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmST);
    tma_prefetch_desc(&tmSW);
  }
  if (warp == 1) {
    tmem_alloc<1>(smem_u32(misc), Plan::kTmemCols);
    tmem_relinquish<1>();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(misc);
  if (ks > 1) cluster_arrive();  // this CTA runs: its shared memory may be written
  grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    uint32_t issued_mask = 0, issued_parity = 0;
    bool ok = true;
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      ok = __all_sync(0xffffffffu, mbar_wait_spin(empty_bar(stage), phase ^ 1u, abort_flag, p.limit_ns, kRoleProducer,
                                                  &g_device_error, 4096));
      if (!ok) break;
      if (elect_one()) {
        const uint32_t bar = full_bar(stage);
        mbar_arrive_expect_tx(bar, Plan::kStageBytes);
        tma_load_2d(w_slot(stage), &tmW, bar, kb * 128, tile * 128);
        tma_load_2d(sf_slot(stage), &tmSW, bar, kb * 256, tile);
        tma_load_2d(t_slot(stage), &tmT, bar, kb * 128, 0);
        tma_load_2d(sf_slot(stage) + 2 * kSfTileBytes, &tmST, bar, kb * 256, 0);
      }
      __syncwarp();
      issued_mask |= 1u << stage;
      issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
      if (++stage == ST) {
        stage = 0;
        phase ^= 1u;
      }
    }
    for (int i = 0; i < ST && ok; ++i) {  // no commit-arrive is still on its way
      ok = __all_sync(0xffffffffu, mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.limit_ns, kRoleProducer,
                                             &g_device_error));
      if (++stage == ST) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok) {
      for (int s = 0; s < ST; ++s)
        if (issued_mask & (1u << s))
          mbar_wait(full_bar(s), (issued_parity >> s) & 1u, nullptr, p.limit_ns, kRoleProducer, &g_device_error);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc[2] = {make_idesc_mxf4(128, BN, 0), make_idesc_mxf4(128, BN, 2)};
    bool ok = true;
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      ok = __all_sync(0xffffffffu, mbar_wait_spin(full_bar(stage), phase, abort_flag, p.limit_ns, kRoleMma,
                                                  &g_device_error, 4096));
      if (!ok) break;
      tc_fence_after_sync();
      if (elect_one()) {
        const uint32_t sfa = tmem_base + static_cast<uint32_t>(Plan::kSf0 + stage * 16);
        const uint32_t sfb = sfa + 8;
        const uint64_t sf_desc = smem_desc_plain(sf_slot(stage));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          tmem_copy_scales<1>(sfa + 4 * h, sf_desc + h * (kSfTileBytes / 16));
          tmem_copy_scales<1>(sfb + 4 * h, sf_desc + (2 + h) * (kSfTileBytes / 16));
        }
        const uint64_t wd = smem_desc_sw128(w_slot(stage), 16, 1024);
        const uint64_t td = smem_desc_sw128(t_slot(stage), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_mxf4_ss<1>(tmem_base, wd + kk * 2, td + kk * 2, idesc[kk & 1], sfa + 4 * (kk >> 1),
                         sfb + 4 * (kk >> 1), (kb > kb0 || kk > 0) ? 1u : 0u);
        mma_commit<1>(empty_bar(stage));
        if (kb + 1 == kb1) mma_commit<1>(done_bar);
      }
      __syncwarp();
      if (++stage == ST) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok) {
      if (elect_one()) mma_commit_local<1>(drain_bar);
      __syncwarp();
      mbar_wait(drain_bar, 0, nullptr, p.limit_ns, kRoleMma, &g_device_error);
    }
  }

  // ---------------------------------------------------------------- reduction and epilogue
  // Warps 2..5 hold the accumulator: lane = row of B, column = token.
  const int shift = 31 - __clz(kBM / ks);  // log2 of the rows of B this CTA finishes
  const int rows_per = 1 << shift;
  const uint32_t recv0 = s0 + Plan::kRecvOffset;
  const int tid = static_cast<int>(threadIdx.x) - 64;
  auto bias_of = [&](int col) {
    return p.bias != nullptr && col < p.N ? load_elem<kBiasType<OUT>>(p.bias, col) : 0.0f;
  };
  __syncwarp();
  if (ks > 1) cluster_wait();  // every CTA of the cluster runs
  if (warp >= 2) {
    const uint64_t tile_limit_ns = p.limit_ns + static_cast<uint64_t>(kb1 - kb0) * kWaitPerKBlockNs;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const float bias = ks == 1 ? bias_of(tile * kBM + row) : 0.0f;
    const bool have =
        __all_sync(0xffffffffu, mbar_wait(done_bar, 0, abort_flag, tile_limit_ns, kRoleEpilogue, &g_device_error));
    if (have) {
      tc_fence_after_sync();
      uint32_t r[32];
      tmem_load_32cols(tmem_base + (static_cast<uint32_t>(quarter * 32) << 16), r);
      if (ks == 1) {
        // The activation over all tokens at once: its code runs from a cold instruction cache, so
        // what counts is its length (per token, unrolled: 8.7 us at 16 tokens, 16384 x 4096).
        const int col = tile * kBM + row;
        float v[BN];
#pragma unroll
        for (int j = 0; j < BN; ++j) v[j] = __uint_as_float(r[j]) + bias;
        activate_lane<OUT, BN>(p.act, v);
        if (col < p.N) {
          if (p.R != nullptr) {
#pragma unroll
            for (int j = 0; j < BN; ++j)
              if (j < p.M) v[j] += load_elem<OUT>(p.R, j * p.ldr + col);
          }
#pragma unroll
          for (int j = 0; j < BN; ++j)
            if (j < p.M) store_elem<OUT>(p.C, j * p.ldc + col, v[j]);
        }
      } else {
        const uint32_t dst =
            mapa_shared(recv0, static_cast<uint32_t>(row >> shift)) +
            static_cast<uint32_t>(((slice << shift) + (row & (rows_per - 1))) * Plan::kRecvRow * 4);
#pragma unroll
        for (int j = 0; j < BN; j += 4)
          if (j < p.M) st_cluster_v4(dst + static_cast<uint32_t>(j * 4), r[j], r[j + 1], r[j + 2], r[j + 3]);
      }
    }
    tc_fence_before_sync();
  }
  __syncwarp();
  if (ks > 1)
    cluster_sync_all();  // all partial sums are in place
  else
    __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc<1>(tmem_base, Plan::kTmemCols);
  if (ks == 1 || tid < 0 || *abort_flag != 0u) return;
  // This CTA's rows of B by the tokens: a thread keeps one row and takes every ks-th four tokens.
  const int col = tile * kBM + (slice << shift) + (tid & (rows_per - 1));
  if (col >= p.N) return;
  const float bias = bias_of(col);
  const uint32_t mine = recv0 + static_cast<uint32_t>((tid & (rows_per - 1)) * Plan::kRecvRow * 4);
  const uint32_t slice_bytes = static_cast<uint32_t>((Plan::kRecvRow * 4) << shift);
  for (int t0 = (tid >> shift) * 4; t0 < p.M; t0 += ks * 4) {
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int q = 0; q < ks; ++q) {
      const uint4 x = ld_shared_v4(mine + static_cast<uint32_t>(q) * slice_bytes + static_cast<uint32_t>(t0 * 4));
      f2_add_to(v[0], v[1], __uint_as_float(x.x), __uint_as_float(x.y));
      f2_add_to(v[2], v[3], __uint_as_float(x.z), __uint_as_float(x.w));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += bias;
    activate_lane<OUT, 4>(p.act, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t token = t0 + j;
      if (token < p.M) {
        if (p.R != nullptr) v[j] += load_elem<OUT>(p.R, token * p.ldr + col);
        store_elem<OUT>(p.C, token * p.ldc + col, v[j]);
      }
    }
  }
}

// K == 0: C = act(bias[col]) + R[row, col] (each element read and written by one thread).
template <int OUT>
__global__ void mx_fill_empty_k_kernel(const MxGemmParams p) {
  grid_dependency_wait();
  const int64_t total = static_cast<int64_t>(p.M) * p.N;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = i / p.N, c = i % p.N;
    float v = p.bias != nullptr ? load_elem<kBiasType<OUT>>(p.bias, c) : 0.0f;
    v = activate<OUT != kTypeF32>(p.act, v);
    if (p.R != nullptr) v += load_elem<OUT>(p.R, r * p.ldr + c);
    store_elem<OUT>(p.C, r * p.ldc + c, v);
  }
}

}  // namespace tlg
