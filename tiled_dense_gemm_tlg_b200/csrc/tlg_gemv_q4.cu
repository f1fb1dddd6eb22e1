// Products of a few rows (tokens) with integer 4-bit weights:
//
//   C = act(X . W^T + bias) + residual,  W[n, k] = (q[n, k] - z[n, k / group]) s[n, k / group]
//
// Reading the weights (half a byte each) is all the work there is for one token, so the kernel is built
// around a stream of weights: a CTA takes a block of W's rows, its warps share K in units of 256
// or 128, and TMA brings their units (128 or 64 bytes of a row, and the tokens' elements) into a ring of each
// group of warps, without any barrier across the CTA until the groups' sums are added at the end.
//
// The products run on the tensor core (mma.sync m16n8k16, W's rows as its M, tokens as its N): eight
// tokens at a time cost what one does, and the CUDA cores, which convert 4 bits to 16, have no time for
// the products as well.  (tcgen05 reads its operands from shared memory: the converted weights, four
// times the bytes, would have to go there first.)  Conversion: the four bits of an element placed in the
// mantissa of 1024 (fp16) or 128 (bf16) make 1024 + q, and subtracting 1024 + z is exact.  Products of
// q - z with X are exact in fp32 and summed in fp32 over a group; the scale multiplies the group's sum,
// in fp32, so no weight is rounded.
//
// A lane holds word t of a 32-element block of rows g and g + 8 (t = lane % 4, g = lane / 4), so a word's eight
// elements i and i + 4 are pairs of one mma operand register: the k order of the operands is a permutation,
// the same for X, whose pairs are put together by byte permutes.
//
// What bounds it: latency with few warps.  127 registers a thread and the rings leave 14 warps to an SM; they issue 1.8 of
// 4 instructions a cycle (16 tokens, 16384 x 4096), tensor pipe, shared memory and DRAM are at a fifth to a third.  Of
// the 7.7 cycles from one instruction of a warp to its next 1.6 go to memory (units that have not landed, the panel's
// scales), 1.4 to the latency of the instruction before, 1.0 to a busy pipe, 0.6 to barriers; the rest is issue.  And 256
// tiles on 296 places leave some SMs with one where others have two.  About 50 instructions stand for 512 weights (16
// rows by 32 k), 22 of them the conversion.  bf16, groups of 128, back to back in a graph: one token 4096 x 4096 4.6 us,
// 16384 x 4096 11.4 us (2.9 TB/s of weights), eight tokens 12.1, sixteen 16.0.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "tlg.h"
#include "tlg_mxgemm_kernel.cuh"
#include "tlg_rows.cuh"
#include "tlg_variants.cuh"

namespace tlg {
namespace {

constexpr uint64_t kWaitLimitNs = 1000000000ull;  // 1 s per pipeline wait
constexpr int kQ4Warps = 8;
constexpr int kQ4Panel = 64;     // groups whose scales are held in shared memory at a time

struct Q4Params {
  const uint8_t *Q;
  int64_t ldq;
  const uint16_t *S;
  const uint8_t *Z;  // or nullptr: 8
  const uint16_t *X;
  int64_t ldx;
  int M, N, K;
  int group_log2, groups;
  int x_vec;  // X may be read 16 bytes at a time
  int x_tma;  // and comes by TMA
  int token_blocks;
  void *C;
  int64_t ldc;
  int out_f32;
  const void *bias;  // X's type
  int act;
  const void *R;     // C's type
  int64_t ldr;
};

// (v & mask) | magic in one instruction: both constants in registers.
__device__ __forceinline__ uint32_t q4_place(uint32_t v, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(magic));
  return r;
}

template <int T>
__device__ __forceinline__ uint32_t q4_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (T == kTypeF16)
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int T>
__device__ __forceinline__ void q4_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const float (&c)[4]) {
  if constexpr (T == kTypeF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Shared memory of a CTA: WK rings of ST slots, each a unit of kRows rows of W and of 8 NT tokens (boxes of 64
// elements), the panel's scales, and the barriers.  NT == 0: a single token, which all columns of the
// products share.
template <int NT, int R, int WK>
struct Q4Plan {
  static constexpr int kWR = kQ4Warps / WK;  // warps that share a ring
  static constexpr int kRows = kWR * 16 * R;
  static constexpr int kTokens = NT == 0 ? 1 : 8 * NT;
  static constexpr int kBlocks = NT == 2 ? 4 : 8;  // of 32 k in a unit
  static constexpr int kUnit = kBlocks * 32;
  static constexpr int kStages = NT == 0 && R == 1 ? 4 : NT == 2 && WK == 4 ? 3 : 2;
  static constexpr uint32_t kWRow = kBlocks * 16;
  static constexpr uint32_t kWBytes = kRows * kWRow;
  static constexpr uint32_t kXBox = NT * 1024;
  static constexpr uint32_t kXBytes = NT == 0 ? kUnit * 2 : kBlocks / 2 * kXBox;
  static constexpr uint32_t kXOffset = WK * kStages * kWBytes;
  static constexpr uint32_t kScaleOffset = kXOffset + WK * kStages * kXBytes;
  // Row stride of the scales, in words; odd, so that eight rows lie in different banks.
  static constexpr uint32_t kScaleLd = kQ4Panel + 1;
  static constexpr uint32_t kBarOffset = kScaleOffset + (kRows * kScaleLd * 4 + 7) / 8 * 8;
  static constexpr uint32_t kDynamicBytes = kBarOffset + WK * kStages * 16 + 16;
  static_assert(kWBytes % 1024 == 0 && (NT == 0 || kXBytes % 1024 == 0), "swizzled boxes are 1024-byte aligned");
  static_assert(2 * (kDynamicBytes + 1024) <= 233472, "two CTAs to an SM");
  static_assert(kXOffset >= WK * kRows * kTokens * 4, "the rings' sums fit them");
};

// NT: blocks of 8 tokens, 0 for one token; R: blocks of 16 rows of W to a warp; WK: groups of warps that
// share K, each of kWR warps with a ring of its own; GC: blocks of 32 k that have one scale (1, 2, 4).
template <int T, int NT, int R, int WK, int GC>
__global__ void __launch_bounds__(32 * kQ4Warps, 2)
    gemv_q4_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Q4Params p) {
  using Plan = Q4Plan<NT, R, WK>;
  constexpr int ST = Plan::kStages, WR = Plan::kWR, kRows = Plan::kRows, kUnit = Plan::kUnit;
  constexpr int NC = NT == 0 ? 1 : NT;  // blocks of 8 columns
  constexpr uint32_t kMagic = T == kTypeF16 ? 0x64006400u : 0x43004300u;
  extern __shared__ __align__(1024) uint8_t q4_smem[];
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int wr = warp % WR, wk = warp / WR;
  const int g = lane >> 2, t = lane & 3;
  const int tile = static_cast<int>(blockIdx.x) / p.token_blocks;
  const int token0 = (static_cast<int>(blockIdx.x) - tile * p.token_blocks) * Plan::kTokens;
  const int tokens = min(p.M - token0, Plan::kTokens);
  const int n0 = tile * kRows;
  const uint32_t s0 = smem_u32(q4_smem);
  auto w_slot = [&](int s) { return s0 + static_cast<uint32_t>(wk * ST + s) * Plan::kWBytes; };
  auto x_slot = [&](int s) { return s0 + Plan::kXOffset + static_cast<uint32_t>(wk * ST + s) * Plan::kXBytes; };
  auto full_bar = [&](int s) { return s0 + Plan::kBarOffset + static_cast<uint32_t>((wk * ST + s) * 16); };
  auto empty_bar = [&](int s) { return full_bar(s) + 8u; };
  // a word for each row and group: the scale's bits low, the zero point high
  uint32_t *scales = reinterpret_cast<uint32_t *>(q4_smem + Plan::kScaleOffset);
  volatile uint32_t *abort_flag = reinterpret_cast<uint32_t *>(q4_smem + Plan::kDynamicBytes - 16);

  if (lane == 0 && wr == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), WR);
    }
    if (warp == 0) *abort_flag = 0u;
    fence_mbar_init();
    if (p.K > 0) tma_prefetch_desc(&tmW);
    if (p.K > 0 && p.x_tma) tma_prefetch_desc(&tmX);
  }
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();

  const int units = (p.K + kUnit - 1) / kUnit;
  const int mine = units > wk ? (units - wk + WK - 1) / WK : 0;  // units wk, wk + WK, ..
  // X comes by TMA where it may and the unit is whole.
  auto tma_x = [&](int i) { return p.x_tma != 0 && (wk + i * WK + 1) * kUnit <= p.K; };
  // One lane of the group asks for its i-th unit; TMA fills with zeros what lies outside the matrices.
  auto issue = [&](int i, int slot) {
    const int k = (wk + i * WK) * kUnit;
    const uint32_t bar = full_bar(slot);
    mbar_arrive_expect_tx(bar, Plan::kWBytes + (tma_x(i) ? Plan::kXBytes : 0u));
    tma_load_2d(w_slot(slot), &tmW, bar, k / 2, n0);
    if (tma_x(i)) {
      if constexpr (NT == 0) {
        tma_load_2d(x_slot(slot), &tmX, bar, k, token0);
      } else {
#pragma unroll
        for (int b = 0; b < Plan::kBlocks / 2; ++b)
          tma_load_2d(x_slot(slot) + b * Plan::kXBox, &tmX, bar, k + b * 64, token0);
      }
    }
  };
  const bool issuer = wr == 0 && lane == 0;
  if (issuer) {
    for (int i = 0; i < min(ST, mine); ++i) issue(i, i);
  }
  // Without TMA: the group's lanes write the unit's X as TMA would have.
  auto fill_x = [&](int i, int slot) {
    constexpr int kPieces = kUnit / 8;  // of 16 bytes, of a token
    constexpr int kMine = (Plan::kTokens * kPieces + WR * 32 - 1) / (WR * 32), kBatch = kMine < 8 ? kMine : 8;
    const uint32_t x = x_slot(slot);
    const int k0 = (wk + i * WK) * kUnit;
    for (int b0 = 0; b0 < kMine; b0 += kBatch) {
      uint4 v[kBatch];  // a batch's loads are in flight together
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int e = (b0 + b) * WR * 32 + wr * 32 + lane, m = e / kPieces, k = k0 + e % kPieces * 8;
        const uint16_t *from = p.X + static_cast<int64_t>(token0 + m) * p.ldx + k;
        const int left = m < tokens ? min(max(p.K - k, 0), 8) : 0;
        v[b] = make_uint4(0, 0, 0, 0);
        if (p.x_vec && left == 8) {
          v[b] = __ldg(reinterpret_cast<const uint4 *>(from));
        } else if (left > 0) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            w[j] = ld_u16_pred(from + 2 * j, 2 * j < left) | ld_u16_pred(from + 2 * j + 1, 2 * j + 1 < left) << 16;
          v[b] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int e = (b0 + b) * WR * 32 + wr * 32 + lane, m = e / kPieces, q = e % kPieces;
        const uint32_t to = NT == 0 ? x + q * 16
                                    : x + (q >> 3) * Plan::kXBox + static_cast<uint32_t>(m * 128 + (((q & 7) ^ (m & 7)) * 16));
        if (e < Plan::kTokens * kPieces)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(v[b].x), "r"(v[b].y), "r"(v[b].z), "r"(v[b].w)
                       : "memory");
      }
    }
  };
  if (mine > 0 && mine <= ST && !tma_x(mine - 1)) fill_x(mine - 1, mine - 1);  // under the wait for the scales
  // Whether the i-th unit's X is written by the lanes when its turn comes.
  auto by_lanes = [&](int i) { return !tma_x(i) && !(mine <= ST && i == mine - 1); };
  auto group_sync = [&]() {
    if constexpr (WR == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + wk), "n"(WR * 32) : "memory");
  };

  // What a lane reads of a slot: word t of block c of W's rows g, g + 8, .., and 8 elements of block c of a
  // token; the block's place is an exclusive-or of address bits (the boxes' swizzle).  Column g of the
  // products is token 4 (g % 2) + g / 2: the two tokens of a quarter-warp then lie in different banks.
  const int col_token = 4 * (g & 1) + (g >> 1);
  const uint32_t w_at = static_cast<uint32_t>((wr * 16 * R + g) * Plan::kWRow + (Plan::kBlocks == 8 ? g : (g >> 1) & 3) * 16 + t * 4);
  const uint32_t x_at = NT == 0 ? t * 16 : static_cast<uint32_t>(col_token * 128 + (t ^ col_token) * 16);

  // The row whose sums this thread finishes, and its bias, loaded ahead of their use.
  static_assert(32 * kQ4Warps % kRows == 0, "a thread keeps its row");
  const int last_row = static_cast<int>(threadIdx.x) % kRows;
  const float bias = p.bias != nullptr && n0 + last_row < p.N ? load_elem<T>(p.bias, n0 + last_row) : 0.0f;

  float total[R][NC][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) total[r][n][j] = 0.0f;

  const int panel_units = max(1, static_cast<int>(std::min<int64_t>(int64_t(kQ4Panel) << p.group_log2, int64_t(1) << 30) / kUnit));
  // opaque, so that they stay in registers
  uint32_t mask = 0x000f000fu, magic = kMagic;
  asm volatile("" : "+r"(mask), "+r"(magic));
  bool ok = true;
  int slot = 0, i = 0;
  uint32_t phase = 0;
  for (int u0 = 0; u0 < units; u0 += panel_units) {
    const int u1 = min(units, u0 + panel_units);
    const int first_group = static_cast<int>((static_cast<int64_t>(u0) * kUnit) >> p.group_log2);
    if (u0 > 0) __syncthreads();  // the last panel's scales are read
    // scales and zero points of the panel, 0 past the last row: a warp takes an eighth of the rows, all
    // loads of 32 groups in flight at once
    const int held = min(p.groups - first_group, kQ4Panel);
    for (int j = lane; j < (held + 7) / 8 * 8; j += 32) {  // a unit's blocks past K have no group: their scale is 0
      constexpr int kMine = kRows / kQ4Warps;
      uint32_t v[kMine], z[kMine];
#pragma unroll
      for (int r = 0; r < kMine; ++r) {
        const int n = n0 + warp * kMine + r;
        const int64_t at = static_cast<int64_t>(n) * p.groups + first_group + j;
        v[r] = n < p.N && j < held ? p.S[at] : 0u;
        z[r] = 8;
      }
      if (p.Z != nullptr) {
#pragma unroll
        for (int r = 0; r < kMine; ++r) {
          const int n = n0 + warp * kMine + r;
          if (n < p.N && j < held) z[r] = p.Z[static_cast<int64_t>(n) * p.groups + first_group + j];
        }
      }
#pragma unroll
      for (int r = 0; r < kMine; ++r) scales[(warp * kMine + r) * Plan::kScaleLd + j] = v[r] | (z[r] & 15u) << 16;
    }
    __syncthreads();
    for (; ok && wk + i * WK < u1; ++i) {
      const int u = wk + i * WK;
      // Refills the slot of the unit before this one, which the group has had time to leave.
      if (issuer && i > 0 && i - 1 + ST < mine) {
        const int last = slot == 0 ? ST - 1 : slot - 1;
        const uint32_t last_phase = slot == 0 ? phase ^ 1u : phase;
        ok = mbar_wait(empty_bar(last), last_phase, abort_flag, kWaitLimitNs, kRoleProducer, &g_device_error);
        if (ok) issue(i - 1 + ST, last);
      }
      ok = __all_sync(0xffffffffu, ok && mbar_wait(full_bar(slot), phase, abort_flag, kWaitLimitNs, kRoleMma, &g_device_error));
      if (!ok) break;
      if (by_lanes(i)) {
        fill_x(i, slot);
        group_sync();
      }
      const uint32_t w = w_slot(slot) + w_at, x = x_slot(slot) + x_at;
      const uint32_t *unit_scales = scales + (wr * 16 * R + g) * Plan::kScaleLd + ((u * kUnit) >> p.group_log2) - first_group;
      float acc[R][NC][4];
      uint32_t zero[R][2];
      float scale[R][2];
#pragma unroll
      for (int c = 0; c < Plan::kBlocks; ++c) {
        if (c % GC == 0) {
          const uint32_t *s = unit_scales + (GC < 4 ? c / GC : (c * 32) >> p.group_log2);
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t v = s[(r * 16 + h * 8) * Plan::kScaleLd];
              zero[r][h] = kMagic + (v >> 16) * 0x10001u;
              float none;
              unpack2<T>(v, scale[r][h], none);
            }
        }
        uint32_t b[NC][4];
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const uint4 v = ld_shared_v4(NT == 0 ? x + c * 64 : (x ^ ((c & 1) * 64)) + (c >> 1) * Plan::kXBox + n * 1024);
          b[n][0] = __byte_perm(v.x, v.z, 0x5410);  // elements 0 and 4
          b[n][1] = __byte_perm(v.x, v.z, 0x7632);  // 1 and 5
          b[n][2] = __byte_perm(v.y, v.w, 0x5410);  // 2 and 6
          b[n][3] = __byte_perm(v.y, v.w, 0x7632);  // 3 and 7
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          uint32_t a[2][4];  // [half of the block][operand register]
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t v = ld_shared_u32((w ^ (c * 16)) + (r * 16 + h * 8) * Plan::kWRow);
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i >> 1][h + 2 * (i & 1)] = q4_sub<T>(q4_place(v >> (4 * i), mask, magic), zero[r][h]);
          }
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (c % GC == 0)
              q4_mma<T>(acc[r][n], a[0], b[n][0], b[n][1], none);
            else
              q4_mma<T>(acc[r][n], a[0], b[n][0], b[n][1], acc[r][n]);
            q4_mma<T>(acc[r][n], a[1], b[n][2], b[n][3], acc[r][n]);
          }
          if (c % GC == GC - 1) {
            const float s0 = scale[r][0], s1 = scale[r][1];
#pragma unroll
            for (int n = 0; n < NC; ++n) {
              float(&a)[4] = acc[r][n], (&d)[4] = total[r][n];
              f2_unpack(f2_fma(f2_splat(s0), f2_pack(a[0], a[1]), f2_pack(d[0], d[1])), d[0], d[1]);
              f2_unpack(f2_fma(f2_splat(s1), f2_pack(a[2], a[3]), f2_pack(d[2], d[3])), d[2], d[3]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty_bar(slot));
      if (++slot == ST) {
        slot = 0;
        phase ^= 1u;
      }
    }
    if constexpr (WR > 1) {  // after a wait that ran out: warps that share a ring still meet where the others may wait
      if (!ok)
        for (int e = max(i, u0 > wk ? (u0 - wk + WK - 1) / WK : 0); wk + e * WK < u1; ++e)
          if (by_lanes(e)) group_sync();
    }
  }
  // After a wait that ran out: what was asked for lands before shared memory goes away.
  if (!ok && issuer) {
    for (int e = 0; e < ST && i + e < mine; ++e) {
      mbar_wait(full_bar(slot), phase, nullptr, kWaitLimitNs, kRoleProducer, &g_device_error);
      if (++slot == ST) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }

  // The sums of the warps that share K, added in order: [wk][token][row], in the rings' place.
  __syncthreads();
  float *sums = reinterpret_cast<float *>(q4_smem);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = t * 2 + (j & 1);
        const int m = NT == 0 ? col : n * 8 + 4 * (col & 1) + (col >> 1), row = wr * 16 * R + r * 16 + g + (j >> 1) * 8;
        if (m < tokens) sums[(wk * tokens + m) * kRows + row] = total[r][n][j];
      }
  __syncthreads();
  const int n = n0 + last_row;
  if (n >= p.N) return;
  for (int m = static_cast<int>(threadIdx.x) / kRows; m < tokens; m += 32 * kQ4Warps / kRows) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < WK; ++w) v += sums[(w * tokens + m) * kRows + last_row];
    v += bias;
    const int64_t token = token0 + m;
    if (p.out_f32) {
      v = activate<false>(p.act, v);
      if (p.R != nullptr) v += load_elem<kTypeF32>(p.R, token * p.ldr + n);
      store_elem<kTypeF32>(p.C, token * p.ldc + n, v);
    } else {
      v = activate<true>(p.act, v);
      if (p.R != nullptr) v += load_elem<T>(p.R, token * p.ldr + n);
      store_elem<T>(p.C, token * p.ldc + n, v);
    }
  }
}

// ------------------------------------------------------------------ host side

template <int T, int NT, int R, int WK, int GC>
tlg_status launch_q4(int dev, Q4Params p, cudaStream_t s) {
  using Plan = Q4Plan<NT, R, WK>;
  constexpr auto kernel = gemv_q4_kernel<T, NT, R, WK, GC>;
  static bool ready[kMaxDevices];
  static std::mutex mutex;
  {
    std::lock_guard<std::mutex> lock(mutex);
    if (!ready[dev]) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan::kDynamicBytes) != cudaSuccess) {
        cudaGetLastError();
        return TLG_ERR_CUDA;
      }
      ready[dev] = true;
    }
  }
  p.token_blocks = (p.M + Plan::kTokens - 1) / Plan::kTokens;
  const int64_t tiles = (p.N + Plan::kRows - 1) / Plan::kRows;
  if (tiles * p.token_blocks > kMaxExtent) return TLG_ERR_UNSUPPORTED;
  CUtensorMap w = {}, x = {};
  if (p.K > 0) {
    const uint64_t row = static_cast<uint64_t>(row_bytes(TLG_MX_E2M1, p.K));
    if (!encode_2d(&w, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.Q, row, static_cast<uint64_t>(p.N),
                   p.N > 1 ? static_cast<uint64_t>(p.ldq) : row, Plan::kWRow, Plan::kRows,
                   Plan::kBlocks == 8 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
      return TLG_ERR_CUDA;
    if (p.x_tma && !encode_2d(&x, T == kTypeF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.X,
                              static_cast<uint64_t>(p.K), static_cast<uint64_t>(p.M),
                              static_cast<uint64_t>(p.M > 1 ? p.ldx : (int64_t(p.K) + 7) / 8 * 8) * 2, NT == 0 ? Plan::kUnit : 64,
                              Plan::kTokens, NT == 0 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B))
      return TLG_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.token_blocks));
  cfg.blockDim = dim3(32 * kQ4Warps);
  cfg.dynamicSmemBytes = Plan::kDynamicBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, w, x, p) != cudaSuccess) {
    cudaGetLastError();
    return TLG_ERR_CUDA;
  }
  return TLG_OK;
}

template <int T, int NT, int R, int WK>
tlg_status launch_q4_group(int dev, const Q4Params &p, cudaStream_t s) {
  if (p.group_log2 == 5) return launch_q4<T, NT, R, WK, 1>(dev, p, s);
  if (p.group_log2 == 6) return launch_q4<T, NT, R, WK, 2>(dev, p, s);
  return launch_q4<T, NT, R, WK, 4>(dev, p, s);
}

template <int T>
tlg_status launch_q4_shape(int dev, int sms, const Q4Params &p, cudaStream_t s) {
  const bool wide = p.N >= 64 * sms;
  if (p.M == 1) return wide ? launch_q4_group<T, 0, 2, 4>(dev, p, s) : launch_q4_group<T, 0, 1, 8>(dev, p, s);
  if (p.M <= 8) return wide ? launch_q4_group<T, 1, 2, 4>(dev, p, s) : launch_q4_group<T, 1, 1, 8>(dev, p, s);
  return wide ? launch_q4_group<T, 2, 2, 4>(dev, p, s) : launch_q4_group<T, 2, 1, 8>(dev, p, s);
}

}  // namespace

TLG_DEFINE_ERROR_WORD_READER(error_word_gemv)

}  // namespace tlg

using namespace tlg;

extern "C" {

tlg_status tlg_gemv_q4(int64_t M, int64_t N, int64_t K, tlg_type type, const void *X, int64_t ldx, const void *Q,
                       int64_t ldq, const void *S, const uint8_t *Z, int64_t group, const tlg_fused_epilogue *epilogue,
                       void *C, int64_t ldc, tlg_type out, void *stream) {
  if (M < 0 || N < 0 || K < 0 || (type != TLG_TYPE_F16 && type != TLG_TYPE_BF16) || (out != TLG_TYPE_F32 && out != type))
    return TLG_ERR_INVALID_ARG;
  if (group < 32 || (group & (group - 1)) != 0) return TLG_ERR_INVALID_ARG;
  if (M > kMaxExtent || N > kMaxExtent || K > kMaxExtent || group > (int64_t(1) << 31)) return TLG_ERR_UNSUPPORTED;
  tlg_fused_epilogue e = {};
  if (epilogue != nullptr) e = *epilogue;
  if (!valid_activation(e.activation)) return TLG_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return TLG_OK;
  const int64_t esz = type_bytes(out), groups = (K + group - 1) / group, qrow = row_bytes(TLG_MX_E2M1, K);
  Range rc, rx = {}, rq = {}, rs = {}, rz = {}, rb = {}, rr = {};
  tlg_status st = check_matrix(C, M, N, ldc, esz, &rc);
  if (st != TLG_OK) return st;
  if (K > 0) {
    st = check_matrix(X, M, K, ldx, 2, &rx);
    if (st != TLG_OK) return st;
    if (Q == nullptr || S == nullptr || ldq < qrow) return TLG_ERR_INVALID_ARG;
    if (!aligned16(Q) || (N > 1 && ldq % 16 != 0) || reinterpret_cast<uintptr_t>(S) % 2 != 0) return TLG_ERR_ALIGNMENT;
    if (ldq > kMaxLd || (N > 1 && N - 1 > (int64_t(1) << 60) / ldq)) return TLG_ERR_UNSUPPORTED;
    extent(Q, N, qrow, ldq, 1, &rq.lo, &rq.hi);
    extent(S, N, groups, groups, 2, &rs.lo, &rs.hi);
    if (Z != nullptr) extent(Z, N, groups, groups, 1, &rz.lo, &rz.hi);
  }
  if (e.bias != nullptr) {
    if (reinterpret_cast<uintptr_t>(e.bias) % 2 != 0) return TLG_ERR_ALIGNMENT;
    rb.lo = reinterpret_cast<uintptr_t>(e.bias);
    rb.hi = rb.lo + static_cast<uintptr_t>(2 * N);
  }
  if (e.residual != nullptr) {
    st = check_matrix(e.residual, M, N, e.ldr, esz, &rr);
    if (st != TLG_OK) return st;
    if (meets(rc, rr) && !(e.residual == C && e.ldr == ldc)) return TLG_ERR_INVALID_ARG;
  }
  for (const Range &r : {rx, rq, rs, rz, rb})
    if (meets(rc, r)) return TLG_ERR_INVALID_ARG;
  int dev = 0;
  DeviceInfo info;
  st = current_device(&dev, &info);
  if (st != TLG_OK) return st;
  for (const void *q : {static_cast<const void *>(C), K > 0 ? X : nullptr, K > 0 ? Q : nullptr, K > 0 ? S : nullptr,
                        K > 0 ? static_cast<const void *>(Z) : nullptr, e.bias, e.residual})
    if (q != nullptr && !device_accessible(q, dev)) return TLG_ERR_INVALID_ARG;
  Q4Params p = {};
  p.Q = static_cast<const uint8_t *>(Q);
  p.ldq = ldq;
  p.S = static_cast<const uint16_t *>(S);
  p.Z = K > 0 ? Z : nullptr;
  p.X = static_cast<const uint16_t *>(X);
  p.ldx = ldx;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.groups = static_cast<int>(groups);
  while ((int64_t(1) << p.group_log2) < group) ++p.group_log2;
  p.x_vec = aligned16(X) && (M == 1 || ldx % 8 == 0);
  // Of few tokens TMA is slow to fetch rows that are not whole lines apart (two, 3000 x 1000 weights: 5.0 us, 3.0
  // with plain loads); of more than eight the plain loads take longer (16, 16384 x 16392: 72 us against 60).
  p.x_tma = p.x_vec && (M == 1 || M > 8 || ldx % 64 == 0);
  p.C = C;
  p.ldc = ldc;
  p.out_f32 = out == TLG_TYPE_F32;
  p.bias = e.bias;
  p.act = e.activation;
  p.R = e.residual;
  p.ldr = e.ldr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return type == TLG_TYPE_F16 ? launch_q4_shape<kTypeF16>(dev, info.sm_count, p, s)
                              : launch_q4_shape<kTypeBF16>(dev, info.sm_count, p, s);
}

}  // extern "C"
