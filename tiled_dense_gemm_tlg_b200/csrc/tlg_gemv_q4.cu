// Products of a few rows (tokens) with integer 4-bit weights:
//
//   C = act(X . W^T + bias) + residual,  W[n, k] = (q[n, k] - z[n, k / group]) s[n, k / group]
//
// Reading the weights (half a byte each) is all the work there is for one token, so the kernel is built
// around a stream of weights: a CTA takes 16 R rows of W, its eight warps share K in units of 128, and
// each warp copies its units (64 bytes of a row) asynchronously into a ring of its own, without any
// barrier between warps until their sums are added at the end.
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
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "tlg.h"
#include "tlg_mxgemm_kernel.cuh"
#include "tlg_rows.cuh"

namespace tlg {
namespace {

constexpr int kQ4Warps = 8;
constexpr int kQ4Unit = 128;     // k of a unit
constexpr int kQ4Panel = 128;    // groups whose scales are held in shared memory at a time

struct Q4Params {
  const uint8_t *Q;
  int64_t ldq;
  const uint16_t *S;
  const uint8_t *Z;  // or nullptr: 8
  const uint16_t *X;
  int64_t ldx;
  int M, N, K;
  int group_log2, groups;
  int x_vec;  // X may be copied 16 bytes at a time
  int token_blocks;
  void *C;
  int64_t ldc;
  int out_f32;
  const void *bias;  // X's type
  int act;
  const void *R;     // C's type
  int64_t ldr;
};

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

// Copies 16 bytes to shared memory asynchronously, only the first `size` of them read, zeros behind.
__device__ __forceinline__ void q4_copy(uint32_t dst, const void *src, int size) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}

// Slots of a ring.
template <int NT, int WK>
constexpr int kQ4Stages = WK == kQ4Warps ? 8 : NT == 1 ? 6 : 5;

// Bytes of a slot: a unit of WR * 16 R rows of W, 64 bytes of each, and of X's tokens, 256 of each.
__host__ __device__ constexpr int q4_slot(int rows, int tokens) { return rows * 64 + tokens * 256; }
// Row stride of the scales in shared memory, in words; odd, so that eight rows lie in different banks.
__host__ __device__ constexpr int q4_scale_ld(int groups) { return (groups < kQ4Panel ? groups : kQ4Panel) | 1; }

// NT: blocks of 8 tokens; R: blocks of 16 rows of W to a warp; WK: warps that share K, each group of
// WR = 8 / WK warps with a ring of its own, in which X is shared; GC: blocks of 32 k that have one scale in a
// unit (1, 2, 4).
template <int T, int NT, int R, int WK, int GC>
__global__ void __launch_bounds__(32 * kQ4Warps) gemv_q4_kernel(const Q4Params p) {
  constexpr int ST = kQ4Stages<NT, WK>;
  constexpr int WR = kQ4Warps / WK;
  constexpr int kRows = WR * 16 * R;  // of a CTA
  constexpr uint32_t kMagic = T == kTypeF16 ? 0x64006400u : 0x43004300u;
  extern __shared__ __align__(16) uint8_t q4_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wr = warp % WR, wk = warp / WR;
  const int g = lane >> 2, t = lane & 3;
  const int tile = static_cast<int>(blockIdx.x) / p.token_blocks;
  const int token0 = (static_cast<int>(blockIdx.x) - tile * p.token_blocks) * (8 * NT);
  const int tokens = min(p.M - token0, 8 * NT);
  const int n0 = tile * kRows;
  const int slot_bytes = q4_slot(kRows, tokens);
  const uint32_t ring = smem_u32(q4_smem) + static_cast<uint32_t>(wk * ST * slot_bytes);
  const int scale_ld = q4_scale_ld(p.groups);
  // a word for each row and group: the scale's bits low, the zero point high
  uint32_t *scales = reinterpret_cast<uint32_t *>(q4_smem + WK * ST * slot_bytes);
  grid_dependency_wait();
  grid_launch_dependents();

  const int blocks = (p.K + 31) / 32;  // of a row of W
  // this lane's part of a unit of W: block t of rows g, g + 8, ..
  const int row0 = n0 + wr * 16 * R + g;
  const uint8_t *w_from = p.Q + row0 * p.ldq + t * 16;
  auto issue = [&](int unit, int slot) {
    const uint32_t w = ring + static_cast<uint32_t>(slot * slot_bytes + wr * 1024 * R), x = ring + static_cast<uint32_t>(slot * slot_bytes + kRows * 64);
    const int k0 = unit * kQ4Unit;
    // W: block c of row r at (c ^ r / 2 % 4) of the row's four places
#pragma unroll
    for (int i = 0; i < 2 * R; ++i) {
      const int r = i * 8 + g;
      const bool in = row0 + i * 8 < p.N && unit * 4 + t < blocks;
      q4_copy(w + static_cast<uint32_t>(r * 64 + ((t ^ ((r >> 1) & 3)) * 16)),
              in ? w_from + i * 8 * p.ldq + static_cast<int64_t>(unit) * 64 : p.Q, in ? 16 : 0);
    }
    // X: 8 elements of token m at (q ^ 4 (m % 2)) of its 16 places
    for (int i = wr * 32 + lane; i < tokens * 16; i += WR * 32) {
      const int m = i >> 4, q = i & 15, k = k0 + q * 8;
      const uint32_t to = x + static_cast<uint32_t>(m * 256 + ((q ^ ((m & 1) << 2)) * 16));
      const uint16_t *from = p.X + (token0 + m) * p.ldx + k;
      const int left = min(max(p.K - k, 0), 8);
      if (p.x_vec) {
        q4_copy(to, left > 0 ? from : p.X, left * 2);
      } else {
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[j] = ld_u16_pred(from + 2 * j, 2 * j < left) | ld_u16_pred(from + 2 * j + 1, 2 * j + 1 < left) << 16;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                     : "memory");
      }
    }
  };

  float total[R][NT][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) total[r][n][j] = 0.0f;

  const int units = (p.K + kQ4Unit - 1) / kQ4Unit;
  const int panel_units = max(1, static_cast<int>(std::min<int64_t>(int64_t(kQ4Panel) << p.group_log2, int64_t(1) << 30) / kQ4Unit));
  for (int u0 = 0; u0 < units; u0 += panel_units) {
    const int u1 = min(units, u0 + panel_units);
    const int first_group = static_cast<int>((static_cast<int64_t>(u0) * kQ4Unit) >> p.group_log2);
    if (u0 > 0) __syncthreads();  // the last panel's scales are read
#pragma unroll
    for (int s = 0; s < ST - 1; ++s) {
      const int u = u0 + wk + s * WK;
      if (u < u1) issue(u, s);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // scales and zero points of the panel, 0 past the last row: a warp takes 2 WR R rows, all loads of 32
    // groups in flight at once
    const int held = min(p.groups - first_group, kQ4Panel);
    for (int j = lane; j < held; j += 32) {
      constexpr int kMine = kRows / kQ4Warps;
      uint32_t v[kMine], z[kMine];
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int n = n0 + warp * kMine + i;
        const int64_t at = static_cast<int64_t>(n) * p.groups + first_group + j;
        v[i] = n < p.N ? p.S[at] : 0u;
        z[i] = n < p.N && p.Z != nullptr ? p.Z[at] : 8u;
      }
#pragma unroll
      for (int i = 0; i < kMine; ++i) scales[(warp * kMine + i) * scale_ld + j] = v[i] | (z[i] & 15u) << 16;
    }
    __syncthreads();
    int slot = 0;
    for (int first = u0; first < u1; first += WK) {  // the warps that share a ring go through it together
      const int u = first + wk;
      asm volatile("cp.async.wait_group %0;" ::"n"(ST - 2) : "memory");
      // every copy into this slot has landed, and the slot before is read
      if constexpr (WR > 1)
        __syncthreads();
      else
        __syncwarp();
      const int ahead = u + (ST - 1) * WK;
      if (ahead < u1) issue(ahead, slot == 0 ? ST - 1 : slot - 1);
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (u >= u1) break;
      const uint32_t w = ring + static_cast<uint32_t>(slot * slot_bytes + wr * 1024 * R), x = ring + static_cast<uint32_t>(slot * slot_bytes + kRows * 64);
      float acc[R][NT][4];
      uint32_t zero[R][2];
      float scale[R][2];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c % GC == 0) {
          const int j = static_cast<int>((static_cast<int64_t>(u) * kQ4Unit + c * 32) >> p.group_log2) - first_group;
          const uint32_t *s = scales + wr * 16 * R * scale_ld + min(j, held - 1);  // blocks past K have no group; their X is 0
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t v = s[(r * 16 + h * 8 + g) * scale_ld];
              zero[r][h] = kMagic + (v >> 16) * 0x10001u;
              float none;
              unpack2<T>(v, scale[r][h], none);
            }
        }
        uint32_t b[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int m = n * 8 + g;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (m < tokens) v = ld_shared_v4(x + static_cast<uint32_t>(m * 256 + (((c * 4 + t) ^ ((m & 1) << 2)) * 16)));
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
            const int row = r * 16 + h * 8 + g;
            const uint32_t v = ld_shared_u32(w + static_cast<uint32_t>(row * 64 + ((c ^ ((row >> 1) & 3)) * 16) + t * 4));
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i >> 1][h + 2 * (i & 1)] = q4_sub<T>(((v >> (4 * i)) & 0x000f000fu) | kMagic, zero[r][h]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
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
            for (int n = 0; n < NT; ++n) {
              total[r][n][0] = fmaf(s0, acc[r][n][0], total[r][n][0]);
              total[r][n][1] = fmaf(s0, acc[r][n][1], total[r][n][1]);
              total[r][n][2] = fmaf(s1, acc[r][n][2], total[r][n][2]);
              total[r][n][3] = fmaf(s1, acc[r][n][3], total[r][n][3]);
            }
          }
        }
      }
      slot = slot == ST - 1 ? 0 : slot + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
  }

  // The sums of the warps that share K, added in order: [wk][token][row], in the rings' place.
  __syncthreads();
  float *sums = reinterpret_cast<float *>(q4_smem);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int m = n * 8 + t * 2 + (j & 1), row = wr * 16 * R + r * 16 + g + (j >> 1) * 8;
        if (m < tokens) sums[(wk * tokens + m) * kRows + row] = total[r][n][j];
      }
  __syncthreads();
  for (int i = threadIdx.x; i < tokens * kRows; i += 32 * kQ4Warps) {
    const int m = i / kRows, row = i - m * kRows, n = n0 + row;
    if (n >= p.N) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < WK; ++w) v += sums[(w * tokens + m) * kRows + row];
    if (p.bias != nullptr) v += load_elem<T>(p.bias, n);
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
  constexpr auto kernel = gemv_q4_kernel<T, NT, R, WK, GC>;
  constexpr int kRows = kQ4Warps / WK * 16 * R, kStages = kQ4Stages<NT, WK>;
  constexpr int kMost = WK * kStages * q4_slot(kRows, 8 * NT) + kRows * q4_scale_ld(kQ4Panel) * 4;
  static_assert(kMost <= 232448, "shared memory per CTA exceeded");
  static_assert(kStages * q4_slot(kRows, 1) >= kRows * 4, "a slice's sums of a token fit its ring");
  static bool ready[kMaxDevices];
  static std::mutex mutex;
  {
    std::lock_guard<std::mutex> lock(mutex);
    if (!ready[dev]) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) != cudaSuccess) {
        cudaGetLastError();
        return TLG_ERR_CUDA;
      }
      ready[dev] = true;
    }
  }
  const int tokens = std::min(p.M, 8 * NT);
  p.token_blocks = (p.M + 8 * NT - 1) / (8 * NT);
  const int64_t tiles = (p.N + kRows - 1) / kRows;
  if (tiles * p.token_blocks > kMaxExtent) return TLG_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.token_blocks));
  cfg.blockDim = dim3(32 * kQ4Warps);
  cfg.dynamicSmemBytes = WK * kStages * q4_slot(kRows, tokens) + kRows * q4_scale_ld(p.groups) * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
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
tlg_status launch_q4_shape(int dev, const Q4Params &p, cudaStream_t s) {
  if (p.M > 8) return launch_q4_group<T, 2, 1, 2>(dev, p, s);
  if (p.M > 2) return launch_q4_group<T, 1, 1, 2>(dev, p, s);
  return launch_q4_group<T, 1, 1, 8>(dev, p, s);
}

}  // namespace
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
  p.C = C;
  p.ldc = ldc;
  p.out_f32 = out == TLG_TYPE_F32;
  p.bias = e.bias;
  p.act = e.activation;
  p.R = e.residual;
  p.ldr = e.ldr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return type == TLG_TYPE_F16 ? launch_q4_shape<kTypeF16>(dev, p, s)
                              : launch_q4_shape<kTypeBF16>(dev, p, s);
}

}  // extern "C"
