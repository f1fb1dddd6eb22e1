// What the row kernels (microscaled operators, norms) share: a lane's 16 bytes of a row at any alignment,
// a lane's elements of an MX matrix, the sum of partial column sums, and their launch.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "tlg.h"
#include "tlg_mx_device.cuh"
#include "tlg_mx_host.cuh"

namespace tlg {
namespace {

static_assert(kTypeF32 == TLG_TYPE_F32 && kTypeF16 == TLG_TYPE_F16 && kTypeBF16 == TLG_TYPE_BF16,
              "the kernels' type codes are tlg_type's values");
static_assert(kE2M1 == TLG_MX_E2M1 && kE4M3 == TLG_MX_E4M3,
              "the kernels' format codes are tlg_mx_format's values");

// A lane holds 16 bytes of a row: E elements; a warp 32 * E of them (a chunk: 256 columns of
// a 16-bit type, 128 of fp32, so whole groups of four blocks).  16 bytes, not 32: a warp's
// store then covers 512 consecutive bytes, where two stores of 16 bytes 32 apart would each
// fill half of every sector (8192 x 8192 E2M1 to bf16: 53 us with 32 bytes a lane).
template <int T>
constexpr int kLaneElems = 16 / kTypeBytes<T>;

// One matrix of a row kernel: base and row stride in elements.  Kernels are built with VEC (every
// matrix of the call has a base and row stride that are multiples of 16 bytes) and without.
struct RowMat {
  const void *p;
  int64_t ld;
};

// Elements [c0, c0 + 32 E) of a row, E to a lane; zeros from column `cols` on.  Without VEC,
// neighbouring lanes read neighbouring words (lane l: words l, l + 32, ...); finish_load rearranges
// them.  A row of 16-bit elements may start in the middle of a word: word k then holds elements
// 2k - 1 and 2k, and word 0 the piece's last and first one, which are read one by one.  (8000 x 8191
// bf16 to 4 bits: 51 us; all elements one by one 74.)
// FULL: the whole piece lies before `cols`.  first: the first element, where it is apart.
template <int T, bool VEC>
__device__ __forceinline__ bool starts_inside_word(const char *base) {
  return !VEC && kTypeBytes<T> == 2 && (reinterpret_cast<uintptr_t>(base) & 2) != 0;
}

// Elements of a lane's word j of such a piece, and whether they are apart in memory.
struct WordElems {
  int lo, hi;
  bool apart;
  __device__ __forceinline__ WordElems(int j, int lane, bool inside) {
    const int k = j * 32 + lane;
    apart = inside && k == 0;
    lo = apart ? 255 : 2 * k - (inside ? 1 : 0);
    hi = 2 * k + (inside ? 0 : 1);
  }
};

template <int T, bool VEC, bool FULL>
__device__ __forceinline__ void issue_load(const char *base, int left, int lane, uint32_t (&w)[4], uint32_t &first) {
  constexpr int E = kLaneElems<T>;
  if (VEC && (FULL || (lane + 1) * E <= left)) {
    const uint4 a = *reinterpret_cast<const uint4 *>(base + lane * 16);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  } else if constexpr (T == kTypeF32) {
    const int at = VEC ? lane * E : lane;
    constexpr int step = VEC ? 1 : 32;
    const uint32_t *q = reinterpret_cast<const uint32_t *>(base);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = FULL || at + j * step < left ? q[at + j * step] : 0u;
  } else {
    const unsigned short *q = reinterpret_cast<const unsigned short *>(base);
    const bool inside = starts_inside_word<T, VEC>(base);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      WordElems e(j, lane, inside);
      if constexpr (VEC) e.lo = lane * E + 2 * j, e.hi = e.lo + 1;
      // Nothing here waits for a load: a word's two halves are joined in finish_load.
      w[j] = 0;
      if (!e.apart && (FULL || e.hi < left))
        w[j] = *reinterpret_cast<const uint32_t *>(q + e.lo);
      else if (FULL || e.lo < left)
        w[j] = q[e.lo];
    }
    if (!VEC) first = inside && lane == 0 ? q[0] : 0;
  }
}

// `stage`: 512 bytes of shared memory per warp; `inside`: starts_inside_word of the row.
template <int T, bool VEC>
__device__ __forceinline__ void finish_load(int lane, bool inside, uint32_t first, uint32_t *stage, uint32_t (&w)[4]) {
  if constexpr (!VEC) {
    if (kTypeBytes<T> == 2) w[0] |= first << 16;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) stage[j * 32 + lane] = w[j];
    __syncwarp();
    const uint4 a = reinterpret_cast<const uint4 *>(stage)[lane];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    if (kTypeBytes<T> == 2 && inside) {
      const uint32_t n = __shfl_sync(0xffffffffu, w[0], (lane + 1) & 31);
      w[0] = __funnelshift_r(w[0], w[1], 16);
      w[1] = __funnelshift_r(w[1], w[2], 16);
      w[2] = __funnelshift_r(w[2], w[3], 16);
      w[3] = __funnelshift_r(w[3], n, 16);
    }
  }
}

// The reverse: columns from `left` on are not written.
template <int T, bool VEC, bool FULL>
__device__ __forceinline__ void store_lane(char *base, int left, int lane, uint32_t *stage, const uint32_t (&w)[4]) {
  constexpr int E = kLaneElems<T>;
  if (VEC && (FULL || (lane + 1) * E <= left)) {
    *reinterpret_cast<uint4 *>(base + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }
  uint32_t x[4] = {w[0], w[1], w[2], w[3]};
  const bool inside = starts_inside_word<T, VEC>(base);
  if constexpr (!VEC) {
    if (kTypeBytes<T> == 2 && inside) {
      const uint32_t n = __shfl_sync(0xffffffffu, w[3], (lane + 31) & 31);
      x[0] = __funnelshift_r(n, w[0], 16);
      x[1] = __funnelshift_r(w[0], w[1], 16);
      x[2] = __funnelshift_r(w[1], w[2], 16);
      x[3] = __funnelshift_r(w[2], w[3], 16);
    }
    __syncwarp();
    reinterpret_cast<uint4 *>(stage)[lane] = make_uint4(x[0], x[1], x[2], x[3]);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = stage[j * 32 + lane];
  }
  if constexpr (T == kTypeF32) {
    const int at = VEC ? lane * E : lane;
    constexpr int step = VEC ? 1 : 32;
    uint32_t *q = reinterpret_cast<uint32_t *>(base);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (FULL || at + j * step < left) q[at + j * step] = x[j];
  } else {
    unsigned short *q = reinterpret_cast<unsigned short *>(base);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      WordElems e(j, lane, inside);
      if constexpr (VEC) e.lo = lane * E + 2 * j, e.hi = e.lo + 1;
      if (!e.apart && (FULL || e.hi < left)) {
        *reinterpret_cast<uint32_t *>(q + e.lo) = x[j];
      } else {
        if (FULL || e.lo < left) q[e.lo] = static_cast<unsigned short>(x[j]);
        if (FULL || e.hi < left) q[e.hi] = static_cast<unsigned short>(x[j] >> 16);
      }
    }
  }
}

// Elements and scales of an MX matrix.  A row of Q holds `blocks` whole blocks, 16-byte
// aligned.
struct MxMat {
  const uint8_t *q;
  int64_t ldq;
  const uint8_t *s;
  int64_t tiles_x;
  int blocks;
};

template <int FMT, int E>
__device__ __forceinline__ void load_q(const uint8_t *p, uint32_t (&q)[kQWords<FMT, E>]) {
  constexpr int N = kQBytes<FMT, E>;
  if constexpr (N == 8) {
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    q[0] = x.x; q[1] = x.y;
  } else if constexpr (N == 4) {
    q[0] = *reinterpret_cast<const uint32_t *>(p);
  } else {
    q[0] = *reinterpret_cast<const uint16_t *>(p);
  }
}

template <int FMT, int E>
__device__ __forceinline__ void store_q(uint8_t *p, const uint32_t (&q)[kQWords<FMT, E>]) {
  constexpr int N = kQBytes<FMT, E>;
  if constexpr (N == 8)
    *reinterpret_cast<uint2 *>(p) = make_uint2(q[0], q[1]);
  else if constexpr (N == 4)
    *reinterpret_cast<uint32_t *>(p) = q[0];
  else
    *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(q[0]);
}

// A lane's elements of one row of an MX matrix and their scale byte; zeros past the last block.
template <int FMT, int E>
struct MxLane {
  uint32_t q[kQWords<FMT, E>];
  uint32_t byte;
};

// q: the lane's element bytes; s: its scale byte (read only where `in` holds).
template <int FMT, int E>
__device__ __forceinline__ void issue_load_mx(const uint8_t *q, const uint8_t *s, bool in, MxLane<FMT, E> &x) {
#pragma unroll
  for (int j = 0; j < kQWords<FMT, E>; ++j) x.q[j] = 0;
  x.byte = 0;
  if (in) {
    load_q<FMT, E>(q, x.q);
    x.byte = *s;
  }
}

// Scale offset of (row, block 0 of its tile row), the part that depends on the row.
__device__ __forceinline__ int64_t scale_row(uint32_t row, int64_t tile_row_bytes) {
  return (row >> 7) * tile_row_bytes + ((row & 31) * 16 + ((row >> 5) & 3) * 4);
}

// dbias[c] = the sum over `parts` partial sums: each of a CTA's W warps takes every W-th one of 32
// columns, and their sums are added in order.  W = 32 where a narrow matrix has hundreds of
// row splits and a warp's chain of loads takes the time (16384 x 1000 fp16, 592 splits, the whole
// backward call: 24.7 us, 30.5 with 8), else 8, which find room beside the kernel before sooner
// (2000 x 5000: 18.3 us, 20.3 with 32).  T: the type they are added in.
template <int W, typename T = float>
__global__ void __launch_bounds__(32 * W) column_sum_kernel(const float *part, int parts, int64_t cols, float *dbias) {
  __shared__ T sums[W][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  T s = 0;
  if (c < cols) {
#pragma unroll 8
    for (int i = warp; i < parts; i += W) s += part[i * cols + c];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < W; ++i) s += sums[i][lane];
    dbias[c] = static_cast<float>(s);
  }
}

// ------------------------------------------------------------------ host side

// Whether every row starts on 16 bytes (of a single row, the stride does not matter).
bool vec_rows(const void *p, int64_t rows, int64_t ld, int type) {
  return aligned16(p) && (rows == 1 || (ld * type_bytes(type)) % 16 == 0);
}

MxMat mx_mat(const void *Q, int64_t ldq, const void *S, int64_t cols) {
  return {static_cast<const uint8_t *>(Q), ldq, static_cast<const uint8_t *>(S), scale_tiles_x(cols),
          static_cast<int>(mx_blocks(cols))};
}

// Launches as a programmatic dependent of the previous kernel in the stream: every kernel
// here waits for that one to complete before it touches memory, so only launch latency and
// set-up overlap.
template <typename... P, typename... A>
tlg_status launch(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s, int smem, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) != cudaSuccess) {
    cudaGetLastError();
    return TLG_ERR_CUDA;
  }
  return TLG_OK;
}

// Calls f with the type (or format) as a template argument.
template <typename F>
tlg_status with_type(int type, F f) {
  switch (type) {
    case TLG_TYPE_F32: return f(std::integral_constant<int, kTypeF32>());
    case TLG_TYPE_F16: return f(std::integral_constant<int, kTypeF16>());
    default: return f(std::integral_constant<int, kTypeBF16>());
  }
}

template <typename F>
tlg_status with_flag(bool flag, F f) {
  return flag ? f(std::true_type()) : f(std::false_type());
}

template <typename F>
tlg_status with_format(int format, F f) {
  return format == TLG_MX_E2M1 ? f(std::integral_constant<int, kE2M1>()) : f(std::integral_constant<int, kE4M3>());
}

}  // namespace
}  // namespace tlg
