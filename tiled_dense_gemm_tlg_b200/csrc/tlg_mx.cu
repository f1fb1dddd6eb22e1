// Microscaled (MX) elementwise operators: quantisation of a matrix or its transpose,
// dequantisation, the activation that saves its input in 8 bits and the backward pass that
// reads it.  All of them are bound by HBM traffic: every kernel reads each input byte once
// and writes each output byte once, 16 or 32 bytes a lane.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>
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

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;

// A lane holds 32 bytes of a row: E elements; a warp 32 * E of them (a chunk: 512 columns of
// a 16-bit type, 256 of fp32, so whole groups of four blocks).
template <int T>
constexpr int kLaneElems = T == kTypeF32 ? 8 : 16;

// One matrix of a row kernel: base, row stride in elements, and whether rows may be accessed
// 16 bytes at a time.
struct RowMat {
  const void *p;
  int64_t ld;
  int vec;
};

// Elements [c0, c0 + 32 E) of a row, E to a lane; zeros from column `cols` on.  Rows whose
// address is not a multiple of 16 bytes are read element by element, neighbouring lanes on
// neighbouring elements, and rearranged through `stage` (1 KB per warp).
template <int T>
__device__ __forceinline__ void load_lane(const RowMat &m, int64_t row, int64_t c0, int64_t cols,
                                          int lane, uint32_t *stage, uint32_t (&w)[8]) {
  constexpr int E = kLaneElems<T>;
  constexpr int B = kTypeBytes<T>;
  const char *base = static_cast<const char *>(m.p) + (row * m.ld + c0) * B;
  const int64_t left = cols - c0;  // > 0
  if (m.vec) {
    const int at = lane * E;
    if (at + E <= left) {
      const uint4 *q = reinterpret_cast<const uint4 *>(base + lane * 32);
      const uint4 a = q[0], b = q[1];
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
      w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
      return;
    }
    const int n = static_cast<int>(max(left - at, int64_t(0)));
    if constexpr (T == kTypeF32) {
      const uint32_t *q = reinterpret_cast<const uint32_t *>(base) + at;
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = j < n ? q[j] : 0u;
    } else {
      const unsigned short *q = reinterpret_cast<const unsigned short *>(base) + at;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t lo = 2 * j < n ? q[2 * j] : 0u;
        const uint32_t hi = 2 * j + 1 < n ? q[2 * j + 1] : 0u;
        w[j] = lo | (hi << 16);
      }
    }
    return;
  }
  __syncwarp();
  if constexpr (T == kTypeF32) {
    const uint32_t *q = reinterpret_cast<const uint32_t *>(base);
    uint32_t x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i * 32 + lane < left ? q[i * 32 + lane] : 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) stage[i * 32 + lane] = x[i];
  } else {
    const unsigned short *q = reinterpret_cast<const unsigned short *>(base);
    unsigned short x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i * 32 + lane < left ? q[i * 32 + lane] : (unsigned short)0;
#pragma unroll
    for (int i = 0; i < 16; ++i) reinterpret_cast<unsigned short *>(stage)[i * 32 + lane] = x[i];
  }
  __syncwarp();
  const uint4 a = reinterpret_cast<const uint4 *>(stage)[lane * 2];
  const uint4 b = reinterpret_cast<const uint4 *>(stage)[lane * 2 + 1];
  w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

// The reverse of load_lane: columns from `cols` on are not written.
template <int T>
__device__ __forceinline__ void store_lane(const RowMat &m, int64_t row, int64_t c0, int64_t cols,
                                           int lane, uint32_t *stage, const uint32_t (&w)[8]) {
  constexpr int E = kLaneElems<T>;
  constexpr int B = kTypeBytes<T>;
  char *base = static_cast<char *>(const_cast<void *>(m.p)) + (row * m.ld + c0) * B;
  const int64_t left = cols - c0;
  if (m.vec) {
    const int at = lane * E;
    if (at + E <= left) {
      uint4 *q = reinterpret_cast<uint4 *>(base + lane * 32);
      q[0] = make_uint4(w[0], w[1], w[2], w[3]);
      q[1] = make_uint4(w[4], w[5], w[6], w[7]);
      return;
    }
    const int n = static_cast<int>(max(left - at, int64_t(0)));
    if constexpr (T == kTypeF32) {
      uint32_t *q = reinterpret_cast<uint32_t *>(base) + at;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) q[j] = w[j];
    } else {
      unsigned short *q = reinterpret_cast<unsigned short *>(base) + at;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j < n) q[j] = static_cast<unsigned short>(w[j / 2] >> (16 * (j & 1)));
    }
    return;
  }
  __syncwarp();
  reinterpret_cast<uint4 *>(stage)[lane * 2] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4 *>(stage)[lane * 2 + 1] = make_uint4(w[4], w[5], w[6], w[7]);
  __syncwarp();
  if constexpr (T == kTypeF32) {
    uint32_t *q = reinterpret_cast<uint32_t *>(base);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i * 32 + lane < left) q[i * 32 + lane] = stage[i * 32 + lane];
  } else {
    unsigned short *q = reinterpret_cast<unsigned short *>(base);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i * 32 + lane < left) q[i * 32 + lane] = reinterpret_cast<const unsigned short *>(stage)[i * 32 + lane];
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
  constexpr int N = kQWords<FMT, E>;
  if constexpr (N == 4) {
    const uint4 x = *reinterpret_cast<const uint4 *>(p);
    q[0] = x.x; q[1] = x.y; q[2] = x.z; q[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    q[0] = x.x; q[1] = x.y;
  } else {
    q[0] = *reinterpret_cast<const uint32_t *>(p);
  }
}

template <int FMT, int E>
__device__ __forceinline__ void store_q(uint8_t *p, const uint32_t (&q)[kQWords<FMT, E>]) {
  constexpr int N = kQWords<FMT, E>;
  if constexpr (N == 4)
    *reinterpret_cast<uint4 *>(p) = make_uint4(q[0], q[1], q[2], q[3]);
  else if constexpr (N == 2)
    *reinterpret_cast<uint2 *>(p) = make_uint2(q[0], q[1]);
  else
    *reinterpret_cast<uint32_t *>(p) = q[0];
}

// Quantises a lane's elements (w as stored, v their values) and writes elements and scale.
// The lanes of a block (2 of 16-bit elements, 4 of fp32) agree on its largest magnitude by
// shuffles.
template <int T, int FMT>
__device__ __forceinline__ void quantize_lane(const MxMat &o, int64_t row, int64_t c0, int lane,
                                              const uint32_t (&w)[8],
                                              const float (&v)[kLaneElems<T>]) {
  constexpr int E = kLaneElems<T>;
  constexpr int kLanesPerBlock = kMxBlock / E;
  uint32_t m = amax_bits<T, 8>(w);
#pragma unroll
  for (int d = 1; d < kLanesPerBlock; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  const uint32_t byte = scale_byte<FMT>(m);
  uint32_t q[kQWords<FMT, E>];
  encode<FMT, E>(v, inverse_scale(byte), q);
  const int block = static_cast<int>(c0 / kMxBlock) + lane / kLanesPerBlock;
  if (block < o.blocks) {
    uint8_t *dst = const_cast<uint8_t *>(o.q) + row * o.ldq +
                   static_cast<int64_t>(block) * kBlockBytes<FMT> + (lane % kLanesPerBlock) * kQWords<FMT, E> * 4;
    store_q<FMT, E>(dst, q);
  }
  // blocks past the last one, up to a whole group of four, hold no elements: their scale is 0
  if (lane % kLanesPerBlock == 0 && (block >> 2) < o.tiles_x)
    const_cast<uint8_t *>(o.s)[scale_offset(row, block, o.tiles_x)] = static_cast<uint8_t>(byte);
}

// Rows x chunks of a matrix walked by warps, `step` apart, without a division per item.
struct ChunkIter {
  int64_t row;
  int chunk;
  int64_t step_rows;
  int step_chunks, chunks;
  __device__ __forceinline__ ChunkIter(int64_t at, int64_t step, int chunks_) : chunks(chunks_) {
    row = at / chunks_;
    chunk = static_cast<int>(at - row * chunks_);
    step_rows = step / chunks_;
    step_chunks = static_cast<int>(step - step_rows * chunks_);
  }
  __device__ __forceinline__ void next() {
    row += step_rows;
    chunk += step_chunks;
    if (chunk >= chunks) {
      chunk -= chunks;
      ++row;
    }
  }
};

// Quantises X row by row; with ACT also writes Y = act(X).
template <int T, int FMT, bool ACT>
__global__ void __launch_bounds__(kRowThreads)
    quantize_rows_kernel(const RowMat x, const MxMat o, const RowMat y, int act, int64_t rows,
                         int64_t cols, int chunks) {
  constexpr int E = kLaneElems<T>;
  __shared__ __align__(16) uint32_t stage[kRowWarps][256];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kRowWarps;
  for (ChunkIter it(static_cast<int64_t>(blockIdx.x) * kRowWarps + warp, nwarps, chunks);
       it.row < rows; it.next()) {
    const int64_t c0 = static_cast<int64_t>(it.chunk) * (32 * E);
    uint32_t w[8];
    float v[E];
    load_lane<T>(x, it.row, c0, cols, lane, stage[warp], w);
    to_floats<T, E>(w, v);
    quantize_lane<T, FMT>(o, it.row, c0, lane, w, v);
    if constexpr (ACT) {
      activate_lane<T, E>(act, v);
      from_floats<T, E>(v, w);
      store_lane<T>(y, it.row, c0, cols, lane, stage[warp], w);
    }
  }
}

template <int T, int FMT>
__global__ void __launch_bounds__(kRowThreads)
    dequantize_rows_kernel(const MxMat in, const RowMat x, int64_t rows, int64_t cols, int chunks) {
  constexpr int E = kLaneElems<T>;
  constexpr int kLanesPerBlock = kMxBlock / E;
  __shared__ __align__(16) uint32_t stage[kRowWarps][256];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kRowWarps;
  for (ChunkIter it(static_cast<int64_t>(blockIdx.x) * kRowWarps + warp, nwarps, chunks);
       it.row < rows; it.next()) {
    const int64_t c0 = static_cast<int64_t>(it.chunk) * (32 * E);
    const int block = static_cast<int>(c0 / kMxBlock) + lane / kLanesPerBlock;
    uint32_t q[kQWords<FMT, E>] = {};
    uint32_t byte = 0;
    if (block < in.blocks) {
      load_q<FMT, E>(in.q + it.row * in.ldq + static_cast<int64_t>(block) * kBlockBytes<FMT> +
                         (lane % kLanesPerBlock) * kQWords<FMT, E> * 4,
                     q);
      byte = in.s[scale_offset(it.row, block, in.tiles_x)];
    }
    float v[E];
    decode<FMT, E>(q, scale_value(byte), v);
    uint32_t w[8];
    from_floats<T, E>(v, w);
    store_lane<T>(x, it.row, c0, cols, lane, stage[warp], w);
  }
}

// ------------------------------------------------------------------ transposed quantisation

// Quantises X^T, X stored cols x rows (rows of Q are columns of X).  A CTA takes 128 rows of Q
// by 128 columns (four blocks, one scale tile): warp (block, part) reads the block's 32 rows of
// X, each lane 4 bytes of a row (two rows of Q of a 16-bit type, one of fp32), so a thread
// holds whole blocks and finds their scale without any exchange.  Elements then go through
// shared memory, so that each row of Q is written in pieces of four blocks (64 or 128 bytes).
template <int T, int FMT>
__global__ void __launch_bounds__(T == kTypeF32 ? 512 : 256)
    quantize_cols_kernel(const void *X, int64_t ldx, int pair_aligned, const MxMat o, int64_t rows,
                         int64_t cols, int64_t tiles_r, int64_t tiles) {
  constexpr int W = T == kTypeF32 ? 1 : 2;  // rows of Q per lane
  constexpr int kPieces = kBlockBytes<FMT> / 16;  // 16-byte pieces of a block
  constexpr int kRowPieces = 4 * kPieces;
  __shared__ __align__(16) uint4 elems[128 * kRowPieces];
  __shared__ __align__(16) uint8_t scales[512];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blk = warp & 3, part = warp >> 2;
  const int n_in = part * 32 * W + lane * W;
  // 16-byte piece i of row n of the tile; the low bits are permuted so that the eight lanes
  // of one shared-memory pass touch different banks, writing and reading.
  auto place = [](int n, int i) { return (n * kRowPieces + i) ^ ((n >> 1) & 7); };
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t tr = t % tiles_r, tc = t / tiles_r;
    const int64_t n0 = tr * 128 + n_in, k0 = tc * 128 + blk * 32;
    uint32_t w[32];
    if constexpr (T == kTypeF32) {
      const uint32_t *src = static_cast<const uint32_t *>(X) + k0 * ldx + n0;
#pragma unroll
      for (int k = 0; k < 32; ++k) w[k] = n0 < rows && k0 + k < cols ? src[k * ldx] : 0u;
    } else {
      const unsigned short *src = static_cast<const unsigned short *>(X) + k0 * ldx + n0;
      if (pair_aligned && n0 + 1 < rows) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          w[k] = k0 + k < cols ? *reinterpret_cast<const uint32_t *>(src + k * ldx) : 0u;
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const uint32_t lo = n0 < rows && k0 + k < cols ? src[k * ldx] : 0u;
          const uint32_t hi = n0 + 1 < rows && k0 + k < cols ? src[k * ldx + 1] : 0u;
          w[k] = lo | (hi << 16);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < W; ++h) {
      float v[32];
      uint32_t amax;
      if constexpr (T == kTypeF32) {
        amax = amax_bits<T, 32>(w);
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(w[k]);
      } else {
        uint32_t m[1] = {0};
#pragma unroll
        for (int k = 0; k < 32; ++k) m[0] = max_u16x2(m[0], w[k] & 0x7fff7fffu);
        m[0] = h == 0 ? m[0] & 0xffffu : m[0] >> 16;
        amax = amax_bits<T, 1>(m);
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          float lo, hi;
          unpack2<T>(w[k], lo, hi);
          v[k] = h == 0 ? lo : hi;
        }
      }
      const uint32_t byte = scale_byte<FMT>(amax);
      uint32_t q[kQWords<FMT, 32>];
      encode<FMT, 32>(v, inverse_scale(byte), q);
      const int n = n_in + h;
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        elems[place(n, blk * kPieces + i)] = make_uint4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
      scales[(n & 31) * 16 + (n >> 5) * 4 + blk] = static_cast<uint8_t>(byte);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 128 * kRowPieces; i += blockDim.x) {
      const int n = i / kRowPieces, piece = i % kRowPieces;
      const int64_t row = tr * 128 + n;
      const int64_t at = tc * kRowPieces + piece;  // piece of the whole row
      if (row < rows && at < static_cast<int64_t>(o.blocks) * kPieces)
        *reinterpret_cast<uint4 *>(const_cast<uint8_t *>(o.q) + row * o.ldq + at * 16) = elems[place(n, piece)];
    }
    if (threadIdx.x < 128) {
      const int i = threadIdx.x;  // word i of the scale tile: four blocks of row (i % 4) * 32 + i / 4
      if (tr * 128 + (i & 3) * 32 + (i >> 2) < rows)
        reinterpret_cast<uint32_t *>(const_cast<uint8_t *>(o.s) + (tr * o.tiles_x + tc) * 512)[i] =
            reinterpret_cast<const uint32_t *>(scales)[i];
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ backward

// dZ = dY act'(Z), Z from its 8-bit checkpoint, and the column sums of dZ before rounding.
// A CTA owns one chunk of columns and the rows [blockIdx.y * rows_per, +rows_per); its warps
// take rows in turn and keep the sums of their columns in registers.  The warps' sums are
// added in warp order and written to part[blockIdx.y][cols] (or straight to dbias when one
// CTA covers all rows), so the result does not depend on timing.
template <int T, bool SUM>
__global__ void __launch_bounds__(kRowThreads)
    act_backward_kernel(const RowMat dy, const MxMat z, const RowMat dz, int act, int64_t rows,
                        int64_t cols, int64_t rows_per, float *part) {
  constexpr int E = kLaneElems<T>;
  constexpr int kLanesPerBlock = kMxBlock / E;
  __shared__ __align__(16) uint32_t stage[kRowWarps][256];
  __shared__ __align__(16) float sums[SUM ? kRowWarps : 1][SUM ? 32 * E : 4];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * (32 * E);
  const int block = static_cast<int>(c0 / kMxBlock) + lane / kLanesPerBlock;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * rows_per;
  const int64_t r1 = min(rows, r0 + rows_per);
  float acc[E];
#pragma unroll
  for (int j = 0; j < E; ++j) acc[j] = 0.0f;
  for (int64_t r = r0 + warp; r < r1; r += kRowWarps) {
    uint32_t w[8];
    uint32_t q[kQWords<kE4M3, E>] = {};
    uint32_t byte = 0;
    if (block < z.blocks) {
      load_q<kE4M3, E>(z.q + r * z.ldq + static_cast<int64_t>(block) * kBlockBytes<kE4M3> +
                           (lane % kLanesPerBlock) * kQWords<kE4M3, E> * 4,
                       q);
      byte = z.s[scale_offset(r, block, z.tiles_x)];
    }
    load_lane<T>(dy, r, c0, cols, lane, stage[warp], w);
    float v[E], d[E];
    decode<kE4M3, E>(q, scale_value(byte), v);
    to_floats<T, E>(w, d);
    slope_lane<E>(act, v, d);
    if constexpr (SUM) {
#pragma unroll
      for (int j = 0; j < E; j += 2) f2_add_to(acc[j], acc[j + 1], d[j], d[j + 1]);
    }
    from_floats<T, E>(d, w);
    store_lane<T>(dz, r, c0, cols, lane, stage[warp], w);
  }
  if constexpr (SUM) {
#pragma unroll
    for (int j = 0; j < E; j += 4)
      *reinterpret_cast<float4 *>(&sums[warp][lane * E + j]) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
    __syncthreads();
    for (int c = threadIdx.x; c < 32 * E && c0 + c < cols; c += kRowThreads) {
      float s = sums[0][c];
#pragma unroll
      for (int i = 1; i < kRowWarps; ++i) s += sums[i][c];
      part[static_cast<int64_t>(blockIdx.y) * cols + c0 + c] = s;
    }
  }
}

// dbias[c] = the sum over `parts` partial sums, in order.
__global__ void __launch_bounds__(128) column_sum_kernel(const float *part, int parts, int64_t cols, float *dbias) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
  if (c >= cols) return;
  float s = 0.0f;
#pragma unroll 8
  for (int i = 0; i < parts; ++i) s += part[i * cols + c];
  dbias[c] = s;
}

// ------------------------------------------------------------------ host side

RowMat row_mat(const void *p, int64_t ld, int type) {
  return {p, ld, aligned16(p) && (ld * type_bytes(type)) % 16 == 0 ? 1 : 0};
}

MxMat mx_mat(const void *Q, int64_t ldq, const void *S, int64_t cols) {
  return {static_cast<const uint8_t *>(Q), ldq, static_cast<const uint8_t *>(S), scale_tiles_x(cols),
          static_cast<int>(mx_blocks(cols))};
}

// Launches as a programmatic dependent of the previous kernel in the stream: every kernel
// here waits for that one to complete before it touches memory, so only launch latency and
// set-up overlap.
template <typename... P, typename... A>
tlg_status launch(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
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
tlg_status with_format(int format, F f) {
  return format == TLG_MX_E2M1 ? f(std::integral_constant<int, kE2M1>()) : f(std::integral_constant<int, kE4M3>());
}

// Column chunks of a row kernel, and its grid: one warp an item up to eight 256-thread blocks
// an SM, then each warp takes several.
int chunks_of(int type, int64_t cols) {
  const int64_t c = 32 * 32 / type_bytes(type);
  return static_cast<int>((cols + c - 1) / c);
}

dim3 row_grid(int64_t rows, int chunks, int sms) {
  const int64_t blocks = (rows * chunks + kRowWarps - 1) / kRowWarps;
  return dim3(static_cast<unsigned>(std::min<int64_t>(blocks, int64_t(sms) * 8)));
}

// Row splits of the backward kernel: enough CTAs to fill the device, each warp with a few rows.
int backward_splits(int64_t rows, int chunks, int sms) {
  const int64_t want = (int64_t(sms) * 4 + chunks - 1) / chunks;
  const int64_t most = (rows + 4 * kRowWarps - 1) / (4 * kRowWarps);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({want, most, 65535})));
}

}  // namespace
}  // namespace tlg

using namespace tlg;

extern "C" {

tlg_status tlg_mx_size(tlg_mx_format format, int64_t rows, int64_t cols, int64_t *q_row_bytes, size_t *s_bytes) {
  if (q_row_bytes == nullptr || s_bytes == nullptr) return TLG_ERR_INVALID_ARG;
  *q_row_bytes = 0;
  *s_bytes = 0;
  if (!valid_format(format)) return TLG_ERR_INVALID_ARG;
  const tlg_status es = check_extents(rows, cols);
  if (es != TLG_OK) return es;
  *q_row_bytes = row_bytes(format, cols);
  *s_bytes = static_cast<size_t>(scale_bytes(rows, cols));
  return TLG_OK;
}

tlg_status tlg_mx_quantize(tlg_mx_format format, int64_t rows, int64_t cols, tlg_op op, tlg_type type, const void *X,
                           int64_t ldx, void *Q, int64_t ldq, void *S, void *stream) {
  if (!valid_format(format) || !valid_type(type) || (op != TLG_OP_N && op != TLG_OP_T)) return TLG_ERR_INVALID_ARG;
  tlg_status st = check_extents(rows, cols);
  if (st != TLG_OK || rows == 0 || cols == 0) return st;
  const bool t = op == TLG_OP_T;
  Range rx, rq, rs;
  st = check_matrix(X, t ? cols : rows, t ? rows : cols, ldx, type_bytes(type), &rx);
  if (st != TLG_OK) return st;
  st = check_mx(format, rows, cols, Q, ldq, S, &rq, &rs);
  if (st != TLG_OK) return st;
  if (meets(rx, rq) || meets(rx, rs) || meets(rq, rs)) return TLG_ERR_INVALID_ARG;
  DeviceInfo info;
  st = device_ready({X, Q, S}, &info);
  if (st != TLG_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const MxMat o = mx_mat(Q, ldq, S, cols);
  return with_type(type, [&](auto T) {
    return with_format(format, [&](auto F) {
      constexpr int kT = decltype(T)::value, kF = decltype(F)::value;
      if (t) {
        const int64_t tiles_r = (rows + 127) / 128, tiles = tiles_r * o.tiles_x;
        const int pair = (reinterpret_cast<uintptr_t>(X) % 4 == 0 && ldx % 2 == 0) ? 1 : 0;
        return launch(quantize_cols_kernel<kT, kF>, dim3(static_cast<unsigned>(std::min<int64_t>(tiles, 1 << 30))),
                      kT == kTypeF32 ? 512 : 256, s, X, ldx, pair, o, rows, cols, tiles_r, tiles);
      }
      const int chunks = chunks_of(type, cols);
      return launch(quantize_rows_kernel<kT, kF, false>, row_grid(rows, chunks, info.sm_count), kRowThreads, s,
                    row_mat(X, ldx, type), o, RowMat{}, 0, rows, cols, chunks);
    });
  });
}

tlg_status tlg_mx_dequantize(tlg_mx_format format, int64_t rows, int64_t cols, const void *Q, int64_t ldq,
                             const void *S, tlg_type type, void *X, int64_t ldx, void *stream) {
  if (!valid_format(format) || !valid_type(type)) return TLG_ERR_INVALID_ARG;
  tlg_status st = check_extents(rows, cols);
  if (st != TLG_OK || rows == 0 || cols == 0) return st;
  Range rx, rq, rs;
  st = check_matrix(X, rows, cols, ldx, type_bytes(type), &rx);
  if (st != TLG_OK) return st;
  st = check_mx(format, rows, cols, Q, ldq, S, &rq, &rs);
  if (st != TLG_OK) return st;
  if (meets(rx, rq) || meets(rx, rs)) return TLG_ERR_INVALID_ARG;
  DeviceInfo info;
  st = device_ready({X, Q, S}, &info);
  if (st != TLG_OK) return st;
  const MxMat in = mx_mat(Q, ldq, S, cols);
  const int chunks = chunks_of(type, cols);
  return with_type(type, [&](auto T) {
    return with_format(format, [&](auto F) {
      return launch(dequantize_rows_kernel<decltype(T)::value, decltype(F)::value>,
                    row_grid(rows, chunks, info.sm_count), kRowThreads, static_cast<cudaStream_t>(stream), in,
                    row_mat(X, ldx, type), rows, cols, chunks);
    });
  });
}

tlg_status tlg_act_forward_mx(int64_t rows, int64_t cols, tlg_activation activation, tlg_type type, const void *Z,
                              int64_t ldz, void *Y, int64_t ldy, void *Q, int64_t ldq, void *S, void *stream) {
  if (!valid_activation(activation) || !valid_type(type)) return TLG_ERR_INVALID_ARG;
  tlg_status st = check_extents(rows, cols);
  if (st != TLG_OK || rows == 0 || cols == 0) return st;
  Range rz, ry, rq, rs;
  st = check_matrix(Z, rows, cols, ldz, type_bytes(type), &rz);
  if (st != TLG_OK) return st;
  st = check_matrix(Y, rows, cols, ldy, type_bytes(type), &ry);
  if (st != TLG_OK) return st;
  st = check_mx(TLG_MX_E4M3, rows, cols, Q, ldq, S, &rq, &rs);
  if (st != TLG_OK) return st;
  if (meets(ry, rz) && !(Y == Z && ldy == ldz)) return TLG_ERR_INVALID_ARG;
  if (meets(rz, rq) || meets(rz, rs) || meets(ry, rq) || meets(ry, rs) || meets(rq, rs)) return TLG_ERR_INVALID_ARG;
  DeviceInfo info;
  st = device_ready({Z, Y, Q, S}, &info);
  if (st != TLG_OK) return st;
  const MxMat o = mx_mat(Q, ldq, S, cols);
  const int chunks = chunks_of(type, cols);
  return with_type(type, [&](auto T) {
    return launch(quantize_rows_kernel<decltype(T)::value, kE4M3, true>, row_grid(rows, chunks, info.sm_count),
                  kRowThreads, static_cast<cudaStream_t>(stream), row_mat(Z, ldz, type), o, row_mat(Y, ldy, type),
                  static_cast<int>(activation), rows, cols, chunks);
  });
}

tlg_status tlg_act_backward_mx_workspace_size(int64_t rows, int64_t cols, tlg_type type, size_t *bytes) {
  if (bytes == nullptr) return TLG_ERR_INVALID_ARG;
  *bytes = 0;
  if (!valid_type(type)) return TLG_ERR_INVALID_ARG;
  const tlg_status es = check_extents(rows, cols);
  if (es != TLG_OK || rows == 0 || cols == 0) return es;
  int dev = 0;
  DeviceInfo info;
  const tlg_status ds = current_device(&dev, &info);
  if (ds != TLG_OK) return ds;
  const int splits = backward_splits(rows, chunks_of(type, cols), info.sm_count);
  *bytes = splits > 1 ? static_cast<size_t>(splits) * static_cast<size_t>(cols) * 4 : 0;
  return TLG_OK;
}

tlg_status tlg_act_backward_mx(int64_t rows, int64_t cols, tlg_activation activation, tlg_type type, const void *dY,
                               int64_t lddy, const void *Q, int64_t ldq, const void *S, void *dZ, int64_t lddz,
                               float *dbias, void *workspace, size_t workspace_bytes, void *stream) {
  if (!valid_activation(activation) || !valid_type(type)) return TLG_ERR_INVALID_ARG;
  tlg_status st = check_extents(rows, cols);
  if (st != TLG_OK || cols == 0) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Range rb = {0, 0}, rw = {0, 0};
  if (dbias != nullptr) {
    if (reinterpret_cast<uintptr_t>(dbias) % 4 != 0) return TLG_ERR_ALIGNMENT;
    rb.lo = reinterpret_cast<uintptr_t>(dbias);
    rb.hi = rb.lo + static_cast<uintptr_t>(cols) * 4;
  }
  if (workspace != nullptr) {
    if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return TLG_ERR_ALIGNMENT;
    rw.lo = reinterpret_cast<uintptr_t>(workspace);
    rw.hi = rw.lo + workspace_bytes;
  }
  DeviceInfo info;
  if (rows == 0) {  // the sum over no rows
    if (dbias == nullptr) return TLG_OK;
    st = device_ready({dbias}, &info);
    if (st != TLG_OK) return st;
    if (cudaMemsetAsync(dbias, 0, static_cast<size_t>(cols) * 4, s) != cudaSuccess) {
      cudaGetLastError();
      return TLG_ERR_CUDA;
    }
    return TLG_OK;
  }
  Range ry, rz, rq, rs;
  st = check_matrix(dY, rows, cols, lddy, type_bytes(type), &ry);
  if (st != TLG_OK) return st;
  st = check_matrix(dZ, rows, cols, lddz, type_bytes(type), &rz);
  if (st != TLG_OK) return st;
  st = check_mx(TLG_MX_E4M3, rows, cols, Q, ldq, S, &rq, &rs);
  if (st != TLG_OK) return st;
  if (meets(ry, rz) && !(dY == dZ && lddy == lddz)) return TLG_ERR_INVALID_ARG;
  if (meets(rz, rq) || meets(rz, rs)) return TLG_ERR_INVALID_ARG;
  for (const Range &r : {ry, rz, rq, rs})
    if ((dbias != nullptr && meets(rb, r)) || (workspace != nullptr && meets(rw, r))) return TLG_ERR_INVALID_ARG;
  if (dbias != nullptr && workspace != nullptr && meets(rb, rw)) return TLG_ERR_INVALID_ARG;
  st = device_ready({dY, Q, S, dZ, dbias, workspace}, &info);
  if (st != TLG_OK) return st;
  const int chunks = chunks_of(type, cols);
  const int splits = backward_splits(rows, chunks, info.sm_count);
  const int64_t rows_per = (rows + splits - 1) / splits;
  float *part = dbias;
  if (dbias != nullptr && splits > 1) {
    if (workspace == nullptr || workspace_bytes < static_cast<size_t>(splits) * static_cast<size_t>(cols) * 4)
      return TLG_ERR_INVALID_ARG;
    part = static_cast<float *>(workspace);
  }
  const MxMat z = mx_mat(Q, ldq, S, cols);
  const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>(splits));
  st = with_type(type, [&](auto T) {
    constexpr int kT = decltype(T)::value;
    const RowMat dy = row_mat(dY, lddy, type), dz = row_mat(dZ, lddz, type);
    return dbias != nullptr ? launch(act_backward_kernel<kT, true>, grid, kRowThreads, s, dy, z, dz,
                                     static_cast<int>(activation), rows, cols, rows_per, part)
                            : launch(act_backward_kernel<kT, false>, grid, kRowThreads, s, dy, z, dz,
                                     static_cast<int>(activation), rows, cols, rows_per, part);
  });
  if (st != TLG_OK || part == dbias) return st;
  return launch(column_sum_kernel, dim3(static_cast<unsigned>((cols + 127) / 128)), 128, s, part, splits, cols, dbias);
}

}  // extern "C"
