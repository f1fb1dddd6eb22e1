// Microscaled (MX) elementwise operators: quantisation of a matrix or its transpose,
// dequantisation, the activation that saves its input in 8 bits and the backward pass that
// reads it.  All of them are bound by HBM traffic: every kernel reads each input byte once
// and writes each output byte once, 16 bytes a lane where rows are aligned.
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

// The row kernels: a warp owns a stripe of U * 32 * E columns (U pieces of 32 * E) and some of the
// rows [blockIdx.y * rows_per, +rows_per) of its CTA.  Of one row it loads all U pieces before it
// works on the first (16 * U bytes a lane in flight); with the columns fixed, each row costs a
// few pointer steps, and the pieces of a row are constant distances apart in every matrix.  (An
// item-at-a-time walk over rows and pieces spent 13 instructions an element on quantising, most
// of them on addresses.)  2^across of a CTA's warps lie side by side, the others take the next
// rows.
template <int T, int U>
struct Stripe {
  static constexpr int E = kLaneElems<T>;
  static constexpr int kPiece = 32 * E;              // columns of a piece
  static constexpr int kPieceScales = kPiece / kMxBlock / 4 * 512;  // bytes between two pieces' scales
  uint32_t c0;    // first column
  int left;       // columns from c0 on, 0 for a warp past the last one
  int block;      // this lane's block in piece 0
  uint32_t r, step, r1;  // this warp's rows: r, r + step, ... below r1
  __device__ __forceinline__ Stripe(uint32_t rows, uint32_t cols, uint32_t rows_per, int across, int lane, int warp) {
    const int side = warp & ((1 << across) - 1);
    const uint32_t at = ((blockIdx.x << across) + static_cast<uint32_t>(side)) * (kPiece * U);
    const uint32_t r0 = blockIdx.y * rows_per;
    const bool in = at < cols;
    c0 = in ? at : 0;
    left = in ? static_cast<int>(min(cols - c0, uint32_t(kPiece * U))) : 0;
    block = static_cast<int>(c0 / kMxBlock) + lane * E / kMxBlock;
    r1 = in ? min(rows, r0 + rows_per) : 0;
    r = r0 + (warp >> across);
    step = kRowWarps >> across;
  }
  // Bytes of this lane's elements in a row of an ordinary matrix / of an MX matrix.
  __device__ __forceinline__ int64_t at(int lane, bool vec) const {
    return static_cast<int64_t>(c0) * kTypeBytes<T> + (vec ? lane * 16 : 0);
  }
  template <int FMT>
  __device__ __forceinline__ int64_t q_at(int lane) const {
    return static_cast<int64_t>(c0 / E) * kQBytes<FMT, E> + lane * kQBytes<FMT, E>;
  }
};

// Scale offset of (row, block 0 of its tile row), the part that depends on the row.
__device__ __forceinline__ int64_t scale_row(uint32_t row, int64_t tile_row_bytes) {
  return (row >> 7) * tile_row_bytes + ((row & 31) * 16 + ((row >> 5) & 3) * 4);
}

// CTAs an SM.  Rows that are not aligned wait for shared memory as well as for their loads: 16-bit ones
// do best with five (8000 x 8191 bf16 to 4 bits 51 us, 66 with three), fp32 ones, whose registers
// would spill, with three (4000 x 8191: 37 us, 51 with five).
constexpr int quantize_ctas(int type, bool vec) { return vec ? 4 : type == kTypeF32 ? 3 : 5; }

// Quantises X row by row; with ACT also writes Y = act(X).  The lanes of a block (4 of 16-bit
// elements, 8 of fp32) agree on its largest magnitude by shuffles.
template <int T, int FMT, bool ACT, bool VEC, int U>
__global__ void __launch_bounds__(kRowThreads, quantize_ctas(T, VEC))
    quantize_rows_kernel(const RowMat x, const MxMat o, const RowMat y, int act, uint32_t rows,
                         uint32_t cols, uint32_t rows_per, int across) {
  using St = Stripe<T, U>;
  constexpr int E = St::E, B = kTypeBytes<T>;
  constexpr int kLanesPerBlock = kMxBlock / E;
  // Rows read element by element are loaded a row ahead, over the shared-memory round trip of the
  // row before (4000 x 3001 fp32 to 4 bits: 12.4 us, 13.6 without); with whole 16-byte loads the
  // registers are better spent on a fourth CTA (8192 x 16384 bf16: 53.6 us against 60).
  constexpr bool kAheadOne = !VEC;
  __shared__ __align__(16) uint32_t stage[VEC ? 1 : kRowWarps][128];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t *st = stage[VEC ? 0 : warp];
  const St s(rows, cols, rows_per, across, lane, warp);
  const int64_t tile_row = o.tiles_x * 512;
  const char *src = static_cast<const char *>(x.p) + static_cast<int64_t>(s.r) * x.ld * B + s.at(0, false);
  char *dst = static_cast<char *>(const_cast<void *>(y.p)) + static_cast<int64_t>(s.r) * y.ld * B + s.at(0, false);
  uint8_t *oq = const_cast<uint8_t *>(o.q) + static_cast<int64_t>(s.r) * o.ldq + s.template q_at<FMT>(lane);
  uint8_t *os = const_cast<uint8_t *>(o.s) + scale_offset(0, s.block, o.tiles_x);
  // Whole stripes (all but the last) need no column checks.
  auto run = [&](auto full) {
    constexpr bool kFull = decltype(full)::value;
    uint32_t next[U][4], first_next[U] = {};  // the row to work on next
    bool inside_next = false;
    auto issue = [&]() {
      inside_next = starts_inside_word<T, VEC>(src);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (kFull || u * St::kPiece < s.left)
          issue_load<T, VEC, kFull>(src + u * (St::kPiece * B), s.left - u * St::kPiece, lane, next[u], first_next[u]);
      src += s.step * x.ld * B;
    };
    if (kAheadOne && s.r < s.r1) issue();
    for (uint32_t r = s.r; r < s.r1; r += s.step) {
      if (!kAheadOne) issue();
      uint32_t w[U][4], first[U];
      const bool inside = inside_next;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        first[u] = first_next[u];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[u][j] = next[u][j];
      }
      if (kAheadOne && r + s.step < s.r1) issue();
      const int64_t sr = scale_row(r, tile_row);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (kFull || u * St::kPiece < s.left) {
          float v[E];
          finish_load<T, VEC>(lane, inside, first[u], st, w[u]);
          to_floats<T, E>(w[u], v);
          uint32_t m = amax_bits<T, 4>(w[u]);
#pragma unroll
          for (int d = 1; d < kLanesPerBlock; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
          const uint32_t byte = scale_byte<FMT>(m);
          uint32_t q[kQWords<FMT, E>];
          encode<FMT, E>(v, inverse_scale(byte), q);
          const int block = s.block + u * (St::kPiece / kMxBlock);
          if (kFull || block < o.blocks) store_q<FMT, E>(oq + u * (32 * kQBytes<FMT, E>), q);
          // blocks past the last one, up to a whole group of four, hold no elements: their scale is 0
          if (lane % kLanesPerBlock == 0 && (kFull || (block >> 2) < o.tiles_x))
            os[sr + u * St::kPieceScales] = static_cast<uint8_t>(byte);
          if constexpr (ACT) {
            activate_lane<T, E>(act, v);
            from_floats<T, E>(v, w[u]);
            store_lane<T, VEC, kFull>(dst + u * (St::kPiece * B), s.left - u * St::kPiece, lane, st, w[u]);
          }
        }
      }
      oq += s.step * o.ldq;
      if constexpr (ACT) dst += s.step * y.ld * B;
    }
  };
  if (s.left == St::kPiece * U)
    run(std::true_type());
  else
    run(std::false_type());
}

template <int T, int FMT, bool VEC, int U>
__global__ void __launch_bounds__(kRowThreads, 4)
    dequantize_rows_kernel(const MxMat in, const RowMat x, uint32_t rows, uint32_t cols, uint32_t rows_per, int across) {
  using St = Stripe<T, U>;
  constexpr int E = St::E, B = kTypeBytes<T>;
  __shared__ __align__(16) uint32_t stage[VEC ? 1 : kRowWarps][128];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t *st = stage[VEC ? 0 : warp];
  const St s(rows, cols, rows_per, across, lane, warp);
  const int64_t tile_row = in.tiles_x * 512;
  char *dst = static_cast<char *>(const_cast<void *>(x.p)) + static_cast<int64_t>(s.r) * x.ld * B + s.at(0, false);
  const uint8_t *iq = in.q + static_cast<int64_t>(s.r) * in.ldq + s.template q_at<FMT>(lane);
  const uint8_t *is = in.s + scale_offset(0, s.block, in.tiles_x);
  // Whole stripes (all but the last) need no column checks.
  auto run = [&](auto full) {
    constexpr bool kFull = decltype(full)::value;
    for (uint32_t r = s.r; r < s.r1; r += s.step) {
      MxLane<FMT, E> q[U];
      const int64_t sr = scale_row(r, tile_row);
#pragma unroll
      for (int u = 0; u < U; ++u)
        issue_load_mx<FMT, E>(iq + u * (32 * kQBytes<FMT, E>), is + sr + u * St::kPieceScales,
                              kFull || s.block + u * (St::kPiece / kMxBlock) < in.blocks, q[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (kFull || u * St::kPiece < s.left) {
          float v[E];
          uint32_t w[4];
          decode<FMT, E>(q[u].q, scale_value(q[u].byte), v);
          from_floats<T, E>(v, w);
          store_lane<T, VEC, kFull>(dst + u * (St::kPiece * B), s.left - u * St::kPiece, lane, st, w);
        }
      }
      dst += s.step * x.ld * B;
      iq += s.step * in.ldq;
    }
  };
  if (s.left == St::kPiece * U)
    run(std::true_type());
  else
    run(std::false_type());
}

// ------------------------------------------------------------------ transposed quantisation

// Quantises X^T, X stored cols x rows (rows of Q are columns of X).  A CTA takes 128 rows of Q
// by 128 columns (four blocks, one scale tile): warp (block, part) reads the block's 32 rows of
// X, each lane 4 bytes of a row (two rows of Q of a 16-bit type, one of fp32), so a thread
// holds whole blocks and finds their scale without any exchange.  Elements then go through
// shared memory, so that each row of Q is written in pieces of four blocks (64 or 128 bytes).
// The 32 loads of a thread are all in flight at once; three CTAs an SM (768 or 1024 threads) let one
// load while others convert (8192 x 8192 bf16 to 4 bits: 31.4 us, 34.9 with four and 37.9 with the two
// that the registers ptxas would take allow; its bytes take 26).
template <int T, int FMT>
__global__ void __launch_bounds__(T == kTypeF32 ? 512 : 256, T == kTypeF32 ? 2 : 3)
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
    if (pair_aligned && tr * 128 + 128 <= rows && tc * 128 + 128 <= cols) {
      // A whole tile: no element is checked.
      const char *src = static_cast<const char *>(X) + (k0 * ldx + n0) * kTypeBytes<T>;
      const int64_t step = ldx * kTypeBytes<T>;
#pragma unroll
      for (int k = 0; k < 32; ++k, src += step) w[k] = *reinterpret_cast<const uint32_t *>(src);
    } else if constexpr (T == kTypeF32) {
      const uint32_t *src = static_cast<const uint32_t *>(X) + k0 * ldx + n0;
#pragma unroll
      for (int k = 0; k < 32; ++k) w[k] = n0 < rows && k0 + k < cols ? src[k * ldx] : 0u;
    } else {
      const unsigned short *src = static_cast<const unsigned short *>(X) + k0 * ldx + n0;
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const uint32_t lo = n0 < rows && k0 + k < cols ? src[k * ldx] : 0u;
        const uint32_t hi = n0 + 1 < rows && k0 + k < cols ? src[k * ldx + 1] : 0u;
        w[k] = lo | (hi << 16);
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
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 32; ++k) m = max_abs2<T>(m, w[k]);
        amax = magnitude_bits<T>(h == 0 ? m & 0xffffu : m >> 16);
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

// Copies 16 bytes to shared memory asynchronously, in this thread's current group.
__device__ __forceinline__ void copy_async_16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows a warp of the backward kernel has on their way while it works on one.
constexpr int kAhead = 2;

// dZ = dY act'(Z), Z from its 8-bit checkpoint, and the column sums of dZ before rounding.
// Each warp keeps the sums of its stripe's columns in registers.  The warps' sums are
// added in warp order and written to part[blockIdx.y][cols] (or straight to dbias when one
// CTA covers all rows), so the result does not depend on timing.
//
// Two input streams, the sums and the derivative leave no registers for loads in flight, so
// whole stripes of aligned rows come through shared memory, 16 bytes a lane of the next kAhead
// rows copied asynchronously (8192 x 8192 bf16, SiLU: 74 us loading to registers, 1.4 times the
// time of its bytes).  The scales, a byte for 32 elements, are loaded a row ahead.
template <int T, bool SUM, bool VEC, int U>
__global__ void __launch_bounds__(kRowThreads, VEC ? 4 : 3)
    act_backward_kernel(const RowMat dy, const MxMat z, const RowMat dz, int act, uint32_t rows,
                        uint32_t cols, uint32_t rows_per, int across, float *part) {
  using St = Stripe<T, U>;
  constexpr int E = St::E, B = kTypeBytes<T>;
  constexpr int kQ = kQBytes<kE4M3, E>;
  constexpr int kCols = St::kPiece * U;
  struct Ahead {
    uint4 dy[kAhead + 1][U][kRowThreads];
    uint8_t q[kAhead + 1][kRowWarps][U * 32 * kQ];
  };
  union Shared {
    Ahead ahead[VEC ? 1 : 0];
    uint32_t stage[VEC ? 0 : kRowWarps][128];
    float sums[kRowWarps][SUM ? kCols : 4];
  };
  __shared__ __align__(16) Shared sh;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const St s(rows, cols, rows_per, across, lane, warp);
  const int64_t tile_row = z.tiles_x * 512;
  const char *src = static_cast<const char *>(dy.p) + static_cast<int64_t>(s.r) * dy.ld * B + s.at(0, false);
  char *dst = static_cast<char *>(const_cast<void *>(dz.p)) + static_cast<int64_t>(s.r) * dz.ld * B + s.at(0, false);
  const uint8_t *zq = z.q + static_cast<int64_t>(s.r) * z.ldq + s.template q_at<kE4M3>(lane);
  float acc[U][E];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = 0; j < E; ++j) acc[u][j] = 0.0f;
  // One piece of a row: w holds dY's elements, q and byte Z's.
  auto work = [&](int u, uint32_t(&w)[4], const uint32_t(&q)[kQWords<kE4M3, E>], uint32_t byte) {
    float v[E], d[E];
    decode<kE4M3, E>(q, scale_value(byte), v);
    to_floats<T, E>(w, d);
    slope_lane<E>(act, v, d);
    if constexpr (SUM) {
#pragma unroll
      for (int j = 0; j < E; j += 2) f2_add_to(acc[u][j], acc[u][j + 1], d[j], d[j + 1]);
    }
    from_floats<T, E>(d, w);
  };
  if (VEC && s.left == kCols) {
    if constexpr (VEC) {
      Ahead &a = sh.ahead[0];
      const int tid = threadIdx.x;
      const uint8_t *zs = z.s + scale_offset(0, s.block, z.tiles_x);
      const char *fsrc = src + lane * 16;  // of the row to fetch next
      const uint8_t *fq = zq - lane * kQ + lane * 16;
      uint32_t fr = s.r;
      auto fetch = [&](int slot) {
        if (fr < s.r1) {
#pragma unroll
          for (int u = 0; u < U; ++u) copy_async_16(&a.dy[slot][u][tid], fsrc + u * (St::kPiece * B));
          if (lane * 16 < U * 32 * kQ) copy_async_16(&a.q[slot][warp][lane * 16], fq);
        }
        copy_async_commit();
        fr += s.step;
        fsrc += s.step * dy.ld * B;
        fq += s.step * z.ldq;
      };
      uint32_t bytes[U];
      auto fetch_scales = [&](uint32_t r) {
        if (r < s.r1) {
#pragma unroll
          for (int u = 0; u < U; ++u) bytes[u] = zs[scale_row(r, tile_row) + u * St::kPieceScales];
        }
      };
      int slot = 0;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) fetch(i);
      fetch_scales(s.r);
      for (uint32_t r = s.r; r < s.r1; r += s.step) {
        copy_async_wait<kAhead - 1>();
        __syncwarp();  // every lane's copies of this row have landed, and the row before is read
        fetch(slot == 0 ? kAhead : slot - 1);  // into the slot of the row before
        uint32_t now[U];
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = bytes[u];
        fetch_scales(r + s.step);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint4 x = a.dy[slot][u][tid];
          uint32_t w[4] = {x.x, x.y, x.z, x.w};
          uint32_t q[kQWords<kE4M3, E>];
          load_q<kE4M3, E>(&a.q[slot][warp][(u * 32 + lane) * kQ], q);
          work(u, w, q, now[u]);
          store_lane<T, true, true>(dst + u * (St::kPiece * B), kCols, lane, nullptr, w);
        }
        dst += s.step * dz.ld * B;
        slot = slot == kAhead ? 0 : slot + 1;
      }
      copy_async_wait<0>();
    }
  } else {
    uint32_t *st = VEC ? nullptr : sh.stage[VEC ? 0 : warp];
    const uint8_t *zs = z.s + scale_offset(0, s.block, z.tiles_x);
    for (uint32_t r = s.r; r < s.r1; r += s.step) {
      uint32_t w[U][4], first[U] = {};
      MxLane<kE4M3, E> q[U];
      const int64_t sr = scale_row(r, tile_row);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        issue_load_mx<kE4M3, E>(zq + u * (32 * kQ), zs + sr + u * St::kPieceScales,
                                s.block + u * (St::kPiece / kMxBlock) < z.blocks, q[u]);
        if (u * St::kPiece < s.left)
          issue_load<T, VEC, false>(src + u * (St::kPiece * B), s.left - u * St::kPiece, lane, w[u], first[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u * St::kPiece < s.left) {
          finish_load<T, VEC>(lane, starts_inside_word<T, VEC>(src), first[u], st, w[u]);
          work(u, w[u], q[u].q, q[u].byte);
          store_lane<T, VEC, false>(dst + u * (St::kPiece * B), s.left - u * St::kPiece, lane, st, w[u]);
        }
      }
      src += s.step * dy.ld * B;
      dst += s.step * dz.ld * B;
      zq += s.step * z.ldq;
    }
  }
  if constexpr (SUM) __syncthreads();  // every warp is done with its part of the shared memory
  if constexpr (SUM) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < E; j += 4)
        *reinterpret_cast<float4 *>(&sh.sums[warp][u * St::kPiece + lane * E + j]) =
            make_float4(acc[u][j], acc[u][j + 1], acc[u][j + 2], acc[u][j + 3]);
    __syncthreads();
    const int span = kCols << across;  // the CTA's columns
    const uint32_t first = blockIdx.x * static_cast<uint32_t>(span);
    for (int c = threadIdx.x; c < span && first + c < cols; c += kRowThreads) {
      const int side = c / kCols;
      float t = sh.sums[side][c % kCols];
      for (int i = side + (1 << across); i < kRowWarps; i += 1 << across) t += sh.sums[i][c % kCols];
      part[static_cast<int64_t>(blockIdx.y) * cols + (first + c)] = t;
    }
  }
}

// dbias[c] = the sum over `parts` partial sums: each of a CTA's W warps takes every W-th one of 32
// columns, and their sums are added in order.  W = 32 where a narrow matrix has hundreds of
// row splits and a warp's chain of loads takes the time (16384 x 1000 fp16, 592 splits, the whole
// backward call: 24.7 us, 30.5 with 8), else 8, which find room beside the kernel before sooner
// (2000 x 5000: 18.3 us, 20.3 with 32).
template <int W>
__global__ void __launch_bounds__(32 * W) column_sum_kernel(const float *part, int parts, int64_t cols, float *dbias) {
  __shared__ float sums[W][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int i = warp; i < parts; i += W) s += part[i * cols + c];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < W; ++i) s += sums[i][lane];
    dbias[c] = s;
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
tlg_status with_flag(bool flag, F f) {
  return flag ? f(std::true_type()) : f(std::false_type());
}

template <typename F>
tlg_status with_format(int format, F f) {
  return format == TLG_MX_E2M1 ? f(std::integral_constant<int, kE2M1>()) : f(std::integral_constant<int, kE4M3>());
}

// Pieces of a row a warp loads at once: several where there are rows enough to fill the
// device all the same, one in small calls.
constexpr int kWide = 4, kWideBackward = 2;

// log2 of the warps of a CTA side by side.  Two in the backward kernel: half the row splits, and
// so half the partial sums (8192 x 16384 bf16, SiLU: 129 us, 142 with one, 134 with eight); the
// others do not care.
constexpr int kAcross = 0, kAcrossBackward = 1;

// A row kernel's grid: column stripes x row splits, about `per_sm` CTAs an SM.
struct RowGrid {
  int u, across;
  dim3 grid;
  uint32_t rows_per;
};

RowGrid row_grid(int64_t rows, int64_t cols, int type, int wide, int most_across, int least_rows, int sms, int per_sm) {
  const int64_t piece = 32 * 16 / type_bytes(type);
  RowGrid g;
  const int64_t items = (rows + kRowWarps - 1) / kRowWarps * ((cols + piece * wide - 1) / (piece * wide));
  g.u = items >= 2 * int64_t(sms) ? wide : 1;
  const int64_t stripes = (cols + piece * g.u - 1) / (piece * g.u);
  // as many warps side by side as leave at most a tenth of them without columns
  g.across = most_across;
  while (g.across > 0 && ((stripes + (int64_t(1) << g.across) - 1) >> g.across << g.across) * 10 > stripes * 11)
    --g.across;
  const int64_t step = kRowWarps >> g.across;
  const int64_t ctas_x = (stripes + (int64_t(1) << g.across) - 1) >> g.across;
  const int64_t row_groups = (rows + step - 1) / step;  // a row to each warp of a CTA
  // Row groups a CTA takes: few enough for per_sm CTAs an SM, and from there on what is done first:
  // the busiest SM's k CTAs take k times as long as one with all the SM's bandwidth, and fewer of
  // them hide less of each other's latency (the 1.5 / k, which ranks 4000 x 3001 fp32 back from
  // 4 bits, 13.8 us with 432 CTAs of seven groups and 16.6 with 504 of six, and 4096 x 4096 bf16 to
  // 4 bits, better with 512 of four than with 296 of seven).
  const int64_t most = std::max<int64_t>(1, std::min<int64_t>(int64_t(sms) * per_sm / ctas_x, 65535));
  const int64_t fewest = std::max<int64_t>({1, (row_groups + most - 1) / most, std::min<int64_t>(least_rows, row_groups)});
  int64_t take = fewest;
  double best = 0;
  for (int64_t c = fewest; c <= 2 * fewest && c < fewest + 16; ++c) {
    const int64_t ctas = ctas_x * ((row_groups + c - 1) / c);
    const double k = static_cast<double>((ctas + sms - 1) / sms);
    const double cost = static_cast<double>(c) * (k + 1.5);
    if (best == 0 || cost < best) {
      best = cost;
      take = c;
    }
  }
  g.rows_per = static_cast<uint32_t>(take * step);
  g.grid = dim3(static_cast<unsigned>(ctas_x), static_cast<unsigned>((rows + g.rows_per - 1) / g.rows_per));
  return g;
}

// The same for the backward kernel, whose splits each leave a partial column sum: at least two
// rows to a warp, and as many CTAs an SM as its registers allow.
RowGrid backward_grid(int64_t rows, int64_t cols, int type, bool vec, int sms) {
  return row_grid(rows, cols, type, kWideBackward, kAcrossBackward, 2, sms, vec ? 4 : 3);
}

// And for quantising: 16-bit rows that are not aligned fill the SM with more CTAs of one piece instead
// (8000 x 8191 bf16 with SiLU: 94 us, 103 with four pieces and three CTAs).
constexpr int quantize_width(int type, bool vec) { return vec || type == kTypeF32 ? kWide : 1; }

RowGrid quantize_grid(int64_t rows, int64_t cols, int type, bool vec, int sms) {
  return row_grid(rows, cols, type, quantize_width(type, vec), kAcross, 1, sms, quantize_ctas(type, vec));
}

// Workspace bytes of its partial sums; the caller does not know which matrices will be aligned.
size_t backward_workspace(int64_t rows, int64_t cols, int type, int sms) {
  const unsigned splits = std::max(backward_grid(rows, cols, type, true, sms).grid.y,
                                   backward_grid(rows, cols, type, false, sms).grid.y);
  return splits > 1 ? static_cast<size_t>(splits) * static_cast<size_t>(cols) * 4 : 0;
}

// Calls f with the pieces a warp takes, 1 or WIDE.
template <int WIDE, typename F>
tlg_status with_width(int u, F f) {
  if constexpr (WIDE > 1) {
    if (u != 1) return f(std::integral_constant<int, WIDE>());
  }
  return f(std::integral_constant<int, 1>());
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
        const int pairs = reinterpret_cast<uintptr_t>(X) % 4 == 0 && ldx * type_bytes(type) % 4 == 0 ? 1 : 0;
        return launch(quantize_cols_kernel<kT, kF>, dim3(static_cast<unsigned>(std::min<int64_t>(tiles, 1 << 30))),
                      kT == kTypeF32 ? 512 : 256, s, X, ldx, pairs, o, rows, cols, tiles_r, tiles);
      }
      const bool vec = vec_rows(X, rows, ldx, type);
      const RowGrid g = quantize_grid(rows, cols, type, vec, info.sm_count);
      return with_flag(vec, [&](auto V) {
        return with_width<quantize_width(kT, decltype(V)::value)>(g.u, [&](auto U) {
          return launch(quantize_rows_kernel<kT, kF, false, decltype(V)::value, decltype(U)::value>, g.grid,
                        kRowThreads, s, RowMat{X, ldx}, o, RowMat{}, 0, rows, cols, g.rows_per, g.across);
        });
      });
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
  const bool vec = vec_rows(X, rows, ldx, type);
  const RowGrid g = row_grid(rows, cols, type, kWide, kAcross, 1, info.sm_count, 4);
  return with_type(type, [&](auto T) {
    return with_format(format, [&](auto F) {
      return with_flag(vec, [&](auto V) {
        return with_width<kWide>(g.u, [&](auto U) {
          return launch(
              dequantize_rows_kernel<decltype(T)::value, decltype(F)::value, decltype(V)::value, decltype(U)::value>,
              g.grid, kRowThreads, static_cast<cudaStream_t>(stream), in, RowMat{X, ldx}, rows, cols, g.rows_per, g.across);
        });
      });
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
  const bool vec = vec_rows(Z, rows, ldz, type) && vec_rows(Y, rows, ldy, type);
  const RowGrid g = quantize_grid(rows, cols, type, vec, info.sm_count);
  return with_type(type, [&](auto T) {
    return with_flag(vec, [&](auto V) {
      return with_width<quantize_width(decltype(T)::value, decltype(V)::value)>(g.u, [&](auto U) {
        return launch(quantize_rows_kernel<decltype(T)::value, kE4M3, true, decltype(V)::value, decltype(U)::value>,
                      g.grid, kRowThreads, static_cast<cudaStream_t>(stream), RowMat{Z, ldz}, o, RowMat{Y, ldy},
                      static_cast<int>(activation), rows, cols, g.rows_per, g.across);
      });
    });
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
  *bytes = backward_workspace(rows, cols, type, info.sm_count);
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
  const bool vec = vec_rows(dY, rows, lddy, type) && vec_rows(dZ, rows, lddz, type);
  const RowGrid g = backward_grid(rows, cols, type, vec, info.sm_count);
  const int splits = static_cast<int>(g.grid.y);
  float *part = dbias;
  if (dbias != nullptr && splits > 1) {
    if (workspace == nullptr || workspace_bytes < backward_workspace(rows, cols, type, info.sm_count))
      return TLG_ERR_INVALID_ARG;
    part = static_cast<float *>(workspace);
  }
  const MxMat z = mx_mat(Q, ldq, S, cols);
  st = with_type(type, [&](auto T) {
    constexpr int kT = decltype(T)::value;
    return with_flag(dbias != nullptr, [&](auto SUM) {
      return with_flag(vec, [&](auto V) {
        return with_width<kWideBackward>(g.u, [&](auto U) {
          return launch(act_backward_kernel<kT, decltype(SUM)::value, decltype(V)::value, decltype(U)::value>, g.grid,
                        kRowThreads, s, RowMat{dY, lddy}, z, RowMat{dZ, lddz}, static_cast<int>(activation), rows,
                        cols, g.rows_per, g.across, part);
        });
      });
    });
  });
  if (st != TLG_OK || part == dbias) return st;
  const dim3 sum_grid(static_cast<unsigned>((cols + 31) / 32));
  return splits > 128 ? launch(column_sum_kernel<32>, sum_grid, 1024, s, part, splits, cols, dbias)
                      : launch(column_sum_kernel<8>, sum_grid, 256, s, part, splits, cols, dbias);
}

}  // extern "C"
