// The root-mean-square norm with the residual's addition, its output in the inputs' type or as a
// microscaled (MX) matrix, and its backward pass.
//
//   forward:  h = x + r,  s = 1 / sqrt(mean(h^2) + eps),  y = h s w
//   backward: with x^ = h s and g = dy w,  dx = s (g - x^ mean(g x^)) + dh,  dw = sum over rows of dy x^
//
// Both are bound by HBM traffic: a row is read once, held in registers while its sum is taken, and
// written once.  `nw` warps share a row; each has up to U pieces of 32 lanes x 16 bytes side by side.
// CTAs are persistent and load their next row before they wait for the sum of this one, so that the
// reduction's latency (two barriers, shuffles) runs under the next row's loads; the weights stay in
// registers.  From HBM, back to back: 8192 x 8192 bf16 with a residual 92 us for 537 MB (5.8 TB/s), to 8 bits about
// 77 us; backward 16384 x 4096 bf16 with dH 89 us for 537 MB (6.0 TB/s, its column sum of 4 us among them).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "tlg.h"
#include "tlg_rows.cuh"

namespace tlg {
namespace {

constexpr int64_t kNormMaxCols = 16384;

// How a row is spread: warps of a CTA, warps to a row (a CTA of more takes several rows at a time),
// pieces to a warp.
struct NormShape {
  int u, warps, nw;
};

// Eight warps with more pieces rather than sixteen, so that an SM has several CTAs whose barriers do not meet
// (1000 x 3001 fp32, forward: 17.8 us with sixteen warps of two pieces).
NormShape norm_shape(int64_t cols, int type) {
  const int64_t piece = 32 * 16 / type_bytes(type);
  const int pieces = static_cast<int>((cols + piece - 1) / piece);
  if (pieces <= 8) {
    int nw = 1;
    while (nw < pieces) nw *= 2;
    return {1, 8, nw};
  }
  if (pieces <= 32) return {(pieces + 7) / 8, 8, 8};
  return {pieces <= 48 ? 3 : pieces <= 64 ? 4 : 8, 16, 16};
}

// Rows are loaded a row ahead where the registers hold two.
template <int U>
constexpr bool kNormAhead = U <= 4;

// A lane's part of one row: U pieces of 32 lanes x 16 bytes side by side, as loaded.
template <int U>
struct RowPart {
  uint32_t w[U][4], first[U];
};

// Rows of one matrix from a warp's first column on: a cursor that steps from row to row.
template <int T>
struct RowCursor {
  char *p;
  int64_t step;  // bytes from one of the warp's rows to its next
  __device__ __forceinline__ RowCursor(const RowMat &m, int64_t row, int64_t row_step, int c0)
      : p(static_cast<char *>(const_cast<void *>(m.p)) + (row * m.ld + c0) * kTypeBytes<T>),
        step(row_step * m.ld * kTypeBytes<T>) {}
};

// Calls f(u, full) for every piece that has columns; `left`: columns from the warp's first one on.  Whole
// pieces, all but the last as a rule, need no check of columns.
template <int T, int U, typename F>
__device__ __forceinline__ void for_pieces(int left, F f) {
  constexpr int kPiece = 32 * kLaneElems<T>;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (left >= (u + 1) * kPiece)
      f(u, std::true_type());
    else if (left > u * kPiece)
      f(u, std::false_type());
  }
}

template <int T, bool VEC, int U>
__device__ __forceinline__ void load_row(const char *p, int left, int lane, RowPart<U> &part) {
  constexpr int kPiece = 32 * kLaneElems<T>;
  for_pieces<T, U>(left, [&](int u, auto full) {
    part.first[u] = 0;
    issue_load<T, VEC, decltype(full)::value>(p + u * 512, left - u * kPiece, lane, part.w[u], part.first[u]);
  });
}

// Piece u's values, zeros past the last column.
template <int T, bool VEC, int U, int E>
__device__ __forceinline__ void row_values(RowPart<U> &part, int u, const char *p, int lane, uint32_t *stage, float (&v)[E]) {
  finish_load<T, VEC>(lane, starts_inside_word<T, VEC>(p + u * 512), part.first[u], stage, part.w[u]);
  to_floats<T, E>(part.w[u], v);
}

// d[j] = a[j] * b[j] and so on, two at a time.
template <int E>
__device__ __forceinline__ void mul_to(float (&d)[E], const float (&a)[E], const float (&b)[E]) {
#pragma unroll
  for (int j = 0; j < E; j += 2) f2_unpack(f2_mul(f2_pack(a[j], a[j + 1]), f2_pack(b[j], b[j + 1])), d[j], d[j + 1]);
}

template <int E>
__device__ __forceinline__ void scale_to(float (&d)[E], const float (&a)[E], float c) {
#pragma unroll
  for (int j = 0; j < E; j += 2) f2_unpack(f2_mul(f2_pack(a[j], a[j + 1]), f2_splat(c)), d[j], d[j + 1]);
}

template <int E>
__device__ __forceinline__ void add_to(float (&d)[E], const float (&a)[E]) {
#pragma unroll
  for (int j = 0; j < E; j += 2) f2_add_to(d[j], d[j + 1], a[j], a[j + 1]);
}

// (lo, hi) += sums of a[j] * b[j] over even and odd j.
template <int E>
__device__ __forceinline__ void dot_to(float &lo, float &hi, const float (&a)[E], const float (&b)[E]) {
  uint64_t s = f2_pack(lo, hi);
#pragma unroll
  for (int j = 0; j < E; j += 2) s = f2_fma(f2_pack(a[j], a[j + 1]), f2_pack(b[j], b[j + 1]), s);
  f2_unpack(s, lo, hi);
}

// The sum of x over the nw warps of a row, in every lane of them.  part: an entry for each warp; the same
// entries are written again only behind the next call's barrier.
__device__ __forceinline__ float row_sum(float x, int warp, int lane, int nw, float *part) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
  if (nw == 1) return x;
  if (lane == 0) part[warp] = x;
  __syncthreads();
  x = part[(warp & ~(nw - 1)) + (lane & (nw - 1))];
  for (int d = nw / 2; d > 0; d /= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

// CTAs of an SM: what the registers of a row, and of the next, allow.
constexpr int norm_ctas(int u, int warps, bool vec) { return warps != 8 ? 1 : u <= 2 && vec ? 4 : 2; }

struct NormArgs {
  RowMat x, r, h, y;  // r.p, h.p: may be nullptr
  MxMat q;
  const void *w;
  float *rstd;        // may be nullptr
  float eps;
  int64_t rows;
  int cols, nw;
};

// FMT: kE2M1 or kE4M3 for an MX matrix, -1 for Y in the inputs' type.
template <int T, bool VEC, int U, int WARPS, int FMT>
__global__ void __launch_bounds__(32 * WARPS, norm_ctas(U, WARPS, VEC)) norm_forward_kernel(const NormArgs a) {
  constexpr int E = kLaneElems<T>, kPiece = 32 * E;
  __shared__ __align__(16) uint32_t stage_all[VEC ? 1 : WARPS][128];
  __shared__ float sums[2][WARPS];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  uint32_t *stage = stage_all[VEC ? 0 : warp];
  const int at_once = WARPS / a.nw;  // rows of a CTA
  const int c0 = (warp & (a.nw - 1)) * kPiece * U, left = a.cols - c0;
  grid_dependency_wait();
  grid_launch_dependents();
  int64_t row = static_cast<int64_t>(blockIdx.x) * at_once + warp / a.nw;
  const int64_t row_step = static_cast<int64_t>(gridDim.x) * at_once;
  const int rounds = static_cast<int>((a.rows - static_cast<int64_t>(blockIdx.x) * at_once + row_step - 1) / row_step);
  RowCursor<T> x(a.x, row, row_step, c0), r(a.r, row, row_step, c0), h(a.h, row, row_step, c0), y(a.y, row, row_step, c0);
  const bool has_r = a.r.p != nullptr, has_h = a.h.p != nullptr;
  RowPart<U> nx, nr, wp;
  const char *w0 = static_cast<const char *>(a.w) + static_cast<int64_t>(c0) * kTypeBytes<T>;
  load_row<T, VEC, U>(w0, left, lane, wp);
  const char *fx = x.p, *fr = r.p;  // of the row to fetch
  auto fetch = [&](int64_t at) {
    if (at < a.rows) {
      load_row<T, VEC, U>(fx, left, lane, nx);
      if (has_r) load_row<T, VEC, U>(fr, left, lane, nr);
    }
    fx += x.step;
    fr += r.step;
  };
  if (kNormAhead<U>) fetch(row);
  for_pieces<T, U>(left, [&](int u, auto) {
    finish_load<T, VEC>(lane, starts_inside_word<T, VEC>(w0 + u * 512), wp.first[u], stage, wp.w[u]);
  });
  for (int i = 0; i < rounds; ++i, row += row_step) {
    const bool in = row < a.rows;
    if (!kNormAhead<U>) fetch(row);
    float v[U][E];
    float lo = 0.0f, hi = 0.0f;
    if (in) {
      for_pieces<T, U>(left, [&](int u, auto) {
        row_values<T, VEC, U, E>(nx, u, x.p, lane, stage, v[u]);
        if (has_r) {
          float b[E];
          row_values<T, VEC, U, E>(nr, u, r.p, lane, stage, b);
          add_to<E>(v[u], b);
        }
      });
    }
    if (kNormAhead<U>) fetch(row + row_step);
    if (in) {
      for_pieces<T, U>(left, [&](int u, auto full) {
        dot_to<E>(lo, hi, v[u], v[u]);
        if (has_h) {
          uint32_t o[4];
          from_floats<T, E>(v[u], o);
          store_lane<T, VEC, decltype(full)::value>(h.p + u * 512, left - u * kPiece, lane, stage, o);
        }
      });
    }
    const float sum = row_sum(lo + hi, warp, lane, a.nw, sums[i & 1]);
    if (in) {
      const float s = __frsqrt_rn(sum / static_cast<float>(a.cols) + a.eps);
      if (a.rstd != nullptr && c0 == 0 && lane == 0) a.rstd[row] = s;
      for_pieces<T, U>(left, [&](int u, auto full) {
        constexpr bool kFull = decltype(full)::value;
        float w[E], o[E];
        to_floats<T, E>(wp.w[u], w);
        scale_to<E>(o, v[u], s);
        mul_to<E>(o, o, w);
        if constexpr (FMT < 0) {
          uint32_t b[4];
          from_floats<T, E>(o, b);
          store_lane<T, VEC, kFull>(y.p + u * 512, left - u * kPiece, lane, stage, b);
        } else {
          constexpr int kFmt = FMT < 0 ? 0 : FMT;
          constexpr int kLanesPerBlock = kMxBlock / E;
          uint32_t m = 0;
#pragma unroll
          for (int j = 0; j < E; ++j) {
            if (!kFull && lane * E + j >= left - u * kPiece) o[j] = 0.0f;  // also where the row's factor is not finite
            m = max(m, __float_as_uint(o[j]) & 0x7fffffffu);
          }
#pragma unroll
          for (int d = 1; d < kLanesPerBlock; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
          const uint32_t byte = scale_byte<kFmt>(m);
          uint32_t q[kQWords<kFmt, E>];
          encode<kFmt, E>(o, inverse_scale(byte), q);
          const int at = c0 + u * kPiece;
          const int block = at / kMxBlock + lane * E / kMxBlock;
          if (kFull || block < a.q.blocks)
            store_q<kFmt, E>(const_cast<uint8_t *>(a.q.q) + row * a.q.ldq + (at / E + lane) * kQBytes<kFmt, E>, q);
          if (lane % kLanesPerBlock == 0 && (kFull || (block >> 2) < a.q.tiles_x))
            const_cast<uint8_t *>(a.q.s)[scale_offset(row, block, a.q.tiles_x)] = static_cast<uint8_t>(byte);
        }
      });
    }
    x.p += x.step;
    r.p += r.step;
    h.p += h.step;
    y.p += y.step;
  }
}

struct NormBackArgs {
  RowMat dy, h, dh, dx;  // dh.p: may be nullptr
  const void *w;
  const float *rstd;
  float *part;           // a row of partial sums for each CTA, or dweight itself; may be nullptr
  int64_t rows;
  int cols, nw;
};

// The end of both backward kernels: a CTA's row of partial sums for dw.  acc: the lane's sums, piece u of it at
// column c0 + u * kPiece; where a CTA takes several rows at once (U == 1) its warps' sums are added in order.
template <int T, int U, int WARPS>
__device__ __forceinline__ void leave_sums(const NormBackArgs &a, const float (&acc)[U][kLaneElems<T>], int c0, int left,
                                           int warp, int lane) {
  constexpr int E = kLaneElems<T>, kPiece = 32 * E;
  __shared__ __align__(16) float columns[U == 1 ? WARPS : 1][U == 1 ? kPiece : 4];
  if (a.part == nullptr) return;
  float *part = a.part + static_cast<int64_t>(blockIdx.x) * a.cols;
  if constexpr (U == 1) {
#pragma unroll
    for (int j = 0; j < E; j += 4)
      *reinterpret_cast<float4 *>(&columns[warp][lane * E + j]) = make_float4(acc[0][j], acc[0][j + 1], acc[0][j + 2], acc[0][j + 3]);
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += 32 * WARPS) {
      float t = 0.0f;
      for (int q = 0; q < WARPS / a.nw; ++q) t += columns[q * a.nw + c / kPiece][c % kPiece];
      part[c] = t;
    }
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < E; j += 4) {
        const int c = u * kPiece + lane * E + j;
        if (a.cols % 4 == 0 && reinterpret_cast<uintptr_t>(a.part) % 16 == 0) {
          if (c < left) *reinterpret_cast<float4 *>(part + c0 + c) = make_float4(acc[u][j], acc[u][j + 1], acc[u][j + 2], acc[u][j + 3]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (c + k < left) part[c0 + c + k] = acc[u][j + k];
        }
      }
  }
}

// dX of one piece: g = dy w, xh = h s, and dh, or nullptr.
template <int E>
__device__ __forceinline__ void finish_dx(float (&g)[E], const float (&xh)[E], float dot, float s) {
#pragma unroll
  for (int j = 0; j < E; j += 2)
    f2_unpack(f2_fma(f2_splat(-dot), f2_pack(xh[j], xh[j + 1]), f2_pack(g[j], g[j + 1])), g[j], g[j + 1]);
  scale_to<E>(g, g, s);
}

// Backward kernel.  Three streams, the sums for dw and the row between its two uses leave no registers for
// loads in flight, and one row ahead is too little of them (16384 x 4096 bf16: 122 us), so rows come through
// shared memory: a ring of SLOTS rows to a warp, copied asynchronously, each lane's 16 bytes its own.  WORDS:
// rows that are aligned to 4 bytes only are copied by words, neighbouring lanes on neighbouring ones, which
// rearranges them on the way.  The sums for dw stay in registers, row after row in order; CTAs leave their
// sums in `part`, which column_sum_kernel adds in order, so the result does not depend on timing, and in 64 bits, which
// costs nothing: 1000 x 3001 fp32 13.9 us with both, dw 5e-8 of its size off, 1.3e-7 with fp32.
template <int T, int U, int WARPS>
struct NormRing {
  static constexpr int kSlots = U == 8 ? 1 : U == 4 || WARPS * U > 24 ? 2 : 3;
  static constexpr int kStream = U * 512;                      // bytes of a warp's part of a row
  static constexpr int kSlot = 3 * kStream;                    // dY, H, dH
  static constexpr int kWarp = kSlots * kSlot;
  static constexpr int kDynamicBytes = WARPS * (kWarp + kSlots * 4 + (16 - kSlots * 4 % 16) % 16);
  static constexpr int kCtas = WARPS == 8 ? (U == 1 ? 4 : 2) : 1;
  static constexpr int kStaticBytes = WARPS * (512 + 8 + (U == 1 ? 1024 : 2));
  static_assert(kCtas * (kDynamicBytes + kStaticBytes + 1024) <= 233472, "CTAs of an SM");
};

template <int T, bool WORDS, int U, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, NormRing<T, U, WARPS>::kCtas) norm_backward_ring_kernel(const NormBackArgs a) {
  using Ring = NormRing<T, U, WARPS>;
  constexpr int E = kLaneElems<T>, B = kTypeBytes<T>, kPiece = 32 * E, ST = Ring::kSlots;
  constexpr bool kKeep = U <= 2;  // dy w and h s stay in registers between their uses
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ __align__(16) uint32_t stage_all[WORDS ? WARPS : 1][128];
  __shared__ float sums[2][WARPS];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  uint32_t *stage = stage_all[WORDS ? warp : 0];
  uint8_t *ring = ring_smem + warp * Ring::kWarp;
  float *factors = reinterpret_cast<float *>(ring_smem + WARPS * Ring::kWarp) + warp * ST;
  const int at_once = WARPS / a.nw;
  const int c0 = (warp & (a.nw - 1)) * kPiece * U, left = a.cols - c0;
  grid_dependency_wait();
  grid_launch_dependents();
  int64_t row = static_cast<int64_t>(blockIdx.x) * at_once + warp / a.nw;
  const int64_t row_step = static_cast<int64_t>(gridDim.x) * at_once;
  const int rounds = static_cast<int>((a.rows - static_cast<int64_t>(blockIdx.x) * at_once + row_step - 1) / row_step);
  RowCursor<T> y(a.dy, row, row_step, c0), h(a.h, row, row_step, c0), d(a.dh, row, row_step, c0), x(a.dx, row, row_step, c0);
  const bool has_d = a.dh.p != nullptr;
  const char *w0 = static_cast<const char *>(a.w) + static_cast<int64_t>(c0) * B;
  RowPart<U> wp;
  load_row<T, !WORDS, U>(w0, left, lane, wp);

  auto copy = [&](uint8_t *to, const char *from) {
    for_pieces<T, U>(left, [&](int u, auto full) {
      const int have = (left - u * kPiece) * B;  // bytes of the piece's columns
      if constexpr (!WORDS) {
        const int size = decltype(full)::value ? 16 : min(max(have - lane * 16, 0), 16);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to + u * 512 + lane * 16)),
                     "l"(size > 0 ? from + u * 512 + lane * 16 : from), "r"(size)
                     : "memory");
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = (j * 32 + lane) * 4;
          const int size = decltype(full)::value ? 4 : min(max(have - at, 0), 4);
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(to + u * 512 + at)),
                       "l"(size > 0 ? from + u * 512 + at : from), "r"(size)
                       : "memory");
        }
      }
    });
  };
  int64_t next = row;  // to fetch
  auto fetch = [&](int slot) {
    if (next < a.rows) {
      uint8_t *to = ring + slot * Ring::kSlot;
      copy(to, y.p);
      copy(to + Ring::kStream, h.p);
      if (has_d) copy(to + 2 * Ring::kStream, d.p);
      if (lane == 0)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(factors + slot)), "l"(a.rstd + next) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    next += row_step;
    y.p += y.step;
    h.p += h.step;
    d.p += d.step;
  };
#pragma unroll
  for (int q = 0; q < ST - 1; ++q) fetch(q);
  for_pieces<T, U>(left, [&](int u, auto) {
    finish_load<T, !WORDS>(lane, starts_inside_word<T, !WORDS>(w0 + u * 512), wp.first[u], stage, wp.w[u]);
  });
  float acc[U][E];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = 0; j < E; ++j) acc[u][j] = 0.0f;
  int slot = 0;
  for (int i = 0; i < rounds; ++i, row += row_step) {
    const bool in = row < a.rows;
    if constexpr (ST == 1) {
      __syncwarp();
      fetch(0);
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncwarp();
    } else {
      asm volatile("cp.async.wait_group %0;" ::"n"(ST - 2) : "memory");
      __syncwarp();  // every lane's copies of this row have landed, and the row before is read
      fetch(slot == 0 ? ST - 1 : slot - 1);
    }
    const uint8_t *at = ring + slot * Ring::kSlot + lane * 16;
    auto values = [&](int u, int stream, float(&v)[E]) {
      const uint4 q = *reinterpret_cast<const uint4 *>(at + stream * Ring::kStream + u * 512);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      to_floats<T, E>(w, v);
    };
    const float s = factors[slot];
    float lo = 0.0f, hi = 0.0f;
    float g[kKeep ? U : 1][E], xh[kKeep ? U : 1][E];
    if (in) {
      for_pieces<T, U>(left, [&](int u, auto) {
        const int k = kKeep ? u : 0;
        float w[E], t[E];
        values(u, 0, g[k]);
        values(u, 1, xh[k]);
        to_floats<T, E>(wp.w[u], w);
        scale_to<E>(xh[k], xh[k], s);
        mul_to<E>(t, g[k], xh[k]);
        add_to<E>(acc[u], t);
        mul_to<E>(g[k], g[k], w);
        dot_to<E>(lo, hi, g[k], xh[k]);
      });
    }
    const float dot = row_sum(lo + hi, warp, lane, a.nw, sums[i & 1]) / static_cast<float>(a.cols);
    if (in) {
      for_pieces<T, U>(left, [&](int u, auto full) {
        const int k = kKeep ? u : 0;
        float b[E];
        if constexpr (!kKeep) {
          values(u, 0, g[k]);
          values(u, 1, xh[k]);
          to_floats<T, E>(wp.w[u], b);
          mul_to<E>(g[k], g[k], b);
          scale_to<E>(xh[k], xh[k], s);
        }
        finish_dx<E>(g[k], xh[k], dot, s);
        if (has_d) {
          values(u, 2, b);
          add_to<E>(g[k], b);
        }
        uint32_t o[4];
        from_floats<T, E>(g[k], o);
        store_lane<T, !WORDS, decltype(full)::value>(x.p + u * 512, left - u * kPiece, lane, stage, o);
      });
    }
    x.p += x.step;
    slot = slot == ST - 1 ? 0 : slot + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  leave_sums<T, U, WARPS>(a, acc, c0, left, warp, lane);
}

// The same for 16-bit rows at odd places, which no asynchronous copy takes: loaded to registers, a row ahead
// where they hold two.
template <int T, int U, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) norm_backward_odd_kernel(const NormBackArgs a) {
  constexpr int E = kLaneElems<T>, kPiece = 32 * E;
  __shared__ __align__(16) uint32_t stage_all[WARPS][128];
  __shared__ float sums[2][WARPS];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  uint32_t *stage = stage_all[warp];
  const int at_once = WARPS / a.nw;
  const int c0 = (warp & (a.nw - 1)) * kPiece * U, left = a.cols - c0;
  grid_dependency_wait();
  grid_launch_dependents();
  int64_t row = static_cast<int64_t>(blockIdx.x) * at_once + warp / a.nw;
  const int64_t row_step = static_cast<int64_t>(gridDim.x) * at_once;
  const int rounds = static_cast<int>((a.rows - static_cast<int64_t>(blockIdx.x) * at_once + row_step - 1) / row_step);
  RowCursor<T> y(a.dy, row, row_step, c0), h(a.h, row, row_step, c0), d(a.dh, row, row_step, c0), x(a.dx, row, row_step, c0);
  const bool has_d = a.dh.p != nullptr;
  RowPart<U> ny, nh, nd, wp;
  float ns = 0.0f;
  const char *w0 = static_cast<const char *>(a.w) + static_cast<int64_t>(c0) * kTypeBytes<T>;
  load_row<T, false, U>(w0, left, lane, wp);
  const char *fy = y.p, *fh = h.p, *fd = d.p;
  auto fetch = [&](int64_t at) {
    if (at < a.rows) {
      load_row<T, false, U>(fy, left, lane, ny);
      load_row<T, false, U>(fh, left, lane, nh);
      ns = a.rstd[at];
    }
    fy += y.step;
    fh += h.step;
  };
  auto fetch_d = [&](int64_t at) {
    if (has_d && at < a.rows) load_row<T, false, U>(fd, left, lane, nd);
    fd += d.step;
  };
  if (kNormAhead<U>) {
    fetch(row);
    fetch_d(row);
  }
  for_pieces<T, U>(left, [&](int u, auto) {
    finish_load<T, false>(lane, starts_inside_word<T, false>(w0 + u * 512), wp.first[u], stage, wp.w[u]);
  });
  float acc[U][E];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int j = 0; j < E; ++j) acc[u][j] = 0.0f;
  for (int i = 0; i < rounds; ++i, row += row_step) {
    const bool in = row < a.rows;
    if (!kNormAhead<U>) {
      fetch(row);
      fetch_d(row);
    }
    const float s = ns;
    float lo = 0.0f, hi = 0.0f;
    float g[U][E], xh[U][E];  // dy w and h s
    if (in) {
      for_pieces<T, U>(left, [&](int u, auto) {
        float w[E], t[E];
        row_values<T, false, U, E>(ny, u, y.p, lane, stage, g[u]);
        row_values<T, false, U, E>(nh, u, h.p, lane, stage, xh[u]);
        to_floats<T, E>(wp.w[u], w);
        scale_to<E>(xh[u], xh[u], s);
        mul_to<E>(t, g[u], xh[u]);
        add_to<E>(acc[u], t);
        mul_to<E>(g[u], g[u], w);
        dot_to<E>(lo, hi, g[u], xh[u]);
      });
    }
    if (kNormAhead<U>) fetch(row + row_step);
    const float dot = row_sum(lo + hi, warp, lane, a.nw, sums[i & 1]) / static_cast<float>(a.cols);
    if (in) {
      for_pieces<T, U>(left, [&](int u, auto full) {
        finish_dx<E>(g[u], xh[u], dot, s);
        if (has_d) {
          float b[E];
          row_values<T, false, U, E>(nd, u, d.p, lane, stage, b);
          add_to<E>(g[u], b);
        }
        uint32_t o[4];
        from_floats<T, E>(g[u], o);
        store_lane<T, false, decltype(full)::value>(x.p + u * 512, left - u * kPiece, lane, stage, o);
      });
    }
    if (kNormAhead<U>) fetch_d(row + row_step);
    y.p += y.step;
    h.p += h.step;
    d.p += d.step;
    x.p += x.step;
  }
  leave_sums<T, U, WARPS>(a, acc, c0, left, warp, lane);
}

// ------------------------------------------------------------------ host side

// Calls f with the pieces and warps of norm_shape.
template <int T, typename F>
tlg_status with_shape(const NormShape &n, F f) {
  using W8 = std::integral_constant<int, 8>;
  using W16 = std::integral_constant<int, 16>;
  using U1 = std::integral_constant<int, 1>;
  using U2 = std::integral_constant<int, 2>;
  using U3 = std::integral_constant<int, 3>;
  using U4 = std::integral_constant<int, 4>;
  if (n.warps == 8) return n.u == 1 ? f(U1(), W8()) : n.u == 2 ? f(U2(), W8()) : n.u == 3 ? f(U3(), W8()) : f(U4(), W8());
  if constexpr (T == kTypeF32) {
    if (n.u == 8) return f(std::integral_constant<int, 8>(), W16());
  }
  return n.u == 3 ? f(U3(), W16()) : f(U4(), W16());
}

unsigned norm_grid(const NormShape &n, int64_t rows, int sms, int per_sm) {
  const int64_t at_once = n.warps / n.nw;
  return static_cast<unsigned>(std::min<int64_t>((rows + at_once - 1) / at_once, int64_t(sms) * per_sm));
}

// CTAs of the backward kernels, each of which leaves a row of partial sums.
unsigned ring_ctas(const NormShape &n, int64_t rows, int sms) {
  return norm_grid(n, rows, sms, n.warps != 8 ? 1 : n.u == 1 ? 4 : 2);
}

unsigned odd_ctas(const NormShape &n, int64_t rows, int sms) { return norm_grid(n, rows, sms, n.warps == 8 ? 2 : 1); }

// Workspace bytes of their partial sums; the caller does not know which matrices will be aligned.
size_t norm_workspace(int64_t rows, int64_t cols, int type, int sms) {
  const NormShape n = norm_shape(cols, type);
  const unsigned ctas = std::max(ring_ctas(n, rows, sms), odd_ctas(n, rows, sms));
  return ctas > 1 ? static_cast<size_t>(ctas) * static_cast<size_t>(cols) * 4 : 0;
}

template <int T, bool WORDS, int U, int WARPS>
tlg_status launch_ring(int dev, unsigned ctas, cudaStream_t s, const NormBackArgs &a) {
  constexpr auto kernel = norm_backward_ring_kernel<T, WORDS, U, WARPS>;
  constexpr int kBytes = NormRing<T, U, WARPS>::kDynamicBytes;
  static bool ready[kMaxDevices];
  static std::mutex mutex;
  {
    std::lock_guard<std::mutex> lock(mutex);
    if (!ready[dev]) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes) != cudaSuccess) {
        cudaGetLastError();
        return TLG_ERR_CUDA;
      }
      ready[dev] = true;
    }
  }
  return launch(kernel, dim3(ctas), 32 * WARPS, s, kBytes, a);
}

// Whether every row starts on 4 bytes.
bool word_rows(const void *p, int64_t rows, int64_t ld, int type) {
  return reinterpret_cast<uintptr_t>(p) % 4 == 0 && (rows == 1 || (ld * type_bytes(type)) % 4 == 0);
}

tlg_status check_norm(int64_t rows, int64_t cols, int type) {
  if (!valid_type(type)) return TLG_ERR_INVALID_ARG;
  const tlg_status st = check_extents(rows, cols);
  if (st != TLG_OK) return st;
  return cols > kNormMaxCols ? TLG_ERR_UNSUPPORTED : TLG_OK;
}

// Whether a matrix, if it is there, may be accessed 16 bytes at a time.
bool vec_or_none(const void *p, int64_t rows, int64_t ld, int type) {
  return p == nullptr || vec_rows(p, rows, ld, type);
}

tlg_status check_vector(const void *p, int64_t n, int64_t esz, Range *r) {
  if (p == nullptr) return TLG_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(esz) != 0) return TLG_ERR_ALIGNMENT;
  r->lo = reinterpret_cast<uintptr_t>(p);
  r->hi = r->lo + static_cast<uintptr_t>(n * esz);
  return TLG_OK;
}

// The forward pass; format < 0: Y, else Q and S.
tlg_status norm_forward(int64_t rows, int64_t cols, int type, const void *X, int64_t ldx, const void *R, int64_t ldr,
                        const void *weight, float eps, void *H, int64_t ldh, void *Y, int64_t ldy, int format, void *Q,
                        int64_t ldq, void *S, float *rstd, void *stream) {
  tlg_status st = check_norm(rows, cols, type);
  if (st != TLG_OK) return st;
  if (!(eps >= 0.0f) || std::isinf(eps) || (format >= 0 && !valid_format(format))) return TLG_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return TLG_OK;
  const int64_t esz = type_bytes(type);
  Range in[3] = {}, out[4] = {};  // X, R, weight; H, Y or Q, S, rstd
  st = check_matrix(X, rows, cols, ldx, esz, &in[0]);
  if (st == TLG_OK && R != nullptr) st = check_matrix(R, rows, cols, ldr, esz, &in[1]);
  if (st == TLG_OK) st = check_vector(weight, cols, esz, &in[2]);
  if (st == TLG_OK && H != nullptr) st = check_matrix(H, rows, cols, ldh, esz, &out[0]);
  if (st == TLG_OK) {
    st = format < 0 ? check_matrix(Y, rows, cols, ldy, esz, &out[1]) : check_mx(format, rows, cols, Q, ldq, S, &out[1], &out[2]);
  }
  if (st == TLG_OK && rstd != nullptr) st = check_vector(rstd, rows, 4, &out[3]);
  if (st != TLG_OK) return st;
  // H and Y may be X or R themselves: an element is read by the lane that writes it, before it does.
  auto same = [&](const void *o, int64_t ldo, int i) {
    return i == 0 ? o == X && ldo == ldx : i == 1 && o == R && ldo == ldr;
  };
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 3; ++i)
      if (meets(out[o], in[i]) && !(o == 0 && same(H, ldh, i)) && !(o == 1 && format < 0 && same(Y, ldy, i)))
        return TLG_ERR_INVALID_ARG;
    for (int k = 0; k < o; ++k)
      if (meets(out[o], out[k])) return TLG_ERR_INVALID_ARG;
  }
  DeviceInfo info;
  st = device_ready({X, R, weight, H, Y, Q, S, rstd}, &info);
  if (st != TLG_OK) return st;
  const NormShape n = norm_shape(cols, type);
  NormArgs a = {{X, ldx}, {R, ldr}, {H, ldh}, {Y, ldy}, format < 0 ? MxMat{} : mx_mat(Q, ldq, S, cols), weight, rstd, eps, rows,
                static_cast<int>(cols), n.nw};
  const bool vec = aligned16(weight) && vec_rows(X, rows, ldx, type) && vec_or_none(R, rows, ldr, type) &&
                   vec_or_none(H, rows, ldh, type) && vec_or_none(Y, rows, ldy, type);
  // Few rows: a CTA for each, which loads no row ahead of its own (1000 x 3000 fp32: 8.7 us, 13.6 with 296).
  const int per_sm = norm_ctas(n.u, n.warps, vec);
  const unsigned grid = norm_grid(n, rows, info.sm_count, (vec || type == TLG_TYPE_F32) && rows * n.nw <= 64 * int64_t(info.sm_count) ? 64 : per_sm);
  return with_type(type, [&](auto T) {
    constexpr int kT = decltype(T)::value;
    return with_flag(vec, [&](auto V) {
      return with_shape<kT>(n, [&](auto U, auto W) {
        constexpr int kU = decltype(U)::value, kW = decltype(W)::value;
        constexpr bool kV = decltype(V)::value;
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        if (format < 0) return launch(norm_forward_kernel<kT, kV, kU, kW, -1>, dim3(grid), 32 * kW, s, 0, a);
        if (format == TLG_MX_E2M1) return launch(norm_forward_kernel<kT, kV, kU, kW, kE2M1>, dim3(grid), 32 * kW, s, 0, a);
        return launch(norm_forward_kernel<kT, kV, kU, kW, kE4M3>, dim3(grid), 32 * kW, s, 0, a);
      });
    });
  });
}

}  // namespace
}  // namespace tlg

using namespace tlg;

extern "C" {

tlg_status tlg_rmsnorm_forward(int64_t rows, int64_t cols, tlg_type type, const void *X, int64_t ldx, const void *R,
                               int64_t ldr, const void *weight, float eps, void *H, int64_t ldh, void *Y, int64_t ldy,
                               float *rstd, void *stream) {
  return norm_forward(rows, cols, type, X, ldx, R, ldr, weight, eps, H, ldh, Y, ldy, -1, nullptr, 0, nullptr, rstd, stream);
}

tlg_status tlg_rmsnorm_forward_mx(int64_t rows, int64_t cols, tlg_type type, const void *X, int64_t ldx, const void *R,
                                  int64_t ldr, const void *weight, float eps, void *H, int64_t ldh,
                                  tlg_mx_format format, void *Q, int64_t ldq, void *S, float *rstd, void *stream) {
  if (!valid_format(format)) return TLG_ERR_INVALID_ARG;
  return norm_forward(rows, cols, type, X, ldx, R, ldr, weight, eps, H, ldh, nullptr, 0, format, Q, ldq, S, rstd, stream);
}

tlg_status tlg_rmsnorm_backward_workspace_size(int64_t rows, int64_t cols, tlg_type type, size_t *bytes) {
  if (bytes == nullptr) return TLG_ERR_INVALID_ARG;
  *bytes = 0;
  const tlg_status st = check_norm(rows, cols, type);
  if (st != TLG_OK || rows == 0 || cols == 0) return st;
  int dev = 0;
  DeviceInfo info;
  const tlg_status ds = current_device(&dev, &info);
  if (ds != TLG_OK) return ds;
  *bytes = norm_workspace(rows, cols, type, info.sm_count);
  return TLG_OK;
}

tlg_status tlg_rmsnorm_backward(int64_t rows, int64_t cols, tlg_type type, const void *dY, int64_t lddy, const void *H,
                                int64_t ldh, const void *weight, const float *rstd, const void *dH, int64_t lddh,
                                void *dX, int64_t lddx, float *dweight, void *workspace, size_t workspace_bytes,
                                void *stream) {
  tlg_status st = check_norm(rows, cols, type);
  if (st != TLG_OK || cols == 0) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  DeviceInfo info;
  Range rw = {}, rk = {};
  if (dweight != nullptr) {
    st = check_vector(dweight, cols, 4, &rw);
    if (st != TLG_OK) return st;
  }
  if (workspace != nullptr) {
    if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return TLG_ERR_ALIGNMENT;
    rk.lo = reinterpret_cast<uintptr_t>(workspace);
    rk.hi = rk.lo + workspace_bytes;
  }
  if (rows == 0) {  // the sum over no rows
    if (dweight == nullptr) return TLG_OK;
    st = device_ready({dweight}, &info);
    if (st != TLG_OK) return st;
    if (cudaMemsetAsync(dweight, 0, static_cast<size_t>(cols) * 4, s) != cudaSuccess) {
      cudaGetLastError();
      return TLG_ERR_CUDA;
    }
    return TLG_OK;
  }
  const int64_t esz = type_bytes(type);
  Range ry, rh, rwt, rr, rd = {}, rx;
  st = check_matrix(dY, rows, cols, lddy, esz, &ry);
  if (st == TLG_OK) st = check_matrix(H, rows, cols, ldh, esz, &rh);
  if (st == TLG_OK) st = check_vector(weight, cols, esz, &rwt);
  if (st == TLG_OK) st = check_vector(rstd, rows, 4, &rr);
  if (st == TLG_OK && dH != nullptr) st = check_matrix(dH, rows, cols, lddh, esz, &rd);
  if (st == TLG_OK) st = check_matrix(dX, rows, cols, lddx, esz, &rx);
  if (st != TLG_OK) return st;
  if (meets(rx, ry) && !(dX == dY && lddx == lddy)) return TLG_ERR_INVALID_ARG;
  if (dH != nullptr && meets(rx, rd) && !(dX == dH && lddx == lddh)) return TLG_ERR_INVALID_ARG;
  if (meets(rx, rh) || meets(rx, rwt) || meets(rx, rr)) return TLG_ERR_INVALID_ARG;
  for (const Range &r : {ry, rh, rwt, rr, rd, rx})
    if (meets(rw, r) || meets(rk, r)) return TLG_ERR_INVALID_ARG;
  if (meets(rw, rk)) return TLG_ERR_INVALID_ARG;
  st = device_ready({dY, H, weight, rstd, dH, dX, dweight, workspace}, &info);
  if (st != TLG_OK) return st;
  int dev = 0;
  st = current_device(&dev, &info);
  if (st != TLG_OK) return st;
  auto rows_are = [&](bool (*fit)(const void *, int64_t, int64_t, int), const void *w) {
    return fit(w, 1, 0, type) && fit(dY, rows, lddy, type) && fit(H, rows, ldh, type) &&
           (dH == nullptr || fit(dH, rows, lddh, type)) && fit(dX, rows, lddx, type);
  };
  const bool vec = rows_are(vec_rows, weight), words = rows_are(word_rows, weight);
  const NormShape n = norm_shape(cols, type);
  const unsigned ctas = vec || words ? ring_ctas(n, rows, info.sm_count) : odd_ctas(n, rows, info.sm_count);
  float *part = dweight;
  if (dweight != nullptr && ctas > 1) {
    if (workspace == nullptr || workspace_bytes < norm_workspace(rows, cols, type, info.sm_count)) return TLG_ERR_INVALID_ARG;
    part = static_cast<float *>(workspace);
  }
  const NormBackArgs a = {{dY, lddy}, {H, ldh}, {dH, lddh}, {dX, lddx}, weight, rstd, part, rows, static_cast<int>(cols), n.nw};
  st = with_type(type, [&](auto T) {
    constexpr int kT = decltype(T)::value;
    if (vec || words) {
      return with_shape<kT>(n, [&](auto U, auto W) {
        constexpr int kU = decltype(U)::value, kW = decltype(W)::value;
        return vec ? launch_ring<kT, false, kU, kW>(dev, ctas, s, a) : launch_ring<kT, true, kU, kW>(dev, ctas, s, a);
      });
    }
    if constexpr (kT != kTypeF32) {
      return with_shape<kT>(n, [&](auto U, auto W) {
        constexpr int kU = decltype(U)::value, kW = decltype(W)::value;
        return launch(norm_backward_odd_kernel<kT, kU, kW>, dim3(ctas), 32 * kW, s, 0, a);
      });
    }
    return TLG_ERR_ALIGNMENT;  // fp32 rows are aligned to words
  });
  if (st != TLG_OK || part == dweight) return st;
  const dim3 sum_grid(static_cast<unsigned>((cols + 31) / 32));
  return ctas > 128 ? launch(column_sum_kernel<32, double>, sum_grid, 1024, s, 0, part, static_cast<int>(ctas), cols, dweight)
                    : launch(column_sum_kernel<8, double>, sum_grid, 256, s, 0, part, static_cast<int>(ctas), cols, dweight);
}

}  // extern "C"
