// Host-side argument checks shared by the microscaled (MX) entry points.
#pragma once

#include <cstdint>
#include <initializer_list>

#include "tlg_host.cuh"
#include "tlg_mx_device.cuh"

namespace tlg {

constexpr int64_t kMaxExtent = 0x7fffffff - 256;  // rows, cols
constexpr int64_t kMaxLd = int64_t(1) << 36;

inline bool valid_type(int t) { return t == TLG_TYPE_F32 || t == TLG_TYPE_F16 || t == TLG_TYPE_BF16; }
inline bool valid_format(int f) { return f == TLG_MX_E2M1 || f == TLG_MX_E4M3; }
inline bool valid_activation(int a) { return a >= TLG_ACT_NONE && a <= TLG_ACT_GELU_TANH; }
inline int64_t type_bytes(int t) { return t == TLG_TYPE_F32 ? 4 : 2; }
inline int64_t row_bytes(int f, int64_t cols) { return mx_blocks(cols) * (f == TLG_MX_E2M1 ? 16 : 32); }
inline int64_t scale_tiles_x(int64_t cols) { return (mx_blocks(cols) + 3) / 4; }
inline int64_t scale_bytes(int64_t rows, int64_t cols) { return (rows + 127) / 128 * scale_tiles_x(cols) * 512; }

struct Range {
  uintptr_t lo, hi;
};

// A rows x cols matrix of esz-byte elements: pointer, alignment, stride and span.
inline tlg_status check_matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t esz, Range *out) {
  if (p == nullptr || ld < cols) return TLG_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(esz) != 0) return TLG_ERR_ALIGNMENT;
  if (ld > kMaxLd || (rows > 1 && rows - 1 > ((int64_t(1) << 60) / esz) / ld)) return TLG_ERR_UNSUPPORTED;
  extent(p, rows, cols, ld, esz, &out->lo, &out->hi);
  return TLG_OK;
}

// The elements and scales of a rows x cols MX matrix.
inline tlg_status check_mx(int f, int64_t rows, int64_t cols, const void *Q, int64_t ldq, const void *S, Range *q, Range *s) {
  if (Q == nullptr || S == nullptr || ldq < row_bytes(f, cols)) return TLG_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(S) || (rows > 1 && ldq % 16 != 0)) return TLG_ERR_ALIGNMENT;
  if (ldq > kMaxLd || (rows > 1 && rows - 1 > (int64_t(1) << 60) / ldq)) return TLG_ERR_UNSUPPORTED;
  extent(Q, rows, row_bytes(f, cols), ldq, 1, &q->lo, &q->hi);
  s->lo = reinterpret_cast<uintptr_t>(S);
  s->hi = s->lo + static_cast<uintptr_t>(scale_bytes(rows, cols));
  return TLG_OK;
}

inline bool meets(const Range &a, const Range &b) { return overlaps(a.lo, a.hi, b.lo, b.hi); }

inline tlg_status check_extents(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return TLG_ERR_INVALID_ARG;
  if (rows > kMaxExtent || cols > kMaxExtent) return TLG_ERR_UNSUPPORTED;
  return TLG_OK;
}

inline tlg_status device_ready(std::initializer_list<const void *> ptrs, DeviceInfo *info) {
  int dev = 0;
  const tlg_status ds = current_device(&dev, info);
  if (ds != TLG_OK) return ds;
  for (const void *p : ptrs)
    if (p != nullptr && !device_accessible(p, dev)) return TLG_ERR_INVALID_ARG;
  return TLG_OK;
}

}  // namespace tlg
