// Host-side helpers shared by the library's entry points: the device probe, pointer and
// extent checks, and TMA descriptor encoding.  Defined in tlg_gemm.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <mutex>

#include "tlg.h"

namespace tlg {

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  bool probed = false;
  bool supported = false;
  int sm_count = 0;
};

// Guards the library's per-device state.
extern std::mutex g_mutex;

// The current device and what it is; TLG_ERR_UNSUPPORTED unless it is an sm_100.
tlg_status current_device(int *dev, DeviceInfo *info);

// A pointer the kernels may read or write: device memory of `dev`, or managed memory.
bool device_accessible(const void *p, int dev);

bool aligned16(const void *p);

// Byte range [lo, hi) touched by a rows x cols matrix with row stride ld (rows, cols >= 1).
void extent(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t esz, uintptr_t *lo,
            uintptr_t *hi);

bool overlaps(uintptr_t a0, uintptr_t a1, uintptr_t b0, uintptr_t b1);

// A 2-D tensor map of `outer` rows of `inner` elements, row_bytes apart (current_device
// must have succeeded before).
bool encode_2d(CUtensorMap *tm, CUtensorMapDataType dtype, const void *base, uint64_t inner,
               uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
               CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);

}  // namespace tlg
