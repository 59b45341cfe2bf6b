// api_common.hpp -- what the translation units of the C ABI share: alignment
// of addresses, the status of a launch, and the device's size.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvfp4.h"

namespace nvfp4 {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int launch_status()
{
    hipError_t e = hipGetLastError();
    return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH;
}

// Compute units of the current device (0: none).
inline int device_cus()
{
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
    return n;
}

// Tiles of 256 x 256 outputs that one grid holds: 512 threads each, and a
// grid has fewer than 2^32 threads.
constexpr int64_t kMostBigTiles = int64_t(1) << 22;

// Whether `stride` elements hold `rows` rows of `cols`, `ld` apart (ld >= cols
// >= 0; ld * rows may pass 64 bits).
inline bool holds(int64_t stride, int64_t rows, int64_t ld, int64_t cols)
{
    if (rows == 0) return stride >= 0;
    return stride >= cols && (rows == 1 || (stride - cols) / (rows - 1) >= ld);
}

// Pass and sizes of a grouped product.
inline int check_grouped(int32_t pass, int64_t E, int64_t T, int64_t N, int64_t K)
{
    if (pass != NVFP4_FPROP && pass != NVFP4_DGRAD && pass != NVFP4_WGRAD) return NVFP4_ERR_MODE;
    if (E < 0 || T < 0 || N < 0 || K < 0 || N % 8 || K % 8) return NVFP4_ERR_SHAPE;
    const int64_t lim = int64_t(1) << 31;
    if (E >= lim || T >= lim || N >= lim || K >= lim) return NVFP4_ERR_SHAPE;
    const int64_t cols = pass == NVFP4_FPROP ? N : K;
    const int64_t row_tiles = pass == NVFP4_WGRAD ? E * ((N + 255) / 256) : T / 256 + E + 1;
    const int64_t col_tiles = (cols + 255) / 256;  // (the product of the two may pass 64 bits)
    return col_tiles == 0 || row_tiles <= (kMostBigTiles - 1) / col_tiles ? NVFP4_OK : NVFP4_ERR_SHAPE;
}

}  // namespace nvfp4
