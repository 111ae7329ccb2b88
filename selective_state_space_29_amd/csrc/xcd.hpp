// The order in which a launch's workgroups take its items, without any GPU header: host code can count on it.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define MSCAN_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MSCAN_HOST_DEVICE inline
#endif

namespace mscan {

// Workgroups go to the 8 XCDs in turn. Workgroup `id` of n takes item xcd_item(id, n): every item once, each
// XCD one stretch of neighbouring items, no stretch more than one item longer than another.
MSCAN_HOST_DEVICE int64_t xcd_item(int64_t id, int64_t n) {
    const int64_t each = n / 8, more = n % 8, xcd = id % 8;
    return xcd * each + (xcd < more ? xcd : more) + id / 8;
}

}  // namespace mscan

#undef MSCAN_HOST_DEVICE
