// Which 16-byte granules of a row a bulk copy may take (host and device).
#pragma once
#include <stddef.h>
#include <stdint.h>

#ifdef __CUDACC__
#define VH_HD __host__ __device__ __forceinline__
#else
#define VH_HD inline
#endif

namespace vh {

// The granules that a row at address b of `bytes` bytes touches, without those that reach past the tensor's bytes
// [start, end): [lo, hi), empty where none is left.  What the row holds outside is read element by element (a row
// shorter than a granule may lie there altogether, and with it rows that are neither the first nor the last).
VH_HD void copy_window(uintptr_t b, uint32_t bytes, uintptr_t start, uintptr_t end, uintptr_t& lo, uintptr_t& hi) {
    lo = b & ~uintptr_t(15);
    if (lo < start) lo = (start + 15) & ~uintptr_t(15);
    hi = (b + bytes + 15) & ~uintptr_t(15);
    if (hi > end) hi = end & ~uintptr_t(15);
    if (hi < lo) hi = lo;
}

// Elements [0, head) and [tail, n) of that row lie outside [lo, hi); `size`: bytes of an element.
VH_HD void outside_window(uintptr_t b, uint32_t bytes, int size, uintptr_t lo, uintptr_t hi, int& head, int& tail) {
    const int n = (int)(bytes / (uint32_t)size);
    head = lo > b ? (int)(lo - b) / size : 0;
    tail = hi > b ? (int)(hi - b) / size : 0;
    if (head > n) head = n;
    if (tail > n) tail = n;
    if (tail < head) tail = head;
}

}  // namespace vh
