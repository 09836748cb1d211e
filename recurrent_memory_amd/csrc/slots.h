// Rows of a batch that name the same page of a pool.
#pragma once

#include <hip/hip_runtime.h>

namespace dr {

// Row b's page, and whether a row before b, or one after it, names that page too.
// Every wave scans the list by itself, 256 entries at a time, so that the answer is
// wave-uniform without a barrier; that is quadratic in B, and made for batches of up to
// some thousand rows (a step of 256 fp32 channels: 1024 rows 9 us with or without slots,
// 4096 rows 25 us against 8, 16384 rows 272 against 15, 65536 rows 3.9 ms against 48 us).
// Called by whole waves.  The first 256 are loaded along with the row's own entry, before
// either is looked at, so that a batch of up to 256 rows waits once.
__device__ __forceinline__ int slot_of_row(const int* __restrict__ slots, int B, int b, bool* earlier,
                                           bool* later) {
    const int lane = threadIdx.x & 63;
    int s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = slots[min(64 * j + lane, B - 1)];
    const int slot = slots[b];
    bool e = false, l = false;
    for (int i0 = 0;;) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + 64 * j + lane;      // beyond the list: entry B - 1 again, not counted
            e |= s[j] == slot && i < b;
            l |= s[j] == slot && i > b && i < B;
        }
        i0 += 256;
        if (i0 >= B) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = slots[min(i0 + 64 * j + lane, B - 1)];
    }
    *earlier = __ballot(e) != 0;
    *later = __ballot(l) != 0;
    return slot;
}

// The first row after b that names page `slot`, or B.  Called by whole waves.
__device__ __forceinline__ int next_sharer(const int* __restrict__ slots, int B, int b, int slot) {
    const int lane = threadIdx.x & 63;
    for (int i0 = b + 1; i0 < B; i0 += 64) {
        const uint64_t found = __ballot(i0 + lane < B && slots[min(i0 + lane, B - 1)] == slot);
        if (found != 0) return i0 + __ffsll(static_cast<unsigned long long>(found)) - 1;
    }
    return B;
}

}  // namespace dr
