// Single-token decode update on the pages of a pool: row b's states are those of
// page slots[b], [H,d_v,d_k].
//
// The work and the bound are the dense kernel's (8 bytes of HBM traffic per state
// element): one workgroup per (row, head), and decode_row() does the step.  What
// is added is one dependent load (the slot, before the state's address is known)
// and, beside the state's own loads, a scan of the slot list for rows that share
// the page: the first of them takes the others' tokens too, in order, so that two
// workgroups never touch one state and a page named twice gets its two tokens one
// after the other.
#include "decode_row.h"
#include "slots.h"

namespace dr {
namespace {

template <int VAR, typename E, int DK, int DV>
__global__ __launch_bounds__(kDecodeThreads) void decode_slots_kernel(DecodeArgs p, int n_pages,
                                                                      const int* slots) {
    const int h = blockIdx.x % p.H;
    int b = blockIdx.x / p.H;
    const int slot = slots[b];
    if (slot < 0 || slot >= n_pages) return;   // padding row: nothing read, nothing written
    bool earlier, later;
    slot_sharers(slots, p.B, b, slot, &earlier, &later);
    if (earlier) return;
    float* S = p.S + (static_cast<int64_t>(slot) * p.H + h) * DV * DK;
    decode_row<VAR, E, DK, DV>(p, b * p.H + h, S);
    while (later) {
        b = next_sharer(slots, p.B, b, slot);
        if (b == p.B) break;
        decode_row<VAR, E, DK, DV>(p, b * p.H + h, S);
    }
}

template <int VAR, typename E>
hipError_t launch_dims(const DecodeArgs& a, int n_pages, const int* slots, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.B) * static_cast<unsigned>(a.H));
    const dim3 block(kDecodeThreads);
    if (a.dk == 128 && a.dv == 128)
        hipLaunchKernelGGL((decode_slots_kernel<VAR, E, 128, 128>), grid, block, 0, s, a, n_pages, slots);
    else if (a.dk == 128 && a.dv == 64)
        hipLaunchKernelGGL((decode_slots_kernel<VAR, E, 128, 64>), grid, block, 0, s, a, n_pages, slots);
    else if (a.dk == 64 && a.dv == 128)
        hipLaunchKernelGGL((decode_slots_kernel<VAR, E, 64, 128>), grid, block, 0, s, a, n_pages, slots);
    else
        hipLaunchKernelGGL((decode_slots_kernel<VAR, E, 64, 64>), grid, block, 0, s, a, n_pages, slots);
    return hipGetLastError();
}

template <int VAR>
hipError_t launch_dtype(int dtype, const DecodeArgs& a, int n_pages, const int* slots, hipStream_t s) {
    return dtype == 0 ? launch_dims<VAR, F32>(a, n_pages, slots, s)
                      : launch_dims<VAR, BF16>(a, n_pages, slots, s);
}

}  // namespace

hipError_t launch_decode_slots(int variant, int dtype, const DecodeArgs& a, int n_pages,
                               const int* slots, hipStream_t s) {
    switch (variant) {
        case 0: return launch_dtype<0>(dtype, a, n_pages, slots, s);
        case 1: return launch_dtype<1>(dtype, a, n_pages, slots, s);
        case 2: return launch_dtype<2>(dtype, a, n_pages, slots, s);
        case 3: return launch_dtype<3>(dtype, a, n_pages, slots, s);
        default: return launch_dtype<4>(dtype, a, n_pages, slots, s);
    }
}

}  // namespace dr
