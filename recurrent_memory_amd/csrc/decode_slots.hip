// Single-token decode update on the pages of a pool: row b's states are those of
// page slots[b], [H,d_v,d_k].
//
// The work and the bound are the dense kernel's (8 bytes of HBM traffic per state
// element): one workgroup per (row, head), and decode_row() does the step.  What
// is added is one dependent load (the slot, before the state's address is known)
// and a scan of the slot list for rows that share the page: the first of them takes
// the others' tokens too, in order, so that two workgroups never touch one state and
// a page named twice gets its two tokens one after the other.  Every wave scans the whole
// list: nothing to speak of for the batches of a server, but quadratic (4 heads of width
// 64: 1024 rows 27 us against 25 dense, 4096 rows 169 against 91, 16384 rows 1.27 ms
// against 0.40, 65536 rows 16.4 ms against 1.6).
#include "decode_row.h"
#include "slots.h"

namespace dr {
namespace {

// Four waves a SIMD: the compiler gives the forms with a vector of decays or steps (2, 4) a
// few registers too many by itself.  64 rows of 16 heads of width 128, states from HBM: a
// step size per channel 35.4 us, 38.0 with three waves; channel-wise decay in fp32 36.2 and
// 38.0 (both spill two registers at four waves; in bf16 the compiler finds 128 by itself).
// 256 rows, streamed, are the same or up to 2% slower.  The split gates (3) stay at three
// waves and 137 registers: 37.8 us, at four 38.0; 256 rows 105 us, at four 108.
template <int VAR, typename E, int DK, int DV, bool NT>
__global__ __launch_bounds__(kDecodeThreads, VAR == 2 || VAR == 4 ? 4 : 1) void decode_slots_kernel(DecodeArgs p, int n_pages,
                                                                      const int* slots) {
    const int h = blockIdx.x % p.H;
    int b = blockIdx.x / p.H;
    bool earlier, later;
    const int slot = slot_of_row(slots, p.B, b, &earlier, &later);
    if (slot < 0 || slot >= n_pages || earlier) return;   // padding rows: nothing read, nothing written
    float* S = p.S + (static_cast<int64_t>(slot) * p.H + h) * DV * DK;
    do {
        // taken as new in every turn, so that the rows' addresses are not kept in registers
        // from one to the next (147 instead of 128 with a decay per head, one wave less on each SIMD)
        asm volatile("" : "+s"(S));
        decode_row<VAR, E, DK, DV, NT>(p, b * p.H + h, S);
        if (later) b = next_sharer(slots, p.B, b, slot);
    } while (later && b < p.B);
}

// From half of the last-level cache on, the states of a call will not be there at the
// next token, and non-temporal accesses stream them faster: 128 MiB of states 55 us
// against 63 us plain, 256 MiB 107 against 116 us (other layers' states between the
// tokens).  Smaller ones may still be there, if little else runs between: 64 MiB of
// states 23 us non-temporal, 21 us plain.  The host counts all rows, those that pad the
// batch too: it cannot see the slots, and a large batch with few live rows streams.
constexpr int64_t kStreamBytes = int64_t(128) << 20;

template <int VAR, typename E, int DK, int DV>
hipError_t launch_widths(const DecodeArgs& a, int n_pages, const int* slots, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.B) * static_cast<unsigned>(a.H));
    const dim3 block(kDecodeThreads);
    if (static_cast<int64_t>(a.B) * a.H * DK * DV * 4 >= kStreamBytes)
        hipLaunchKernelGGL((decode_slots_kernel<VAR, E, DK, DV, true>), grid, block, 0, s, a, n_pages, slots);
    else
        hipLaunchKernelGGL((decode_slots_kernel<VAR, E, DK, DV, false>), grid, block, 0, s, a, n_pages, slots);
    return hipGetLastError();
}

template <int VAR, typename E>
hipError_t launch_dims(const DecodeArgs& a, int n_pages, const int* slots, hipStream_t s) {
    if (a.dk == 128 && a.dv == 128) return launch_widths<VAR, E, 128, 128>(a, n_pages, slots, s);
    if (a.dk == 128) return launch_widths<VAR, E, 128, 64>(a, n_pages, slots, s);
    if (a.dv == 128) return launch_widths<VAR, E, 64, 128>(a, n_pages, slots, s);
    return launch_widths<VAR, E, 64, 64>(a, n_pages, slots, s);
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
