// Single-token decode update over dense states [B,H,d_v,d_k]: one workgroup per
// (batch, head) state matrix; the step itself is decode_row().
#include "decode_row.h"

namespace dr {
namespace {

template <int VAR, typename E, int DK, int DV>
__global__ __launch_bounds__(kDecodeThreads) void decode_kernel(DecodeArgs p) {
    const int bh = blockIdx.x;  // b * H + h
    decode_row<VAR, E, DK, DV>(p, bh, p.S + static_cast<int64_t>(bh) * DV * DK);
}

template <int VAR, typename E>
hipError_t launch_decode_dims(const DecodeArgs& a, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.B) * static_cast<unsigned>(a.H));
    const dim3 block(kDecodeThreads);
    if (a.dk == 128 && a.dv == 128) hipLaunchKernelGGL((decode_kernel<VAR, E, 128, 128>), grid, block, 0, s, a);
    else if (a.dk == 128 && a.dv == 64) hipLaunchKernelGGL((decode_kernel<VAR, E, 128, 64>), grid, block, 0, s, a);
    else if (a.dk == 64 && a.dv == 128) hipLaunchKernelGGL((decode_kernel<VAR, E, 64, 128>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((decode_kernel<VAR, E, 64, 64>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <int VAR>
hipError_t launch_decode_dtype(int dtype, const DecodeArgs& a, hipStream_t s) {
    return dtype == 0 ? launch_decode_dims<VAR, F32>(a, s) : launch_decode_dims<VAR, BF16>(a, s);
}

}  // namespace

hipError_t launch_decode(int variant, int dtype, const DecodeArgs& a, hipStream_t s) {
    switch (variant) {
        case 0: return launch_decode_dtype<0>(dtype, a, s);
        case 1: return launch_decode_dtype<1>(dtype, a, s);
        case 2: return launch_decode_dtype<2>(dtype, a, s);
        case 3: return launch_decode_dtype<3>(dtype, a, s);
        default: return launch_decode_dtype<4>(dtype, a, s);
    }
}

}  // namespace dr
