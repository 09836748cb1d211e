// Gated linear recurrence h_t = exp(g_t) h_{t-1} + beta_t x_t per channel, its
// backward pass and its single-token step.
//
// Forward and backward: one lane per channel walks the tokens in order, with the
// state in a register.  HBM-bound work (4 and 7 values per element), here bound by
// the latency of each token's loads.
#include "common.h"
#include "kernels.h"
#include "slots.h"

namespace dr {
namespace {

constexpr int kBlock = 16;          // tokens per row of `states`
constexpr int kSeqThreads = 64;
constexpr int kStepThreads = 256;

template <typename E, bool BETA>
__global__ __launch_bounds__(kSeqThreads) void linrec_fwd_kernel(LinrecArgs p) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kSeqThreads + threadIdx.x;  // b * D + c
    if (i >= static_cast<int64_t>(p.B) * p.D) return;
    const int64_t b = i / p.D, c = i % p.D;
    const int64_t blocks = (static_cast<int64_t>(p.T) + kBlock - 1) / kBlock;
    float h = p.h0 != nullptr ? p.h0[i] : 0.f;
    for (int64_t t = 0; t < p.T; ++t) {
        const int64_t at = (b * p.T + t) * p.D + c;
        if (p.states != nullptr && t % kBlock == 0) p.states[(b * blocks + t / kBlock) * p.D + c] = h;
        float u = load_elem<E>(p.x, at);
        if constexpr (BETA) u *= load_elem<E>(p.beta, at);
        h = fmaf(__expf(load_elem<E>(p.g, at)), h, u);
        store_elem<E>(p.o, at, h);
    }
    if (p.hT != nullptr) p.hT[i] = h;
}

template <typename E, bool BETA>
__global__ __launch_bounds__(kSeqThreads) void linrec_bwd_kernel(LinrecBwdArgs p) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kSeqThreads + threadIdx.x;
    if (i >= static_cast<int64_t>(p.B) * p.D) return;
    const int64_t b = i / p.D, c = i % p.D;
    const int64_t blocks = (static_cast<int64_t>(p.T) + kBlock - 1) / kBlock;
    float r = p.dhT != nullptr ? p.dhT[i] : 0.f;      // gradient arriving at h_t from later tokens
    for (int64_t j = blocks - 1; j >= 0; --j) {
        const int64_t t0 = j * kBlock;
        const int n = static_cast<int>(p.T - t0 < kBlock ? p.T - t0 : kBlock);
        float before[kBlock];                          // h_{t-1} of the block's tokens
        float h = p.states[(b * blocks + j) * p.D + c];
#pragma unroll
        for (int k = 0; k < kBlock; ++k) {
            before[k] = h;
            if (k < n) {
                const int64_t at = (b * p.T + t0 + k) * p.D + c;
                float u = load_elem<E>(p.x, at);
                if constexpr (BETA) u *= load_elem<E>(p.beta, at);
                h = fmaf(__expf(load_elem<E>(p.g, at)), h, u);
            }
        }
#pragma unroll
        for (int k = kBlock - 1; k >= 0; --k) {
            if (k >= n) continue;
            const int64_t at = (b * p.T + t0 + k) * p.D + c;
            const float e = r + load_elem<E>(p.dO, at);
            r = __expf(load_elem<E>(p.g, at)) * e;
            store_elem<E>(p.dg, at, r * before[k]);
            if constexpr (BETA) {
                store_elem<E>(p.dx, at, load_elem<E>(p.beta, at) * e);
                store_elem<E>(p.dbeta, at, load_elem<E>(p.x, at) * e);
            } else {
                store_elem<E>(p.dx, at, e);
            }
        }
    }
    if (p.dh0 != nullptr) p.dh0[i] = r;
}

// One token per sequence.  A workgroup takes 256 * V channels of one row; rows
// that share a page are all taken by the first of them, in order.
template <typename E, bool BETA, int V>
__global__ __launch_bounds__(kStepThreads) void linrec_step_kernel(LinrecStepArgs p, int per_row) {
    int b = blockIdx.x / per_row;
    const int c = ((blockIdx.x % per_row) * kStepThreads + threadIdx.x) * V;
    int page = b;
    bool later = false;
    if (p.slots != nullptr) {
        page = p.slots[b];
        if (page < 0 || page >= p.n_pages) return;
        bool earlier;
        slot_sharers(p.slots, p.B, b, page, &earlier, &later);
        if (earlier) return;
    }
    if (c >= p.D) return;
    float* hp = p.h + static_cast<int64_t>(page) * p.D + c;
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = hp[v];
    while (true) {
        const int64_t at = static_cast<int64_t>(b) * p.D + c;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float u = load_elem<E>(p.x, at + v);
            if constexpr (BETA) u *= load_elem<E>(p.beta, at + v);
            h[v] = fmaf(__expf(load_elem<E>(p.g, at + v)), h[v], u);
            store_elem<E>(p.o, at + v, h[v]);
        }
        if (!later) break;
        b = next_sharer(p.slots, p.B, b, page);
        if (b == p.B) break;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) hp[v] = h[v];
}

template <typename E>
hipError_t launch_fwd_dtype(const LinrecArgs& a, hipStream_t s) {
    const int64_t rows = static_cast<int64_t>(a.B) * a.D;
    const dim3 grid(static_cast<unsigned>((rows + kSeqThreads - 1) / kSeqThreads)), block(kSeqThreads);
    if (a.beta != nullptr) hipLaunchKernelGGL((linrec_fwd_kernel<E, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((linrec_fwd_kernel<E, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <typename E>
hipError_t launch_bwd_dtype(const LinrecBwdArgs& a, hipStream_t s) {
    const int64_t rows = static_cast<int64_t>(a.B) * a.D;
    const dim3 grid(static_cast<unsigned>((rows + kSeqThreads - 1) / kSeqThreads)), block(kSeqThreads);
    if (a.beta != nullptr) hipLaunchKernelGGL((linrec_bwd_kernel<E, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((linrec_bwd_kernel<E, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <typename E, bool BETA>
hipError_t launch_step_beta(const LinrecStepArgs& a, hipStream_t s) {
    // four channels a lane where rows start on whole vectors, one otherwise
    const int V = a.D % 4 == 0 ? 4 : 1;
    const int per_row = (a.D + kStepThreads * V - 1) / (kStepThreads * V);
    const dim3 grid(static_cast<unsigned>(a.B) * static_cast<unsigned>(per_row)), block(kStepThreads);
    if (V == 4) hipLaunchKernelGGL((linrec_step_kernel<E, BETA, 4>), grid, block, 0, s, a, per_row);
    else hipLaunchKernelGGL((linrec_step_kernel<E, BETA, 1>), grid, block, 0, s, a, per_row);
    return hipGetLastError();
}

template <typename E>
hipError_t launch_step_dtype(const LinrecStepArgs& a, hipStream_t s) {
    return a.beta != nullptr ? launch_step_beta<E, true>(a, s) : launch_step_beta<E, false>(a, s);
}

}  // namespace

size_t linrec_fwd_workspace_bytes(int, int, int, int) { return 0; }
size_t linrec_bwd_workspace_bytes(int, int, int, int) { return 0; }

hipError_t launch_linrec_fwd(int dtype, const LinrecArgs& a, hipStream_t s) {
    return dtype == 0 ? launch_fwd_dtype<F32>(a, s) : launch_fwd_dtype<BF16>(a, s);
}

hipError_t launch_linrec_bwd(int dtype, const LinrecBwdArgs& a, hipStream_t s) {
    return dtype == 0 ? launch_bwd_dtype<F32>(a, s) : launch_bwd_dtype<BF16>(a, s);
}

hipError_t launch_linrec_step(int dtype, const LinrecStepArgs& a, hipStream_t s) {
    return dtype == 0 ? launch_step_dtype<F32>(a, s) : launch_step_dtype<BF16>(a, s);
}

}  // namespace dr
