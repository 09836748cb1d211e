// Host-side validation shared by the entry points of the C ABI: byte ranges and
// overlap, descriptor, gate, workspace and device checks.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "../../include/deltarule.h"

namespace dr {
namespace abi {

struct Span {
    uintptr_t lo = 0, hi = 0;  // [lo, hi); empty when lo == hi
};

inline Span span_of(const void* p, int64_t elems, int64_t elem_bytes) {
    Span s;
    if (p != nullptr) {
        s.lo = reinterpret_cast<uintptr_t>(p);
        s.hi = s.lo + static_cast<uintptr_t>(elems * elem_bytes);
    }
    return s;
}

inline bool overlap(const Span& a, const Span& b) {
    return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Elements of each operand for a descriptor (T tokens per sequence), and the
// number of query/key heads.
struct Sizes {
    int64_t qk, v, beta, wgate, g, state;
    int Hk;
};

inline dr_status check_desc(const dr_desc* d, bool decode, Sizes* sz) {
    if (d == nullptr) return DR_E_NULLPTR;
    if (d->variant < DR_DELTANET || d->variant > DR_FG2) return DR_E_UNSUPPORTED;
    if (d->dtype != DR_F32 && d->dtype != DR_BF16) return DR_E_UNSUPPORTED;
    if (d->B < 1 || d->H < 1 || d->T < 1) return DR_E_SHAPE;
    if (decode && d->T != 1) return DR_E_SHAPE;
    if ((d->d_k != 64 && d->d_k != 128) || (d->d_v != 64 && d->d_v != 128)) return DR_E_UNSUPPORTED;
    if (d->chunk != 64) return DR_E_UNSUPPORTED;
    if (d->H_k < 0 || d->H_k > d->H || (d->H_k > 0 && d->H % d->H_k != 0)) return DR_E_SHAPE;
    sz->Hk = d->H_k == 0 ? d->H : d->H_k;
    const int64_t tok = static_cast<int64_t>(d->B) * d->T * d->H;
    // Keep every element index inside int64, every grid below 2^31 threads
    // (the widest grids: 8 value tiles of 256 threads per head, and one
    // 512-thread workgroup per 64-token chunk of every head in the backward)
    // and the kernels' 32-bit offsets within a chunk (64 rows of H_k heads of
    // d_k elements) below 2^31.
    if (tok > (int64_t(1) << 34)) return DR_E_SHAPE;
    const int64_t heads = static_cast<int64_t>(d->B) * d->H;
    if (heads > (int64_t(1) << 20)) return DR_E_SHAPE;
    if (heads * ((d->T + 63) / 64) > (int64_t(1) << 22)) return DR_E_SHAPE;
    if (static_cast<int64_t>(d->H) * 64 * 128 > (int64_t(1) << 31) - 1) return DR_E_SHAPE;
    sz->qk = static_cast<int64_t>(d->B) * d->T * sz->Hk * d->d_k;
    sz->v = tok * d->d_v;
    sz->beta = (d->variant == DR_GDN2 || d->variant == DR_FG2) ? tok * d->d_k : tok;
    sz->wgate = d->variant == DR_GDN2 ? tok * d->d_v : 0;
    sz->g = d->variant == DR_DELTANET ? 0 : (d->variant == DR_GDN ? tok : tok * d->d_k);
    sz->state = static_cast<int64_t>(d->B) * d->H * d->d_v * d->d_k;
    return DR_OK;
}

inline dr_status check_gate_ptrs(const dr_desc* d, const void* beta, const void* wgate, const void* g) {
    if (beta == nullptr) return DR_E_NULLPTR;
    if (d->variant == DR_GDN2) {
        if (wgate == nullptr) return DR_E_NULLPTR;
    } else if (wgate != nullptr) {
        return DR_E_UNSUPPORTED;
    }
    if (d->variant == DR_DELTANET) {
        if (g != nullptr) return DR_E_UNSUPPORTED;
    } else if (g == nullptr) {
        return DR_E_NULLPTR;
    }
    return DR_OK;
}

// The caller's workspace: present and large enough when one is needed,
// 256-byte aligned, and disjoint from every tensor argument.
inline dr_status check_workspace(size_t need, const void* ws, size_t ws_bytes, const Span* spans, int n) {
    if (need == 0) return DR_OK;
    if (ws == nullptr || ws_bytes < need) return DR_E_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return DR_E_ALIGN;
    Span w;
    w.lo = reinterpret_cast<uintptr_t>(ws);
    w.hi = w.lo + need;
    for (int i = 0; i < n; ++i)
        if (overlap(w, spans[i])) return DR_E_ALIAS;
    return DR_OK;
}

inline std::atomic<int> g_arch_state[64];  // per device: 0 unknown, 1 gfx950, 2 other

inline dr_status check_device() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) {
        (void)hipGetLastError();
        return DR_E_DEVICE;
    }
    if (dev < 64) {
        const int st = g_arch_state[dev].load(std::memory_order_acquire);
        if (st == 1) return DR_OK;
        if (st == 2) return DR_E_DEVICE;
    }
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) {
        (void)hipGetLastError();
        return DR_E_DEVICE;
    }
    const bool ok = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    if (dev < 64) g_arch_state[dev].store(ok ? 1 : 2, std::memory_order_release);
    return ok ? DR_OK : DR_E_DEVICE;
}

}  // namespace abi
}  // namespace dr
