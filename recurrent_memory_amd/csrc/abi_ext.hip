// C ABI of the gated linear recurrence and of the pool of state pages: host-side
// validation and dispatch.  See include/deltarule_ext.h for the contract.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/deltarule_ext.h"
#include "abi_checks.h"
#include "kernels.h"

namespace {

using namespace dr::abi;

// Elements of the recurrence's operands.
struct LinrecSizes {
    int64_t seq, row, states;  // [B,T,D], [B,D], [B,ceil(T/16),D]
};

dr_status check_linrec_desc(const dr_linrec_desc* d, bool step, LinrecSizes* sz) {
    if (d == nullptr) return DR_E_NULLPTR;
    if (d->dtype != DR_F32 && d->dtype != DR_BF16) return DR_E_UNSUPPORTED;
    if (d->B < 1 || d->T < 1 || d->D < 1) return DR_E_SHAPE;
    if (step && d->T != 1) return DR_E_SHAPE;
    // element indices stay far inside int64, channel numbers inside int32 and
    // grids below 2^32 threads
    if (d->B > (1 << 20) || d->D > (1 << 24)) return DR_E_SHAPE;
    sz->row = static_cast<int64_t>(d->B) * d->D;
    if (sz->row > (int64_t(1) << 31) - 1) return DR_E_SHAPE;
    if (d->T > (int64_t(1) << 40) / sz->row) return DR_E_SHAPE;
    sz->seq = sz->row * d->T;
    sz->states = sz->row * ((d->T - 1) / DR_LINREC_BLOCK + 1);
    return DR_OK;
}

// The outputs lie clear of every input and of one another, except where two
// pointers are equal and the pair is listed as allowed in place.
dr_status check_outputs(const Span* in, int n_in, const Span* out, int n_out, int inplace_out = -1,
                        int inplace_in = -1) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j) {
            if (i == inplace_out && j == inplace_in && out[i].lo == in[j].lo) continue;
            if (overlap(out[i], in[j])) return DR_E_ALIAS;
        }
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return DR_E_ALIAS;
    }
    return DR_OK;
}

dr_status check_pages_desc(const dr_pages_desc* d) {
    if (d == nullptr) return DR_E_NULLPTR;
    if (d->page < 1 || d->n_pages < 1 || d->n_pages > DR_MAX_PAGES) return DR_E_SHAPE;
    if (d->n < 0 || d->n > DR_MAX_PAGES) return DR_E_SHAPE;
    if (d->page > (int64_t(1) << 40) / d->n_pages) return DR_E_SHAPE;
    return DR_OK;
}

// Lists of page numbers may start at any int32 (a part of a longer list).
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

dr_status launched(hipError_t e) { return e == hipSuccess ? DR_OK : DR_E_LAUNCH; }

}  // namespace

extern "C" {

int dr_ext_version(void) { return DR_EXT_VERSION; }

dr_status delta_linrec_fwd_workspace_bytes(const dr_linrec_desc* desc, size_t* bytes) {
    try {
        if (bytes == nullptr) return DR_E_NULLPTR;
        LinrecSizes sz;
        const dr_status st = check_linrec_desc(desc, false, &sz);
        if (st != DR_OK) return st;
        *bytes = dr::linrec_fwd_workspace_bytes(desc->dtype, desc->B, desc->T, desc->D);
        return DR_OK;
    } catch (...) {
        return DR_E_LAUNCH;
    }
}

dr_status delta_linrec_fwd(const dr_linrec_desc* desc, const void* x, const void* g,
                           const void* beta, const float* h0, void* o, float* h_T, float* states,
                           void* workspace, size_t workspace_bytes, void* stream) {
    try {
        LinrecSizes sz;
        dr_status st = check_linrec_desc(desc, false, &sz);
        if (st != DR_OK) return st;
        if (x == nullptr || g == nullptr || o == nullptr) return DR_E_NULLPTR;
        const void* ptrs[] = {x, g, beta, h0, o, h_T, states};
        for (const void* p : ptrs)
            if (p != nullptr && !aligned16(p)) return DR_E_ALIGN;
        const int64_t eb = desc->dtype == DR_F32 ? 4 : 2;
        const Span all[] = {span_of(x, sz.seq, eb),  span_of(g, sz.seq, eb),  span_of(beta, sz.seq, eb),
                            span_of(h0, sz.row, 4),  span_of(o, sz.seq, eb),  span_of(h_T, sz.row, 4),
                            span_of(states, sz.states, 4)};
        st = check_outputs(all, 4, all + 4, 3, 1, 3);
        if (st != DR_OK) return st;
        const size_t need = dr::linrec_fwd_workspace_bytes(desc->dtype, desc->B, desc->T, desc->D);
        st = check_workspace(need, workspace, workspace_bytes, all, 7);
        if (st != DR_OK) return st;

        st = check_device();
        if (st != DR_OK) return st;
        dr::LinrecArgs a{desc->B, desc->T, desc->D, x, g, beta, h0, o, h_T, states};
        a.ws = workspace;
        return launched(dr::launch_linrec_fwd(desc->dtype, a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return DR_E_LAUNCH;
    }
}

dr_status delta_linrec_bwd_workspace_bytes(const dr_linrec_desc* desc, size_t* bytes) {
    try {
        if (bytes == nullptr) return DR_E_NULLPTR;
        LinrecSizes sz;
        const dr_status st = check_linrec_desc(desc, false, &sz);
        if (st != DR_OK) return st;
        *bytes = dr::linrec_bwd_workspace_bytes(desc->dtype, desc->B, desc->T, desc->D);
        return DR_OK;
    } catch (...) {
        return DR_E_LAUNCH;
    }
}

dr_status delta_linrec_bwd(const dr_linrec_desc* desc, const void* x, const void* g,
                           const void* beta, const float* states, const void* dO,
                           const float* dh_T, void* dx, void* dg, void* dbeta, float* dh0,
                           void* workspace, size_t workspace_bytes, void* stream) {
    try {
        LinrecSizes sz;
        dr_status st = check_linrec_desc(desc, false, &sz);
        if (st != DR_OK) return st;
        if (x == nullptr || g == nullptr || states == nullptr || dO == nullptr || dx == nullptr ||
            dg == nullptr)
            return DR_E_NULLPTR;
        if ((beta == nullptr) != (dbeta == nullptr))
            return beta == nullptr ? DR_E_UNSUPPORTED : DR_E_NULLPTR;
        const void* ptrs[] = {x, g, beta, states, dO, dh_T, dx, dg, dbeta, dh0};
        for (const void* p : ptrs)
            if (p != nullptr && !aligned16(p)) return DR_E_ALIGN;
        const int64_t eb = desc->dtype == DR_F32 ? 4 : 2;
        const Span all[] = {span_of(x, sz.seq, eb),     span_of(g, sz.seq, eb), span_of(beta, sz.seq, eb),
                            span_of(states, sz.states, 4), span_of(dO, sz.seq, eb), span_of(dh_T, sz.row, 4),
                            span_of(dx, sz.seq, eb),    span_of(dg, sz.seq, eb), span_of(dbeta, sz.seq, eb),
                            span_of(dh0, sz.row, 4)};
        st = check_outputs(all, 6, all + 6, 4);
        if (st != DR_OK) return st;
        const size_t need = dr::linrec_bwd_workspace_bytes(desc->dtype, desc->B, desc->T, desc->D);
        st = check_workspace(need, workspace, workspace_bytes, all, 10);
        if (st != DR_OK) return st;

        st = check_device();
        if (st != DR_OK) return st;
        dr::LinrecBwdArgs a{desc->B, desc->T, desc->D, x, g, beta, states, dO, dh_T, dx, dg, dbeta, dh0};
        a.ws = workspace;
        return launched(dr::launch_linrec_bwd(desc->dtype, a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return DR_E_LAUNCH;
    }
}

dr_status delta_linrec_step(const dr_linrec_desc* desc, const void* x, const void* g,
                            const void* beta, float* h, int32_t n_pages, const int32_t* slots,
                            void* o, void* stream) {
    try {
        LinrecSizes sz;
        dr_status st = check_linrec_desc(desc, true, &sz);
        if (st != DR_OK) return st;
        if (x == nullptr || g == nullptr || h == nullptr || o == nullptr) return DR_E_NULLPTR;
        if (n_pages < 1) return DR_E_SHAPE;
        if (slots == nullptr ? n_pages != desc->B : n_pages > DR_MAX_PAGES || desc->B > DR_MAX_PAGES)
            return DR_E_SHAPE;
        const void* ptrs[] = {x, g, beta, h, o};
        for (const void* p : ptrs)
            if (p != nullptr && !aligned16(p)) return DR_E_ALIGN;
        if (!aligned4(slots)) return DR_E_ALIGN;
        const int64_t eb = desc->dtype == DR_F32 ? 4 : 2;
        const Span in[] = {span_of(x, sz.row, eb), span_of(g, sz.row, eb), span_of(beta, sz.row, eb),
                           span_of(slots, desc->B, 4)};
        const Span out[] = {span_of(h, static_cast<int64_t>(n_pages) * desc->D, 4), span_of(o, sz.row, eb)};
        st = check_outputs(in, 4, out, 2);
        if (st != DR_OK) return st;

        st = check_device();
        if (st != DR_OK) return st;
        const dr::LinrecStepArgs a{desc->B, desc->D, n_pages, x, g, beta, h, slots, o};
        return launched(dr::launch_linrec_step(desc->dtype, a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return DR_E_LAUNCH;
    }
}

dr_status delta_decode_slots(const dr_desc* desc, const void* q, const void* k, const void* v,
                             const void* beta, const void* wgate, const void* g, float* pool,
                             int32_t n_pages, const int32_t* slots, void* o, void* stream) {
    try {
        Sizes sz;
        dr_status st = check_desc(desc, true, &sz);
        if (st != DR_OK) return st;
        if (q == nullptr || k == nullptr || v == nullptr || o == nullptr || pool == nullptr ||
            slots == nullptr)
            return DR_E_NULLPTR;
        st = check_gate_ptrs(desc, beta, wgate, g);
        if (st != DR_OK) return st;
        if (n_pages < 1 || n_pages > DR_MAX_PAGES || desc->B > DR_MAX_PAGES) return DR_E_SHAPE;
        const void* ptrs[] = {q, k, v, beta, wgate, g, pool, o};
        for (const void* p : ptrs)
            if (p != nullptr && !aligned16(p)) return DR_E_ALIGN;
        if (!aligned4(slots)) return DR_E_ALIGN;
        const int64_t eb = desc->dtype == DR_F32 ? 4 : 2;
        const int64_t page = static_cast<int64_t>(desc->H) * desc->d_v * desc->d_k;
        const Span in[] = {span_of(q, sz.qk, eb),        span_of(k, sz.qk, eb), span_of(v, sz.v, eb),
                           span_of(beta, sz.beta, eb),   span_of(wgate, sz.wgate, eb),
                           span_of(g, sz.g, eb),         span_of(slots, desc->B, 4)};
        const Span out[] = {span_of(pool, page * n_pages, 4), span_of(o, sz.v, eb)};
        st = check_outputs(in, 7, out, 2);
        if (st != DR_OK) return st;

        st = check_device();
        if (st != DR_OK) return st;
        const dr::DecodeArgs a{desc->B, desc->H, desc->d_k, desc->d_v, q, k, v, beta, wgate, g, pool, o,
                               sz.Hk};
        return launched(dr::launch_decode_slots(desc->variant, desc->dtype, a, n_pages, slots,
                                                static_cast<hipStream_t>(stream)));
    } catch (...) {
        return DR_E_LAUNCH;
    }
}

dr_status delta_pages_copy(const dr_pages_desc* desc, float* pool, const int32_t* dst,
                           const float* src_pool, int32_t src_pages, const int32_t* src,
                           void* stream) {
    try {
        dr_status st = check_pages_desc(desc);
        if (st != DR_OK) return st;
        if (pool == nullptr || src_pool == nullptr) return DR_E_NULLPTR;
        if (desc->n > 0 && (dst == nullptr || src == nullptr)) return DR_E_NULLPTR;
        if (src_pages < 1 || src_pages > DR_MAX_PAGES || desc->page > (int64_t(1) << 40) / src_pages)
            return DR_E_SHAPE;
        if (src_pool == pool && src_pages != desc->n_pages) return DR_E_SHAPE;
        if (!aligned16(pool) || !aligned16(src_pool) || !aligned4(dst) || !aligned4(src)) return DR_E_ALIGN;
        const Span in[] = {span_of(src_pool, desc->page * src_pages, 4), span_of(dst, desc->n, 4),
                           span_of(src, desc->n, 4)};
        const Span out[] = {span_of(pool, desc->page * desc->n_pages, 4)};
        st = check_outputs(in, 3, out, 1, 0, 0);
        if (st != DR_OK) return st;
        if (desc->n == 0) return DR_OK;

        st = check_device();
        if (st != DR_OK) return st;
        const dr::PagesCopyArgs a{desc->page, desc->n_pages, src_pages, desc->n, pool, dst, src_pool, src};
        return launched(dr::launch_pages_copy(a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return DR_E_LAUNCH;
    }
}

dr_status delta_pages_compact(const dr_pages_desc* desc, float* pool, const int32_t* slots,
                              int32_t* slots_out, int32_t* n_live, void* stream) {
    try {
        dr_status st = check_pages_desc(desc);
        if (st != DR_OK) return st;
        if (pool == nullptr || n_live == nullptr) return DR_E_NULLPTR;
        if (desc->n > 0 && (slots == nullptr || slots_out == nullptr)) return DR_E_NULLPTR;
        if (!aligned16(pool) || !aligned4(slots) || !aligned4(slots_out) || !aligned4(n_live)) return DR_E_ALIGN;
        const Span in[] = {span_of(slots, desc->n, 4)};
        const Span out[] = {span_of(pool, desc->page * desc->n_pages, 4), span_of(slots_out, desc->n, 4),
                            span_of(n_live, 1, 4)};
        st = check_outputs(in, 1, out, 3);
        if (st != DR_OK) return st;

        st = check_device();
        if (st != DR_OK) return st;
        const dr::PagesCompactArgs a{desc->page, desc->n_pages, desc->n, pool, slots, slots_out, n_live};
        return launched(dr::launch_pages_compact(a, static_cast<hipStream_t>(stream)));
    } catch (...) {
        return DR_E_LAUNCH;
    }
}

}  // extern "C"
