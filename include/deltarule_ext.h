/*
 * deltarule_ext.h — further entry points of libdeltarule.so: the gated linear
 * recurrence, and the pool of state pages that serving keeps between calls.
 *
 * The conventions of deltarule.h hold here too: device pointers on the current
 * HIP device, dense and row-major, 16-byte aligned; the caller owns every
 * buffer; workspaces as (workspace, workspace_bytes), 256-byte aligned and
 * disjoint from every tensor argument; a hipStream_t as the last argument;
 * calls enqueue and return; host-side validation before any HIP call; errors as
 * a dr_status; results that do not depend on timing.
 *
 * What the host cannot see, the page numbers in device memory, is checked by
 * the kernels: a number outside the pool never reaches memory, with the effect
 * stated at each entry point.
 */
#ifndef DELTARULE_EXT_H
#define DELTARULE_EXT_H

#include "deltarule.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Version of this header; dr_ext_version() returns that of the loaded library. */
#define DR_EXT_VERSION 1
int dr_ext_version(void);

/* ---- gated linear recurrence ------------------------------------------------
 *
 * A state per channel instead of a matrix per head.  For channel c and token t
 *
 *   h_t = exp(g_t) h_{t-1} + beta_t x_t        o_t = h_t
 *
 * with a log-decay g_t <= 0 and a write gate beta_t per channel and token.  It
 * is the delta rule's decay and write without the read that makes a matrix
 * memory error-correcting.  A decay that is zero in fp32 (g = -inf; any g below
 * -87.4) forgets everything before its token, infinities and NaN too (a
 * document's border in a packed sequence), and lets no gradient past it, whatever
 * arrives: dg is 0 there.  Elsewhere an infinity or NaN stays in its channel, as
 * the formula has it.  There is no floor.  g > 0 is not refused, but the decays of
 * up to 384 consecutive tokens are multiplied up, and their product must stay
 * inside fp32.  Tokens with g = 0 and x = 0 leave the
 * state as it is (the padding of a short sequence in a batch).
 *
 * States, decays and sums are fp32 whatever the dtype; o and the gradients are
 * rounded once.
 */
typedef struct {
    int32_t B;     /* sequences, 1 .. 2^20                                      */
    int32_t T;     /* tokens per sequence, >= 1 (1 for delta_linrec_step)       */
    int32_t D;     /* channels, any number from 1 to 2^24                       */
    int32_t dtype; /* dr_dtype of x, g, beta, o, dO and their gradients         */
} dr_linrec_desc;  /* and B * D <= 2^31 - 1, B * T * D <= 2^40 (DR_E_SHAPE)     */

/* Tokens from one row of `states` to the next. */
#define DR_LINREC_BLOCK 16

/*
 * delta_linrec_fwd — the recurrence over whole sequences.
 *
 *   x, g   [B, T, D] dtype;  beta [B, T, D] dtype or NULL (1)
 *   h0     [B, D] fp32, the state before the first token; NULL means zero
 *   o      [B, T, D] dtype (written)
 *   h_T    [B, D] fp32 (written), the state after the last token; NULL if not
 *          wanted; may be h0 (in place)
 *   states [B, ceil(T / DR_LINREC_BLOCK), D] fp32 (written): row j is the state
 *          before token j * DR_LINREC_BLOCK.  What delta_linrec_bwd needs of
 *          this call; NULL if not wanted
 *   Outputs must not overlap any input or one another (h_T = h0 excepted).
 */
dr_status delta_linrec_fwd_workspace_bytes(const dr_linrec_desc* desc, size_t* bytes);
dr_status delta_linrec_fwd(const dr_linrec_desc* desc, const void* x, const void* g,
                           const void* beta, const float* h0, void* o, float* h_T, float* states,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * delta_linrec_bwd — gradients of delta_linrec_fwd.  With e_t the gradient that
 * arrives at h_t (e_t = dO_t + exp(g_{t+1}) e_{t+1}, dh_T added at the last token):
 *
 *   dx_t = beta_t e_t    dbeta_t = x_t e_t    dg_t = exp(g_t) h_{t-1} e_t
 *   dh0  = exp(g_1) e_1
 *
 *   x, g, beta  as given to delta_linrec_fwd
 *   states      as delta_linrec_fwd wrote it for these inputs
 *   dO     [B, T, D] dtype;  dh_T [B, D] fp32 or NULL (0)
 *   dx, dg [B, T, D] dtype (written);  dbeta [B, T, D] dtype (written), NULL
 *          exactly when beta is NULL
 *   dh0    [B, D] fp32 (written); NULL if not wanted
 *   Outputs must not overlap any input or one another.
 */
dr_status delta_linrec_bwd_workspace_bytes(const dr_linrec_desc* desc, size_t* bytes);
dr_status delta_linrec_bwd(const dr_linrec_desc* desc, const void* x, const void* g,
                           const void* beta, const float* states, const void* dO,
                           const float* dh_T, void* dx, void* dg, void* dbeta, float* dh0,
                           void* workspace, size_t workspace_bytes, void* stream);

/* ---- pool of state pages ----------------------------------------------------
 *
 * A pool is n_pages pages of `page` floats each; a page holds the state of one
 * sequence: [H, d_v, d_k] of the delta rule, [D] of the linear recurrence.
 * Sequences name their pages by slot numbers: lists of int32 in device memory,
 * which need be aligned to 4 bytes only.
 */
#define DR_MAX_PAGES 65536   /* pages of a pool, and entries of a list of slots */

/*
 * delta_linrec_step — one token per sequence.
 *
 *   desc->T must be 1;  x, g [B, D] dtype;  beta [B, D] dtype or NULL
 *   h      pool [n_pages, D] fp32, updated in place
 *   slots  [B] int32: row b's state is page slots[b].  A row whose slot lies
 *          outside the pool (-1, say, for the rows that pad a batch) is skipped:
 *          its row of o is left as it was.  Rows that name the same page are
 *          applied one after the other, in the order of b.  NULL: row b's state
 *          is page b, and n_pages must be B.  Every row looks through the list for
 *          others of its page: meant for batches of up to some thousand rows (4096
 *          rows of 256 channels 25 us, 65536 rows 3.9 ms)
 *   o      [B, D] dtype (written)
 *   Neither o nor h may overlap any input or each other.
 */
dr_status delta_linrec_step(const dr_linrec_desc* desc, const void* x, const void* g,
                            const void* beta, float* h, int32_t n_pages, const int32_t* slots,
                            void* o, void* stream);

/*
 * delta_decode_slots — delta_decode on the pages of a pool.
 *
 *   desc and q, k, v, beta, wgate, g, o  as for delta_decode (T = 1)
 *   pool   [n_pages, H, d_v, d_k] fp32, updated in place
 *   slots  [B] int32, as for delta_linrec_step (required): rows outside the pool
 *          are skipped, rows that share a page act in the order of b; up to some
 *          thousand rows
 *   Neither o nor pool may overlap any input or each other.
 */
dr_status delta_decode_slots(const dr_desc* desc, const void* q, const void* k, const void* v,
                             const void* beta, const void* wgate, const void* g, float* pool,
                             int32_t n_pages, const int32_t* slots, void* o, void* stream);

typedef struct {
    int64_t page;    /* floats per page, any number >= 1                          */
    int32_t n_pages; /* pages of the pool, 1 .. DR_MAX_PAGES                      */
    int32_t n;       /* entries of the list, 0 .. DR_MAX_PAGES                    */
} dr_pages_desc;     /* limit: page * n_pages <= 2^40 (DR_E_SHAPE)                */

/*
 * delta_pages_copy — copies, forks and clears pages.  Entry i copies page src[i]
 * of src_pool to page dst[i] of pool; src[i] = -1 clears page dst[i] to zero (the
 * state of a new sequence).  Any other number outside its pool makes the entry
 * do nothing.
 *
 *   pool      [n_pages, page] fp32, the destination
 *   src_pool  [src_pages, page] fp32: pool itself (src_pages = n_pages), or
 *             another pool, disjoint from it (a batch of prefilled states, say)
 *   dst, src  [n] int32 (NULL if n = 0)
 *
 * The entries act as if one after the other, in order: a page may be named any
 * number of times on either side.  Lists in which no destination is named twice
 * or is also a source (every list of forks into free pages) are copied at once;
 * one such entry makes the call apply its whole list in order, at 0.3 to 1 us an
 * entry (4000 pages of 8 KiB: 18 us at once, 1.95 ms in order).  A move, a copy
 * and then the clear of its source, is quicker as two calls.
 */
dr_status delta_pages_copy(const dr_pages_desc* desc, float* pool, const int32_t* dst,
                           const float* src_pool, int32_t src_pages, const int32_t* src,
                           void* stream);

/*
 * delta_pages_compact — moves the live pages of a pool to its front.
 *
 *   pool      [n_pages, page] fp32, in place
 *   slots     [n] int32: the pages of the live sequences, in any order; numbers
 *             outside the pool (-1) are sequences that have ended; sequences
 *             that share a page keep sharing it
 *   slots_out [n] int32 (written): where each sequence's page is now, -1 for the
 *             ended ones; must not overlap slots
 *   n_live    [1] int32 (written): the number of live pages L
 *
 * Afterwards the live pages are pages 0 .. L-1.  A live page below L stays where
 * it is; the k-th lowest live page at or above L goes to the k-th lowest free
 * page below L.  Pages L and up are free, their content unspecified.
 */
dr_status delta_pages_compact(const dr_pages_desc* desc, float* pool, const int32_t* slots,
                              int32_t* slots_out, int32_t* n_live, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DELTARULE_EXT_H */
