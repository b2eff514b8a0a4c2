/*
 * gdn_recurrent.h - C ABI of the recurrent-state operators of libgdn (AMD
 * Instinct MI355X, gfx950), beside the chunked gated delta rule of gdn.h:
 *
 *   gdn_linattn_fwd, gdn_linattn_bwd   linear attention with a decay for each
 *                                      head, over whole prompts
 *   gdn_linattn_step                   its form for single tokens
 *   gdn_recurrent_step                 the gated delta rule for single tokens
 *   gdn_pages_copy, gdn_pages_fork,    the pages of a state cache: copying,
 *   gdn_pages_compact                  forking and freeing, compacting
 *
 * A state is K x V (key-major) in fp32. A cache is a pool of pages, one page
 * holding the H states of one sequence ([n_pages][H][K][V]); operators that
 * take a pool find a sequence's page through an int32 page number. A number
 * outside [0, n_pages) means "no page": nothing is read (zero state) or
 * written through it, so no page list can cause an access out of range.
 *
 * Conventions are those of gdn.h: pointers marked device are HIP device
 * memory owned by the caller, 16-byte aligned; inputs are never written;
 * nothing is allocated or synchronised; all work goes on the given stream;
 * every check runs before the first HIP call; the status codes are
 * gdn_status.
 */
#ifndef GDN_RECURRENT_H
#define GDN_RECURRENT_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Linear attention with a decay for each head. For head h of H, with
 * d = e^{decay[h]} and a state S in K x V,
 *
 *     S_t = d S_{t-1} + k_t v_t^T          o_t = scale * S_t^T q_t
 *
 * or, over a whole sequence with entry state S_0 (t counted from 1),
 *
 *     o_i = scale * [ sum_{j <= i} d^{i-j} (q_i . k_j) v_j + d^i S_0^T q_i ]
 *
 * decay holds log decays, decay[h] <= 0 (0: no decay; -inf: only a token's
 * own k v^T). Powers of d are taken of differences of positions only, so no
 * intermediate exceeds the values themselves.
 *
 * q, k and v may each have fewer heads than H (Hq, Hk, Hv dividing H): head h
 * reads head h / (H / Hx). Rows (the K or V values of one token and head) are
 * contiguous; tokens and heads may lie at any distance that keeps every row
 * 16-byte aligned (strides in elements); a token stride of 32 MiB or more,
 * or 65536 heads, is GDN_ERR_UNSUPPORTED. So is work that a launch cannot
 * hold, 2^32 threads: 256 for each head of each segment of a sequence (1024
 * in the backward), and a quarter of the values of gradients of shared heads.
 *
 * Sequences are the B rows of T tokens (n_units = 0) or packed documents of
 * one row, offsets as in gdn_desc (a sequence's tokens are contiguous).
 */
typedef struct {
    int32_t B, T, H, Hq, Hk, Hv;
    int32_t K, V;                      /* 64 or 128, each */
    int32_t dtype;                     /* q, k, v: GDN_DTYPE_* */
    int32_t o_dtype;                   /* o: GDN_DTYPE_* */
    float scale;
    int32_t n_units;                   /* 0: rows; else documents (B = 1) */
    int64_t q_stride[2], k_stride[2], v_stride[2];   /* elements: token, head */
    const int32_t* offsets_host;       /* host   [n_units + 1] */
    const int32_t* offsets_dev;        /* device [n_units + 1] */
} gdn_linattn_desc;

/*
 * gdn_linattn_fwd - a whole prompt.
 *   q, k, v        device, as the descriptor says
 *   decay          device fp32 [H]
 *   s_in           device fp32 [units][H][K][V], or a pool of n_pages pages
 *                  with in_pages device int32 [units]; NULL: zero states
 *   s_out          device fp32, likewise with out_pages; NULL: not wanted.
 *                  May be s_in (each sequence's state is replaced); two
 *                  sequences must not write one page, nor one write a page
 *                  that another reads
 *   n_pages        pages of both pools (ignored without page lists)
 *   o              device [tokens][H][V] in o_dtype, contiguous; apart from
 *                  all else
 *   workspace      as for gdn_chunk_fwd (size query with NULL)
 * Products with bf16 inputs run on bf16 MFMA with fp32 accumulation; the
 * values computed on the way are split into two bf16 terms (scores and the
 * state, where they meet q and v; decayed v, where it enters the state of a
 * segment that returns none) or three (decayed v elsewhere). Two terms hold 16
 * bits: o is right to about 2^-16 of the sum of its absolute terms, 8 bits
 * more than a bf16 o is rounded to and 8 fewer than an fp32 o holds; the same
 * goes for the per-head gradients that are summed for shared heads. A returned
 * state keeps fp32 accuracy. fp32 inputs run on fp32 MFMA. Inputs must be
 * finite: masked products are multiplied by zero, so a value that is not
 * reaches o up to 31 tokens before it too.
 */
gdn_status gdn_linattn_fwd(const gdn_linattn_desc* desc, const void* q, const void* k, const void* v,
                           const float* decay, const float* s_in, const int32_t* in_pages, float* s_out,
                           const int32_t* out_pages, int32_t n_pages, void* o, void* workspace,
                           size_t* workspace_bytes, hipStream_t stream);

/*
 * gdn_linattn_bwd - the gradients of gdn_linattn_fwd (without pages) for
 * dL/do = dout and dL/d(final state) = dht. With D_t = dL/dS_t,
 *
 *     D_t = d D_{t+1} + scale q_t do_t^T  (D_T also + dht)
 *     dq_t = scale S_t do_t,  dk_t = D_t v_t,  dv_t = D_t^T k_t,  dS_0 = d D_1
 *
 *   dout        device [tokens][H][V] in desc->dtype, contiguous
 *   s_in, dht   device fp32 [units][H][K][V] or NULL (zero)
 *   dq, dk, dv  device, contiguous [tokens][Hq][K], [tokens][Hk][K],
 *               [tokens][Hv][V] in desc->dtype: sums over the heads that share
 *               one, each rounded once
 *   dh0         device fp32 [units][H][K][V] or NULL; may be dht or s_in
 *               (each sequence's state is replaced), but not overlap them
 *               otherwise (GDN_ERR_INVALID)
 * decay is a constant: it has no gradient. desc->o_dtype is not used.
 */
gdn_status gdn_linattn_bwd(const gdn_linattn_desc* desc, const void* q, const void* k, const void* v,
                           const float* decay, const float* s_in, const void* dout, const float* dht, void* dq,
                           void* dk, void* dv, float* dh0, void* workspace, size_t* workspace_bytes,
                           hipStream_t stream);

/*
 * Single tokens: N sequences, one token each. Row n of q, k, v belongs to
 * page pages[n] of the pool (pages NULL: page n), whose states are advanced
 * in place. Rows without a page get o = 0. No two rows may name one page.
 * N * H >= 2^24 is GDN_ERR_UNSUPPORTED.
 */
typedef struct {
    int32_t N, H, Hq, Hk, Hv;
    int32_t K, V;                      /* 64 or 128, each; gdn_recurrent_step: 128 */
    int32_t dtype, o_dtype;
    float scale;
    int32_t n_pages;
    int64_t q_stride[2], k_stride[2], v_stride[2];   /* elements: row, head */
} gdn_step_desc;

/*
 * gdn_linattn_step - S = d S + k v^T, o = scale * S^T q.
 *   state  device fp32 [n_pages][H][K][V], updated in place
 *   o      device [N][H][V] in o_dtype, apart from all else
 */
gdn_status gdn_linattn_step(const gdn_step_desc* desc, const void* q, const void* k, const void* v,
                            const float* decay, const int32_t* pages, float* state, void* o, hipStream_t stream);

/*
 * gdn_recurrent_step - the gated delta rule of gdn.h for one token:
 *     S~ = Diag(b^g) S,  r = v - S~^T k,  S = S~ + beta k r^T,  o = scale * S^T q
 *   g      device fp32 [N][H], or [N][H][K] with gate_kind = GDN_GATE_PER_KEY
 *   beta   device [N][H] in desc->dtype
 *   flags  GDN_FLAG_QK_L2NORM, GDN_FLAG_BETA_SIGMOID as in gdn_chunk_fwd
 * q and k may have fewer heads than H, as in gdn_linattn_desc.
 */
gdn_status gdn_recurrent_step(const gdn_step_desc* desc, int32_t gate_kind, int32_t use_exp2, const void* q,
                              const void* k, const void* v, const float* g, const void* beta, const int32_t* pages,
                              float* state, void* o, int32_t flags, hipStream_t stream);

/*
 * The pages of a cache. A pool is [n_layers][n_pages] pages of page_bytes
 * (a multiple of 16), contiguous; a page number stands for that page in
 * every layer. Page lists and tables are device int32.
 *
 * gdn_pages_copy - dst page dst_pages[i] = src page src_pages[i], every
 * layer, i < n. Pairs with a page out of range are skipped. The pools may be
 * one; the destinations must then be distinct and no source.
 */
gdn_status gdn_pages_copy(void* dst_pool, int32_t dst_n_pages, const void* src_pool, int32_t src_n_pages,
                          int32_t n_layers, int64_t page_bytes, const int32_t* dst_pages, const int32_t* src_pages,
                          int32_t n, hipStream_t stream);

/*
 * gdn_pages_fork - every slot i of a batch of beams continues slot parent[i]
 * (outside [0, n_slots): slot i ends). table[n_slots] holds the slots' pages,
 * distinct. The lowest child of a slot keeps its page; each further child
 * gets a copy in a free page, taken in order from the pages of the slots
 * without children (ascending slot), then from spare[n_spare] (entries out of
 * range are passed over). A child of a slot without a page gets none, and so
 * does one that finds no free page left.
 *   new_table  device int32 [n_slots], page or -1
 *   left       device int32 [n_slots + n_spare]: the free pages not taken, in
 *              order, then -1
 *   workspace  device int32 [gdn_pages_workspace_ints(n_slots)]
 * The inputs are not changed: new_table, left and workspace that overlap one
 * of them or each other are GDN_ERR_INVALID. n_slots <= 8192, n_spare <= 8192
 * (GDN_ERR_UNSUPPORTED beyond).
 */
gdn_status gdn_pages_fork(void* pool, int32_t n_layers, int32_t n_pages, int64_t page_bytes, const int32_t* table,
                          const int32_t* parent, int32_t n_slots, const int32_t* spare, int32_t n_spare,
                          int32_t* new_table, int32_t* left, int32_t* workspace, hipStream_t stream);

/*
 * gdn_pages_compact - moves the pages that table[n_slots] names into
 * [0, count), count being their number: pages below count stay, the others
 * move, in ascending order, into the holes in ascending order. Slots may
 * share a page; entries out of range stay -1.
 *   new_table  device int32 [n_slots]
 *   count      device int32 [1]
 *   workspace  device int32 [gdn_pages_workspace_ints(n_pages)]
 * These three may not overlap table or each other (GDN_ERR_INVALID).
 * n_pages <= 2^17 (GDN_ERR_UNSUPPORTED beyond).
 */
gdn_status gdn_pages_compact(void* pool, int32_t n_layers, int32_t n_pages, int64_t page_bytes, const int32_t* table,
                             int32_t n_slots, int32_t* new_table, int32_t* count, int32_t* workspace,
                             hipStream_t stream);

/* int32 entries of the workspace for n slots (fork) or n pages (compact) */
size_t gdn_pages_workspace_ints(int32_t n);

#ifdef __cplusplus
}
#endif

#endif /* GDN_RECURRENT_H */
