/*
 * gdn_mixer.h - C ABI of the operators that stand around the recurrent layers
 * of gdn.h and gdn_recurrent.h (AMD Instinct MI355X, gfx950):
 *
 *   gdn_conv_fwd, _bwd, _step       the short causal convolution of each channel
 *                                   in front of a recurrent layer
 *   gdn_scan_fwd, _bwd, _step       the selective state space scan: a recurrent
 *                                   layer with a decay for each channel, state
 *                                   and token
 *   gdn_qk_rotary_fwd, _bwd         norms of queries and keys for each head, and
 *                                   the rotation by position, in one pass
 *
 * Conventions are those of gdn.h and gdn_recurrent.h: pointers marked device
 * are HIP device memory owned by the caller, 16-byte aligned; inputs are never
 * written; nothing is allocated or synchronised; all work goes on the given
 * stream; every check runs before the first HIP call; the status codes are
 * gdn_status; a page number outside [0, n_pages) means "no page". Outputs are
 * apart from the inputs and from each other unless said otherwise. dtype is
 * GDN_DTYPE_F32 or GDN_DTYPE_BF16. Work that a launch cannot hold (2^32 threads)
 * is GDN_ERR_UNSUPPORTED, and so are token strides of 2^24 bytes or more in a
 * scan.
 *
 * Sequences are the B rows of T tokens (n_units = 0) or packed documents of
 * one row, offsets as in gdn_desc (none is empty).
 */
#ifndef GDN_MIXER_H
#define GDN_MIXER_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The short causal convolution. For channel d of D and W taps,
 *
 *     z_t = bias[d] + sum_{j < W} weight[d][j] x_{t-W+1+j}[d]
 *     y_t = z_t, or z_t sigmoid(z_t) with silu
 *
 * A sequence's state is the W - 1 inputs in front of its next token, oldest
 * first, in the inputs' type ([W-1][D]): nothing in it is rounded. Products
 * and sums are fp32; y is rounded once.
 */
typedef struct {
    int32_t B, T, D;                   /* D a multiple of 8 */
    int32_t W;                         /* 2, 3 or 4 */
    int32_t dtype;                     /* x, y, states */
    int32_t w_dtype;                   /* weight [D][W] and bias [D] */
    int32_t silu;
    int32_t n_units;                   /* 0: rows; else documents (B = 1) */
    int64_t x_stride;                  /* elements from a token to the next, 16-byte aligned */
    const int32_t* offsets_host;       /* host   [n_units + 1] */
    const int32_t* offsets_dev;        /* device [n_units + 1] */
} gdn_conv_desc;

/*
 * gdn_conv_fwd - whole prompts.
 *   x         device, tokens of D channels at x_stride
 *   weight    device [D][W];  bias device [D] or NULL, both in w_dtype
 *   s_in      device [units][W-1][D], or a pool of n_pages such pages with
 *             in_pages device int32 [units]; NULL: zeros
 *   s_out     device, likewise with out_pages; NULL: not wanted. May be s_in
 *             (each sequence's state is replaced); two sequences must not write
 *             one page, nor one write a page that another reads (without page
 *             lists states that overlap by part are GDN_ERR_INVALID)
 *   y         device [tokens][D], contiguous
 */
gdn_status gdn_conv_fwd(const gdn_conv_desc* desc, const void* x, const void* weight, const void* bias,
                        const void* s_in, const int32_t* in_pages, void* s_out, const int32_t* out_pages,
                        int32_t n_pages, void* y, hipStream_t stream);

/*
 * gdn_conv_bwd - the gradients of gdn_conv_fwd (without pages) for dL/dy =
 * dout and dL/d(final state) = dfinal, both in dtype, contiguous (dfinal may
 * be NULL: zero).
 *   dx        device [tokens][D] in dtype
 *   dweight   device fp32 [D][W];  dbias device fp32 [D] or NULL (not wanted)
 *   dinitial  device [units][W-1][D] in dtype, or NULL
 *   workspace as for gdn_chunk_fwd (size query with NULL)
 * Sums over tokens are fp32, in an order that the sizes alone fix.
 */
gdn_status gdn_conv_bwd(const gdn_conv_desc* desc, const void* x, const void* weight, const void* bias,
                        const void* s_in, const void* dout, const void* dfinal, void* dx, float* dweight,
                        float* dbias, void* dinitial, void* workspace, size_t* workspace_bytes, hipStream_t stream);

/*
 * gdn_conv_step - one token of N sequences. desc->B = N and T = 1, n_units =
 * 0. Row n belongs to page pages[n] (pages NULL: page n), whose inputs are
 * shifted in place; rows without a page get y = 0. No two rows may name one
 * page.
 *   state     device [n_pages][W-1][D] in dtype
 *   y         device [N][D]
 */
gdn_status gdn_conv_step(const gdn_conv_desc* desc, const void* x, const void* weight, const void* bias,
                         const int32_t* pages, int32_t n_pages, void* state, void* y, hipStream_t stream);

/*
 * The selective state space scan. For channel d of D with S states, in group
 * g = d / (D / G), h [D][S] and everything in fp32,
 *
 *     dt'_t = dt_t[d] + dt_bias[d], through softplus if asked for
 *     h_t[d][s] = e^{dt'_t A[d][s]} h_{t-1}[d][s] + dt'_t u_t[d] B_t[g][s]
 *     y_t[d] = sum_s C_t[g][s] h_t[d][s] + skip[d] u_t[d]
 *     out_t[d] = y_t[d], or y_t[d] gate_t[d] sigmoid(gate_t[d])
 *
 * All values must be finite. A decay is one fp32 exponential (about 2^-23, and
 * as much of its exponent), so that a state which hardly decays drifts by up to
 * that a token (but for gdn_scan_step, which adds what a weak decay takes).
 */
typedef struct {
    int32_t B, T, D, G;                /* D / G a multiple of 8 */
    int32_t S;                         /* 8, 16, 32 or 64 */
    int32_t dtype;                     /* u, dt, B, C, gate, out */
    int32_t softplus;
    int32_t n_units;
    int64_t u_stride, dt_stride, gate_stride;        /* elements: token */
    int64_t b_stride[2], c_stride[2];                /* elements: token, group */
    const int32_t* offsets_host;
    const int32_t* offsets_dev;
} gdn_scan_desc;

/*
 * gdn_scan_fwd - whole prompts.
 *   u, dt, gate  device, tokens of D channels (gate may be NULL)
 *   A            device fp32 [D][S]
 *   B, C         device, tokens of G rows of S
 *   skip         device fp32 [D] or NULL;  dt_bias device fp32 [D] or NULL
 *   s_in, s_out  device fp32 [units][D][S] or pools with pages, as in
 *                gdn_conv_fwd
 *   h            device fp32 [gdn_scan_h_rows(desc)][D][S] or NULL: what
 *                gdn_scan_bwd needs of the states (those that every 16th token
 *                of a sequence is entered with)
 *   out          device [tokens][D]
 *   workspace    as for gdn_chunk_fwd
 */
gdn_status gdn_scan_fwd(const gdn_scan_desc* desc, const void* u, const void* dt, const float* A, const void* B,
                        const void* C, const float* skip, const void* gate, const float* dt_bias, const float* s_in,
                        const int32_t* in_pages, float* s_out, const int32_t* out_pages, int32_t n_pages, float* h,
                        void* out, void* workspace, size_t* workspace_bytes, hipStream_t stream);

/* rows of h; negative for a descriptor that gdn_scan_fwd refuses */
int64_t gdn_scan_h_rows(const gdn_scan_desc* desc);

/*
 * gdn_scan_bwd - the gradients of gdn_scan_fwd for dL/dout = dout (device
 * [tokens][D] in dtype) and dL/d(final state) = dht (fp32 [units][D][S] or
 * NULL), with h as that call wrote it. With E the gradient that arrives from
 * the next token,
 *
 *     g_t = C_t dy_t + E_{t+1},  E_t = e^{dt'_t A} g_t   (E_{T+1} = dht, dh0 = E_1)
 *
 *   du, ddt, dgate   device [tokens][D] in dtype (dgate NULL exactly if gate is)
 *   dB, dC           device [tokens][G][S] in dtype: sums over a group's
 *                    channels, rounded once
 *   dA, dskip, ddt_bias  device fp32 [D][S], [D], [D]; the latter two or NULL
 *   dh0              device fp32 [units][D][S] or NULL; may be dht
 * No atomics: results repeat bit for bit.
 */
gdn_status gdn_scan_bwd(const gdn_scan_desc* desc, const void* u, const void* dt, const float* A, const void* B,
                        const void* C, const float* skip, const void* gate, const float* dt_bias, const float* h,
                        const void* dout, const float* dht, void* du, void* ddt, float* dA, void* dB, void* dC,
                        float* dskip, void* dgate, float* ddt_bias, float* dh0, void* workspace,
                        size_t* workspace_bytes, hipStream_t stream);

/*
 * gdn_scan_step - one token of N sequences (desc->B = N, T = 1, n_units = 0)
 * on states in pages, as in gdn_conv_step.
 *   state     device fp32 [n_pages][D][S], updated in place
 *   out       device [N][D]; rows without a page get 0
 */
gdn_status gdn_scan_step(const gdn_scan_desc* desc, const void* u, const void* dt, const float* A, const void* B,
                         const void* C, const float* skip, const void* gate, const float* dt_bias,
                         const int32_t* pages, int32_t n_pages, float* state, void* out, hipStream_t stream);

/*
 * Norms of queries and keys and their rotation. Every row x of D values (a
 * token's head) becomes, with r = 1 / sqrt(mean x^2 + eps) (GDN_NORM_RMS),
 * 1 / sqrt(sum x^2 + eps) (GDN_NORM_L2) or 1 (GDN_NORM_NONE),
 *
 *     n = r x weight
 *     (n_a, n_b) -> amplitude (n_a cos - n_b sin, n_b cos + n_a sin)
 *
 * for the R / 2 pairs i of its first R values, a = i and b = i + R/2, or a = 2i
 * and b = 2i + 1 with interleaved; values from R on stay n. The angle of pair i
 * is position * freqs[i], multiplied and reduced to a turn in 64 bits: off by
 * up to 2^-51 of itself, 2^-24 of a turn after 2^27 turns.
 */
enum { GDN_NORM_NONE = 0, GDN_NORM_RMS = 1, GDN_NORM_L2 = 2 };
typedef struct {
    int32_t B, T, Hq, Hk;
    int32_t D;                         /* a multiple of 8, at most 256 */
    int32_t R;                         /* a multiple of 8, at most D; 0: no rotation */
    int32_t dtype;                     /* q, k and their gradients */
    int32_t w_dtype;                   /* q_weight, k_weight [D] */
    int32_t norm;                      /* GDN_NORM_* */
    int32_t interleaved;
    int32_t pos_i64;                   /* positions are int64, not int32 */
    float eps, amplitude;
    int64_t q_stride[2], k_stride[2];  /* elements: token, head */
} gdn_rotary_desc;

/*
 * gdn_qk_rotary_fwd
 *   q, k       device, B T tokens of Hq and Hk rows (strides as in
 *              gdn_linattn_desc)
 *   freqs      device fp64 [R/2], radians a token
 *   positions  device int32 or int64 [B T]; NULL: a token's place in its row.
 *              Both aligned to their own values, so that they may be slices
 *   q_weight, k_weight  device [D] in w_dtype, or NULL
 *   q_out, k_out        device [tokens][H][D], contiguous. q_out may be q, and
 *              k_out k, where these are contiguous
 */
gdn_status gdn_qk_rotary_fwd(const gdn_rotary_desc* desc, const void* q, const void* k, const double* freqs,
                             const void* positions, const void* q_weight, const void* k_weight, void* q_out,
                             void* k_out, hipStream_t stream);

/*
 * gdn_qk_rotary_bwd - the gradients for dL/dq_out = dq_out and dk_out (device
 * [tokens][H][D], contiguous); q and k are the forward's inputs.
 *   dq, dk     device, contiguous; may be dq_out and dk_out
 *   dq_weight, dk_weight  device fp32 [D]; NULL exactly where the weight is
 *   workspace  as for gdn_chunk_fwd
 */
gdn_status gdn_qk_rotary_bwd(const gdn_rotary_desc* desc, const void* q, const void* k, const double* freqs,
                             const void* positions, const void* q_weight, const void* k_weight, const void* dq_out,
                             const void* dk_out, void* dq, void* dk, float* dq_weight, float* dk_weight,
                             void* workspace, size_t* workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_MIXER_H */
