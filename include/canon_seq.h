/*
 * canon_seq.h — operators of sequence models on AMD MI355X (gfx950) whose
 * sums, like the reductions and scans of canon.h, each follow one fixed
 * expression: embedding lookup and its gradient (a canonical reduction by
 * key), the short causal convolution, and the selective state space scan,
 * with their backward passes and their forms for single tokens.  Part of
 * libcanon.
 *
 * What is computed:
 *
 *   embedding        out[t,:] = scale * W[ids[t],:]; a zero row where ids[t]
 *                    is outside [0, rows).
 *   embedding_grad   dW[v,:] = scale * PW(dout[t,:] over the t with
 *                    ids[t] = v, ascending), PW the pairwise tree of canon.h
 *                    in 32-bit additions; zero for a row that no id names.
 *                    Accumulating: dW[v,:] + that, and rows that no id names
 *                    are left as they are.
 *   causal_conv      p[t,d] = bias[d] + sum_j weight[d,j] x[t-(taps-1)+j, d]
 *                    (j ascending), out = p or p * sigmoid(p).  Rows before
 *                    the sequence's first are the initial state's, or zero.
 *   selective_scan   dl = delta + delta_bias, or softplus of that
 *                    a[t,d,n] = exp(dl[t,d] A[d,n])
 *                    h[t,d,n] = a h[t-1,d,n] + dl u[t,d] B[t,g,n]
 *                    y[t,d]   = sum_n C[t,g,n] h[t,d,n] + D[d] u[t,d]
 *                    out      = y, or y * z * sigmoid(z)
 *                    with g = d / (channels / groups).  The recurrence is
 *                    evaluated in chunks of CANON_SCAN_CHUNK rows from the
 *                    sequence's first row: inside a chunk h folds from the
 *                    chunk's start state H, and the next chunk's start state
 *                    is exp(A sum dl) H + S (S alone where H is zero), where
 *                    S is the chunk's fold from zero.  A sequence's outputs
 *                    therefore do not depend on
 *                    the other sequences of the call, on how it is packed or
 *                    on how the work is spread; cutting a sequence at a
 *                    multiple of CANON_SCAN_CHUNK rows and passing the state
 *                    on changes no bit.
 *
 * Everything is computed in 32 bits and rounded once where it is stored.  No
 * value is ever combined by an atomic, so each call is reproducible bit for
 * bit.  An infinite u, dl or B of the scan leaves the channel's outputs from that
 * row on not finite; which of them are infinite and which NaN is not specified.
 *
 * Conventions are those of canon.h: device pointers on the current HIP
 * device, work enqueued on `stream`, argument errors returned before anything
 * is enqueued, `ws` a caller-owned 256-byte aligned workspace whose contents
 * on entry are ignored (calls that may run concurrently must not share one),
 * nothing kept between calls.  No call waits on another workgroup, allocates,
 * or synchronises, so every call may be captured into a graph.  In addition:
 *   - Limits, beyond which calls return CANON_EUNSUPPORTED: seqs, rows and
 *     tokens below 2^30, a table's rows below 2^31, channels and columns below
 *     2^24, and what keeps a launch below 2^32 threads:
 *       embedding        tokens times the 16-byte accesses of a row (elements,
 *                        of rows shorter than one) at most 2^34 - 2^10
 *       causal_conv      seqs ceil(rows / 8), or, packed, seqs + rows / 8, times
 *                        channels at most 2^40; times channels / 4 (backward
 *                        / 2; / 1 where channels are no multiple of 4 or rows
 *                        not aligned to 4 elements) at most 2^32 - 2^24
 *       selective_scan   with S the states rounded up to 4, 8 or 16: row pitches
 *                        below 2^24 elements; the convolution's 2^40;
 *                        chunks (seqs ceil(rows / CANON_SCAN_CHUNK), packed
 *                        seqs + rows / CANON_SCAN_CHUNK, single rows seqs) times
 *                        groups ceil(channels / groups / 64) below 2^24; seqs
 *                        ceil(channels S / 64) below 2^26; backward also groups
 *                        S times the rows of all sequences at most 2^30 and
 *                        channels (S + 2) at most 2^26
 *     (sequences without rows count as one run or chunk).
 *   - Activations (dtype) are float32, bfloat16 or float16 and are passed as
 *     canon_rows_t: element (sequence s, row t, column d) is at
 *     p + s * seq + t * row + d elements.  Columns are contiguous, strides are
 *     at least 0 for inputs; the rows of an output must not overlap.  Any
 *     element alignment is accepted; 16-byte aligned rows are fastest.
 *   - Sequences.  starts == NULL: `seqs` sequences of `rows` rows each.
 *     Otherwise the sequences are packed in `rows` rows (canon_rows_t.seq is
 *     ignored): sequence s is rows starts[s] <= t < starts[s+1], with
 *     seqs + 1 ascending device values; rows outside [starts[0],
 *     starts[seqs]) are neither read nor written.  Values outside [0, rows]
 *     are taken as the nearest of the two.
 *   - Parameters, their gradients and scan states are float32 and contiguous
 *     unless said otherwise; the convolution's states have the type dtype.
 *   - Outputs do not overlap inputs unless said otherwise.
 */
#ifndef CANON_SEQ_H
#define CANON_SEQ_H

#include "canon.h"

#ifdef __cplusplus
extern "C" {
#endif

#define CANON_SEQ_VERSION 1
int canon_seq_version(void);

typedef enum { CANON_F32 = 0, CANON_BF16 = 1, CANON_F16 = 2 } canon_dtype_t;

typedef struct {
    void* p;      /* NULL: absent */
    int64_t seq;  /* elements from one sequence to the next */
    int64_t row;  /* elements from one row to the next */
} canon_rows_t;

/* ------------------------------------------------------------- embedding */
/* weight   device, `rows` rows of `width` elements, row pitch ld_weight
 * ids      device, `tokens` ids (64-bit if id_bytes is 8, 32-bit if 4)
 * out      device, tokens rows of width elements, row pitch ld_out
 * weight and out have the type dtype. */
canon_status_t canon_embedding(int dtype, const void* weight, size_t ld_weight, size_t rows,
                               size_t width, const void* ids, int id_bytes, size_t tokens,
                               float scale, void* out, size_t ld_out, void* stream);

/* dout     device, tokens rows of width elements of dtype, row pitch ld_dout
 * dw       device, rows x width, type dw_dtype (dtype or CANON_F32), pitch
 *          ld_dw
 * padding_id  an id whose row takes no gradient; -1: none
 * accumulate  0: every row of dw is written; 1: added to dw as above
 * Limits: tokens < 2^30, rows <= 2^31 - 512 (CANON_EUNSUPPORTED). */
size_t canon_embedding_grad_workspace_bytes(size_t tokens, size_t rows, size_t width);
canon_status_t canon_embedding_grad(int dtype, const void* dout, size_t ld_dout, const void* ids,
                                    int id_bytes, size_t tokens, size_t rows, size_t width,
                                    float scale, int64_t padding_id, int accumulate, int dw_dtype,
                                    void* dw, size_t ld_dw, void* ws, size_t ws_bytes,
                                    void* stream);

/* ----------------------------------------------------------- causal conv */
#define CANON_MAX_TAPS 8

typedef struct {
    int64_t dtype;    /* canon_dtype_t of x, out, states and their gradients */
    int64_t taps;     /* 1 .. CANON_MAX_TAPS */
    int64_t silu;     /* 0: out = p; 1: out = p sigmoid(p) */
    int64_t param_dtype; /* of weight and bias: dtype or CANON_F32 */
    int64_t seqs, rows, channels;
    const int32_t* starts;
    canon_rows_t x, out;
    const void* weight; /* channels x taps */
    const void* bias;   /* channels, or NULL */
    const void* init_state; /* seqs x (taps-1) x channels, oldest row first, or NULL (zero) */
    void* final_state;  /* the same shape: the last taps-1 rows seen, or NULL */
    /* backward */
    canon_rows_t dout, dx;
    float* dweight;     /* channels x taps */
    float* dbias;       /* channels, or NULL */
    const void* d_final_state; /* gradient of final_state, or NULL (zero) */
    void* d_init_state; /* or NULL */
} canon_conv_t;

/* Reads x, weight, bias, init_state; writes out, final_state (which may be
 * init_state's buffer).  out == x is refused. */
canon_status_t canon_causal_conv(const canon_conv_t* c, void* stream);

/* Reads x, weight, bias, init_state, dout, d_final_state; writes dx, dweight,
 * dbias, d_init_state.  dweight and dbias are summed over each chunk of
 * CANON_CONV_CHUNK rows of a sequence, rows ascending, then over the chunks:
 * number i to lane i mod 16, each lane in order, the lanes by the pairwise tree.
 * Chunk c of sequence s has the number s ceil(rows / CANON_CONV_CHUNK) + c, or,
 * packed, s + floor(starts[s] / CANON_CONV_CHUNK) + c: there the bits of these
 * two sums depend on where the sequences lie. */
#define CANON_CONV_CHUNK 32
size_t canon_causal_conv_grad_workspace_bytes(size_t seqs, size_t rows, int packed,
                                              size_t channels, size_t taps);
canon_status_t canon_causal_conv_grad(const canon_conv_t* c, void* ws, size_t ws_bytes,
                                      void* stream);

/* One row of each of `seqs` sequences (rows is ignored): x and out have one
 * row per sequence (canon_rows_t.seq apart).  Reads init_state, writes
 * final_state, which may be the same buffer (updated in place). */
canon_status_t canon_causal_conv_step(const canon_conv_t* c, void* stream);

/* -------------------------------------------------- selective state space */
#define CANON_SCAN_CHUNK 64
/* Largest number of states per channel. */
#define CANON_MAX_STATES 16

typedef struct {
    int64_t dtype;    /* canon_dtype_t of the canon_rows_t below */
    int64_t softplus; /* 1: dl = softplus(delta + delta_bias) */
    int64_t seqs, rows, channels, groups, states;
    const int32_t* starts;
    canon_rows_t u, delta, z, out; /* channels columns; z.p may be NULL */
    canon_rows_t B, C;             /* groups x states columns */
    const float* A;          /* channels x states */
    const float* D;          /* channels, or NULL (zero) */
    const float* delta_bias; /* channels, or NULL (zero) */
    const float* init_state; /* seqs x channels x states, or NULL (zero) */
    float* final_state;      /* the same shape, or NULL */
    float* chunk_states;     /* canon_selective_scan_states(...) elements that
                                the forward pass writes for the backward pass,
                                16-byte aligned, or NULL */
    /* backward */
    canon_rows_t dout, du, ddelta, dz, dB, dC;
    float *dA, *dD, *ddelta_bias; /* dD, ddelta_bias may be NULL */
    const float* d_final_state;   /* or NULL (zero) */
    float* d_init_state;          /* or NULL */
} canon_selective_scan_t;

/* Reads u, delta, z, B, C, A, D, delta_bias, init_state; writes out,
 * final_state (which may be init_state's buffer), chunk_states. */
size_t canon_selective_scan_states(size_t seqs, size_t rows, int packed, size_t channels,
                                   size_t states);
size_t canon_selective_scan_workspace_bytes(size_t seqs, size_t rows, int packed, size_t channels,
                                            size_t states);
canon_status_t canon_selective_scan(const canon_selective_scan_t* c, void* ws, size_t ws_bytes,
                                    void* stream);

/* Reads the forward pass's inputs (without init_state), its chunk_states,
 * dout and d_final_state; writes du, ddelta, dz (with z), dB, dC, dA, dD,
 * ddelta_bias, d_init_state.  Every sum over rows or channels, and the fold of
 * the gradient backwards (over whole sequences, or in chunks as above), is one
 * fixed expression of the shapes and the sequences' places.  dA, dD and
 * ddelta_bias are summed over each chunk of CANON_SCAN_CHUNK rows, then over the
 * chunks as the convolution's, numbered likewise.  channels is at least 1
 * (CANON_EINVAL). */
size_t canon_selective_scan_grad_workspace_bytes(size_t seqs, size_t rows, int packed,
                                                 size_t channels, size_t groups, size_t states);
canon_status_t canon_selective_scan_grad(const canon_selective_scan_t* c, void* ws,
                                         size_t ws_bytes, void* stream);

/* One row of each of `seqs` sequences (rows is ignored; canon_rows_t.seq
 * apart): h from init_state (NULL: zero), written to final_state, which may
 * be the same buffer (updated in place). */
canon_status_t canon_selective_scan_step(const canon_selective_scan_t* c, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CANON_SEQ_H */
