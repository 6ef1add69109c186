/*
 * canon_layer.h — operators of a recurrent language model's layers on AMD MI355X
 * (gfx950), beside those of canon_seq.h: layer norm with the residual sum, the
 * gated linear recurrence, and sampling of the next token.  Part of libcanon.
 *
 * What is computed:
 *
 *   layer_norm       s = x, or x + residual rounded to the type dtype;
 *                    m = mean(s), v = mean((s - m)^2), r = 1 / sqrt(v + eps),
 *                    out = (s - m) r weight + bias, over the columns of each row.
 *                    Of any size of the deviations whose r is a float; the
 *                    row's sum has to be one too.
 *   layer_norm_grad  with n = (s - m) r and g = dout weight:
 *                    dx = r (g - mean(g) - n mean(g n)) + dsum (the gradient that
 *                    reaches s itself; of both x and residual),
 *                    dweight = sum dout n, dbias = sum dout, over the rows.
 *   gated_recurrence r = sigmoid(gate), i = sigmoid(input_gate) or 1,
 *                    a = exp(-decay r), c = sqrt(1 - a^2), or, without decay,
 *                    a = r, c = 1 - r;
 *                    h[t,d] = a h[t-1,d] + c i x[t,d], out = h.
 *                    Gradients are the formula's; where c is 0 (an a of 1), the
 *                    slope of the square root counts as 0.  a is 1 + e with e in
 *                    32 bits: one near 0 is off by some 2^-24, and an a of 0 (a
 *                    gate of minus infinity without decay) leaves nothing of any
 *                    finite h[t-1].
 *   sample           w[j] = exp((logits[j] - max) / temperature), held as a multiple
 *                    of 2^-S, S = 62 - ceil(log2 vocab), 50 at most; tokens ranked by
 *                    logits, the lowest index first among equals; kept are
 *                      the top_k first ones (0: all),
 *                      of those the fewest first ones whose weights add up to top_p
 *                      of the sum (one at least; 1 or more: all),
 *                      of those the ones whose weight is at least min_p;
 *                    the token is the first one in index order at which the sum of
 *                    the kept weights up to it exceeds u times their whole sum.
 *                    (top_p and u times a sum: in 64-bit floats.)
 *
 * Everything is computed in 32 bits and rounded once where it is stored, but for
 * the recurrence's carried state and the sampling's weights, in 64.  Each sum is
 * one fixed expression of the shapes, and sums of sampling weights are sums of
 * integers, so each call is reproducible bit for bit.  In particular:
 *   - a row's norm depends on its width, type and values alone, not on the rows
 *     around it, strides or alignment;
 *   - the recurrence is evaluated in chunks of CANON_RECUR_CHUNK rows from the
 *     sequence's first row: inside a chunk h folds from the chunk's start state, and
 *     the next chunk starts from P H + S, P the product of the a and S the chunk's
 *     fold from zero; the same way over blocks of CANON_RECUR_BLOCK rows.  So a
 *     sequence's outputs do not depend on the other sequences, on packing or on how
 *     the work is spread, and cutting a sequence at a multiple of CANON_RECUR_BLOCK
 *     rows and passing the state on changes no bit;
 *   - sums over rows (dweight, dbias, ddecay) go by chunks of rows and then over the
 *     chunks as the convolution's of canon_seq.h; ddecay's depend on the number of
 *     sequences, rows and channels.
 *
 * Conventions are those of canon_seq.h: canon_rows_t, dtype, sequences and starts,
 * workspaces, streams, capture and errors; columns are contiguous, any element
 * alignment is accepted.
 */
#ifndef CANON_LAYER_H
#define CANON_LAYER_H

#include "canon_seq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define CANON_LAYER_VERSION 1
int canon_layer_version(void);

/* ------------------------------------------------------------- layer norm */
typedef struct {
    int64_t dtype;       /* canon_dtype_t of the canon_rows_t below */
    int64_t param_dtype; /* of weight and bias: dtype or CANON_F32 */
    int64_t seqs, rows, width;
    double eps; /* at least 0, at most the largest float */
    canon_rows_t x, residual; /* residual.p may be NULL (none) */
    canon_rows_t sum;         /* s, with residual only; .p may be NULL (not wanted) */
    canon_rows_t out;
    const void* weight;       /* width */
    const void* bias;         /* width, or NULL (zero) */
    float* stats;             /* seqs x rows x 2: m and r, or NULL (not wanted) */
    /* backward */
    canon_rows_t dout, dsum, dx; /* dsum.p may be NULL (zero) */
    float *dweight, *dbias;      /* width; dbias may be NULL */
} canon_norm_t;

/* seqs x rows rows (there is no `starts`: rows are independent).  Reads x, residual,
 * weight, bias; writes sum, out, stats.  out and sum may each be x's or residual's
 * buffer with the same strides (in place), not each other's.
 * Limits (CANON_EUNSUPPORTED): seqs, rows and seqs x rows < 2^30, width < 2^24,
 * backward also max(512, seqs rows / 64) times ceil(width / 1024) below 2^24. */
canon_status_t canon_layer_norm(const canon_norm_t* c, void* stream);

/* Reads x (the s of the forward pass), weight, stats, dout, dsum; writes dx,
 * dweight, dbias.  residual, sum, out, bias and eps are not read.  dx may be the buffer
 * of dout or dsum with the same strides, not x's. */
size_t canon_layer_norm_grad_workspace_bytes(size_t seqs, size_t rows, size_t width);
canon_status_t canon_layer_norm_grad(const canon_norm_t* c, void* ws, size_t ws_bytes,
                                     void* stream);

/* ------------------------------------------------- gated linear recurrence */
#define CANON_RECUR_CHUNK 8
#define CANON_RECUR_BLOCK 512

typedef struct {
    int64_t dtype; /* canon_dtype_t of the canon_rows_t below */
    int64_t seqs, rows, channels;
    const int32_t* starts;
    canon_rows_t x, gate, input_gate, out; /* input_gate.p may be NULL (i = 1) */
    const float* decay;      /* channels, finite, not negative, or NULL (a = sigmoid(gate)) */
    const float* init_state; /* seqs x channels, or NULL (zero) */
    float* final_state;      /* the same shape, or NULL */
    float* kept_states;      /* canon_gated_recurrence_states(...) elements that the
                                forward pass writes for the backward pass, or NULL */
    /* backward */
    canon_rows_t dout, dx, dgate, dinput_gate; /* dinput_gate with input_gate */
    float* ddecay;               /* channels, with decay */
    const float* d_final_state;  /* or NULL (zero) */
    float* d_init_state;         /* or NULL */
} canon_recur_t;

/* Reads x, gate, input_gate, decay, init_state; writes out, final_state (which may be
 * init_state's buffer), kept_states.  out may be the buffer of none of the inputs.  An
 * x, gate or input_gate that is not finite can leave its channel's outputs from that
 * row on not finite (a gate of minus or plus infinity is its limit, and one that
 * makes c zero shuts out finite x only).
 * Limits (CANON_EUNSUPPORTED): those of canon_seq.h on seqs, rows and channels;
 * row pitches below 2^24 elements (but for single rows); blocks (seqs ceil(rows /
 * CANON_RECUR_BLOCK), packed seqs + rows / CANON_RECUR_BLOCK, single rows seqs) times
 * ceil(channels / 64) below 2^22. */
size_t canon_gated_recurrence_states(size_t seqs, size_t rows, int packed, size_t channels);
size_t canon_gated_recurrence_workspace_bytes(size_t seqs, size_t rows, int packed,
                                              size_t channels);
canon_status_t canon_gated_recurrence(const canon_recur_t* c, void* ws, size_t ws_bytes,
                                      void* stream);

/* Reads the forward pass's inputs (without init_state), its kept_states, dout and
 * d_final_state; writes dx, dgate, dinput_gate, ddecay, d_init_state.  No output may be
 * an input's buffer. */
size_t canon_gated_recurrence_grad_workspace_bytes(size_t seqs, size_t rows, int packed,
                                                   size_t channels);
canon_status_t canon_gated_recurrence_grad(const canon_recur_t* c, void* ws, size_t ws_bytes,
                                           void* stream);

/* One row of each of `seqs` sequences (rows is ignored; canon_rows_t.seq apart): h from
 * init_state (NULL: zero), written to final_state, which may be the same buffer.  out may
 * be the buffer of x, gate or input_gate with the same strides. */
canon_status_t canon_gated_recurrence_step(const canon_recur_t* c, void* stream);

/* --------------------------------------------------------------- sampling */
typedef struct {
    int64_t dtype; /* canon_dtype_t of logits */
    int64_t rows, vocab;
    const void* logits; /* rows of vocab elements, row pitch ld >= 0 */
    int64_t ld;
    const float* u; /* rows random numbers in [0, 1); others count as the nearest */
    /* per row, or NULL: the value beside it for every row */
    const float* temperature; /* not above 0: the largest logit's token */
    const int32_t* top_k;     /* not above 0: no limit */
    const float* top_p;
    const float* min_p;
    double temperature_all, top_p_all, min_p_all;
    int64_t top_k_all;
    void* ids;        /* rows, 64-bit if id_bytes is 8, 32-bit if 4 */
    int64_t id_bytes;
} canon_sample_t;

/* Logits of minus infinity and NaN are masked: never chosen.  A row with nothing else
 * gives -1.  Where the largest logit is plus infinity, the infinite ones have weight 1
 * and the others 0.  A min_p above 1 counts as 1.
 * Limits (CANON_EUNSUPPORTED): rows < 2^22, vocab < 2^24. */
size_t canon_sample_workspace_bytes(size_t rows, size_t vocab);
canon_status_t canon_sample(const canon_sample_t* c, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CANON_LAYER_H */
