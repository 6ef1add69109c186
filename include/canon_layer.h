/*
 * canon_layer.h — operators of a recurrent language model's layers on AMD MI355X
 * (gfx950), beside those of canon_seq.h: layer norm with the residual sum.  Part
 * of libcanon.
 *
 * What is computed:
 *
 *   layer_norm       s = x, or x + residual rounded to the type dtype;
 *                    m = mean(s), v = mean((s - m)^2), r = 1 / sqrt(v + eps),
 *                    out = (s - m) r weight + bias, over the columns of each row.
 *   layer_norm_grad  with n = (s - m) r and g = dout weight:
 *                    dx = r (g - mean(g) - n mean(g n)) + dsum (the gradient that
 *                    reaches s itself; of both x and residual),
 *                    dweight = sum dout n, dbias = sum dout, over the rows.
 *
 * Everything is computed in 32 bits and rounded once where it is stored.  Each sum is
 * one fixed expression of the shapes, so each call is reproducible bit for bit.  In
 * particular:
 *   - a row's norm depends on its width, type and values alone, not on the rows
 *     around it, strides or alignment;
 *   - sums over rows (dweight, dbias) go by chunks of rows and then over the
 *     chunks as the convolution's of canon_seq.h.
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
    double eps;
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
 * Limits (CANON_EUNSUPPORTED): seqs, rows < 2^30, seqs x rows < 2^31, width < 2^24,
 * backward also max(512, seqs rows / 64) times ceil(width / 1024) below 2^24. */
canon_status_t canon_layer_norm(const canon_norm_t* c, void* stream);

/* Reads x (the s of the forward pass), weight, stats, dout, dsum; writes dx,
 * dweight, dbias.  residual, sum, out, bias and eps are not read.  dx may be the buffer
 * of dout or dsum with the same strides, not x's. */
size_t canon_layer_norm_grad_workspace_bytes(size_t seqs, size_t rows, size_t width);
canon_status_t canon_layer_norm_grad(const canon_norm_t* c, void* ws, size_t ws_bytes,
                                     void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CANON_LAYER_H */
