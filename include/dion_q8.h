/*
 * dion_q8.h -- the 8-bit linear layer around the orthonormalized step: the
 * operators that read and write a layer's activations, weights and gradients
 * in 8-bit floating point with one power-of-two scale for each block of 128
 * values along the contraction.
 *
 * A linear layer Y = X W^T whose weight W (n x k) the step trains runs as
 *
 *   dion_rms_norm_q8        X8      <- quantized rows of norm(residual stream)
 *   dion_q8_matmul          Y       <- X8 W8^T
 *   dion_q8_quantize        dY8, dY8^T  from dY (rows for dX, columns for dW)
 *   dion_q8_matmul          dX      <- dY8 (W8^T)^T,   dW <- dY8^T (X8^T)^T
 *   dion_rms_norm_backward  the norm's gradient from dX
 *   dion_step_batched       X <- the step on dW (bf16 or float32)
 *   dion_q8_quantize        W8, W8^T from the new weights (square blocks)
 *
 * Quantized matrix: rows x cols bytes of one 8-bit format (row pitch a multiple
 * of 16 bytes, base 16-byte aligned) and the scales of its 1 x 128 blocks,
 * rows x ceil(cols / 128) bytes (row pitch a multiple of 4 bytes, base 4-byte
 * aligned, every row readable up to the next multiple of 4 bytes), or of its
 * 128 x 128 blocks, ceil(rows / 128) x ceil(cols / 128).
 * Scale byte e stands for 2^(e - 127) (byte 255 for NaN).  A block with
 * largest finite magnitude a has the smallest 2^e (e >= -127) with
 * a <= 448 * 2^e for E4M3 and a <= 57344 * 2^e for E5M2, and 2^0 if a = 0; a
 * value is divided by it (exactly) and rounded once, to nearest even.
 * Infinities and NaN become the format's NaN and leave the block's other
 * values as they are.
 *
 * The conventions of dion.h hold (caller-owned device memory, no allocation,
 * no synchronization, host-side argument checks before any launch) except
 * that matrices have row pitches, in elements, and may have any alignment that
 * their type has unless stated otherwise.  Pitches may exceed the row length;
 * rows must not overlap.
 */
#ifndef DION_Q8_H
#define DION_Q8_H

#include "dion.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DION_E4M3 = 0,              /* largest value 448, no infinity */
    DION_E5M2 = 1               /* largest value 57344 */
} dion_q8_format;

/*
 * Quantizes `batch` matrices x [batch, rows, cols] (type dt, row pitch ldx,
 * matrix pitch sx).  Either or both of
 *   q, s    the matrix, blocks along its rows (q pitches ldq, sq; s pitches
 *           lds, ss)
 *   qt, st  its transpose cols x rows, blocks along the rows of the
 *           transpose, that is down the columns of x
 * are written from one read of x; the pair that is not wanted is NULL.
 * square = 0: 1 x 128 blocks; 1: 128 x 128 blocks, and then qt is exactly the
 * transpose of q, with the transposed scales.
 * rstd, weight (both or neither; batch must be 1): x[i][j] stands for
 * x[i][j] * rstd[i] * weight[j], each product rounded to float32: the output
 * of dion_rms_norm_q8 recomputed from its h and rstd, for the transposed copy
 * that a weight gradient reads.  weight has type wdt.
 * Zero rows or columns write nothing.
 */
dion_status dion_q8_quantize(int batch, int rows, int cols, dion_dtype dt, const void* x, long long ldx, long long sx,
                             const float* rstd, const void* weight, dion_dtype wdt, int square, dion_q8_format fmt,
                             void* q, long long ldq, long long sq, void* s, long long lds, long long ss, void* qt,
                             long long ldqt, long long sqt, void* st, long long ldst, long long sst,
                             void* cuda_stream);

/*
 * C (m x n, type cdt, pitch ldc) = A B^T, A (m x k) and B (n x k) quantized
 * matrices of formats afmt and bfmt with scales sa, sb; a_square, b_square: the
 * scales are those of 128 x 128 blocks (else of 1 x 128 blocks).  Products of
 * 8-bit values are accumulated in float32 on the tensor cores, which apply the
 * scales, and rounded once to cdt.  k = 0 writes zeros; m = 0 or n = 0 nothing.
 * status (nullable): a device int, OR-ed with 4 if the kernel gave up waiting
 * on one of its own barriers (C is then undefined; see dion_get_status).  The
 * library never clears it.
 */
dion_status dion_q8_matmul(int m, int n, int k, const void* a, long long lda, dion_q8_format afmt, const void* sa,
                           long long ldsa, int a_square, const void* b, long long ldb, dion_q8_format bfmt,
                           const void* sb, long long ldsb, int b_square, void* c, long long ldc, dion_dtype cdt,
                           int* status, void* cuda_stream);

/*
 * Root-mean-square norm of each row, with the residual's addition before it
 * and the quantization of its result after it:
 *   h = x + residual (rounded to dt)      y = h * rstd * weight
 *   rstd = 1 / sqrt(mean(h^2) + eps)      q, s = quantized rows of y
 * x, residual, h [rows, cols] of type dt; residual and h are NULL together
 * (h = x then), or h may be x or residual itself.  weight [cols] of type wdt.
 * Sums and products are in float32.  rstd [rows] float32 is written for the
 * backward pass (nullable).  Zero rows or columns write nothing.
 */
dion_status dion_rms_norm_q8(int rows, int cols, dion_dtype dt, const void* x, long long ldx, const void* residual,
                             long long ldr, const void* weight, dion_dtype wdt, float eps, void* h, long long ldh,
                             dion_q8_format fmt, void* q, long long ldq, void* s, long long lds, float* rstd,
                             void* cuda_stream);

/* Workspace bytes of dion_rms_norm_backward (rows, cols >= 0). */
dion_status dion_rms_norm_backward_workspace_size(int rows, int cols, size_t* bytes);

/*
 * Gradient of the norm with respect to h and weight, for dy = dL/dy:
 *   xhat = h * rstd, g = dy * weight
 *   dx = rstd * (g - xhat * mean(g * xhat)) + dh       dw = sum of dy * xhat
 * dh (nullable) is the gradient that reaches h past the norm, added in the
 * same pass; dx is then the gradient of both x and residual.  dy, h, dh, dx
 * [rows, cols] of type dt; dx may be dy or dh itself.  dw [cols] float32, its
 * sum over the rows taken in a fixed order (the same bits every time).
 * Up to 2048 rows, 8192 columns and 2^21 elements, with dx apart from dy and
 * from h, no workspace is used, and it may be NULL.  Apart: the address ranges
 * do not meet, or the pitches are the same and no element is shared.
 */
dion_status dion_rms_norm_backward(int rows, int cols, dion_dtype dt, const void* dy, long long lddy, const void* h,
                                   long long ldh, const float* rstd, const void* weight, dion_dtype wdt,
                                   const void* dh, long long lddh, void* dx, long long lddx, float* dw,
                                   void* workspace, size_t workspace_bytes, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* DION_Q8_H */
