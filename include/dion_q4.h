/*
 * dion_q4.h -- serving the weights that the step trains in 4 bits: their
 * quantization with one scale for each group of values along a row, and the
 * product with a few rows of activations (single tokens), whose time is that of
 * reading the weights.
 *
 *   dion_q4_quantize      W4 <- W, once
 *   dion_rms_norm_q8      x8 <- the residual stream (or any plain rows)
 *   dion_q4_matmul        y  <- x W4^T
 *   dion_q4_dequantize    W4's values, where many rows are to be multiplied
 *                         (dion_q8_quantize and dion_q8_matmul take them)
 *
 * 4-bit matrix (n x k): whole numbers q in -8..7, each held as q + 8, and a
 * bfloat16 scale for each group of 32, 64 or 128 along a row; q * scale is the
 * value.  Row r of the data is ceil(k / 128) chunks of 64 bytes (row pitch ldq a
 * multiple of 16 bytes, base 16-byte aligned), one for each 128 columns: its
 * 32-bit word 4 t + j (little endian) holds columns 32 j + 8 t +
 * (0, 2, 4, 6, 1, 3, 5, 7), from its low four bits up.  So 16 bytes are one
 * lane's operands of eight tensor-core products, without a shuffle, and each
 * product lies inside a group.  Columns past k hold zero (8).
 * Scales [n, ceil(k / group)], row pitch lds elements.
 *
 * The conventions of dion.h hold, except that matrices have row pitches, in
 * elements (bytes for 4-bit data), and may have any alignment that their type
 * has unless stated otherwise.  Rows must not overlap.
 */
#ifndef DION_Q4_H
#define DION_Q4_H

#include "dion_q8.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Quantizes x [rows, cols] (type dt, pitch ldx): scale = bfloat16(amax / 7),
 * q = x / scale rounded to nearest even, both divisions in float32; a group
 * whose scale rounds to zero holds zeros, one with an infinity or NaN gets the
 * scale NaN.  Every byte of the rows' chunks is written.
 */
dion_status dion_q4_quantize(int rows, int cols, int group, dion_dtype dt, const void* x, long long ldx, void* q,
                             long long ldq, void* s, long long lds, void* cuda_stream);

/* y [rows, cols] (type dt, pitch ldy) = q * scale, rounded once. */
dion_status dion_q4_dequantize(int rows, int cols, int group, const void* q, long long ldq, const void* s,
                               long long lds, dion_dtype dt, void* y, long long ldy, void* cuda_stream);

/* Types of dion_q4_matmul's x. */
typedef enum {
    DION_X_F32 = 0,
    DION_X_BF16 = 1,
    DION_X_E4M3 = 2,            /* quantized rows of dion_q8.h: bytes and 1 x 128 scales */
    DION_X_E5M2 = 3
} dion_x_type;

/*
 * y (m x n, type ydt, pitch ldy) = x W^T, x (m x k, pitch ldx; sx, ldsx: the
 * scales of 8-bit rows, else ignored) and W a 4-bit matrix n x k.  x is exact but
 * for values far below the largest of a row's 128 columns, which are off by 2^-39
 * of that one at most (float32: by 2^-24 of themselves too); products are exact,
 * summed in float32, a group at a time, in an order that depends on the sizes
 * alone, and rounded once.  A group's sum meets its scale before x's power of two
 * (the largest of 128 columns is raised to between 2^14 and 2^15): a scale below 2^102, of
 * weights below 3.5e31, cannot overflow there; a larger one may give an infinity
 * where x is small enough for a finite result.  Made for few rows: beyond 32 (16
 * of float32; fewer for k beyond 16384, down to 4 and 2) the weights are read
 * again for each as many.  k = 0 writes zeros, m = 0 or n = 0 nothing.  m up to
 * 65535, k up to 131072.
 */
dion_status dion_q4_matmul(int m, int n, int k, dion_x_type xt, const void* x, long long ldx, const void* sx,
                           long long ldsx, int group, const void* q, long long ldq, const void* s, long long lds,
                           dion_dtype ydt, void* y, long long ldy, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* DION_Q4_H */
