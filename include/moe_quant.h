/*
 * moe_quant.h -- products of a few rows with a 4-bit weight matrix and group
 * scales on AMD Instinct MI355X (gfx950).
 *
 *   Y[t][n] = sum_k X[t][k] * q[k][n] * scale[k / group][n]
 *
 * The codes q are in [-8, 7] and each scale is one fp16 number per `group`
 * consecutive rows of a column: the INT4 form of the compressed layer's
 * residual factors (MOE_RESID_INT4_G32 in moe.h is group = 32), for any
 * linear projection of a model that decodes a few tokens at a time.  Sums
 * run in FP32 from exact products; Y is rounded once.
 *
 * Error codes, streams and moe_last_error() as in moe.h.
 */
#ifndef CEFN_MOE_QUANT_H
#define CEFN_MOE_QUANT_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* 1 <= n_in, n_out <= 2^24 and n_in * n_out <= 2^31; group 32, 64 or 128 (the
 * last group of a column may be short); x_dtype MOE_F16 or MOE_BF16, the type
 * of X and Y. */
typedef struct {
  int32_t n_in;    /* length of a row of X */
  int32_t n_out;   /* length of a row of Y */
  int32_t group;   /* rows of the weight matrix that share a scale */
  int32_t x_dtype; /* moe_dtype */
} moe_quant_config;

/* The matrix, row-major [n_in][n_out], in one of two forms (exactly one of q
 * and values is given), read only during moe_quant_create:
 *   q       int8, codes in [-8, 7], with
 *   scale   fp16 bits [ceil(n_in / group)][n_out], finite;
 *   values  MOE_F32, MOE_F16 or MOE_BF16 (values_dtype), finite: quantised by
 *           the rule of MOE_RESID_INT4_G32 in moe.h with `group` in place of 32.
 * on_device = 0: host pointers; 1: device pointers on the current device. */
typedef struct {
  const int8_t* q;
  const uint16_t* scale;
  const void* values;
  int32_t values_dtype;
  int32_t on_device;
} moe_quant_weights;

typedef struct moe_quant moe_quant;

/* Pack the matrix into library-owned memory on the current device.  Work on
 * device sources is ordered after what `stream` holds.  Synchronous.
 * MOE_ERR_INVALID_ARG for a code outside [-8, 7]. */
int moe_quant_create(const moe_quant_config* cfg, const moe_quant_weights* weights, void* stream, moe_quant** out);

/* Y = X W for T rows, T >= 0.  X: device [T] rows ldx >= n_in elements apart;
 * Y: device [T] rows ldy >= n_out elements apart; elements between the rows
 * are neither read nor written.  X and Y may not overlap.  Any T is taken, 32
 * rows a launch: each launch reads the matrix once, so this entry is for few
 * rows.  X on 16-byte boundaries with n_in and ldx multiples of 8 is read
 * fastest; every other alignment of the type is accepted.  A row with an
 * infinity or a NaN gives NaN in its row of Y and leaves the others alone.
 * Enqueue only (no allocation, no synchronisation, no state): a handle's calls
 * may overlap on several streams, and may be captured into a HIP graph.  The
 * handle's device must be current. */
int moe_quant_matvec(const moe_quant* h, const void* X, int64_t ldx, int32_t T, void* Y, int64_t ldy,
                     void* stream);

/* The stored codes and scales, host buffers in the layout of
 * moe_quant_weights (either may be NULL).  Synchronous. */
int moe_quant_read(const moe_quant* h, int8_t* q, uint16_t* scale);

/* Bytes of the codes and scales as stored on the device, padding included. */
int64_t moe_quant_bytes(const moe_quant* h);

/* Free the handle (synchronises its device first).  NULL is a no-op. */
int moe_quant_destroy(moe_quant* h);

#ifdef __cplusplus
}
#endif
#endif /* CEFN_MOE_QUANT_H */
