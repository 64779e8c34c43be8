/*
 * ttc_block.h - what stands between the tensor-train layers of a transformer
 * block: layer norm with the residual sum, attention over a sliding window
 * with a few first tokens that stay visible, and the orthogonalised update of
 * the cores.  Same library, same conventions as ttc.h: device pointers to
 * caller-owned memory, 16-byte aligned, row-major; workspaces from the
 * caller; everything enqueued on `stream`, no allocation, no synchronisation
 * and no memset, so every call can be captured into a HIP graph; errors come
 * back before anything is launched; every sum runs in a fixed order, so
 * results are bitwise reproducible.  Buffers of one call must not overlap
 * unless a comment allows it.
 */
#ifndef TTC_BLOCK_H
#define TTC_BLOCK_H

#include "ttc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- layer norm ---------------------------------------------------------- */

/* Rows of n elements.  x_dtype (TTC_F32 or TTC_BF16) is the type of the
 * residual stream: x, res, h, dh, dx.  y_dtype (TTC_F32, TTC_BF16 or TTC_FP8)
 * is the type of what the next layer takes: y and dy.  Statistics, gamma,
 * beta and their gradients are fp32. */
typedef struct {
  int32_t n;       /* row length, 1 .. TTC_NORM_MAX_N */
  int32_t x_dtype; /* ttc_dtype of x, res, h, dh, dx  */
  int32_t y_dtype; /* ttc_dtype of y, dy              */
  float eps;       /* added to the variance, >= 0     */
} ttc_norm_desc;

#define TTC_NORM_MAX_N (1 << 20)

/* Bytes of saved (mean and reciprocal deviation of each row, written by the
 * forward, read by the backward) and of the backward's scratch (partial sums
 * of the weight gradients).  Host-only. */
ttc_status ttc_norm_workspace(const ttc_norm_desc* desc, int64_t T,
                              size_t* saved_bytes, size_t* scratch_bytes);

/*
 * Forward: h = x + res (rounded to x_dtype), y = (h - mean) * rstd * gamma +
 * beta with mean and variance of each row of the rounded h.
 *   x, res - T x n (x_dtype); res NULL: h = x
 *   gamma, beta - n fp32
 *   h - T x n (x_dtype), overwritten; required with res, ignored (may be
 *       NULL) without
 *   y - T x n (y_dtype), overwritten; e4m3: magnitudes over 448 become 448
 *   saved - at least ttc_norm_workspace() bytes
 * A row that holds a NaN or an infinity gives a NaN row.  T = 0 does nothing.
 */
ttc_status ttc_norm_fwd(const ttc_norm_desc* desc, int64_t T, const void* x,
                        const void* res, const float* gamma, const float* beta,
                        void* h, void* y, void* saved, size_t saved_bytes,
                        ttc_stream_t stream);

/*
 * Backward.  With xhat = (h - mean) rstd and u = dy gamma:
 *   dx = (u - mean(u) - xhat mean(u xhat)) rstd + dh    (dh NULL: 0)
 *   dgamma = sum over rows of dy xhat,  dbeta = sum over rows of dy
 * dx is the gradient of x and of res alike.
 *   dy - T x n (y_dtype);  h, gamma, saved - as in the forward (h = x there
 *        when res was NULL)
 *   dh - T x n (x_dtype): the gradient that reaches h from elsewhere, or NULL
 *   dx - T x n (x_dtype), overwritten;  dgamma, dbeta - n fp32, overwritten
 * T = 0 writes zero dgamma and dbeta.
 */
ttc_status ttc_norm_bwd(const ttc_norm_desc* desc, int64_t T, const void* dy,
                        const void* h, const float* gamma, const void* dh,
                        const void* saved, size_t saved_bytes, void* dx,
                        float* dgamma, float* dbeta, void* scratch,
                        size_t scratch_bytes, ttc_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TTC_BLOCK_H */
