/*
 * gptq_matmul.h -- C ABI of libgptq.so: products of packed layers on NVIDIA B200 (sm_100a),
 * grouped by expert and with low-rank adapters, and their gradients.
 *
 * The conventions of gptq.h hold: the caller owns all device memory, every call is
 * asynchronous on `stream`, argument errors are returned before anything is enqueued, and
 * what only the device can see (row ranges, indices) is reported in the status word.
 */
#ifndef GPTQ_MATMUL_H
#define GPTQ_MATMUL_H

#include "gptq.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * gptq_packed -- a packed layer, or the packed layers of several experts, as the products
 * below read it: the words of gptq_pack_codes with the scales (and g_idx) of the
 * quantisation call, laid out as those calls write them. Expert e's weights are
 *   W^[e][n][k] = scales[e][n][group(k)] (code[e][n][k] - 2^(bits-1)).
 *
 *   words      device uint32, row (e, n) at words + (e N + n) ld_words,
 *              ld_words >= ceil(K bits / 32). Rows that start on 16-byte boundaries
 *              (words 16-byte aligned, ld_words % 4 == 0) are read fastest.
 *   scales     device fp32 [experts][N] (groupsize 0) or
 *              [experts][N][ceil(K / groupsize)]. An infinite or NaN scale makes its channel's
 *              outputs infinite or NaN (of the input gradient: its group's columns).
 *   g_idx      device int32 [experts][K], the group of each column (each in
 *              [0, ceil(K / groupsize)), else GPTQ_ERR_ARG in the status word), or NULL:
 *              column k in group k / groupsize. A layer quantised in natural order or with
 *              static groups has that g_idx too: give NULL for it. Its groups are looked up
 *              column by column, at up to twelve times the time.
 *   experts    1..512; a plain projection is one expert.
 *   N, K       1..GPTQ_MAX_DIM.  bits 2, 3, 4 or 8.  groupsize 0, 32, 64 or 128.
 */
typedef struct {
    const uint32_t *words;
    int64_t ld_words;
    const float *scales;
    const int32_t *g_idx;
    int experts, N, K, bits, groupsize;
} gptq_packed;

/*
 * gptq_matmul_grouped -- products grouped by expert over a packed layer:
 * Y[t] = W^_e X[t] for the rows offsets[e] <= t < offsets[e + 1] (the pages stop at
 * packed storage; this is the product that reads it).
 *
 *   Y        device [M][ldy], ldy >= N; X device [M][ldx], ldx >= K; both of dtype
 *            GPTQ_BF16 or GPTQ_F16, 2-byte aligned, not overlapping. Rows on 16-byte
 *            boundaries are read fastest. M 0..2^30.
 *   offsets  device int32 [experts + 1], non-decreasing inside [0, M], or NULL (one
 *            expert, all M rows). Ranges may be empty. Rows of Y outside
 *            [offsets[0], offsets[experts]) are left as they were. Offsets out of order
 *            or out of range: nothing is written, GPTQ_ERR_ARG in the status word.
 *   Arithmetic: fp32 sums. With groupsize 0 the codes enter exactly and the scale in
 *            fp32 at the end; with input groups each weight s (c - z) is rounded once to
 *            dtype, as a dequantised layer in dtype would hold it. The result is rounded
 *            once to dtype. Results do not change from call to call on the same inputs.
 *   status   device int32 or NULL (then a refused device-side argument leaves no trace
 *            but unwritten rows); GPTQ_ERR_TIMEOUT if a bounded wait ran out.
 *   Errors: GPTQ_ERR_ARG for sizes, strides, dtype, alignment or NULL pointers.
 */
GPTQ_API gptq_status gptq_matmul_grouped(void *Y, int64_t ldy, const void *X, int64_t ldx, int dtype,
                                         int64_t M, const gptq_packed *W, const int32_t *offsets,
                                         int32_t *status, void *stream);

/*
 * gptq_matmul_grouped_dx -- the gradient of gptq_matmul_grouped's rows:
 * dX[t] = W^_e^T dY[t]. Backpropagation through packed layers to the layer whose gradient
 * gptq_first_order_shift takes. dX [M][lddx], lddx >= K; dY [M][lddy], lddy >= N;
 * otherwise as gptq_matmul_grouped, but every weight s (c - z) is rounded once to dtype
 * (the scale changes along this contraction).
 */
GPTQ_API gptq_status gptq_matmul_grouped_dx(void *dX, int64_t lddx, const void *dY, int64_t lddy,
                                            int dtype, int64_t M, const gptq_packed *W,
                                            const int32_t *offsets, int32_t *status, void *stream);

/*
 * gptq_matmul_grouped_dw -- the gradients of the experts' weights:
 * dW[e] = sum over offsets[e] <= t < offsets[e + 1] of dY[t]^T X[t] (added to dW[e] when
 * accumulate != 0). fp32; the G of gptq_first_order_shift.
 *
 *   dW       device fp32 [experts][N][K]; an expert without rows gets zeros (or keeps
 *            its values when accumulating).
 *   dY, X    device [M][lddy >= N], [M][ldx >= K], dtype GPTQ_BF16 or GPTQ_F16.
 *   offsets, status, errors: as gptq_matmul_grouped.
 *   Rows are added in order, in chains of 512 on the tensor cores and in fp32 to nearest
 *   across chains; results do not change from call to call.
 */
GPTQ_API gptq_status gptq_matmul_grouped_dw(float *dW, const void *dY, int64_t lddy, const void *X,
                                            int64_t ldx, int dtype, int64_t M, int N, int K,
                                            int experts, const int32_t *offsets, int accumulate,
                                            int32_t *status, void *stream);

/*
 * gptq_matmul_lora -- low-rank adapters of many requests beside one packed projection:
 * Y[t] = W^ X[t] + alpha[a] B[a] (A[a] X[t]), a = ids[r] for the rows
 * offsets[r] <= t < offsets[r + 1] of request r; ids[r] = -1: no adapter.
 *
 *   W        one packed layer (experts == 1).
 *   A        device [adapters][rank][K]; B device [adapters][N][rank]; both of dtype,
 *            16-byte aligned, dense. rank a multiple of 8, 8..128 (pad with zeros).
 *            adapters 1..65535.
 *   alpha    device fp32 [adapters].
 *   offsets  device int32 [requests + 1] and ids device int32 [requests], requests
 *            1..65535; several requests may share an adapter. Offsets and ids are
 *            checked as a whole as in gptq_matmul_grouped (ids in [-1, adapters)); rows
 *            outside [offsets[0], offsets[requests]) are left as they were.
 *   ws       gptq_lora_workspace_size(0, M, N, K, requests, adapters, rank) bytes.
 *   Arithmetic: fp32 sums; alpha A X has the range of fp32 for either dtype and enters the
 *            output with 16 bits (fp16 up to 8 rows, and in runs of fewer than 16 rows of an
 *            adapter: 24). Up to 8 rows, W^ enters as in gptq_matmul_grouped; above, each
 *            weight is rounded once to dtype.
 *   Others as gptq_matmul_grouped. GPTQ_ERR_WORKSPACE for the workspace.
 */
GPTQ_API gptq_status gptq_matmul_lora(void *Y, int64_t ldy, const void *X, int64_t ldx, int dtype,
                                      int64_t M, const gptq_packed *W, const void *A, const void *B,
                                      const float *alpha, int adapters, int rank,
                                      const int32_t *offsets, const int32_t *ids, int requests,
                                      void *ws, size_t ws_bytes, int32_t *status, void *stream);

/*
 * gptq_matmul_lora_backward -- the gradients of gptq_matmul_lora (W^ is frozen):
 *   dX[t]  = W^^T dY[t] + A[a]^T U[t],       U[t] = alpha[a] B[a]^T dY[t]
 *   dA[a]  = sum of U[t] X[t]^T,  dB[a] = sum of dY[t] T[t]^T,  T[t] = alpha[a] A[a] X[t]
 * over the rows of every request that uses adapter a.
 *
 *   dX       device [M][lddx] of dtype, or NULL (not wanted). Rows outside the requests
 *            are left as they were.
 *   dA, dB   device fp32 [adapters][rank][K], [adapters][N][rank], or NULL; written, not
 *            added to: zeros for an adapter that no row uses.
 *   X        may be NULL when neither dA nor dB is wanted.
 *   ws       gptq_lora_workspace_size(1, M, N, K, requests, adapters, rank) bytes.
 *   Others as gptq_matmul_lora; T and U enter dA and dB with 24 bits (bf16), or with 22 and no
 *   step coarser than 2^-39 of the adapter's largest value (fp16); dA and dB are fp32 sums in a
 *   fixed order. Where dY or X is infinite, they may hold NaN in the place of infinities.
 */
GPTQ_API gptq_status gptq_matmul_lora_backward(void *dX, int64_t lddx, float *dA, float *dB,
                                               const void *dY, int64_t lddy, const void *X,
                                               int64_t ldx, int dtype, int64_t M,
                                               const gptq_packed *W, const void *A, const void *B,
                                               const float *alpha, int adapters, int rank,
                                               const int32_t *offsets, const int32_t *ids,
                                               int requests, void *ws, size_t ws_bytes,
                                               int32_t *status, void *stream);

/* gptq_lora_workspace_size -- bytes of the calls above (backward 0 or 1); 0 for sizes that
 * they refuse. The workspace needs no initialisation and keeps nothing between calls; calls
 * that overlap on the GPU each need their own. */
GPTQ_API size_t gptq_lora_workspace_size(int backward, int64_t M, int N, int K, int requests,
                                         int adapters, int rank);

#ifdef __cplusplus
}
#endif
#endif /* GPTQ_MATMUL_H */
