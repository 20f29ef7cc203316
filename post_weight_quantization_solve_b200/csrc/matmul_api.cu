// C ABI entry points of the packed-weight products: argument checks, sizing, dispatch.
#include <nvtx3/nvToolsExt.h>

#include "matmul.cuh"

namespace gptq {
gptq_status matmul_tc(const MatmulArg &m, int dir, int dtype, int bits, cudaStream_t st);
gptq_status matmul_token(const MatmulArg &m, int dtype, int bits, cudaStream_t st);
gptq_status matmul_dw(float *G, const void *dY, int64_t lddy, const void *X, int64_t ldx, int dtype,
                      int64_t M, int N, int K, int E, const int32_t *offsets, int accumulate,
                      int32_t *status, cudaStream_t st);
size_t lora_workspace(bool backward, int64_t M, int N, int K, int R, int L, int rank);
gptq_status matmul_lora(MatmulArg m, const void *A, const void *B, const float *alpha, int dtype, int bits,
                        void *ws, cudaStream_t st);
gptq_status matmul_lora_backward(MatmulArg m, float *dA, float *dB, const void *X, int64_t ldx, const void *A,
                                 const void *B, const float *alpha, int dtype, int bits, void *ws,
                                 cudaStream_t st);

// Whether a forward product has so few rows that reading the words is all that counts: the token
// kernel reads them once for every 8 rows of a range, the tiled one once for 128 or more, at a
// higher cost a word. One range of 14,336 x 4,096 (4 bits, groups of 128): 8 rows 26 against 29 us,
// 16 rows 42 against 29. Experts, by mean rows a range (64 of 1,024 x 2,048): 1 row 22 against
// 31 us, 2 rows 31 against 43, 4 rows 43 against 43, 8 rows 67 against 55.
bool matmul_few_rows(int64_t M, int E) { return E == 1 ? M <= 8 : M <= 4 * (int64_t)E; }
}  // namespace gptq

using namespace gptq;

namespace {
constexpr int64_t MAX_ROWS = int64_t(1) << 30;

struct Range {
    explicit Range(const char *name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

bool rows_ok(const void *p, int64_t ld, int cols) { return p && aligned(p, 2) && ld >= cols; }

bool packed_ok(const gptq_packed *W) {
    if (!W || !W->words || !W->scales || !aligned(W->words, 4) || !aligned(W->scales, 4)) return false;
    if (W->experts < 1 || W->experts > MATMUL_MAX_EXPERTS) return false;
    if (W->N < 1 || W->N > GPTQ_MAX_DIM || W->K < 1 || W->K > GPTQ_MAX_DIM) return false;
    if (W->bits != 2 && W->bits != 3 && W->bits != 4 && W->bits != 8) return false;
    if (W->groupsize != 0 && W->groupsize != 32 && W->groupsize != 64 && W->groupsize != 128) return false;
    if (W->g_idx && (W->groupsize == 0 || !aligned(W->g_idx, 4))) return false;
    return W->ld_words >= ((int64_t)W->K * W->bits + 31) / 32;
}

bool dtype_ok(int d) { return d == GPTQ_BF16 || d == GPTQ_F16; }

PackedArg packed_arg(const gptq_packed *W) {
    PackedArg a{};
    a.words = W->words;
    a.ldw = W->ld_words;
    a.scales = W->scales;
    a.g_idx = W->g_idx;
    a.E = W->experts;
    a.N = W->N;
    a.K = W->K;
    a.groups = W->groupsize ? (W->K + W->groupsize - 1) / W->groupsize : 0;
    a.gshift = W->groupsize == 32 ? 5 : W->groupsize == 64 ? 6 : 7;
    return a;
}

gptq_status grouped(int dir, void *Y, int64_t ldy, const void *X, int64_t ldx, int dtype, int64_t M,
                    const gptq_packed *W, const int32_t *offsets, int32_t *status, void *stream) {
    if (!packed_ok(W) || !dtype_ok(dtype) || M < 0 || M > MAX_ROWS) return GPTQ_ERR_ARG;
    if (!offsets && W->experts != 1) return GPTQ_ERR_ARG;
    if (!aligned(offsets, 4) || !aligned(status, 4)) return GPTQ_ERR_ARG;
    if (M == 0) return GPTQ_OK;
    if (!rows_ok(Y, ldy, dir == 0 ? W->N : W->K) || !rows_ok(X, ldx, dir == 0 ? W->K : W->N))
        return GPTQ_ERR_ARG;
    MatmulArg m{};
    m.w = packed_arg(W);
    m.X = X; m.ldx = ldx;
    m.Y = Y; m.ldy = ldy;
    m.offsets = offsets;
    m.M = M;
    m.status = status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dir == 0 && matmul_few_rows(M, W->experts)) return matmul_token(m, dtype, W->bits, st);
    return matmul_tc(m, dir, dtype, W->bits, st);
}

bool lora_sizes_ok(int64_t M, int N, int K, int R, int L, int rank) {
    return M >= 0 && M <= MAX_ROWS && N >= 1 && N <= GPTQ_MAX_DIM && K >= 1 && K <= GPTQ_MAX_DIM && R >= 1 &&
           R <= 65535 && L >= 1 && L <= 65535 && rank >= 8 && rank <= 128 && rank % 8 == 0;
}

bool lora_ok(const gptq_packed *W, int dtype, int64_t M, const void *A, const void *B, const float *alpha,
             int L, int rank, const int32_t *offsets, const int32_t *ids, int R, const int32_t *status) {
    if (!packed_ok(W) || W->experts != 1 || !dtype_ok(dtype)) return false;
    if (!lora_sizes_ok(M, W->N, W->K, R, L, rank)) return false;
    if (!A || !B || !alpha || !offsets || !ids) return false;
    return aligned(A, 16) && aligned(B, 16) && aligned(alpha, 4) && aligned(offsets, 4) && aligned(ids, 4) &&
           aligned(status, 4);
}
}  // namespace

extern "C" {

gptq_status gptq_matmul_grouped(void *Y, int64_t ldy, const void *X, int64_t ldx, int dtype, int64_t M,
                                const gptq_packed *W, const int32_t *offsets, int32_t *status, void *stream) {
    Range range("gptq_matmul_grouped");
    return grouped(0, Y, ldy, X, ldx, dtype, M, W, offsets, status, stream);
}

gptq_status gptq_matmul_grouped_dx(void *dX, int64_t lddx, const void *dY, int64_t lddy, int dtype, int64_t M,
                                   const gptq_packed *W, const int32_t *offsets, int32_t *status,
                                   void *stream) {
    Range range("gptq_matmul_grouped_dx");
    return grouped(1, dX, lddx, dY, lddy, dtype, M, W, offsets, status, stream);
}

gptq_status gptq_matmul_grouped_dw(float *dW, const void *dY, int64_t lddy, const void *X, int64_t ldx,
                                   int dtype, int64_t M, int N, int K, int experts, const int32_t *offsets,
                                   int accumulate, int32_t *status, void *stream) {
    Range range("gptq_matmul_grouped_dw");
    if (!dW || !aligned(dW, 4) || !dtype_ok(dtype) || M < 0 || M > MAX_ROWS) return GPTQ_ERR_ARG;
    if (N < 1 || N > GPTQ_MAX_DIM || K < 1 || K > GPTQ_MAX_DIM) return GPTQ_ERR_ARG;
    if (experts < 1 || experts > MATMUL_MAX_EXPERTS || (!offsets && experts != 1)) return GPTQ_ERR_ARG;
    if ((accumulate != 0 && accumulate != 1) || !aligned(offsets, 4) || !aligned(status, 4)) return GPTQ_ERR_ARG;
    if (M > 0 && (!rows_ok(dY, lddy, N) || !rows_ok(X, ldx, K))) return GPTQ_ERR_ARG;
    return matmul_dw(dW, dY, lddy, X, ldx, dtype, M, N, K, experts, offsets, accumulate, status,
                     static_cast<cudaStream_t>(stream));
}

gptq_status gptq_matmul_lora(void *Y, int64_t ldy, const void *X, int64_t ldx, int dtype, int64_t M,
                             const gptq_packed *W, const void *A, const void *B, const float *alpha,
                             int adapters, int rank, const int32_t *offsets, const int32_t *ids, int requests,
                             void *ws, size_t ws_bytes, int32_t *status, void *stream) {
    Range range("gptq_matmul_lora");
    if (!lora_ok(W, dtype, M, A, B, alpha, adapters, rank, offsets, ids, requests, status)) return GPTQ_ERR_ARG;
    if (M == 0) return GPTQ_OK;
    if (!rows_ok(Y, ldy, W->N) || !rows_ok(X, ldx, W->K)) return GPTQ_ERR_ARG;
    if (!ws || !aligned(ws, 256) || ws_bytes < lora_workspace(false, M, W->N, W->K, requests, adapters, rank))
        return GPTQ_ERR_WORKSPACE;
    MatmulArg m{};
    m.w = packed_arg(W);
    m.X = X; m.ldx = ldx;
    m.Y = Y; m.ldy = ldy;
    m.offsets = offsets;
    m.M = M;
    m.lora.ids = ids;
    m.lora.R = requests;
    m.lora.L = adapters;
    m.lora.rank = rank;
    m.status = status;
    return matmul_lora(m, A, B, alpha, dtype, W->bits, ws, static_cast<cudaStream_t>(stream));
}

gptq_status gptq_matmul_lora_backward(void *dX, int64_t lddx, float *dA, float *dB, const void *dY, int64_t lddy,
                                      const void *X, int64_t ldx, int dtype, int64_t M, const gptq_packed *W,
                                      const void *A, const void *B, const float *alpha, int adapters, int rank,
                                      const int32_t *offsets, const int32_t *ids, int requests, void *ws,
                                      size_t ws_bytes, int32_t *status, void *stream) {
    Range range("gptq_matmul_lora_backward");
    if (!lora_ok(W, dtype, M, A, B, alpha, adapters, rank, offsets, ids, requests, status)) return GPTQ_ERR_ARG;
    if (!aligned(dA, 4) || !aligned(dB, 4)) return GPTQ_ERR_ARG;
    if (M > 0) {
        if (!rows_ok(dY, lddy, W->N) || (dX && !rows_ok(dX, lddx, W->K))) return GPTQ_ERR_ARG;
        if ((dA || dB) && !rows_ok(X, ldx, W->K)) return GPTQ_ERR_ARG;
    }
    if (!dX && !dA && !dB) return GPTQ_OK;
    if (!ws || !aligned(ws, 256) || ws_bytes < lora_workspace(true, M, W->N, W->K, requests, adapters, rank))
        return GPTQ_ERR_WORKSPACE;
    MatmulArg m{};
    m.w = packed_arg(W);
    m.X = dY; m.ldx = lddy;
    m.Y = dX; m.ldy = lddx;
    m.offsets = offsets;
    m.M = M;
    m.lora.ids = ids;
    m.lora.R = requests;
    m.lora.L = adapters;
    m.lora.rank = rank;
    m.status = status;
    return matmul_lora_backward(m, dA, dB, X, ldx, A, B, alpha, dtype, W->bits, ws,
                                static_cast<cudaStream_t>(stream));
}

size_t gptq_lora_workspace_size(int backward, int64_t M, int N, int K, int requests, int adapters, int rank) {
    if ((backward != 0 && backward != 1) || !lora_sizes_ok(M, N, K, requests, adapters, rank)) return 0;
    return lora_workspace(backward != 0, M, N, K, requests, adapters, rank);
}

}  // extern "C"
