// Low-rank adapters beside a packed projection: the rank-space rows, the requests of each
// adapter, and the calls that put the pieces together.
//
//   T[t] = alpha_a A_a X[t]        (forward, and the gradient of B)
//   U[t] = alpha_a B_a^T dY[t]     (gradients of X and A)
//
// Both are a thin product rows x [rank][inner], bound by reading the rows (long prompts) or the
// adapters (requests that decode, each with an adapter of its own). The result leaves as three bf16
// parts side by side that add up to the fp32 sum, which the products that follow read as matrix
// operands. The gradients of fp16 adapters have fp16 rows as their other operand, so k_rank_scale makes
// an fp16 pair of T or U, scaled by the power of two that brings the adapter's largest value below
// 2^15: 22 bits, and no step coarser than 2^-39 of that largest value, whatever its size. Tiles of rows are cut inside each request, so a tile has one adapter.
//   k_rank_tc    prompts: the adapter is the A operand of tcgen05 (rank lanes), 64 rows the B
//                operand, both by tiled copies in steps of 128 columns.
//   k_rank_rows  a few rows, or layouts that tiled copies refuse: fragments of mma.sync m16n8k16
//                straight from global memory; a lane takes 16 bytes (8 neighbouring columns) of
//                its row and of its adapter row, which permutes the contraction index alike on
//                both sides.
// A cluster of up to 8 blocks shares the contraction of a tile when there are few tiles.
// 8,192 rows of 4,096 with rank 64: 24 us, 67 MB at 2.8 TB/s (cold); 48 rows with an adapter each of
// rank 16: 12 us, the latency of one launch and its reads. k_rank_scale: 5 us for 700 rows of rank 32.
// B_a is stored [N][rank]; the backward pass reads it transposed (k_lora_setup).
#include <algorithm>

#include "matmul.cuh"

namespace gptq {

int adapter_parts(int64_t M, int L, int width);
gptq_status adapter_gradients(const AdapterGrad *grads, int count, int rank, int dtype, int64_t M,
                              const int32_t *offsets, const int32_t *ids, const int32_t *list_off,
                              const int32_t *list, int R, int L, int32_t *status, cudaStream_t st);
gptq_status matmul_tc(const MatmulArg &m, int dir, int dtype, int bits, cudaStream_t st);
gptq_status matmul_token(const MatmulArg &m, int dtype, int bits, cudaStream_t st);
bool matmul_few_rows(int64_t M, int E);

struct RankArg {
    const void *X;            // [M][ldx]
    int64_t ldx, M;
    const void *A;            // [L][rank][inner]
    const float *alpha;       // [L]
    const int32_t *offsets, *ids;
    int R, L, rank, inner;
    __nv_bfloat16 *T3;        // [M][LORA_PARTS rank]
    uint32_t *most;           // [L] largest finite |value| of each adapter, as bits, or NULL
    int xvec, avec, split;
    int32_t *status;
};

// One launch makes T or U, or both (blockIdx.y).
struct RankArgs {
    RankArg a[2];
};
struct RankMaps {
    CUtensorMap x[2], a[2];
};

template <typename T>
__device__ __forceinline__ uint4 piece(const T *row, int c, int cols, bool vec) {
    if (row == nullptr || c >= cols) return make_uint4(0u, 0u, 0u, 0u);
    if (vec && c + 8 <= cols) return __ldg(reinterpret_cast<const uint4 *>(row + c));
    uint32_t v[4] = {0u, 0u, 0u, 0u};
    const unsigned short *s = reinterpret_cast<const unsigned short *>(row + c);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (c + e < cols) v[e >> 1] |= (uint32_t)__ldg(s + e) << (16 * (e & 1));
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// The b-th tile of `rows` rows: its first row, its rows and its adapter; none: false. Requests
// without an adapter have no tiles. Offsets and ids are checked as a whole first (refused: status,
// false). Called by every thread of the block; `found` is four ints of shared memory.
__device__ __forceinline__ bool rank_tile(const RankArg &p, int64_t b, int rows, int *found, int &t, int &n,
                                          int &id) {
    if (threadIdx.x < 4) found[threadIdx.x] = 0;
    __syncthreads();
    bool bad = offsets_bad(p.offsets, p.R, p.M, threadIdx.x, blockDim.x);
    bad |= ids_bad(p.ids, p.R, p.L, threadIdx.x, blockDim.x);
    if (bad) found[3] = 1;
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int64_t base = 0;
        for (int s0 = 0; s0 < p.R && base <= b; s0 += 32) {
            const int s = s0 + lane;
            int begin = 0, len = 0, a = -1;
            if (s < p.R) {
                begin = __ldg(p.offsets + s);
                len = __ldg(p.offsets + s + 1) - begin;
                a = __ldg(p.ids + s);
            }
            const int nt = a >= 0 && len > 0 ? (len + rows - 1) / rows : 0;
            int sum = nt;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(~0u, sum, d);
                if (lane >= d) sum += v;
            }
            const int64_t j = b - (base + sum - nt);
            if (j >= 0 && j < nt) {
                found[0] = begin + (int)j * rows;
                found[1] = min(rows, len - (int)j * rows);
                found[2] = a;
            }
            base += __shfl_sync(~0u, sum, 31);
        }
    }
    __syncthreads();
    if (found[3]) {
        if (threadIdx.x == 0) set_status(p.status, GPTQ_ERR_ARG);
        return false;
    }
    t = found[0];
    n = found[1];
    id = found[2];
    return n > 0;
}

// A rank-space value as its parts; the larger of `big` and its size, if it is finite.
__device__ __forceinline__ float store_parts(__nv_bfloat16 *d, int rank, float v, float big) {
    big = isfinite(v) ? fmaxf(big, fabsf(v)) : big;
#pragma unroll
    for (int h = 0; h < LORA_PARTS; ++h) {
        const __nv_bfloat16 x = from_f32<__nv_bfloat16>(v);
        const float f = to_f32(x);
        d[h * rank] = x;
        v = isfinite(f) ? v - f : 0.f;          // an infinite part has no rest
    }
    return big;
}

// By whole warps: bits of positive floats are ordered as they are.
__device__ __forceinline__ void note_most(uint32_t *most, float big) {
    const uint32_t b = __reduce_max_sync(~0u, __float_as_uint(big));
    if ((threadIdx.x & 31) == 0 && b != 0u) atomicMax(most, b);
}

// Block (row tile, part of the contraction): MW warps of 16 rows x KW warps of the contraction;
// a cluster of `split` blocks shares a tile's contraction.
template <typename T, int NR, int MW, int KW>
__global__ void __launch_bounds__(MW * KW * 32) k_rank_rows(const __grid_constant__ RankArgs args) {
    const RankArg &p = args.a[blockIdx.y];
    constexpr int THREADS = MW * KW * 32, ROWS = 16 * MW;
    __shared__ float part[KW][ROWS][NR * 8 + 1];
    __shared__ int found[4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = lane & 3, g = lane >> 2;
    const int mw = warp % MW, kw = warp / MW;
    const uint32_t rank = p.split > 1 ? tc::cluster_ctarank() : 0u;
    grid_dependency();
    int t, n, id;
    // every block of a cluster looks for the same tile, so they agree
    if (!rank_tile(p, blockIdx.x / p.split, ROWS, found, t, n, id)) return;
    const int end = t + n;

    const int r0 = t + mw * 16;
    const T *X = static_cast<const T *>(p.X);
    const T *x0 = r0 + g < end ? X + (int64_t)(r0 + g) * p.ldx : nullptr;
    const T *x1 = r0 + g + 8 < end ? X + (int64_t)(r0 + g + 8) * p.ldx : nullptr;
    const T *A = static_cast<const T *>(p.A) + (int64_t)id * p.rank * p.inner;
    // The matrix unit rounds each sum the same way, so a chain is CHAIN steps (two products each), and
    // the chains are added in fp32 to nearest (one chain of 214 products: U 3.6e-6 off in the mean).
    constexpr int CHAIN = 8;
    float total[NR][4];
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) total[j][i] = 0.f;
    const int steps = (p.inner + 31) / 32;
    const int s0 = (int)((int64_t)steps * rank / p.split), s1 = (int)((int64_t)steps * (rank + 1) / p.split);
    const bool xv = p.xvec != 0, av = p.avec != 0;
    constexpr int AHEAD = NR <= 2 ? 4 : NR <= 4 ? 2 : 1;      // steps in flight
#pragma unroll 1
    for (int chain = s0 + kw; chain < s1; chain += CHAIN * KW) {
        const int end_step = min(s1, chain + CHAIN * KW);
        float acc[NR][4];
#pragma unroll
        for (int j = 0; j < NR; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
#pragma unroll AHEAD
        for (int step = chain; step < end_step; step += KW) {
            const int c = step * 32 + quad * 8;
            const uint4 a = piece<T>(x0, c, p.inner, xv), b = piece<T>(x1, c, p.inner, xv);
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                const int row = j * 8 + g;
                const uint4 w = piece<T>(row < p.rank ? A + (int64_t)row * p.inner : nullptr, c, p.inner, av);
                mma_16816<T>(acc[j], a.x, b.x, a.y, b.y, w.x, w.y);
                mma_16816<T>(acc[j], a.z, b.z, a.w, b.w, w.z, w.w);
            }
        }
#pragma unroll
        for (int j = 0; j < NR; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) total[j][i] += acc[j][i];
    }
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            part[kw][mw * 16 + g + 8 * (i >> 1)][j * 8 + 2 * quad + (i & 1)] = total[j][i];
    __syncthreads();
    const int rows = n;
    for (int i = threadIdx.x; i < rows * NR * 8; i += THREADS) {
        const int row = i / (NR * 8), j = i % (NR * 8);
        float sum = part[0][row][j];
#pragma unroll
        for (int k = 1; k < KW; ++k) sum += part[k][row][j];
        part[0][row][j] = sum;
    }
    if (p.split > 1) tc::cluster_sync();
    else __syncthreads();
    const float alpha = __ldg(p.alpha + id);
    float big = 0.f;
    const int per = (rows * NR * 8 + p.split - 1) / p.split;
    for (int i = (int)rank * per + threadIdx.x; i < min(rows * NR * 8, ((int)rank + 1) * per); i += THREADS) {
        const int row = i / (NR * 8), j = i % (NR * 8);
        float sum = 0.f;
        if (p.split > 1) {
            const uint32_t at = tc::smem_u32(&part[0][row][j]);
            for (int c = 0; c < p.split; ++c)
                sum += __uint_as_float(tc::ld_shared_cluster(tc::mapa_shared(at, c)));
        } else {
            sum = part[0][row][j];
        }
        if (j < p.rank) big = store_parts(p.T3 + ((int64_t)t + row) * LORA_PARTS * p.rank + j, p.rank, alpha * sum, big);
    }
    if (p.most) note_most(p.most + id, big);
    if (p.split > 1) tc::cluster_sync();
}

// ---- prompts -------------------------------------------------------------------------------

namespace {
constexpr int RK_ROWS = 64, RK_BK = 128, RK_STAGES = 4;
constexpr int RK_X = RK_ROWS * RK_BK * 2;               // 16 KB, two boxes of 64 columns
constexpr int RK_A = 128 * RK_BK * 2;                   // 32 KB; only `rank` rows are filled
constexpr int RK_STAGE = RK_X + RK_A;
constexpr int RK_SMEM = RK_STAGES * RK_STAGE + 1024 + 256;
constexpr int RK_THREADS = 192;
constexpr int RK_ACCS = 8, RK_CHAIN = 4;                // accumulators; steps of one
}  // namespace

// Roles: warp 0 tiled copies, warp 1 TMEM and MMAs, warps 2-5 outputs. The lanes past the rank
// multiply what the stage happens to hold; nothing reads them. The tensor core's own accumulation
// rounds each step the same way (one chain of 256 MMAs was 4e-6 off in the mean), so a chain is
// RK_CHAIN steps of 8 MMAs; the chains go to eight accumulators in turn, and the outputs' warps add
// them in fp32 to nearest while the next ones run.
template <typename T>
__global__ void __launch_bounds__(RK_THREADS, 1)
    k_rank_tc(const __grid_constant__ RankMaps maps, const __grid_constant__ RankArgs args) {
    const RankArg &p = args.a[blockIdx.y];
    const CUtensorMap *xmap = &maps.x[blockIdx.y], *amap = &maps.a[blockIdx.y];
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + RK_STAGES * RK_STAGE);
    uint64_t *empty = full + RK_STAGES;
    uint64_t *tfull = empty + RK_STAGES;
    uint64_t *tempty = tfull + RK_ACCS;
    uint64_t *drain = tempty + RK_ACCS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    __shared__ int found[4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = p.split > 1 ? tc::cluster_ctarank() : 0u;
    if (threadIdx.x == 0) {
        for (int s = 0; s < RK_STAGES; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], 1);
        }
        for (int k = 0; k < RK_ACCS; ++k) {
            tc::mbar_init(&tfull[k], 1);
            tc::mbar_init(&tempty[k], (p.rank + 31) / 32);      // the warps that have outputs
        }
        tc::mbar_init(drain, 1);
        *abort = 0;
        tc::fence_mbar_init();
        tc::prefetch_tmap(xmap);
        tc::prefetch_tmap(amap);
    }
    if (warp == 1) tc::tmem_alloc(tmem_slot, RK_ACCS * RK_ROWS);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    grid_dependency();
    int t = 0, n = 0, id = 0;
    // every block of a cluster looks for the same tile, so they agree
    const bool work = rank_tile(p, blockIdx.x / p.split, RK_ROWS, found, t, n, id);
    const int steps = (p.inner + RK_BK - 1) / RK_BK;
    const int s0 = (int)((int64_t)steps * rank / p.split), s1 = (int)((int64_t)steps * (rank + 1) / p.split);
    const int n16 = (n + 15) & ~15;
    float *sums = reinterpret_cast<float *>(smem);       // [row][rank] once the stages are done with
    if (work) {
        if (warp == 0) {
            bool ok = true;
            for (int s = s0; s < s1; ++s) {
                const int i = s - s0, stage = i % RK_STAGES;
                ok = __all_sync(~0u, tc::mbar_wait(&empty[stage], ((i / RK_STAGES) & 1) ^ 1, abort));
                if (!ok) break;
                uint8_t *x = smem + stage * RK_STAGE, *a = x + RK_X;
                if (tc::elect_one()) {
                    tc::mbar_arrive_expect_tx(&full[stage], RK_X + p.rank * 256);
                    tc::tma_load_2d(x, xmap, &full[stage], s * RK_BK, t);
                    tc::tma_load_2d(x + RK_X / 2, xmap, &full[stage], s * RK_BK + 64, t);
                    tc::tma_load_2d(a, amap, &full[stage], s * RK_BK, id * p.rank);
                    tc::tma_load_2d(a + RK_A / 2, amap, &full[stage], s * RK_BK + 64, id * p.rank);
                }
                __syncwarp();
            }
            if (!ok) {                      // loads still in flight land before the block exits
                const long long from = clock64();
                while (clock64() - from < 20000000ll) {
                }
            }
        } else if (warp == 1) {
            const uint32_t idesc = tc::idesc_f16_f32(Half2<T>::kType, 128, n16, 0, 0);
            const uint64_t bd0 = tc::desc_sw128(tc::smem_u32(smem), 16, 1024);
            const uint64_t ad0 = tc::desc_sw128(tc::smem_u32(smem) + RK_X, 16, 1024);
            bool ok = true;
            for (int s = s0; s < s1; ++s) {
                const int i = s - s0, stage = i % RK_STAGES, chain = i / RK_CHAIN, acc = chain % RK_ACCS;
                if (i % RK_CHAIN == 0) {
                    ok = __all_sync(~0u, tc::mbar_wait(&tempty[acc], ((chain / RK_ACCS) & 1) ^ 1, abort));
                    if (!ok) break;
                }
                ok = __all_sync(~0u, tc::mbar_wait(&full[stage], (i / RK_STAGES) & 1, abort));
                if (!ok) break;
                tc::fence_after_sync();
                const uint32_t by = (uint32_t)(stage * RK_STAGE >> 4);
                if (tc::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < RK_BK / 16; ++kk)
                        tc::mma_bf16(tmem + acc * RK_ROWS, ad0 + by + ((kk >> 2) * (RK_A / 2) + (kk & 3) * 32 >> 4),
                                     bd0 + by + ((kk >> 2) * (RK_X / 2) + (kk & 3) * 32 >> 4), idesc,
                                     (i % RK_CHAIN > 0 || kk > 0) ? 1u : 0u);
                    tc::mma_commit(&empty[stage]);
                    if (i % RK_CHAIN == RK_CHAIN - 1 || s == s1 - 1) tc::mma_commit(&tfull[acc]);
                }
                __syncwarp();
            }
            // (also after a time-out: what was issued completes before TMEM is released)
            if (tc::elect_one()) tc::mma_commit(drain);
            __syncwarp();
            volatile int never = 0;
            tc::mbar_wait(drain, 0, &never);
        } else {
            // lane = rank index
            const int quad = warp & 3, j = quad * 32 + lane;
            if (quad * 32 < p.rank) {
                float total[RK_ROWS];
#pragma unroll
                for (int q = 0; q < RK_ROWS; ++q) total[q] = 0.f;
                bool ok = true;
                const int chains = (s1 - s0 + RK_CHAIN - 1) / RK_CHAIN;
                for (int chain = 0; chain < chains; ++chain) {
                    const int acc = chain % RK_ACCS;
                    ok = __all_sync(~0u, tc::mbar_wait(&tfull[acc], (chain / RK_ACCS) & 1, abort));
                    if (!ok) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int c = 0; c < RK_ROWS; c += 16) {
                        if (c >= n16) break;
                        uint32_t v[16];
                        tc::tmem_ld_32x32b_x16(tmem + acc * RK_ROWS + c + ((uint32_t)(quad * 32) << 16), v);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int q = 0; q < 16; ++q) total[c + q] += __uint_as_float(v[q]);
                    }
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&tempty[acc]);
                }
                // into shared memory, over stages that the last products have read
                if (ok && j < p.rank) {
#pragma unroll
                    for (int q = 0; q < RK_ROWS; ++q)
                        if (q < n16) sums[q * p.rank + j] = total[q];
                }
            }
            tc::fence_before_sync();
        }
    }
    __syncwarp();
    __syncthreads();
    if (p.split > 1) tc::cluster_sync();
    // a cluster writes only when every block of it finished (the flags are read after the barrier)
    bool all = work && !*abort;
    if (p.split > 1 && work)
        for (int c = 0; c < p.split; ++c)
            all &= tc::ld_shared_cluster(tc::mapa_shared(tc::smem_u32(const_cast<int *>(abort)), c)) == 0;
    if (all) {
        const float alpha = __ldg(p.alpha + id);
        float big = 0.f;
        const int total = n * p.rank, per = (total + p.split - 1) / p.split;
        for (int i = (int)rank * per + threadIdx.x; i < min(total, ((int)rank + 1) * per); i += RK_THREADS) {
            const int row = i / p.rank, j = i - row * p.rank;
            float sum = 0.f;
            if (p.split > 1) {
                const uint32_t at = tc::smem_u32(&sums[i]);
                for (int c = 0; c < p.split; ++c)
                    sum += __uint_as_float(tc::ld_shared_cluster(tc::mapa_shared(at, c)));
            } else {
                sum = sums[i];
            }
            big = store_parts(p.T3 + ((int64_t)t + row) * LORA_PARTS * p.rank + j, p.rank, alpha * sum, big);
        }
        if (p.most) note_most(p.most + id, big);
    }
    if (p.split > 1) tc::cluster_sync();
    if (*abort && threadIdx.x == 0) set_status(p.status, GPTQ_ERR_TIMEOUT);
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, RK_ACCS * RK_ROWS);
    }
}

template <typename T, int NR>
static gptq_status launch_rank_nr(RankArgs &q, int count, cudaStream_t st) {
    const RankArg &p = q.a[0];
    if (p.M >= 1024) {
        // many rows in a layout that tiled copies refuse: 64 rows a block share the adapter
        constexpr int KW = NR > 8 ? 1 : 2;
        for (int i = 0; i < count; ++i) q.a[i].split = 1;
        return launch_pdl(k_rank_rows<T, NR, 4, KW>, dim3((unsigned)(p.R + p.M / 64), count), 128 * KW, 0, 0, 1, st, q);
    }
    constexpr int KW = NR > 8 ? 4 : 8;
    const int steps = (std::min(p.inner, q.a[count - 1].inner) + 31) / 32;
    int split = 1;
    const int64_t tiles = std::min<int64_t>(p.M, p.R + p.M / 16);
    while (split < 8 && tiles * count * split * 2 <= 2 * device_sms() && steps >= 4 * KW * split) split *= 2;
    for (int i = 0; i < count; ++i) q.a[i].split = split;
    return launch_pdl(k_rank_rows<T, NR, 1, KW>, dim3((unsigned)(tiles * split), count), 32 * KW, 0, 0, split, st, q);
}

template <typename T>
static gptq_status launch_rank(RankArgs &q, int count, int dtype, cudaStream_t st) {
    const RankArg &p = q.a[0];
    // prompts: 64 rows a tile. The bound on short requests is that of tiles that a few rows fill.
    if (p.M >= 256 && p.M >= 16 * (int64_t)p.R) {
        RankMaps maps{};
        bool tiled = true;
        for (int i = 0; i < count; ++i) {
            const RankArg &r = q.a[i];
            tiled = tiled && rows_map(&maps.x[i], r.X, dtype, r.M, r.inner, r.ldx, RK_ROWS) &&
                    rows_map(&maps.a[i], r.A, dtype, (int64_t)r.L * r.rank, r.inner, r.inner, r.rank);
        }
        if (tiled) {
            const int64_t tiles = p.R + p.M / RK_ROWS;
            const int steps = (std::min(p.inner, q.a[count - 1].inner) + RK_BK - 1) / RK_BK;
            int split = 1;
            while (split < 8 && tiles * count * split * 2 <= device_sms() && steps >= 4 * split) split *= 2;
            for (int i = 0; i < count; ++i) q.a[i].split = split;
            return launch_pdl(k_rank_tc<T>, dim3((unsigned)(tiles * split), count), RK_THREADS, RK_SMEM, RK_SMEM, split, st,
                              maps, q);
        }
    }
    if (p.rank <= 8) return launch_rank_nr<T, 1>(q, count, st);
    if (p.rank <= 16) return launch_rank_nr<T, 2>(q, count, st);
    if (p.rank <= 32) return launch_rank_nr<T, 4>(q, count, st);
    if (p.rank <= 64) return launch_rank_nr<T, 8>(q, count, st);
    return launch_rank_nr<T, 16>(q, count, st);
}

// T and U of fp16 rows (blockIdx.y) as pairs for the gradients, eight values a thread. Rows of requests
// without an adapter are left out: nothing reads them.
struct ScaleArg {
    const __nv_bfloat16 *T3[2];
    __half *pair[2];                    // [M][2 rank]
    const uint32_t *most[2];
    const int32_t *offsets, *ids, *list_off;
    int64_t M;
    int R, rank;
    const int32_t *status;
};
__global__ void __launch_bounds__(256) k_rank_scale(const __grid_constant__ ScaleArg p) {
    grid_dependency();
    if (failed(p.status) || __ldcg(p.list_off) < 0) return;
    const int per = p.rank / 8, which = blockIdx.y;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, t = i / per;
    if (t >= p.M || t < __ldg(p.offsets) || t >= __ldg(p.offsets + p.R)) return;
    const int id = __ldg(p.ids + request_of(p.offsets, p.R, (int)t)), j = (int)(i - t * per) * 8;
    if (id < 0) return;
    const int e = 141 - (int)(__ldcg(p.most[which] + id) >> 23);
    const __nv_bfloat16 *src = p.T3[which] + t * LORA_PARTS * p.rank + j;
    uint4 in[LORA_PARTS];
#pragma unroll
    for (int h = 0; h < LORA_PARTS; ++h) in[h] = __ldcg(reinterpret_cast<const uint4 *>(src + h * p.rank));
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float2 v = make_float2(0.f, 0.f);
#pragma unroll
        for (int h = LORA_PARTS - 1; h >= 0; --h) {
            const float2 f = Half2<__nv_bfloat16>::unpack(reinterpret_cast<const uint32_t *>(&in[h])[q]);
            v.x += f.x;
            v.y += f.y;
        }
        v.x = ldexpf(v.x, e);
        v.y = ldexpf(v.y, e);
        hi[q] = Half2<__half>::pack(v.x, v.y);
        const float2 f = Half2<__half>::unpack(hi[q]);
        lo[q] = Half2<__half>::pack(isfinite(f.x) ? v.x - f.x : 0.f, isfinite(f.y) ? v.y - f.y : 0.f);
    }
    __half *d = p.pair[which] + t * 2 * p.rank + j;
    *reinterpret_cast<uint4 *>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4 *>(d + p.rank) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

// What the backward pass needs first. Block 0: the requests of each adapter, in request order
// (list_off [L + 1], list [R]; a warp takes whole adapters, 32 requests at a time; list_off[0] is
// -1 when offsets or ids are refused, which a caller without a status word would not see). The others:
// out[l][j][n] = in[l][n][j], 16-bit elements, 32 x 32 tiles through shared memory.
struct SetupArg {
    const int32_t *offsets, *ids;
    int64_t M;
    int R, L;
    int32_t *list_off, *list, *status;
    uint32_t *most;                     // [2][L], set to zero
    const uint16_t *in;
    uint16_t *out;
    int N, r;
};

__device__ __forceinline__ void adapter_lists(const SetupArg &p) {
    __shared__ int warp_sum[8], base;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < 2 * p.L; i += 256) p.most[i] = 0u;
    const bool bad = __syncthreads_or(ids_bad(p.ids, p.R, p.L, threadIdx.x, 256) ||
                                      offsets_bad(p.offsets, p.R, p.M, threadIdx.x, 256));
    if (bad) {
        if (threadIdx.x == 0) {
            set_status(p.status, GPTQ_ERR_ARG);
            p.list_off[0] = -1;
        }
        return;
    }
    auto uses = [&](int i, int a) { return __ballot_sync(~0u, i < p.R && __ldg(p.ids + i) == a); };
    if (threadIdx.x == 0) p.list_off[0] = base = 0;
    for (int a = warp; a < p.L; a += 8) {
        int n = 0;
#pragma unroll 4
        for (int i = 0; i < p.R; i += 32) n += __popc(uses(i + lane, a));
        if (lane == 0) p.list_off[a + 1] = n;
    }
    __syncthreads();
    // counts to ends
    for (int a0 = 0; a0 < p.L; a0 += 256) {
        const int a = a0 + threadIdx.x;
        int sum = a < p.L ? p.list_off[a + 1] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(~0u, sum, d);
            if (lane >= d) sum += v;
        }
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
        sum += base;
        for (int w = 0; w < warp; ++w) sum += warp_sum[w];
        if (a < p.L) p.list_off[a + 1] = sum;
        __syncthreads();
        if (threadIdx.x == 255) base = sum;
        __syncthreads();
    }
    for (int a = warp; a < p.L; a += 8) {
        int at = p.list_off[a];
        for (int i = 0; i < p.R; i += 32) {
            const unsigned b = uses(i + lane, a);
            if (b >> lane & 1u) p.list[at + __popc(b & ((1u << lane) - 1u))] = i + lane;
            at += __popc(b);
        }
    }
}

__global__ void __launch_bounds__(256) k_lora_setup(const __grid_constant__ SetupArg p) {
    __shared__ uint16_t tile[32][34];
    grid_dependency();
    if (blockIdx.x == 0) {
        adapter_lists(p);
        return;
    }
    const int tn = (p.N + 31) / 32, tr = (p.r + 31) / 32;
    const int64_t b = blockIdx.x - 1;
    const int l = (int)(b / (tn * tr)), rest = (int)(b - (int64_t)l * tn * tr);
    const int n0 = rest % tn * 32, j0 = rest / tn * 32;
    const int64_t base = (int64_t)l * p.N * p.r;
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    for (int i = y; i < 32; i += 8)
        if (n0 + i < p.N && j0 + x < p.r) tile[i][x] = p.in[base + (int64_t)(n0 + i) * p.r + j0 + x];
    __syncthreads();
    for (int i = y; i < 32; i += 8)
        if (j0 + i < p.r && n0 + x < p.N) p.out[base + (int64_t)(j0 + i) * p.N + n0 + x] = tile[x][i];
}

static RankArg rank_arg(__nv_bfloat16 *T3, uint32_t *most, const void *X, int64_t ldx, int64_t M, const void *A, int inner,
                        const float *alpha, const int32_t *offsets, const LoraArg &l, int32_t *status) {
    RankArg p{};
    p.X = X; p.ldx = ldx; p.M = M;
    p.A = A; p.alpha = alpha;
    p.offsets = offsets; p.ids = l.ids;
    p.R = l.R; p.L = l.L; p.rank = l.rank; p.inner = inner;
    p.T3 = T3;
    p.most = most;
    p.xvec = aligned(X, 16) && ldx % 8 == 0;
    p.avec = aligned(A, 16) && inner % 8 == 0;
    p.status = status;
    return p;
}

static gptq_status rank_rows(RankArgs &q, int count, int dtype, cudaStream_t st) {
    return dtype == GPTQ_BF16 ? launch_rank<__nv_bfloat16>(q, count, dtype, st)
                              : launch_rank<__half>(q, count, dtype, st);
}

struct LoraSpace {
    __nv_bfloat16 *T3, *U3;
    __half *T_pair, *U_pair;            // (made for fp16 rows)
    uint32_t *most;                     // [2][L]: T, U
    void *Bt;
    float *parts_a, *parts_b;
    int32_t *list_off, *list;
    size_t bytes;
};

static LoraSpace lora_space(void *ws, bool backward, int64_t M, int N, int K, int R, int L, int rank) {
    Carver c(ws);
    LoraSpace s{};
    s.T3 = c.take<__nv_bfloat16>((size_t)M * LORA_PARTS * rank);
    if (backward) {
        s.U3 = c.take<__nv_bfloat16>((size_t)M * LORA_PARTS * rank);
        s.T_pair = c.take<__half>((size_t)M * 2 * rank);
        s.U_pair = c.take<__half>((size_t)M * 2 * rank);
        s.most = c.take<uint32_t>(2 * (size_t)L);
        s.Bt = c.take<uint16_t>((size_t)L * N * rank);
        // (a single part goes to the gradient itself)
        auto parts = [&](int width) {
            const int n = adapter_parts(M, L, width);
            return n > 1 ? c.take<float>((size_t)n * L * width * rank) : nullptr;
        };
        s.parts_a = parts(K);
        s.parts_b = parts(N);
        s.list_off = c.take<int32_t>(L + 1);
        s.list = c.take<int32_t>(std::max(R, 1));
    }
    s.bytes = round_up(c.off, 256);
    return s;
}

size_t lora_workspace(bool backward, int64_t M, int N, int K, int R, int L, int rank) {
    return lora_space(nullptr, backward, M, N, K, R, L, rank).bytes;
}

gptq_status matmul_lora(MatmulArg m, const void *A, const void *B, const float *alpha, int dtype, int bits,
                        void *ws, cudaStream_t st) {
    const LoraArg &l = m.lora;
    const LoraSpace s = lora_space(ws, false, m.M, m.w.N, m.w.K, l.R, l.L, l.rank);
    RankArgs q{};
    q.a[0] = rank_arg(s.T3, nullptr, m.X, m.ldx, m.M, A, m.w.K, alpha, m.offsets, l, m.status);
    gptq_status r = rank_rows(q, 1, dtype, st);
    if (r != GPTQ_OK) return r;
    m.lora.P = B;
    m.lora.T3 = s.T3;
    if (matmul_few_rows(m.M, 1)) return matmul_token(m, dtype, bits, st);
    return matmul_tc(m, 0, dtype, bits, st);
}

// m.X = dY, m.Y = dX (NULL: not wanted).
gptq_status matmul_lora_backward(MatmulArg m, float *dA, float *dB, const void *X, int64_t ldx, const void *A,
                                 const void *B, const float *alpha, int dtype, int bits, void *ws,
                                 cudaStream_t st) {
    const LoraArg l = m.lora;
    const int N = m.w.N, K = m.w.K;
    const LoraSpace s = lora_space(ws, true, m.M, N, K, l.R, l.L, l.rank);
    const bool need_u = (m.Y || dA) && m.M > 0, need_t = dB && m.M > 0;
    SetupArg setup{m.offsets, l.ids, m.M, l.R, l.L, s.list_off, s.list, m.status, s.most, (const uint16_t *)B, (uint16_t *)s.Bt,
                   N, l.rank};
    const int64_t tiles = need_u ? (int64_t)((N + 31) / 32) * ((l.rank + 31) / 32) * l.L : 0;
    gptq_status r = launch_pdl(k_lora_setup, dim3((unsigned)(1 + tiles)), 256, 0, 0, 1, st, setup);
    if (r != GPTQ_OK) return r;
    const bool pair = dtype == GPTQ_F16;
    uint32_t *t_most = pair && dB ? s.most : nullptr, *u_most = pair && dA ? s.most + l.L : nullptr;
    RankArgs q{};
    int count = 0;
    if (need_u) q.a[count++] = rank_arg(s.U3, u_most, m.X, m.ldx, m.M, s.Bt, N, alpha, m.offsets, l, m.status);
    if (need_t) q.a[count++] = rank_arg(s.T3, t_most, X, ldx, m.M, A, K, alpha, m.offsets, l, m.status);
    if (count > 0) {
        r = rank_rows(q, count, dtype, st);
        if (r != GPTQ_OK) return r;
    }
    AdapterGrad grads[2];
    ScaleArg scale{};
    int wanted = 0;
    auto want = [&](const void *P, int64_t ldp, int np, const __nv_bfloat16 *T3, __half *to, const uint32_t *most,
                    float *out, float *parts, int transposed) {
        if (pair) {
            scale.T3[wanted] = T3;
            scale.pair[wanted] = to;
            scale.most[wanted] = most;
        }
        const int halves = pair ? 2 : LORA_PARTS;
        grads[wanted++] = {P, ldp, np, pair ? (const void *)to : T3, halves * l.rank, halves, most, out, parts, transposed};
    };
    if (dB) want(m.X, m.ldx, N, s.T3, s.T_pair, t_most, dB, s.parts_b, 0);
    if (dA) want(X, ldx, K, s.U3, s.U_pair, u_most, dA, s.parts_a, 1);
    if (pair && wanted > 0 && m.M > 0) {
        scale.offsets = m.offsets; scale.ids = l.ids; scale.list_off = s.list_off;
        scale.M = m.M; scale.R = l.R; scale.rank = l.rank;
        scale.status = m.status;
        r = launch_pdl(k_rank_scale, dim3((unsigned)((m.M * (l.rank / 8) + 255) / 256), wanted), 256, 0, 0, 1, st, scale);
        if (r != GPTQ_OK) return r;
    }
    if (wanted > 0) {
        r = adapter_gradients(grads, wanted, l.rank, dtype, m.M, m.offsets, l.ids, s.list_off, s.list, l.R, l.L,
                              m.status, st);
        if (r != GPTQ_OK) return r;
    }
    if (m.Y && m.M > 0) {
        m.lora.P = A;
        m.lora.T3 = s.U3;
        r = matmul_tc(m, 1, dtype, bits, st);
    }
    return r;
}

}  // namespace gptq
