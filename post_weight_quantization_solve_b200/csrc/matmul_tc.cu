// Packed-weight products on the tensor cores: Y[t] = W^_e X[t] (forward) and
// dX[t] = W^_e^T dY[t] (input gradient) over row ranges of experts, with the low-rank
// adapters of the rows' requests added in the same accumulators.
//
// One tile is 128 output channels (TMEM lanes) x up to 256 rows (TMEM columns): the weights
// are the A operand, so a tile's row count is free (multiples of 16) and a short range of an
// expert costs no more matrix work than it has rows. The contraction runs in steps of 64:
//   forward         a thread unpacks 32 codes of its own channel (lane) and stores them into
//                   TMEM, where the MMA reads A; only the rows X go through shared memory.
//   input gradient  the contraction runs over the packed rows n, so a thread unpacks 32 codes
//                   of one n into a [n][k] tile of shared memory, read as an MN-major A.
// Scales: with one scale a channel the forward product multiplies exact integers c - z and the
// scale enters in fp32 at the end. Where the scale changes along the contraction (input
// groups, the input gradient) or adapters share the accumulators, each weight s (c - z) is
// rounded once to the rows' 16-bit type, as a dequantised layer in that type would hold it.
//
// Adapters: after the steps of W^, each run of rows with one adapter adds
// sum_j P_a[.][j] T[t][j] over the run's columns alone (runs start on 16-column borders, rows
// of the border columns that belong to others are zero in shared memory). T comes as a pair of
// 16-bit halves, so the rank-space rows keep 16 bits.
//
// Roles (320 threads): warps 0-7 unpack and, at a tile's end, write the outputs; warp 8 issues
// the tiled copies of X; warp 9 owns TMEM and issues the MMAs.
#include <algorithm>

#include "matmul.cuh"

namespace gptq {

namespace {
constexpr int MM_LANES = 128;                       // output channels of a tile
constexpr int MM_COLS = 256;                        // most rows of a tile
constexpr int MM_BK = 64;
constexpr int MM_THREADS = 320;
constexpr int MM_B_BYTES = MM_COLS * MM_BK * 2;     // 32 KB
constexpr int MM_A_BYTES = MM_LANES * MM_BK * 2;    // 16 KB (input gradient)
constexpr int MM_BOX = 64 * 64 * 2;                 // one 64 x 64 box of A
constexpr int MM_TABLE = (MATMUL_MAX_EXPERTS + 1) * 4;
constexpr uint32_t MM_TMEM = 512;

template <int DIR>
struct MmShape {
    static constexpr int STAGES = DIR == 0 ? 6 : 4;
    static constexpr int STAGE = DIR == 0 ? MM_B_BYTES : MM_B_BYTES + MM_A_BYTES;
    static constexpr int SMEM = STAGES * STAGE + MM_TABLE + 1024 + 512;
};
}  // namespace

struct MmTcArg {
    MatmulArg m;
    int out, inner;       // output channels and contraction length of this direction
    int cols;             // most rows of a tile (multiple of 16)
    int box_rows;         // rows of one tiled copy of X; 0: plain loads
    int split;            // blocks of a cluster that share a tile's contraction
    int fold;             // scales folded into the weights
    int vec;              // packed rows start on 16-byte boundaries
    int E;                // row ranges
};

// Rows [r0, r0 + rows) x columns [c0, c0 + 64) of X into the swizzled layout of a tiled copy,
// zeros outside [0, row_end) x [0, col_end): the copy for layouts that tiled copies refuse.
template <typename T>
__device__ __forceinline__ void plain_box(uint8_t *dst, const T *x, int64_t ld, int64_t r0, int rows,
                                          int64_t row_end, int c0, int col_end, int tid, int nthr) {
    for (int i = tid; i < rows * 8; i += nthr) {
        const int r = i >> 3, q = i & 7;
        uint32_t v[4] = {0u, 0u, 0u, 0u};
        if (r0 + r < row_end) {
            const unsigned short *src =
                reinterpret_cast<const unsigned short *>(x) + (r0 + r) * ld + c0 + 8 * q;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c0 + 8 * q + e < col_end) v[e >> 1] |= (uint32_t)__ldg(src + e) << (16 * (e & 1));
        }
        *reinterpret_cast<uint4 *>(dst + r * 128 + ((q ^ (r & 7)) << 4)) =
            make_uint4(v[0], v[1], v[2], v[3]);
    }
}

// 16 bytes (8 elements) of a row at p, `left` of them inside; whole pieces only when aligned.
template <typename T>
__device__ __forceinline__ uint4 load8(const T *p, int left, bool vec) {
    if (left >= 8 && vec) return __ldg(reinterpret_cast<const uint4 *>(p));
    uint32_t v[4] = {0u, 0u, 0u, 0u};
    const unsigned short *src = reinterpret_cast<const unsigned short *>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < left) v[e >> 1] |= (uint32_t)__ldg(src + e) << (16 * (e & 1));
    return make_uint4(v[0], v[1], v[2], v[3]);
}

struct MmTile {
    int e, c0;            // range, first output channel
    int64_t t0;           // first row
    int n, n16;           // rows, rounded up to 16
};

// Tile u -> (range, rows, channels), channels fastest: blocks that run together share rows of X.
__device__ __forceinline__ MmTile mm_tile(const MmTcArg &p, const int *table, int tiles_out, int u) {
    MmTile t;
    const int q = u / tiles_out;
    t.c0 = (u - q * tiles_out) * MM_LANES;
    int lo = 0, hi = p.E - 1;                       // last range whose first tile is <= q
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (table[mid] <= q) lo = mid;
        else hi = mid - 1;
    }
    t.e = lo;
    int64_t begin = 0, end = p.m.M;
    if (p.m.offsets) {
        const bool one = p.m.lora.R > 0;            // with adapters the requests are one range
        begin = __ldg(p.m.offsets + (one ? 0 : lo));
        end = __ldg(p.m.offsets + (one ? p.m.lora.R : lo + 1));
    }
    const int cnt = (int)(end - begin);
    const int nt = (cnt + p.cols - 1) / p.cols;
    const int size = ((cnt + nt - 1) / nt + 15) & ~15;
    const int j = q - table[lo];
    t.t0 = begin + (int64_t)j * size;
    t.n = min(size, cnt - j * size);
    t.n16 = (t.n + 15) & ~15;
    return t;
}

template <typename T, int B, int DIR>
__global__ void __launch_bounds__(MM_THREADS, 1)
    k_matmul_tc(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ MmTcArg p) {
    using S = MmShape<DIR>;
    constexpr int PD = B == 8 ? 3 : 4;              // steps of packed words held ahead
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    int *table = reinterpret_cast<int *>(smem + S::STAGES * S::STAGE);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::STAGES * S::STAGE + ((MM_TABLE + 15) & ~15));
    uint64_t *empty = full + S::STAGES;
    uint64_t *tfull = empty + S::STAGES;
    uint64_t *tdone = tfull + 1;
    uint64_t *drain = tdone + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *refuse = reinterpret_cast<int *>(tmem_slot + 2);

    const MatmulArg &m = p.m;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = p.split;
    const uint32_t rank = split > 1 ? tc::cluster_ctarank() : 0u;
    const int group = blockIdx.x / split, ngroups = gridDim.x / split;
    const bool tiled = p.box_rows > 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::STAGES; ++s) {
            tc::mbar_init(&full[s], 8 + (tiled ? 1 : 0));
            tc::mbar_init(&empty[s], 1);
        }
        tc::mbar_init(tfull, 1);
        tc::mbar_init(tdone, 8);
        tc::mbar_init(drain, 1);
        *abort = 0;
        *refuse = 0;
        tc::fence_mbar_init();
        if (tiled) tc::prefetch_tmap(&xmap);
    }
    if (warp == 9) tc::tmem_alloc(tmem_slot, MM_TMEM);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    grid_dependency();

    // the ranges: refused as a whole when they are not ordered inside [0, M]
    bool bad = false;
    const int nranges = m.lora.R > 0 ? m.lora.R : p.E;
    if (m.offsets) bad = offsets_bad(m.offsets, nranges, m.M, threadIdx.x, MM_THREADS);
    if (m.lora.R > 0) bad |= ids_bad(m.lora.ids, m.lora.R, m.lora.L, threadIdx.x, MM_THREADS);
    if (bad) *refuse = 1;
    if (threadIdx.x == 0 && failed(m.status)) *refuse = 2;
    __syncthreads();
    if (warp == 0) {
        // table[e]: tiles of rows before range e
        int base = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            int nt = 0;
            if (e < p.E && *refuse == 0) {
                int64_t cnt = m.M;
                if (m.lora.R > 0) cnt = __ldg(m.offsets + m.lora.R) - __ldg(m.offsets);
                else if (m.offsets) cnt = __ldg(m.offsets + e + 1) - __ldg(m.offsets + e);
                nt = (int)((cnt + p.cols - 1) / p.cols);
            }
            int sum = nt;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(~0u, sum, d);
                if (lane >= d) sum += v;
            }
            if (e < p.E) table[e] = base + sum - nt;
            base += __shfl_sync(~0u, sum, 31);
        }
        if (lane == 0) table[p.E] = base;
    }
    __syncthreads();
    if (split > 1) tc::cluster_sync();      // every block's barriers and refusal are in place
    int skip = *refuse;
    if (split > 1)                          // the blocks of a cluster go by the first one's reading
        skip = (int)tc::ld_shared_cluster(tc::mapa_shared(tc::smem_u32(refuse), 0));
    if (skip == 1 && threadIdx.x == 0) set_status(m.status, GPTQ_ERR_ARG);

    const int tiles_out = (p.out + MM_LANES - 1) / MM_LANES;
    const int tiles = skip ? 0 : table[p.E] * tiles_out;
    const int steps = (p.inner + MM_BK - 1) / MM_BK;
    const int k0 = (int)((int64_t)steps * rank / split), k1 = (int)((int64_t)steps * (rank + 1) / split);
    const bool adapters = m.lora.R > 0 && (int)rank == split - 1;
    const int two_r = 2 * m.lora.rank;
    const int rsteps = (two_r + MM_BK - 1) / MM_BK;
    const T *X = static_cast<const T *>(m.X);

    if (warp < 8) {
        const int tid = threadIdx.x;
        const int nw = (int)(((int64_t)m.w.K * B + 31) / 32);
        const bool vec = p.vec != 0;
        // forward: channel = lane of the warp's TMEM quarter, half of the step's columns
        const int quad = warp & 3, half = warp >> 2;
        // input gradient: row n of the step, chunk of 32 columns of the tile
        const int arow = warp * 8 + ((lane >> 1) & 7), achunk = (lane & 1) + ((lane >> 4) << 1);
        int stage = 0;
        uint32_t phase = 0, tphase = 0;
        for (int u = group; u < tiles; u += ngroups) {
            const MmTile t = mm_tile(p, table, tiles_out, u);
            const int64_t erow = (int64_t)t.e * m.w.N;
            const int32_t *gi = m.w.g_idx ? m.w.g_idx + (int64_t)t.e * m.w.K : nullptr;
            const int ch = t.c0 + quad * 32 + lane;     // forward: this thread's channel
            uint32_t raw[PD][B];
            float sc[PD];
            // words and scale of the step's chunk
            auto fetch = [&](int step, uint32_t (&w)[B], float &s) {
                int n, chunk;
                if constexpr (DIR == 0) {
                    n = ch;
                    chunk = step * 2 + half;
                } else {
                    n = step * MM_BK + arow;
                    chunk = (t.c0 >> 5) + achunk;
                }
                const bool in = n < m.w.N && step < k1;
                load_chunk<B>(in ? m.w.words + (erow + n) * m.w.ldw : nullptr, chunk, nw, vec, w);
                s = 0.f;
                if (p.fold && in && !gi && chunk * 32 < m.w.K)
                    s = __ldg(m.w.scales + (m.w.groups ? (erow + n) * m.w.groups + ((chunk * 32) >> m.w.gshift)
                                                       : erow + n));
            };
#pragma unroll
            for (int d = 0; d < PD; ++d) fetch(k0 + d, raw[d], sc[d]);
            for (int kb = k0; kb < k1; kb += PD) {
#pragma unroll
                for (int d = 0; d < PD; ++d) {
                    const int step = kb + d;
                    if (step >= k1) break;
                    uint32_t v[16];
                    unpack32<B, T>(raw[d], v);
                    if (p.fold) {
                        if (gi) {
                            int n, c;
                            if constexpr (DIR == 0) { n = ch; c = step * 64 + half * 32; }
                            else { n = step * MM_BK + arow; c = t.c0 + achunk * 32; }
                            if (n < m.w.N)
                                scale32_by_index<T>(v, m.w.scales + (erow + n) * m.w.groups, gi, c, m.w.K,
                                                    m.w.groups, m.status);
                        } else {
                            scale32<T>(v, sc[d]);
                        }
                    }
                    fetch(step + PD, raw[d], sc[d]);
                    bool ok = tc::mbar_wait(&empty[stage], phase ^ 1, abort);
                    ok = __all_sync(~0u, ok);
                    if (ok) {
                        uint8_t *st = smem + stage * S::STAGE;
                        if constexpr (DIR == 0) {
                            // the stage's last reader was an MMA that has completed
                            tc::fence_after_sync();
                            tc::tmem_st_32x32b_x16(tmem + MM_COLS + stage * 32 + half * 16 +
                                                       ((uint32_t)(quad * 32) << 16), v);
                            tc::tmem_st_wait();
                        } else {
                            uint8_t *a = st + MM_B_BYTES + (achunk >> 1) * MM_BOX + arow * 128;
                            if (step * MM_BK + arow >= m.w.N) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) v[i] = 0u;
                            }
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                *reinterpret_cast<uint4 *>(a + (((((achunk & 1) << 2) + q) ^ (arow & 7)) << 4)) =
                                    make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                        }
                        if (!tiled)
                            plain_box<T>(st, X, m.ldx, t.t0, t.n16, t.t0 + t.n, step * MM_BK, p.inner, tid, 256);
                        if (DIR == 1 || !tiled) tc::fence_async_shared();
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(&full[stage]);
                    }
                    if (++stage == S::STAGES) { stage = 0; phase ^= 1; }
                }
            }
            if (adapters) {
                const T *P = static_cast<const T *>(m.lora.P);
                const T *T2 = static_cast<const T *>(m.lora.T2);
                const int r = m.lora.rank;
                RunWalk run(m.offsets, m.lora.ids, m.lora.R, (int)t.t0, (int)t.t0 + t.n);
                while (run.next()) {
                    const int b0 = (run.begin - (int)t.t0) & ~15, b1 = ((run.end - (int)t.t0) + 15) & ~15;
                    for (int rs = 0; rs < rsteps; ++rs) {
                        bool ok = tc::mbar_wait(&empty[stage], phase ^ 1, abort);
                        ok = __all_sync(~0u, ok);
                        if (ok) {
                            uint8_t *st = smem + stage * S::STAGE;
                            if constexpr (DIR == 0) {
                                // A: row n of B_a twice over, [hi part | lo part] of the contraction
                                uint32_t v[16];
                                const T *src = P + ((int64_t)run.id * m.w.N + ch) * r;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int q = rs * MM_BK + half * 32 + i * 8;
                                    const uint4 x = ch < m.w.N && q < two_r ? load8<T>(src + (q < r ? q : q - r), 8, true)
                                                                            : make_uint4(0u, 0u, 0u, 0u);
                                    v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
                                }
                                tc::fence_after_sync();
                                tc::tmem_st_32x32b_x16(tmem + MM_COLS + stage * 32 + half * 16 +
                                                           ((uint32_t)(quad * 32) << 16), v);
                                tc::tmem_st_wait();
                            } else {
                                const int q = rs * MM_BK + arow;
                                const int c = t.c0 + achunk * 32;
                                const T *src = P + ((int64_t)run.id * r + (q < r ? q : q - r)) * m.w.K + c;
                                uint8_t *a = st + MM_B_BYTES + (achunk >> 1) * MM_BOX + arow * 128;
                                const bool v8 = (m.w.K & 7) == 0;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int left = q < two_r ? m.w.K - c - 8 * i : 0;
                                    *reinterpret_cast<uint4 *>(a + (((((achunk & 1) << 2) + i) ^ (arow & 7)) << 4)) =
                                        load8<T>(src + 8 * i, left, v8);
                                }
                            }
                            // the run's rows of [hi | lo], zeros for rows of others
                            for (int i = tid; i < (b1 - b0) * 8; i += 256) {
                                const int row = b0 + (i >> 3), q = i & 7, col = rs * MM_BK + 8 * q;
                                const int64_t tr = t.t0 + row;
                                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                                if (tr >= run.begin && tr < run.end && col < two_r)
                                    x = __ldg(reinterpret_cast<const uint4 *>(T2 + tr * two_r + col));
                                *reinterpret_cast<uint4 *>(st + row * 128 + ((q ^ (row & 7)) << 4)) = x;
                            }
                            tc::fence_async_shared();
                            tc::fence_before_sync();
                            __syncwarp();
                            if (lane == 0) tc::mbar_arrive(&full[stage]);
                        }
                        if (++stage == S::STAGES) { stage = 0; phase ^= 1; }
                    }
                }
            }
            // outputs: lane = channel, register = row
            bool ok = tc::mbar_wait(tfull, tphase, abort);
            ok = __all_sync(~0u, ok);
            tphase ^= 1;
            tc::fence_after_sync();
            const bool per_channel = DIR == 0 && !p.fold;
            const float s = per_channel && ch < p.out ? __ldg(m.w.scales + erow + ch) : 1.f;
            T *Y = static_cast<T *>(m.Y);
            if (split == 1) {
                if (ok) {
                    for (int cb = half; cb < t.n16 / 16; cb += 2) {
                        uint32_t r[16];
                        tc::tmem_ld_32x32b_x16(tmem + cb * 16 + ((uint32_t)(quad * 32) << 16), r);
                        tc::tmem_ld_wait();
                        if (ch < p.out) {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (cb * 16 + i < t.n)
                                    Y[(t.t0 + cb * 16 + i) * m.ldy + ch] = from_f32<T>(s * __uint_as_float(r[i]));
                        }
                    }
                }
                tc::fence_before_sync();
            } else {
                // partial sums of the cluster's blocks: [row][channel] in the stages, summed in
                // rank order by the block that writes the row
                float *dump = reinterpret_cast<float *>(smem);
                if (ok) {
                    for (int cb = half; cb < t.n16 / 16; cb += 2) {
                        uint32_t r[16];
                        tc::tmem_ld_32x32b_x16(tmem + cb * 16 + ((uint32_t)(quad * 32) << 16), r);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            dump[(cb * 16 + i) * MM_LANES + quad * 32 + lane] = __uint_as_float(r[i]);
                    }
                }
                tc::fence_before_sync();
                tc::cluster_sync();
                for (int row = (int)rank + split * half; row < t.n; row += 2 * split) {
                    float sum = 0.f;
                    const uint32_t at = tc::smem_u32(dump + row * MM_LANES + quad * 32 + lane);
                    for (int c = 0; c < split; ++c)
                        sum += __uint_as_float(tc::ld_shared_cluster(tc::mapa_shared(at, c)));
                    if (ch < p.out && ok) Y[(t.t0 + row) * m.ldy + ch] = from_f32<T>(s * sum);
                }
                tc::cluster_sync();
                tc::fence_async_shared();       // the stages go back to the tiled copies
                if (lane == 0) tc::mbar_arrive(tdone);
            }
        }
    } else if (warp == 8) {
        int stage = 0, issued = 0;
        uint32_t phase = 0, dphase = 0;
        for (int u = group; u < tiles; u += ngroups) {
            if (lane == 0 && tiled && !*abort) {
                const MmTile t = mm_tile(p, table, tiles_out, u);
                const int boxes = (t.n + p.box_rows - 1) / p.box_rows;
                for (int step = k0; step < k1; ++step) {
                    if (!tc::mbar_wait(&empty[stage], phase ^ 1, abort)) break;
                    tc::mbar_arrive_expect_tx(&full[stage], boxes * p.box_rows * 128);
                    uint8_t *st = smem + stage * S::STAGE;
                    for (int b = 0; b < boxes; ++b)
                        tc::tma_load_2d(st + b * p.box_rows * 128, &xmap, &full[stage], step * MM_BK,
                                        (int)t.t0 + b * p.box_rows);
                    ++issued;
                    if (++stage == S::STAGES) { stage = 0; phase ^= 1; }
                }
                if (adapters) {
                    RunWalk run(m.offsets, m.lora.ids, m.lora.R, (int)t.t0, (int)t.t0 + t.n);
                    while (run.next()) {
                        for (int rs = 0; rs < rsteps; ++rs) {
                            if (!tc::mbar_wait(&empty[stage], phase ^ 1, abort)) break;
                            tc::mbar_arrive(&full[stage]);
                            if (++stage == S::STAGES) { stage = 0; phase ^= 1; }
                        }
                    }
                }
            }
            __syncwarp();
            if (split > 1) {
                tc::cluster_sync();
                tc::cluster_sync();
                if (lane == 0) tc::mbar_wait(tdone, dphase, abort);
                dphase ^= 1;
                __syncwarp();
            }
        }
        if (lane == 0 && tiled && *abort && issued > 0) {
            // loads still in flight land before the block can exit
            const long long from = clock64();
            while (clock64() - from < 20000000ll) {
            }
        }
    } else {
        int stage = 0;
        uint32_t phase = 0;
        for (int u = group; u < tiles; u += ngroups) {
            if (lane == 0 && !*abort) {
                const MmTile t = mm_tile(p, table, tiles_out, u);
                const uint32_t id = tc::idesc_f16_f32(Half2<T>::kType, MM_LANES, t.n16, DIR, 0);
                bool ok = true;
                for (int step = k0; step < k1; ++step) {
                    if (!tc::mbar_wait(&full[stage], phase, abort)) { ok = false; break; }
                    tc::fence_after_sync();
                    const uint32_t sb = tc::smem_u32(smem + stage * S::STAGE);
#pragma unroll
                    for (int kk = 0; kk < MM_BK / 16; ++kk) {
                        const uint64_t bd = tc::desc_sw128(sb + kk * 32, 16, 1024);
                        const uint32_t acc = (step > k0 || kk > 0) ? 1u : 0u;
                        if constexpr (DIR == 0)
                            tc::mma_f16_ts(tmem, tmem + MM_COLS + stage * 32 + kk * 8, bd, id, acc);
                        else
                            tc::mma_bf16(tmem, tc::desc_sw128(sb + MM_B_BYTES + kk * 2048, MM_BOX, 1024), bd, id, acc);
                    }
                    tc::mma_commit(&empty[stage]);
                    if (++stage == S::STAGES) { stage = 0; phase ^= 1; }
                }
                if (ok && adapters) {
                    RunWalk run(m.offsets, m.lora.ids, m.lora.R, (int)t.t0, (int)t.t0 + t.n);
                    while (ok && run.next()) {
                        const int b0 = (run.begin - (int)t.t0) & ~15, b1 = ((run.end - (int)t.t0) + 15) & ~15;
                        const uint32_t rid = tc::idesc_f16_f32(Half2<T>::kType, MM_LANES, b1 - b0, DIR, 0);
                        for (int rs = 0; rs < rsteps; ++rs) {
                            if (!tc::mbar_wait(&full[stage], phase, abort)) { ok = false; break; }
                            tc::fence_after_sync();
                            const uint32_t st = tc::smem_u32(smem + stage * S::STAGE);
                            const uint32_t sb = st + b0 * 128;
                            const int kks = (min(MM_BK, two_r - rs * MM_BK) + 15) / 16;
                            for (int kk = 0; kk < kks; ++kk) {
                                const uint64_t bd = tc::desc_sw128(sb + kk * 32, 16, 1024);
                                if constexpr (DIR == 0)
                                    tc::mma_f16_ts(tmem + b0, tmem + MM_COLS + stage * 32 + kk * 8, bd, rid, 1u);
                                else
                                    tc::mma_bf16(tmem + b0, tc::desc_sw128(st + MM_B_BYTES + kk * 2048, MM_BOX, 1024),
                                                 bd, rid, 1u);
                            }
                            tc::mma_commit(&empty[stage]);
                            if (++stage == S::STAGES) { stage = 0; phase ^= 1; }
                        }
                    }
                }
                if (ok) tc::mma_commit(tfull);
            }
            __syncwarp();
            if (split > 1) {
                tc::cluster_sync();
                tc::cluster_sync();
            }
        }
        if (lane == 0) {
            // every MMA issued completes before TMEM is released
            tc::mma_commit(drain);
            volatile int never = 0;
            tc::mbar_wait(drain, 0, &never);
        }
    }

    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (split > 1) tc::cluster_sync();      // no block leaves while others read its sums
    if (*abort && threadIdx.x == 0) set_status(m.status, GPTQ_ERR_TIMEOUT);
    if (warp == 9) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, MM_TMEM);
    }
}

template <typename T, int B, int DIR>
static gptq_status launch_tc(const CUtensorMap &map, const MmTcArg &p, int blocks, cudaStream_t st) {
    return launch_pdl(k_matmul_tc<T, B, DIR>, dim3(blocks), MM_THREADS, MmShape<DIR>::SMEM, p.split, st,
                      map, p);
}

template <typename T, int DIR>
static gptq_status launch_bits(const CUtensorMap &map, const MmTcArg &p, int bits, int blocks,
                               cudaStream_t st) {
    switch (bits) {
        case 2: return launch_tc<T, 2, DIR>(map, p, blocks, st);
        case 3: return launch_tc<T, 3, DIR>(map, p, blocks, st);
        case 4: return launch_tc<T, 4, DIR>(map, p, blocks, st);
        default: return launch_tc<T, 8, DIR>(map, p, blocks, st);
    }
}

// dir 0: Y = X W^T, 1: dX = dY W.
gptq_status matmul_tc(const MatmulArg &m, int dir, int dtype, int bits, cudaStream_t st) {
    MmTcArg p{};
    p.m = m;
    p.out = dir == 0 ? m.w.N : m.w.K;
    p.inner = dir == 0 ? m.w.K : m.w.N;
    p.E = m.lora.R > 0 ? 1 : m.w.E;
    p.fold = (dir == 1 || m.w.groups > 0 || m.lora.R > 0) ? 1 : 0;
    p.vec = aligned(m.w.words, 16) && m.w.ldw % 4 == 0;
    p.cols = MM_COLS;
    const int sms = device_sms();
    const int64_t tiles_out = (p.out + MM_LANES - 1) / MM_LANES;
    const int steps = (p.inner + MM_BK - 1) / MM_BK;
    // row tiles there can be, at most: one of each range that has a row, and the full ones
    const int64_t row_tiles = std::min<int64_t>(p.E, m.M) + m.M / MM_COLS;
    p.split = 1;
    while (p.split < 8 && tiles_out * row_tiles * p.split * 2 <= sms && steps >= 8 * p.split) p.split *= 2;
    CUtensorMap map{};
    p.box_rows = m.M / p.E <= 32 ? 32 : 64;
    if (!rows_map(&map, m.X, dtype, m.M, p.inner, m.ldx, p.box_rows)) p.box_rows = 0;
    const int64_t groups = std::min<int64_t>(tiles_out * row_tiles, sms / p.split);
    const int blocks = (int)std::max<int64_t>(1, groups) * p.split;
    if (dtype == GPTQ_BF16)
        return dir == 0 ? launch_bits<__nv_bfloat16, 0>(map, p, bits, blocks, st)
                        : launch_bits<__nv_bfloat16, 1>(map, p, bits, blocks, st);
    return dir == 0 ? launch_bits<__half, 0>(map, p, bits, blocks, st)
                    : launch_bits<__half, 1>(map, p, bits, blocks, st);
}

}  // namespace gptq
