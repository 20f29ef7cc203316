// Products over the rows of each range: G_e (+)= sum over t of P[t]^T Q[t], fp32. The experts'
// weight gradients (P = dY, Q = X), and the adapters' gradients, where the range of an adapter
// is the rows of all requests that use it and Q is the rank-space matrix as 16-bit parts side by
// side, whose products are added in the epilogue.
//
// Both operands come straight from row-major matrices: rows are the contraction, so a box of
// 128 rows x 64 columns in the 128-byte swizzle is an MN-major operand. The 128-row steps of a
// range are accumulated in TMEM. Range ends do not fall on step borders: a step that a range ends
// in lands on a barrier of its own, a warp sets the rows that belong to others to zero in shared
// memory, in both operands (infinities in one would meet zeros of the other), and passes it on.
//
// PAIR: two blocks share a tile of 256 columns of P (128 TMEM lanes each) x 256 of Q
// (cta_group::2): each loads its own columns of P and half of Q's, 64 KB a step. Single blocks
// take 128 columns of P x up to 256 of Q: narrow Q (adapters), and products with few tiles.
//
// The tensor core's fp32 accumulation rounds each step the same way, so a chain is 512 rows (32
// MMAs) only: two accumulators in turn, and the epilogue adds each chain to its sums in registers,
// in fp32 to nearest and in order. Mean error over 1,024 rows: 1.7e-6 in one chain, 4.7e-7 in
// chains of 512 (plain fp32 sums: 3.4e-7), 2.5e-7 in chains of 256, at 245, 275 and 310 us side by
// side for eight experts of 4,096 x 4,096 (chains of 512: 338 to 349 us under a full load's clocks, the
// tensor pipe 48 % busy: products wait for accumulators, whose readers wait for TMEM). Nothing is added across blocks, so results do not change from
// run to run.
// Outputs leave through shared memory as tiled stores (or adds) of 32 x 32 boxes: row by row they
// took 25,000 clocks a tile, three times its products. Layouts that tiled stores refuse go row
// by row.
//
// Roles (384 threads): warp 0 tiled copies, warp 1 TMEM and MMAs, warp 2 range ends, warps 4-11
// epilogue (half of the tile's columns each four); where the layout refuses tiled copies, warps 0,
// 2 and 3 make plain ones.
#include <algorithm>

#include "matmul.cuh"

namespace gptq {

namespace {
constexpr int DW_LANES = 128, DW_COLS = 256, DW_BK = 128, DW_MAX_STAGES = 4;
constexpr int DW_BOX = 128 * 64 * 2;                            // 16 KB
constexpr int DW_EPI = 8 * 32 * 33 * 4;                         // one box (or a padded one) a warp
constexpr int DW_FIXED = DW_EPI + 1024 + 256;
constexpr int DW_THREADS = 384;
constexpr int DW_CHAIN = 4;                                     // steps of one accumulator
}  // namespace

struct DwArg {
    const void *P, *Q;        // [M][ldp], [M][ldq]
    int64_t ldp, ldq, M;
    int np, nq;               // their columns
    const int32_t *offsets;   // [R + 1] row ranges, or NULL (all M rows)
    const int32_t *list_off;  // [groups + 1] ranges of each group in list, or NULL (range g)
    const int32_t *list;
    int R, groups, L;
    const int32_t *ids;       // checked with the offsets when given
    int split;                // parts of a group's steps; each writes its own output
    // Q is `parts` parts of `rank` columns side by side, added in the epilogue (1: plain). Where they
    // do not fit a tile together (apart), a tile takes 64 columns of each, a box a part.
    int parts, rank, apart;
    const uint32_t *most;     // Q's groups are scaled by the exponents of these (AdapterGrad), or NULL
    int transposed;           // output [q][p] instead of [p][q]
    int accumulate;
    float *out;               // [split][groups][np][nq'] (or [nq'][np])
    int vec;
    int tstore;               // outputs by tiled stores
    int32_t *status;
};

// One launch does one or two products over the same rows (an adapter's two gradients).
struct DwArgs {
    DwArg a[2];
    int64_t units0, units;    // tiles of the first, of all
    int tiled, stages, boxes; // alike for both: operand ring; boxes of a stage (P's two, then Q's)
};
struct DwMaps {
    CUtensorMap p[2], q[2], o;
};

// The ranges of a group in order, cut to the steps [s0, s1) of one part.
struct StepWalk {
    const DwArg &p;
    int i, iend;              // ranges left
    int skip, left;           // steps to pass over, steps to take
    int64_t row, end;         // the current range
    __device__ __forceinline__ StepWalk(const DwArg &p_, int g, int s0, int s1) : p(p_) {
        i = p.list_off ? __ldg(p.list_off + g) : g;
        iend = p.list_off ? __ldg(p.list_off + g + 1) : g + 1;
        skip = s0;
        left = s1 - s0;
        row = end = 0;
    }
    static __device__ __forceinline__ void range(const DwArg &p, int i, int64_t &b, int64_t &e) {
        const int s = p.list ? __ldg(p.list + i) : i;
        b = p.offsets ? __ldg(p.offsets + s) : 0;
        e = p.offsets ? __ldg(p.offsets + s + 1) : p.M;
    }
    static __device__ __forceinline__ int total(const DwArg &p, int g) {
        int i = p.list_off ? __ldg(p.list_off + g) : g;
        const int iend = p.list_off ? __ldg(p.list_off + g + 1) : g + 1;
        int n = 0;
        for (; i < iend; ++i) {
            int64_t b, e;
            range(p, i, b, e);
            n += (int)((e - b + DW_BK - 1) / DW_BK);
        }
        return n;
    }
    // The next step: its first row and how many rows it has.
    __device__ __forceinline__ bool next(int64_t &r, int &n) {
        if (left <= 0) return false;
        while (row >= end) {
            if (i >= iend) return false;
            range(p, i++, row, end);
            const int steps = (int)((end - row + DW_BK - 1) / DW_BK);
            const int pass = min(skip, steps);
            row += (int64_t)pass * DW_BK;
            skip -= pass;
        }
        r = row;
        n = (int)min((int64_t)DW_BK, end - row);
        row += DW_BK;
        --left;
        return true;
    }
};

// 128 rows x 64 columns from (r0, c0) into a swizzled box; zeros past `rows` or `cols`.
template <typename T>
__device__ __forceinline__ void dw_plain_box(uint8_t *dst, const T *x, int64_t ld, int64_t r0, int rows,
                                             int c0, int cols, bool vec, int tid, int nthr) {
    for (int i = tid; i < DW_BK * 8; i += nthr) {
        const int r = i >> 3, q = i & 7, c = c0 + 8 * q;
        uint32_t v[4] = {0u, 0u, 0u, 0u};
        if (r < rows && c < cols) {
            const T *src = x + (r0 + r) * ld + c;
            if (vec && c + 8 <= cols) {
                const uint4 y = __ldg(reinterpret_cast<const uint4 *>(src));
                v[0] = y.x; v[1] = y.y; v[2] = y.z; v[3] = y.w;
            } else {
                const unsigned short *s = reinterpret_cast<const unsigned short *>(src);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e < cols) v[e >> 1] |= (uint32_t)__ldg(s + e) << (16 * (e & 1));
            }
        }
        *reinterpret_cast<uint4 *>(dst + r * 128 + ((q ^ (r & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

template <typename T, bool PAIR>
__global__ void __launch_bounds__(DW_THREADS, 1)
    k_matmul_dw(const __grid_constant__ DwMaps maps, const __grid_constant__ DwArgs args) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const DwArg &first_arg = args.a[0];
    const int stages = args.stages, stage_bytes = args.boxes * DW_BOX;
    float *epi = reinterpret_cast<float *>(smem + stages * stage_bytes);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + stages * stage_bytes + DW_EPI);
    uint64_t *empty = full + DW_MAX_STAGES;
    uint64_t *tail = empty + DW_MAX_STAGES;     // copies of steps that a range ends in
    uint64_t *tfull = tail + DW_MAX_STAGES;
    uint64_t *tempty = tfull + 2;
    uint64_t *drain = tempty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *refuse = reinterpret_cast<int *>(tmem_slot + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? tc::cluster_ctarank() : 0u;
    if (threadIdx.x == 0) {
        // tiled: the copies' warp of each block, or its warp for range ends; plain: three warps each
        for (int s = 0; s < stages; ++s) {
            tc::mbar_init(&full[s], (args.tiled ? 1 : 3) * (PAIR ? 2 : 1));
            tc::mbar_init(&empty[s], 1);
            tc::mbar_init(&tail[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&tfull[b], 1);
            tc::mbar_init(&tempty[b], PAIR ? 16 : 8);
        }
        tc::mbar_init(drain, 1);
        *abort = 0;
        *refuse = 0;
        tc::fence_mbar_init();
        if (args.tiled) {
            tc::prefetch_tmap(&maps.p[0]);
            tc::prefetch_tmap(&maps.q[0]);
        }
    }
    if (warp == 1) {
        if constexpr (PAIR) tc::tmem_alloc_pair(tmem_slot, 512);
        else tc::tmem_alloc(tmem_slot, 512);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    grid_dependency();
    if (threadIdx.x == DW_THREADS - 1 && failed(first_arg.status)) *refuse = 2;
    bool bad = first_arg.offsets && offsets_bad(first_arg.offsets, first_arg.R, first_arg.M, threadIdx.x, DW_THREADS);
    if (first_arg.ids) bad |= ids_bad(first_arg.ids, first_arg.R, first_arg.L, threadIdx.x, DW_THREADS);
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0) {
        *refuse = 1;
        set_status(first_arg.status, GPTQ_ERR_ARG);
    }
    __syncthreads();
    if constexpr (PAIR) tc::cluster_sync();     // both blocks' barriers and refusal are in place
    int skip = *refuse;
    if constexpr (PAIR) skip = (int)tc::ld_shared_cluster(tc::mapa_shared(tc::smem_u32(refuse), 0));

    constexpr int PW = PAIR ? 2 * DW_LANES : DW_LANES;
    const int64_t units = skip ? 0 : args.units;
    const int64_t first = blockIdx.x / (PAIR ? 2 : 1), by = gridDim.x / (PAIR ? 2 : 1);
    // unit -> product, group, part of its steps, this block's first columns of P and Q (operand),
    // tiles of P fastest
    struct Unit {
        int which, g, part, s0, s1, pc, qc, qb, cols;   // qb boxes of Q from qc, qstep apart; the tile's columns
        int qt, qw, qstep, nout;                        // tile of Q, outputs' columns of a tile, of all
    };
    auto unit = [&](int64_t u) {
        Unit t;
        t.which = u >= args.units0 ? 1 : 0;
        const DwArg &p = args.a[t.which];
        if (t.which) u -= args.units0;
        t.nout = p.parts > 1 ? p.rank : p.nq;
        t.qw = p.apart ? 64 : DW_COLS;
        t.qstep = p.apart ? p.rank : 64;
        // (the host keeps the units below 2^31)
        const unsigned tp = (p.np + PW - 1) / PW, tq = p.apart ? (t.nout + 63) / 64 : (t.nout + DW_COLS - 1) / DW_COLS;
        const unsigned v = (unsigned)u, w = v / tp, x = w / tq;
        t.pc = (int)(v - w * tp) * PW + (int)rank * DW_LANES;
        t.qt = (int)(w - x * tq);
        t.g = (int)(p.split > 1 ? x / (unsigned)p.split : x);
        t.part = (int)x - t.g * p.split;
        const int n = StepWalk::total(p, t.g);
        t.s0 = (int)((int64_t)n * t.part / p.split);
        t.s1 = (int)((int64_t)n * (t.part + 1) / p.split);
        // columns that the MMAs take: multiples of 16 (a pair: all 256, zeros past Q's end)
        t.cols = PAIR ? DW_COLS : p.apart ? p.parts * 64 : min(DW_COLS, (p.nq - t.qt * DW_COLS + 15) & ~15);
        t.qc = t.qt * t.qw + (PAIR ? (int)rank * (DW_COLS / 2) : 0);
        t.qb = PAIR ? 2 : (t.cols + 63) / 64;
        return t;
    };
    auto arrive_full = [&](int stage) {
        if (PAIR && rank != 0) tc::mbar_arrive_remote(tc::mapa_shared(tc::smem_u32(&full[stage]), 0));
        else tc::mbar_arrive(&full[stage]);
    };

    if (warp == 0 && args.tiled) {
        // the whole warp walks, one elected lane issues
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int64_t u = first; u < units && ok; u += by) {
            const Unit t = unit(u);
            StepWalk walk(args.a[t.which], t.g, t.s0, t.s1);
            int64_t r;
            int n;
            const uint32_t bytes = (2 + t.qb) * DW_BOX;
            const CUtensorMap *pmap = &maps.p[t.which], *qmap = &maps.q[t.which];
            while (walk.next(r, n)) {
                ok = __all_sync(~0u, tc::mbar_wait(&empty[stage], phase ^ 1, abort));
                if (!ok) break;
                uint8_t *a = smem + stage * stage_bytes, *b = a + 2 * DW_BOX;
                const int x0 = t.pc, x1 = t.qc, y = (int)r;
                const bool ends = n < DW_BK;
                if (tc::elect_one()) {
                    if (ends || !PAIR) {
                        uint64_t *bar = ends ? &tail[stage] : &full[stage];
                        tc::mbar_arrive_expect_tx(bar, bytes);
                        for (int i = 0; i < 2; ++i) tc::tma_load_2d(a + i * DW_BOX, pmap, bar, x0 + 64 * i, y);
                        for (int i = 0; i < t.qb; ++i) tc::tma_load_2d(b + i * DW_BOX, qmap, bar, x1 + t.qstep * i, y);
                    } else {
                        if (rank == 0) tc::mbar_arrive_expect_tx(&full[stage], 2 * bytes);
                        const uint32_t fb = tc::mapa_shared(tc::smem_u32(&full[stage]), 0);
                        for (int i = 0; i < 2; ++i) tc::tma_load_2d_pair(a + i * DW_BOX, pmap, fb, x0 + 64 * i, y);
                        for (int i = 0; i < 2; ++i) tc::tma_load_2d_pair(b + i * DW_BOX, qmap, fb, x1 + 64 * i, y);
                        if (rank != 0) tc::mbar_arrive_remote(fb);
                    }
                }
                __syncwarp();
                if (++stage == stages) { stage = 0; phase ^= 1; }
            }
        }
        if (!ok) {                          // loads still in flight land before the block exits
            const long long from = clock64();
            while (clock64() - from < 20000000ll) {
            }
        }
    } else if (warp == 2 && args.tiled) {
        // steps that a range ends in: rows n .. the next multiple of 16 belong to others
        int stage = 0;
        uint32_t phases = 0;                // of the tail barriers, a bit a stage
        bool ok = true;
        for (int64_t u = first; u < units && ok; u += by) {
            const Unit t = unit(u);
            StepWalk walk(args.a[t.which], t.g, t.s0, t.s1);
            int64_t r;
            int n;
            while (ok && walk.next(r, n)) {
                if (n < DW_BK) {
                    ok = __all_sync(~0u, tc::mbar_wait(&tail[stage], (phases >> stage) & 1u, abort));
                    if (!ok) break;
                    phases ^= 1u << stage;
                    uint8_t *a = smem + stage * stage_bytes;
                    const int zero = ((n + 15) & ~15) - n, boxes = 2 + t.qb;
                    for (int i = lane; i < zero * 8 * boxes; i += 32) {
                        const int box = i / (zero * 8), j = i - box * zero * 8;
                        *reinterpret_cast<uint4 *>(a + box * DW_BOX + (n + (j >> 3)) * 128 + ((j & 7) << 4)) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    tc::fence_async_shared();
                    __syncwarp();
                    if (lane == 0) arrive_full(stage);
                }
                if (++stage == stages) stage = 0;
            }
        }
    } else if (warp == 1) {
        if (!PAIR || rank == 0) {
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            const uint64_t ad0 = tc::desc_sw128(tc::smem_u32(smem), DW_BOX, 1024);
            const uint64_t bd0 = tc::desc_sw128(tc::smem_u32(smem) + 2 * DW_BOX, DW_BOX, 1024);
            auto commit = [&](uint64_t *bar) {
                if (tc::elect_one()) {
                    if constexpr (PAIR) tc::mma_commit_both(bar);
                    else tc::mma_commit(bar);
                }
                __syncwarp();
            };
            for (int64_t u = first; u < units && ok; u += by) {
                const Unit t = unit(u);
                StepWalk walk(args.a[t.which], t.g, t.s0, t.s1);
                int64_t r;
                int n;
                const uint32_t id = tc::idesc_f16_f32(Half2<T>::kType, PW, t.cols, 1, 1);
                int chain = 0;
                while (ok && walk.next(r, n)) {
                    if (chain == 0) {
                        ok = __all_sync(~0u, tc::mbar_wait(&tempty[acc], acc_phase ^ 1, abort));
                        if (!ok) break;
                    }
                    ok = __all_sync(~0u, tc::mbar_wait(&full[stage], phase, abort));
                    if (!ok) break;
                    tc::fence_after_sync();
                    const uint64_t ad = ad0 + (uint32_t)(stage * stage_bytes >> 4);
                    const uint64_t bd = bd0 + (uint32_t)(stage * stage_bytes >> 4);
                    const uint32_t d = tmem + acc * DW_COLS;
                    const int kks = (n + 15) / 16;
                    if (tc::elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < DW_BK / 16; ++kk) {
                            if (kk >= kks) break;
                            const uint32_t add = (chain > 0 || kk > 0) ? 1u : 0u;
                            if constexpr (PAIR) tc::mma_bf16_pair(d, ad + kk * 128, bd + kk * 128, id, add);
                            else tc::mma_bf16(d, ad + kk * 128, bd + kk * 128, id, add);
                        }
                    }
                    __syncwarp();
                    commit(&empty[stage]);
                    if (++stage == stages) { stage = 0; phase ^= 1; }
                    if (++chain == DW_CHAIN) {
                        commit(&tfull[acc]);
                        chain = 0;
                        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
                    }
                }
                if (ok && chain > 0) {
                    commit(&tfull[acc]);
                    if (++acc == 2) { acc = 0; acc_phase ^= 1; }
                }
            }
            if (tc::elect_one()) {
                if constexpr (PAIR) tc::mma_commit_pair(tc::mapa_shared(tc::smem_u32(drain), 0));
                else tc::mma_commit(drain);
                volatile int never = 0;
                tc::mbar_wait(drain, 0, &never);
            }
        }
    } else if (warp >= 4) {
        const int quad = warp & 3, side = (warp >> 2) - 1;
        uint8_t *box = reinterpret_cast<uint8_t *>(epi) + (warp - 4) * 4096;            // swizzled, or
        float *buf = epi + (warp - 4) * 32 * 33;                                        // [32][33]
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (int64_t u = first; u < units && ok; u += by) {
            const Unit t = unit(u);
            const DwArg &p = args.a[t.which];
            const int nout = t.nout, spacing = p.apart ? 64 : nout;     // of the parts in the accumulator
            // this warp's columns of a tile: up to 128 from `side` times 128 (parts: 64)
            const int own = p.parts > 1 ? 64 : 128;
            float *out = p.out + ((int64_t)t.part * p.groups + t.g) * p.np * nout;
            const int r0 = t.pc + quad * 32, c0 = side * own;
            const int qn = max(0, min(own, min(t.qw, nout - t.qt * t.qw) - c0));            // columns it has
            const int chains = (t.s1 - t.s0 + DW_CHAIN - 1) / DW_CHAIN;                     // none: zeros
            float sum[128];
#pragma unroll
            for (int i = 0; i < 128; ++i) sum[i] = 0.f;
            for (int c = 0; c < chains; ++c) {
                ok = __all_sync(~0u, tc::mbar_wait(&tfull[acc], acc_phase, abort));
                if (!ok) break;
                tc::fence_after_sync();
                const uint32_t at = tmem + acc * DW_COLS + c0 + ((uint32_t)(quad * 32) << 16);
#pragma unroll
                for (int cb = 0; cb < 8; ++cb) {
                    if (cb * 16 >= qn) break;
#pragma unroll 1
                    for (int h = 0; h < p.parts; ++h) {
                        uint32_t v[16];
                        tc::tmem_ld_32x32b_x16(at + cb * 16 + h * spacing, v);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) sum[cb * 16 + i] += __uint_as_float(v[i]);
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR && rank != 0) tc::mbar_arrive_remote(tc::mapa_shared(tc::smem_u32(&tempty[acc]), 0));
                    else tc::mbar_arrive(&tempty[acc]);
                }
                if (++acc == 2) { acc = 0; acc_phase ^= 1; }
            }
            if (!ok) break;
            if (chains == 0 && p.accumulate) continue;
            if (p.most) {                           // 2^(e - 141) as two normal factors
                const int e = (int)(__ldcg(p.most + t.g) >> 23) - 141, e1 = e >> 1, e2 = e - e1;
                const float f1 = __uint_as_float((uint32_t)(127 + e1) << 23), f2 = __uint_as_float((uint32_t)(127 + e2) << 23);
#pragma unroll
                for (int i = 0; i < 128; ++i) sum[i] = sum[i] * f1 * f2;
            }
#pragma unroll
            for (int cb = 0; cb < 4; ++cb) {
                if (cb * 32 >= qn) break;
                const int q0 = t.qt * t.qw + c0 + cb * 32, cols = min(32, qn - cb * 32);
                if (p.tstore) {
                    // row = lane, 16-byte piece q at q ^ (lane & 7), once the box is free again
                    if (lane == 0) tc::bulk_wait_read<0>();
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        *reinterpret_cast<float4 *>(box + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                            make_float4(sum[cb * 32 + 4 * q], sum[cb * 32 + 4 * q + 1], sum[cb * 32 + 4 * q + 2],
                                        sum[cb * 32 + 4 * q + 3]);
                    tc::fence_async_shared();
                    __syncwarp();
                    if (lane == 0 && r0 < p.np) {
                        if (p.accumulate) tc::tma_reduce_add_3d(&maps.o, box, q0, r0, t.g);
                        else tc::tma_store_3d(&maps.o, box, q0, r0, t.g);
                        tc::bulk_commit();
                    }
                } else if (p.transposed) {
                    if (r0 + lane < p.np) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i < cols) {
                                float *d = out + (int64_t)(q0 + i) * p.np + r0 + lane;
                                *d = p.accumulate ? *d + sum[cb * 32 + i] : sum[cb * 32 + i];
                            }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) buf[lane * 33 + i] = sum[cb * 32 + i];
                    __syncwarp();
                    const int rows = min(32, p.np - r0);
                    if (lane < cols) {
                        float *d = out + (int64_t)r0 * nout + q0 + lane;
                        if (p.accumulate) {
#pragma unroll 8
                            for (int i = 0; i < rows; ++i) d[(int64_t)i * nout] += buf[i * 33 + lane];
                        } else {
#pragma unroll 8
                            for (int i = 0; i < rows; ++i) d[(int64_t)i * nout] = buf[i * 33 + lane];
                        }
                    }
                    __syncwarp();
                }
            }
        }
        if (lane == 0) tc::bulk_wait_all();
    } else if (!args.tiled) {
        const int tid = (warp == 0 ? 0 : warp - 1) * 32 + lane;         // warps 0, 2, 3
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int64_t u = first; u < units && ok; u += by) {
            const Unit t = unit(u);
            const DwArg &p = args.a[t.which];
            const T *P = static_cast<const T *>(p.P), *Q = static_cast<const T *>(p.Q);
            StepWalk walk(args.a[t.which], t.g, t.s0, t.s1);
            int64_t r;
            int n;
            while (walk.next(r, n)) {
                ok = __all_sync(~0u, tc::mbar_wait(&empty[stage], phase ^ 1, abort));
                if (!ok) break;
                uint8_t *a = smem + stage * stage_bytes, *b = a + 2 * DW_BOX;
                for (int i = 0; i < 2; ++i)
                    dw_plain_box<T>(a + i * DW_BOX, P, p.ldp, r, n, t.pc + 64 * i, p.np, (p.vec & 1) != 0, tid, 96);
                for (int i = 0; i < t.qb; ++i)
                    dw_plain_box<T>(b + i * DW_BOX, Q, p.ldq, r, n, t.qc + t.qstep * i, p.nq, (p.vec & 2) != 0, tid, 96);
                tc::fence_async_shared();
                __syncwarp();
                if (lane == 0) arrive_full(stage);
                if (++stage == stages) { stage = 0; phase ^= 1; }
            }
        }
    }

    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if constexpr (PAIR) tc::cluster_sync();     // neither block leaves while the pair uses its memory
    if (*abort && threadIdx.x == 0) set_status(first_arg.status, GPTQ_ERR_TIMEOUT);
    if (warp == 1) {
        tc::fence_after_sync();
        if constexpr (PAIR) tc::tmem_dealloc_pair(tmem, 512);
        else tc::tmem_dealloc(tmem, 512);
    }
}

// out[i] = the parts' sum, parts in order, for one or two outputs.
struct SumArg {
    const float *parts[2];
    float *out[2];
    int64_t n[2];
    int split[2];
    const int32_t *list_off;            // -1 first: refused
};
__global__ void __launch_bounds__(256) k_sum_parts(const __grid_constant__ SumArg p, const int32_t *status) {
    grid_dependency();
    if (failed(status) || __ldcg(p.list_off) < 0) return;
    int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int w = i >= p.n[0] ? 1 : 0;
    if (w) i -= p.n[0];
    if (i >= p.n[w]) return;
    float s = 0.f;
    for (int k = 0; k < p.split[w]; ++k) s += p.parts[w][k * p.n[w] + i];
    p.out[w][i] = s;
}

// The outputs [groups][np][nq] as boxes of 32 x 32 of one group.
static bool out_map(CUtensorMap *map, const DwArg &p) {
    EncodeTiled enc = encode_tiled();
    if (!enc || p.parts > 1 || p.split != 1 || !aligned(p.out, 16) || p.nq % 4 != 0) return false;
    const cuuint64_t dim[3] = {(cuuint64_t)p.nq, (cuuint64_t)p.np, (cuuint64_t)p.groups};
    const cuuint64_t stride[2] = {(cuuint64_t)p.nq * 4, (cuuint64_t)p.nq * 4 * p.np};
    const cuuint32_t box[3] = {32, 32, 1}, step[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p.out, dim, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static gptq_status launch_dw(DwArg *a, int count, int dtype, cudaStream_t st) {
    DwMaps maps{};
    DwArgs args{};
    const DwArg &p = a[0];
    auto units = [&](const DwArg &p, int pw) {
        const int nout = p.parts > 1 ? p.rank : p.nq, qw = p.apart ? 64 : DW_COLS;
        return (int64_t)((p.np + pw - 1) / pw) * ((nout + qw - 1) / qw) * p.groups * p.split;
    };
    // pairs where both operands fill their tiles and there are pairs enough for the machine
    const bool pair = count == 1 && p.parts == 1 && p.np > DW_LANES && p.nq > DW_COLS / 2 &&
                      2 * units(p, 2 * DW_LANES) >= device_sms();
    args.tiled = 1;
    for (int i = 0; i < count; ++i) {
        DwArg &p = a[i];
        p.tstore = count == 1 && out_map(&maps.o, p);
        args.tiled &= rows_map(&maps.p[i], p.P, dtype, p.M, p.np, p.ldp, DW_BK) &&
                      rows_map(&maps.q[i], p.Q, dtype, p.M, p.nq, p.ldq, DW_BK);
        p.vec = (aligned(p.P, 16) && p.ldp % 8 == 0 ? 1 : 0) | (aligned(p.Q, 16) && p.ldq % 8 == 0 ? 2 : 0);
        args.a[i] = p;
        args.units += units(p, pair ? 2 * DW_LANES : DW_LANES);
        if (i == 0) args.units0 = args.units;
    }
    if (args.units > 0x7fffffff) return GPTQ_ERR_ARG;
    args.boxes = pair ? 4 : p.apart ? 2 + p.parts : 2 + (std::min(p.nq, DW_COLS) + 63) / 64;
    args.stages = std::min(DW_MAX_STAGES, (int)((SMEM_MOST - DW_FIXED) / (args.boxes * DW_BOX)));
    const size_t smem = (size_t)args.stages * args.boxes * DW_BOX + DW_FIXED;
    const int blocks = (int)std::max<int64_t>(1, std::min<int64_t>(args.units, device_sms() / (pair ? 2 : 1))) * (pair ? 2 : 1);
    if (dtype == GPTQ_BF16)
        return pair ? launch_pdl(k_matmul_dw<__nv_bfloat16, true>, dim3(blocks), DW_THREADS, smem, SMEM_MOST, 2, st, maps, args)
                    : launch_pdl(k_matmul_dw<__nv_bfloat16, false>, dim3(blocks), DW_THREADS, smem, SMEM_MOST, 1, st, maps, args);
    return pair ? launch_pdl(k_matmul_dw<__half, true>, dim3(blocks), DW_THREADS, smem, SMEM_MOST, 2, st, maps, args)
                : launch_pdl(k_matmul_dw<__half, false>, dim3(blocks), DW_THREADS, smem, SMEM_MOST, 1, st, maps, args);
}

// G[e] (+)= dY^T X over the rows of range e.
gptq_status matmul_dw(float *G, const void *dY, int64_t lddy, const void *X, int64_t ldx, int dtype,
                      int64_t M, int N, int K, int E, const int32_t *offsets, int accumulate,
                      int32_t *status, cudaStream_t st) {
    DwArg p{};
    p.P = dY; p.ldp = lddy; p.np = N;
    p.Q = X; p.ldq = ldx; p.nq = K;
    p.M = M;
    p.offsets = offsets;
    p.R = p.groups = E;
    p.split = p.parts = 1;
    p.accumulate = accumulate;
    p.out = G;
    p.status = status;
    return launch_dw(&p, 1, dtype, st);
}

// Parts of an adapter's rows: enough blocks to fill the machine, at least 512 rows a part.
int adapter_parts(int64_t M, int L, int width) {
    const int64_t tiles = (int64_t)L * ((width + DW_LANES - 1) / DW_LANES);
    int64_t s = (device_sms() + tiles - 1) / std::max<int64_t>(1, tiles);
    s = std::min(s, M / 512);
    return (int)std::max<int64_t>(1, std::min<int64_t>(s, 16));
}

// The adapters' gradients, the one or both that are wanted, over the rows of the requests listed for
// each: dB[a][n][j] = sum dY[t][n] T[t][j], dA[a][j][k] = sum U[t][j] X[t][k].
gptq_status adapter_gradients(const AdapterGrad *grads, int count, int rank, int dtype, int64_t M,
                              const int32_t *offsets, const int32_t *ids, const int32_t *list_off,
                              const int32_t *list, int R, int L, int32_t *status, cudaStream_t st) {
    DwArg a[2] = {};
    SumArg sum{};
    sum.list_off = list_off;
    int64_t n = 0;
    for (int i = 0; i < count; ++i) {
        const AdapterGrad &g = grads[i];
        DwArg &p = a[i];
        p.P = g.P; p.ldp = g.ldp; p.np = g.np;
        p.parts = g.halves;
        p.rank = rank;
        p.Q = g.Q; p.ldq = g.ldq; p.nq = p.parts * rank;
        p.most = g.most;
        p.apart = p.nq > DW_COLS;
        p.M = M;
        p.offsets = offsets;
        p.list_off = list_off;
        p.list = list;
        p.R = R;
        p.groups = p.L = L;
        p.ids = ids;
        p.split = adapter_parts(M, L, g.np);
        p.transposed = g.transposed;
        p.out = p.split > 1 ? g.parts : g.out;
        p.status = status;
        if (p.split > 1) {
            sum.parts[i] = g.parts;
            sum.out[i] = g.out;
            sum.n[i] = (int64_t)L * g.np * rank;
            sum.split[i] = p.split;
            n += sum.n[i];
        }
    }
    gptq_status s = launch_dw(a, count, dtype, st);
    if (s != GPTQ_OK || n == 0) return s;
    return launch_pdl(k_sum_parts, dim3((unsigned)((n + 255) / 256)), 256, 0, 0, 1, st, sum, (const int32_t *)status);
}

}  // namespace gptq
