// Packed-weight products on the tensor cores: Y[t] = W^_e X[t] (forward) and
// dX[t] = W^_e^T dY[t] (input gradient) over row ranges of experts, with the low-rank
// adapters of the rows' requests added in the same accumulators.
//
// One tile is 128 output channels (TMEM lanes) x up to 256 rows (TMEM columns): the weights
// are the A operand, so a tile's row count is free (multiples of 16) and a short range of an
// expert costs no more matrix work than it has rows. The contraction runs in steps of 128, one
// stage of the operand rings and one round of barriers each (with steps of 64 the rounds, not the
// MMAs, set the pace: the warp that issues the copies of X needed 690 clocks a round):
//   forward         a thread unpacks 64 codes of its own channel (lane) and stores them into
//                   TMEM, where the MMA reads A; only the rows X go through shared memory.
//   input gradient  the contraction runs over the packed rows n, so a thread unpacks 64 codes
//                   of one n into a [n][k] tile of shared memory, read as an MN-major A.
// PAIR: two blocks share a tile of 256 channels (cta_group::2): each unpacks its own 128
// channels and loads half of the rows' operand, which the pair's MMAs read from both, so the
// operand traffic of an SM halves; that is what bounds the single-block form (one block's
// MMAs alone, without unpacking, ran at 1.25 PFLOP/s on an 8,192 x 4,096 x 14,336 product).
//
// Scales: with one scale a channel the forward product multiplies exact integers c - z and the
// scale enters in fp32 at the end. Where the scale changes along the contraction (input
// groups, the input gradient) or adapters share the accumulators (their terms carry no scale), each
// weight s (c - z) is rounded once to the rows' 16-bit type, as a dequantised layer in that type would
// hold it: bf16 outputs are then 2.4e-3 off 64 bits in the mean instead of 1.7e-3, fp16 2.9e-4 instead
// of 2.1e-4. Two operands a weight would not lose that, at twice the products.
//
// Adapters: after the steps of W^, each run of rows with one adapter adds
// sum_j P_a[.][j] T[t][j] over the run's columns alone (runs are widened to the MMA's column borders,
// the rows there that belong to others are zero in shared memory; an adapter's infinities and NaN,
// which would meet those zeros, and the parts of T one by one, are left out of these steps and added to
// the run's own rows at the end). These steps are bf16 ones for either type of rows: the contraction is
// [P | P] against two parts of T (16 bits), and for fp16 rows, whose P are two bf16 numbers exactly,
// [P's first | P's second | P's first] against T's first, first and second part (16 bits; the outputs
// have 11, and the weights' rounding to fp16 beside it 11). Runs of fewer than 16 rows (requests that decode) are added by the threads that write
// the outputs: as matrix steps they cost about 1.3 us each.
//
// Order: the tiles of a range run rows first, so that blocks that work at the same time read
// different rows of X and the same (few) words; with channels first every block asked the L2
// for the same lines of X at once, and the pair's MMAs waited (54 % tensor-pipe cycles).
//
// Roles (640 threads): warps 0-11 unpack, in three sets of four that take the halves of the steps
// in turn (integer operations issue every other clock, so two warps a scheduler spent most of a
// step in one another's latencies; three do not); warps 12-15 write the outputs; warp 16 issues
// the tiled copies of X; warp 17 owns TMEM and issues the MMAs; warps 18-19 bring the packed words,
// 128 rows x 128 codes (a step) at a time, through a ring of their own that runs ahead across tiles.
// Tiles of at most 128 rows use two accumulators in turn, so a tile's end costs the next one nothing.
//
// 16,384 rows over eight layers of 4,096 -> 14,336, 4 bits: 1.45 to 1.51 ms with the clock that the
// power cap leaves (1.28 to 1.33 PFLOP/s). 512 rows over 32 layers of 2,048 -> 2,816, groups of 128:
// 70 us, about 1,550 clocks a step, of which 870 are issue slots (55 % busy, the integer pipe 46 %): the
// chain of one half-step, wait, read, unpack, wait, store, and what three sets leave of it. Input
// gradient of 8,192 rows over eight layers of 4,096 x 4,096, groups of 128: 319 to 331 us, about 2,200
// clocks a step; the tensor pipe is 47 % busy, the issue slots 54 %.
#pragma once

#include <algorithm>

#include "matmul.cuh"
#include "unpack_turns.h"

namespace gptq {

constexpr int MM_LANES = 128;                       // output channels of a block's tile
constexpr int MM_BK = 128;
constexpr int MM_SETS = UNPACK_SETS;                // of four unpacking warps
constexpr int MM_WARP_OUT = 4 * MM_SETS, MM_WARP_X = MM_WARP_OUT + 4, MM_WARP_MMA = MM_WARP_X + 1,
              MM_WARP_WORDS = MM_WARP_X + 2;
constexpr int MM_THREADS = (MM_WARP_WORDS + 2) * 32;
constexpr int MM_ROWS = 128;                        // rows of X that a block stages (a pair: 256)
constexpr int MM_HALF = MM_ROWS * 64 * 2;           // 64 columns of them, 16 KB
constexpr int MM_B_BYTES = 2 * MM_HALF;
constexpr int MM_A_BYTES = MM_LANES * MM_BK * 2;    // 32 KB (input gradient)
constexpr int MM_BOX = 128 * 64 * 2;                // A: 128 contraction rows x 64 columns
// The runs of one adapter in a tile that are matrix operands, found by the outputs' warps for all.
struct LoraRuns {
    int count;
    int begin[256 / LORA_SHORT], end[256 / LORA_SHORT], id[256 / LORA_SHORT];   // rows of the tile
    uint32_t starts[8], longs[8];       // a bit a row: a run starts, a long one
    int broken;                         // infinities or NaN of an adapter were left out of a step
};

constexpr int MM_CACHED = 256;                       // offsets kept in shared memory
// tiles before each range, the first offsets, and the adapters of a tile's rows (16 bits)
constexpr int MM_TABLE = ((MATMUL_MAX_EXPERTS + 4 + MM_CACHED + 4) * 4 + 256 * 2 + (int)sizeof(LoraRuns) + 15) / 16 * 16;
constexpr uint32_t MM_TMEM = 512;
constexpr int MM_MAX_STAGES = 4;                    // of 64 TMEM columns beside the accumulators

// The infinities and NaN among 8 values set to zero; whether there were any. An exponent of ones
// carries into the sign's place.
template <typename T>
__device__ __forceinline__ uint32_t nonfinite(uint32_t v) {
    constexpr uint32_t e = Half2<T>::kType == 1 ? 0x7f807f80u : 0x7c007c00u;
    return ((v & e) + (Half2<T>::kType == 1 ? 0x00800080u : 0x04000400u)) & 0x80008000u;
}
template <typename T>
__device__ __forceinline__ bool finite_only(uint4 (&y)[8]) {
    uint32_t any = 0u;
    auto clear = [&](uint32_t &v) {
        const uint32_t bad = nonfinite<T>(v);
        any |= bad;
        v &= ~((bad >> 15) * 0xffffu);
    };
#pragma unroll
    for (int j = 0; j < 8; ++j) { clear(y[j].x); clear(y[j].y); clear(y[j].z); clear(y[j].w); }
    return any != 0u;
}

// What finite_only left out, for the rows of the tile's runs, in the accumulators at `at` (this
// thread's channel).
template <typename T, int DIR>
__device__ __noinline__ void add_nonfinite(const LoraArg &l, const LoraRuns *runs, int64_t t0, int ch, int channels,
                                           uint32_t at) {
#pragma unroll 1
    for (int run = 0; run < runs->count; ++run) {
#pragma unroll 1
        for (int row = runs->begin[run]; row < runs->end[run]; ++row) {
            const unsigned short *P = static_cast<const unsigned short *>(l.P) + (int64_t)runs->id[run] * channels * l.rank +
                                      (DIR == 0 ? (int64_t)ch * l.rank : ch);
            const __nv_bfloat16 *t = l.T3 + (t0 + row) * (LORA_PARTS * l.rank);
            float add = 0.f;
            if (ch < channels) {
#pragma unroll 1
                for (int j = l.rank; j > 0; --j, ++t, P += DIR == 0 ? 1 : channels) {
                    const uint32_t v = __ldg(P);
                    if (nonfinite<T>(v) & 0x8000u)
                        add = fmaf(Half2<T>::unpack(v).x, to_f32(t[0]) + to_f32(t[l.rank]), add);
                }
            }
            __syncwarp();
            const uint32_t y = tc::tmem_ld_32x32b_x1(at + row);
            tc::tmem_ld_wait();
            tc::tmem_st_32x32b_x1(at + row, __float_as_uint(__uint_as_float(y) + add));
            tc::tmem_st_wait();
        }
    }
}

// The first bf16 parts of eight fp16 values, or what these leave (for an infinity that is a NaN).
template <typename T>
__device__ __forceinline__ uint4 bf16_part8(uint4 v, bool rest) {
    if constexpr (Half2<T>::kType != 1) {
        using H = Half2<__nv_bfloat16>;
        auto part = [&](uint32_t &x) {
            const float2 f = Half2<T>::unpack(x);
            x = H::pack(f.x, f.y);
            if (rest) {
                const float2 g = H::unpack(x);
                x = H::pack(f.x - g.x, f.y - g.y);
            }
        };
        part(v.x); part(v.y); part(v.z); part(v.w);
    }
    return v;
}

// The ring of packed words: rows of 128 codes (16 B bytes), as a tiled copy with the swizzle of that
// width lays them out (48-byte rows of 3 bits have none). A stage is what is read together: the 128
// channels of a step in the forward product, which two sets read, the 64 rows of half a step in the
// input gradient, which one does. A multiple of three stages: then a set meets the same stages always,
// and is there for every use of them (unpack_turns.h).
template <int B, int DIR>
struct MmRing {
    static constexpr int ROW = 16 * B;
    static constexpr int ROWS = DIR == 0 ? 128 : 64;
    static constexpr int STAGE = ROWS * ROW;
    // the input gradient's operand stages leave less room (4 bits with six stages: 322 us for 321)
    static constexpr int STAGES = B >= (DIR == 0 ? 8 : 4) ? 3 : 6;
    static_assert(STAGES % UNPACK_SETS == 0, "a set's stages are its own");
    static constexpr int WORDS = STAGES * STAGE;
    static constexpr int BYTES = WORDS;
    // byte offset of 16-byte (3 bits: 8-byte) piece q of row r
    static __device__ __forceinline__ int at(int r, int q) {
        return B == 2   ? r * 32 + ((q ^ ((r >> 2) & 1)) << 4)
               : B == 3 ? r * 48 + q * 8
               : B == 4 ? r * 64 + ((q ^ ((r >> 1) & 3)) << 4)
                        : r * 128 + ((q ^ (r & 7)) << 4);
    }
};

struct MmTcArg {
    MatmulArg m;
    int out, inner;       // output channels and contraction length of this direction
    int cols;             // most rows of a tile (multiple of 16)
    int box_rows;         // rows of one tiled copy of X; 0: plain loads
    int stages;           // of the operand ring
    int accs, acc_cols;   // accumulators and their distance
    int split;            // blocks of a cluster that share a tile's contraction
    int fold;             // scales folded into the weights
    int wtiled, yvec;     // packed rows by tiled copies; output rows start on 16-byte boundaries
    int epi;              // bytes of the output staging (or of the partial sums)
    int idx_table;        // g_idx: the scales of each unpacking thread's row stand in shared memory
    int E;                // row ranges
};

gptq_status matmul_tc_bf16(const CUtensorMap &map, const CUtensorMap &wmap, const MmTcArg &p, int dir, int bits, bool pair, int blocks,
                           size_t smem, cudaStream_t st);
gptq_status matmul_tc_fp16(const CUtensorMap &map, const CUtensorMap &wmap, const MmTcArg &p, int dir, int bits, bool pair, int blocks,
                           size_t smem, cudaStream_t st);

int matmul_tc_occupancy(int cluster);

// Rows [r0, r0 + rows) x columns [c0, c0 + 64) of X into the swizzled layout of a tiled copy,
// zeros past row_end or col_end: the copy for layouts that tiled copies refuse.
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

// N bytes (4, 8 or 16) to shared memory, zeros when src is NULL.
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, const void *any) {
    const int bytes = src ? N : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src ? src : any), "n"(N),
                 "r"(bytes)
                 : "memory");
}

struct MmTile {
    int e, c0;            // range, first output channel of this block
    int64_t t0;           // first row
    int n, n16;           // rows, rounded up to the columns an MMA takes (16, a pair 32)
};

// Tile u -> (range, channels, rows), rows fastest.
__device__ __forceinline__ MmTile mm_tile(const MmTcArg &p, const int *table, int tiles_out, int u,
                                          int width, int first, int grain) {
    MmTile t;
    int lo = 0, hi = p.E - 1;                       // last range whose first tile is <= u
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (table[mid] * tiles_out <= u) lo = mid;
        else hi = mid - 1;
    }
    t.e = lo;
    const int *cached = table + MATMUL_MAX_EXPERTS + 4;
    int64_t begin, end;
    if (lo < MM_CACHED) {
        begin = cached[lo];
        end = cached[lo + 1];
    } else {
        begin = __ldg(p.m.offsets + lo);
        end = __ldg(p.m.offsets + lo + 1);
    }
    const int cnt = (int)(end - begin);
    const int nt = (cnt + p.cols - 1) / p.cols;
    const int size = ((cnt + nt - 1) / nt + grain - 1) & -grain;
    const int q = u - table[lo] * tiles_out, c = q / nt, j = q - c * nt;
    t.c0 = c * width + first;
    t.t0 = begin + (int64_t)j * size;
    t.n = min(size, cnt - j * size);
    t.n16 = (t.n + grain - 1) & -grain;
    return t;
}

__device__ __forceinline__ int m_groups(const MmTcArg &p) { return p.m.w.groups; }

// A place in the ring of operand stages.
struct RingPos {
    int stage;
    uint32_t phase;
    __device__ __forceinline__ void jump(int n, int stages) {
        const int s = stage + n, w = s / stages;
        stage = s - w * stages;
        phase ^= w & 1;
    }
    __device__ __forceinline__ void advance(int stages) {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
    }
};

template <typename T, int B, int DIR, bool IDX, bool PAIR>
__global__ void __launch_bounds__(MM_THREADS, 1)
    k_matmul_tc(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                const __grid_constant__ MmTcArg p) {
    using Ring = MmRing<B, DIR>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    constexpr int stage_bytes = MM_B_BYTES + (DIR == 1 ? MM_A_BYTES : 0);
    uint8_t *words = smem + p.stages * stage_bytes;             // the words' ring
    uint8_t *epi = words + Ring::BYTES;
    int *table = reinterpret_cast<int *>(epi + p.epi);
    constexpr int UNPACKERS = MM_WARP_OUT * 32;
    float *own_scales = reinterpret_cast<float *>(epi + p.epi + MM_TABLE);     // [groups][thread]
    uint64_t *full = reinterpret_cast<uint64_t *>(epi + p.epi + MM_TABLE +
                                                  (IDX && p.idx_table ? m_groups(p) * UNPACKERS * 4 : 0));
    uint64_t *empty = full + MM_MAX_STAGES;
    uint64_t *tfull = empty + MM_MAX_STAGES;
    uint64_t *tempty = tfull + 2;
    uint64_t *ready = tempty + 2;                               // partial sums in place / read
    uint64_t *done = ready + 1;
    uint64_t *wfull = done + 1;
    uint64_t *wempty = wfull + Ring::STAGES;
    uint64_t *lfull = wempty + Ring::STAGES;                    // the tile's run list
    uint64_t *lempty = lfull + 1;
    uint64_t *drain = lempty + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *refuse = reinterpret_cast<int *>(tmem_slot + 2);

    const MatmulArg &m = p.m;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stages = p.stages;
    const int split = PAIR ? 1 : p.split;
    const int cluster = PAIR ? 2 : split;
    const uint32_t rank = cluster > 1 ? tc::cluster_ctarank() : 0u;
    const int group = blockIdx.x / cluster, ngroups = gridDim.x / cluster;
    const bool tiled = p.box_rows > 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            tc::mbar_init(&full[s], (PAIR ? 16 : 8) + (tiled ? 1 : 0));
            tc::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&tfull[b], 1);
            tc::mbar_init(&tempty[b], PAIR ? 8 : 4);
        }
        tc::mbar_init(ready, 4 * split);
        tc::mbar_init(done, 4 * split);
        for (int s = 0; s < Ring::STAGES; ++s) {
            tc::mbar_init(&wfull[s], p.wtiled ? 1 : 64);
            tc::mbar_init(&wempty[s], DIR == 0 ? 8 : 4);
        }
        tc::mbar_init(lfull, 4);
        // its readers: the unpacking warps, the X warp where it copies, the MMA warp where it issues
        tc::mbar_init(lempty, MM_WARP_OUT + (tiled ? 1 : 0) + (!PAIR || rank == 0 ? 1 : 0));
        tc::mbar_init(drain, 1);
        *abort = 0;
        *refuse = 0;
        tc::fence_mbar_init();
        if (tiled) tc::prefetch_tmap(&xmap);
        if (p.wtiled) tc::prefetch_tmap(&wmap);
    }
    if (warp == MM_WARP_MMA) {
        if constexpr (PAIR) tc::tmem_alloc_pair(tmem_slot, MM_TMEM);
        else tc::tmem_alloc(tmem_slot, MM_TMEM);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    // With adapters the kernel before this one makes T or follows the one that does; all else that
    // is read was there before it began, so only T waits for it.
    if (m.lora.R == 0) grid_wait();
    grid_release();

    // the ranges: refused as a whole when they are not ordered inside [0, M]. With adapters the
    // requests are one range; without offsets all rows are.
    int *cached = table + MATMUL_MAX_EXPERTS + 4;
    const int nranges = m.lora.R > 0 ? m.lora.R : p.E;
    bool bad = false;
    if (threadIdx.x == MM_THREADS - 1 && failed(m.status)) *refuse = 2;
    if (m.offsets) {
        for (int i = threadIdx.x; i <= nranges; i += MM_THREADS) {
            const int v = __ldg(m.offsets + i);
            bad |= v < 0 || (int64_t)v > m.M || (i > 0 && v < __ldg(m.offsets + i - 1));
            if (m.lora.R > 0) {
                if (i == 0) cached[0] = v;
                if (i == nranges) cached[1] = v;
            } else if (i <= MM_CACHED) {
                cached[i] = v;
            }
        }
    } else if (threadIdx.x < 2) {
        cached[threadIdx.x] = threadIdx.x ? (int)m.M : 0;
    }
    if (m.lora.R > 0) bad |= ids_bad(m.lora.ids, m.lora.R, m.lora.L, threadIdx.x, MM_THREADS);
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0 && bad) *refuse = 1;
    if (warp == 0) {
        // table[e]: tiles of rows before range e
        int base = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            int nt = 0;
            if (e < p.E && !bad) {
                const int cnt = e < MM_CACHED ? cached[e + 1] - cached[e] : __ldg(m.offsets + e + 1) - __ldg(m.offsets + e);
                nt = (cnt + p.cols - 1) / p.cols;
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
    if (cluster > 1) tc::cluster_sync();    // every block's barriers and refusal are in place
    int skip = *refuse;
    if (cluster > 1)                        // the blocks of a cluster go by the first one's reading
        skip = (int)tc::ld_shared_cluster(tc::mapa_shared(tc::smem_u32(refuse), 0));
    if (skip == 1 && threadIdx.x == 0) set_status(m.status, GPTQ_ERR_ARG);

    constexpr int WIDTH = PAIR ? 2 * MM_LANES : MM_LANES;
    constexpr int GRAIN = PAIR ? 32 : 16;           // column counts that an MMA takes
    const int first = PAIR ? (int)rank * MM_LANES : 0;
    const int tiles_out = (p.out + WIDTH - 1) / WIDTH;
    const int tiles = skip ? 0 : table[p.E] * tiles_out;
    const int steps = (p.inner + MM_BK - 1) / MM_BK;
    const int part = PAIR ? 0 : (int)rank;
    const int k0 = (int)((int64_t)steps * part / split), k1 = (int)((int64_t)steps * (part + 1) / split);
    const int nmain = k1 - k0;
    const bool adapters = m.lora.R > 0 && part == split - 1;
    // blocks of `rank` columns in the adapters' contraction; of block 1, P's second part and T's first
    // (fp16), or P and T's second
    constexpr bool SPLIT_P = Half2<T>::kType != 1;
    const int inner_r = (SPLIT_P ? 3 : 2) * m.lora.rank;
    const int rsteps = (inner_r + MM_BK - 1) / MM_BK;
    const T *X = static_cast<const T *>(m.X);
    LoraRuns *runs = reinterpret_cast<LoraRuns *>(table + MATMUL_MAX_EXPERTS + 4 + MM_CACHED + 4 + 128);
    uint32_t lphase = 0;
    // the tile's run list is there; done with it
    auto runs_wait = [&]() { return (bool)__all_sync(~0u, tc::mbar_wait(lfull, lphase, abort)); };
    auto runs_done = [&]() {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(lempty);
        lphase ^= 1;
    };
    // the barrier of a stage that the MMA thread waits on (the first block's, in a pair)
    auto arrive_full = [&](int stage) {
        if (PAIR && rank != 0) tc::mbar_arrive_remote(tc::mapa_shared(tc::smem_u32(&full[stage]), 0));
        else tc::mbar_arrive(&full[stage]);
    };

    if (warp < MM_WARP_OUT) {
        const int set = warp >> 2, wq = warp & 3, tid = threadIdx.x, stid = tid & 127;
        // forward: channel = lane of the warp's TMEM quarter, 64 of the step's columns. Input gradient:
        // one of 64 rows n of the step and half of the block's 128 columns.
        const int arow64 = (wq & 1) * 32 + lane, ahalf = wq >> 1;
        // (halves of a tile's steps in turn, as unpack_turns.h says)
        auto first_half = [&](int turn) { return unpack_first_half(set, turn); };

        // Scales where they fold into the weights: requested one of this thread's steps ahead of the
        // unpacking, across tiles.
        const bool scaled = !IDX && p.fold;
        int fu = group, fturn = 0, fh = first_half(0), fc0 = 0;
        const float *frow = nullptr;                // scales of the channel (forward), of the range
        float ahead[2] = {0.f, 0.f};
        auto fetch_tile = [&]() {
            while (fu < tiles && fh >= 2 * nmain) {
                fu += ngroups;
                fturn = unpack_next_turn(fturn, 2 * nmain);
                fh = first_half(fturn);
            }
            if (fu >= tiles) return;
            const MmTile t = mm_tile(p, table, tiles_out, fu, WIDTH, first, GRAIN);
            fc0 = t.c0;
            const int n = DIR == 0 ? t.c0 + wq * 32 + lane : 0;
            frow = n < m.w.N ? m.w.scales + ((int64_t)t.e * m.w.N + n) * max(m.w.groups, 1) : nullptr;
        };
        auto fetch = [&]() {
            if (fu >= tiles) return;
            const int half = 2 * k0 + fh;           // 64 columns (forward) or rows of the contraction
            const int n = half * 64 + arow64, k = DIR == 0 ? half * 64 : fc0 + ahalf * 64;
            const float *row = DIR == 0 ? frow : n < m.w.N ? frow + (int64_t)n * max(m.w.groups, 1) : nullptr;
            const bool in = row && k < m.w.K, in2 = row && k + 32 < m.w.K;
            const int g = m.w.groups ? k >> m.w.gshift : 0;
            ahead[0] = in ? __ldg(row + g) : 0.f;
            ahead[1] = m.w.gshift == 5 && m.w.groups ? (in2 ? __ldg(row + g + 1) : 0.f) : ahead[0];
            fh += MM_SETS;
            if (fh >= 2 * nmain) fetch_tile();
        };
        if (scaled) {
            fetch_tile();
            fetch();
        }
        int turn = 0;
        RingPos wbase{0, 0}, base{0, 0};            // ring places of the tile's first step
        for (int u = group; u < tiles; u += ngroups) {
            const MmTile t = mm_tile(p, table, tiles_out, u, WIDTH, first, GRAIN);
            const int64_t erow = (int64_t)t.e * m.w.N;
            const int ch = t.c0 + wq * 32 + lane;       // forward: this thread's channel
            RingPos wpos = wbase, pos = base;
            int at = 0, wat = 0;                        // the step that pos stands at, the words' stage
#pragma unroll 1
            for (int h = first_half(turn); h < 2 * nmain; h += MM_SETS) {
                const int side = h & 1;                 // which half of the step
                for (; at < (h >> 1); ++at) {
                    pos.advance(stages);
                    if (DIR == 0) wpos.advance(Ring::STAGES);
                }
                if constexpr (DIR == 1)
                    for (; wat < h; ++wat) wpos.advance(Ring::STAGES);
                const int step = k0 + at;
                const int arow = side * 64 + arow64;
                const float sc[2] = {ahead[0], ahead[1]};
                if (scaled) fetch();
                // by g_idx: where the scales of this lane's columns are, of 32 each
                int place[2] = {0, 0};
                if constexpr (IDX) {
                    if (p.idx_table) {
                        const int32_t *gi = m.w.g_idx + (int64_t)t.e * m.w.K;
                        const int c = DIR == 0 ? step * MM_BK + side * 64 : t.c0 + ahalf * 64;
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            place[q] = group_place(gi, c + 32 * q + lane, m.w.K, m.w.groups, UNPACKERS, m.status);
                    }
                }
                uint32_t raw[2][B];
                bool ok = tc::mbar_wait(&wfull[wpos.stage], wpos.phase, abort);
                {
                    const uint8_t *src = words + wpos.stage * Ring::STAGE;
                    // the row and first 16-byte (8-byte) piece that this thread unpacks
                    const int wrow = DIR == 0 ? wq * 32 + lane : arow64;
                    const int wpiece = (DIR == 0 ? side : ahalf) * (B == 3 ? 3 : B / 2);
                    if constexpr (B == 3) {
#pragma unroll
                        for (int q = 0; q < 3; ++q) {
                            const uint2 y = *reinterpret_cast<const uint2 *>(src + Ring::at(wrow, wpiece + q));
                            raw[(2 * q) / 3][(2 * q) % 3] = y.x;
                            raw[(2 * q + 1) / 3][(2 * q + 1) % 3] = y.y;
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < B / 2; ++q) {
                            const uint4 y = *reinterpret_cast<const uint4 *>(src + Ring::at(wrow, wpiece + q));
                            const uint32_t z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) raw[(4 * q + j) / B][(4 * q + j) % B] = z[j];
                        }
                    }
                }
                // The stage is filled again by a tiled copy, which an arrival alone does not hold back behind
                // reads that are still under way: with other warps' gathers ahead of them (g_idx without a
                // table) the words changed in up to 74 of 100 calls without this fence, in none with it.
                tc::fence_async_shared();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&wempty[wpos.stage]);
                if constexpr (IDX) {
                    // this thread's row of scales, in its own column of the table (forward: once a tile)
                    const int n = DIR == 0 ? ch : step * MM_BK + arow;
                    if (p.idx_table && n < m.w.N && (DIR == 1 || h < MM_SETS)) {
                        const float *row = m.w.scales + (erow + n) * m.w.groups;
#pragma unroll 8
                        for (int q = 0; q < m.w.groups; ++q) own_scales[q * UNPACKERS + tid] = __ldg(row + q);
                    }
                }
                uint32_t v[2][16];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    unpack32<B, T>(raw[q], v[q]);
                    if constexpr (IDX) {
                        const int n = DIR == 0 ? ch : step * MM_BK + arow;
                        const int c = DIR == 0 ? step * MM_BK + side * 64 + 32 * q : t.c0 + ahalf * 64 + 32 * q;
                        if (c < m.w.K) {
                            const int32_t *gi = m.w.g_idx + (int64_t)t.e * m.w.K;
                            if (p.idx_table)
                                scale32_by_table<T>(v[q], own_scales + tid, place[q]);
                            else if (n < m.w.N)
                                scale32_by_index<T, B, true>(v[q], m.w.scales + (erow + n) * m.w.groups, gi, c, m.w.K,
                                                             m.w.groups, m.status);
                        }
                    } else {
                        if (p.fold) scale32<T>(v[q], sc[q]);
                    }
                }
                ok = tc::mbar_wait(&empty[pos.stage], pos.phase ^ 1, abort) && ok;
                ok = __all_sync(~0u, ok);
                if (ok) {
                    uint8_t *st = smem + pos.stage * stage_bytes;
                    if constexpr (DIR == 0) {
                        // the stage's last reader was an MMA that has completed
                        tc::fence_after_sync();
                        uint32_t r[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[j] = v[j >> 4][j & 15];
                        tc::tmem_st_32x32b_x32(tmem + 256 + pos.stage * 64 + side * 32 + ((uint32_t)(wq * 32) << 16), r);
                        tc::tmem_st_wait();
                    } else {
                        uint8_t *a = st + MM_B_BYTES + ahalf * MM_BOX + arow * 128;
                        const bool in = step * MM_BK + arow < m.w.N;
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const uint32_t(&y)[16] = v[q >> 2];
                            const int j = 4 * (q & 3);
                            // (rows past the layer's last: their scale is zero already)
                            *reinterpret_cast<uint4 *>(a + ((q ^ (arow & 7)) << 4)) =
                                !IDX || in ? make_uint4(y[j], y[j + 1], y[j + 2], y[j + 3]) : make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    if (!tiled) {
                        const int rows = PAIR ? t.n16 / 2 : t.n16;
                        plain_box<T>(st + side * MM_HALF, X, m.ldx, t.t0 + (PAIR ? (int)rank * rows : 0), rows, t.t0 + t.n,
                                     step * MM_BK + side * 64, p.inner, stid, 128);
                    }
                    if (DIR == 1 || !tiled) tc::fence_async_shared();
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) arrive_full(pos.stage);
                }
            }
            turn = unpack_next_turn(turn, 2 * nmain);
            wbase.jump(DIR == 0 ? nmain : 2 * nmain, Ring::STAGES);
            base.jump(nmain, stages);
            if (adapters) {
                grid_wait();
                int half = 0;                           // of the adapters' steps, in turn too
                const T *P = static_cast<const T *>(m.lora.P);
                const __nv_bfloat16 *T3 = m.lora.T3;
                const int r = m.lora.rank;
                auto block = [&](int q) { return (q >= r ? 1 : 0) + (SPLIT_P && q >= 2 * r ? 1 : 0); };
                const int count = runs_wait() ? runs->count : 0, halves = 2 * rsteps * count;
                for (int run = 0; run < count; ++run) {
                    const int run_begin = runs->begin[run], run_end = runs->end[run], run_id = runs->id[run];
                    const int b0 = run_begin & -GRAIN, b1 = (run_end + GRAIN - 1) & -GRAIN;
                    const int rows = PAIR ? (b1 - b0) / 2 : b1 - b0;
                    const int row0 = b0 + (PAIR ? (int)rank * rows : 0);
                    for (int hs = 0; hs < 2 * rsteps; ++hs, ++half) {
                        const int side = hs & 1, rs = hs >> 1;
                        RingPos pos = base;
                        if (side) base.advance(stages);
                        if (unpack_adapter_set(turn, half, halves) != set) continue;
                        const int arow = side * 64 + arow64;
                        // this thread's part of A, requested before the stage is free. Forward: row n
                        // of B_a, once for each block of the contraction; input gradient: rows of A_a,
                        // once for each too
                        uint4 y[8];
                        const int qa = rs * MM_BK + (DIR == 0 ? side * 64 : arow);
                        if constexpr (DIR == 0) {
                            const T *src = P + ((int64_t)run_id * m.w.N + ch) * r;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const int q = qa + j * 8;
                                y[j] = ch < m.w.N && q < inner_r
                                           ? bf16_part8<T>(load8<T>(src + q - block(q) * r, 8, true), block(q) == 1)
                                           : make_uint4(0u, 0u, 0u, 0u);
                            }
                        } else {
                            const int c = t.c0 + ahalf * 64;
                            const T *src = P + ((int64_t)run_id * r + qa - block(qa) * r) * m.w.K + c;
                            const bool v8 = (m.w.K & 7) == 0;
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                y[j] = bf16_part8<T>(load8<T>(src + 8 * j, qa < inner_r ? m.w.K - c - 8 * j : 0, v8), block(qa) == 1);
                        }
                        bool ok = tc::mbar_wait(&empty[pos.stage], pos.phase ^ 1, abort);
                        if (finite_only<__nv_bfloat16>(y)) {
                            runs->broken = 1;
                            __threadfence_block();
                        }
                        ok = __all_sync(~0u, ok);
                        if (ok) {
                            uint8_t *st = smem + pos.stage * stage_bytes;
                            if constexpr (DIR == 0) {
                                uint32_t z[32];
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    z[4 * j] = y[j].x; z[4 * j + 1] = y[j].y; z[4 * j + 2] = y[j].z; z[4 * j + 3] = y[j].w;
                                }
                                tc::fence_after_sync();
                                tc::tmem_st_32x32b_x32(tmem + 256 + pos.stage * 64 + side * 32 +
                                                           ((uint32_t)(wq * 32) << 16), z);
                                tc::tmem_st_wait();
                            } else {
                                uint8_t *a = st + MM_B_BYTES + ahalf * MM_BOX + arow * 128;
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    *reinterpret_cast<uint4 *>(a + ((j ^ (arow & 7)) << 4)) = y[j];
                            }
                            // the run's rows of T's parts, zeros for rows of others
                            for (int j = stid; j < rows * 8; j += 128) {
                                const int row = j >> 3, q = j & 7, col = rs * MM_BK + side * 64 + 8 * q;
                                const int tr = row0 + row;
                                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                                if (tr >= run_begin && tr < run_end && col < inner_r) {
                                    const int b = block(col), of = SPLIT_P ? b >> 1 : b;
                                    x = __ldcg(reinterpret_cast<const uint4 *>(T3 + (t.t0 + tr) * (LORA_PARTS * r) + col -
                                                                               (b - of) * r));
                                }
                                *reinterpret_cast<uint4 *>(st + side * MM_HALF + row * 128 + ((q ^ (row & 7)) << 4)) = x;
                            }
                            tc::fence_async_shared();
                            tc::fence_before_sync();
                            __syncwarp();
                            if (lane == 0) arrive_full(pos.stage);
                        }
                    }
                }
                runs_done();
            }
        }
    } else if (warp < MM_WARP_X) {
        // outputs: lane = channel, register = row
        const int wq = warp & 3, etid = threadIdx.x - MM_WARP_OUT * 32;
        int acc = 0;
        uint32_t acc_phase = 0, sum_phase = 0;
        T *Y = static_cast<T *>(m.Y);
        for (int u = group; u < tiles; u += ngroups) {
            const MmTile t = mm_tile(p, table, tiles_out, u, WIDTH, first, GRAIN);
            const int ch = t.c0 + wq * 32 + lane;
            const bool per_channel = DIR == 0 && !p.fold;
            const float s = per_channel && ch < p.out ? __ldg(m.w.scales + (int64_t)t.e * m.w.N + ch) : 1.f;
            // adapters of the rows in short runs (0xffff: none), found while the products run
            bool shorts = false;
            uint16_t *row_ids = reinterpret_cast<uint16_t *>(table + MATMUL_MAX_EXPERTS + 4 + MM_CACHED + 4);
            if (m.lora.R > 0) {
                grid_wait();
                // a bit for each row that starts a run, from its request's adapter and its neighbour's
                bool free = true;
                if (adapters) free = __all_sync(~0u, tc::mbar_wait(lempty, lphase ^ 1, abort));
                asm volatile("bar.sync 1, 128;" ::: "memory");      // the tile before is done with row_ids
                for (int r = etid; r < 256; r += 128) {
                    int id = -1;
                    if (r < t.n) id = __ldg(m.lora.ids + request_of(m.offsets, m.lora.R, (int)t.t0 + r));
                    row_ids[r] = (uint16_t)id;                      // -1 is 0xffff
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
                for (int r = etid; r < 256; r += 128) {
                    const unsigned b = __ballot_sync(~0u, r >= t.n || r == 0 || row_ids[r] != row_ids[r - 1]);
                    if (lane == 0) runs->starts[r >> 5] = b;
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
                int id2[2], begin2[2], len2[2];
                for (int i = 0; i < 2; ++i) {
                    // this row's run: the last start at or before it, the first behind it
                    const int r = etid + 128 * i;
                    int w = r >> 5;
                    uint32_t v = runs->starts[w] & (0xffffffffu >> (31 - (r & 31)));
                    while (v == 0u) v = runs->starts[--w];
                    begin2[i] = w * 32 + 31 - __clz(v);
                    w = r >> 5;
                    v = (r & 31) == 31 ? 0u : runs->starts[w] & (0xfffffffeu << (r & 31));
                    while (v == 0u && w < 7) v = runs->starts[++w];
                    len2[i] = (v ? w * 32 + __ffs(v) - 1 : 256) - begin2[i];
                    id2[i] = r < t.n ? row_ids[r] : 0xffff;
                    const bool some = id2[i] != 0xffff;
                    const unsigned b = __ballot_sync(~0u, some && len2[i] >= LORA_SHORT && begin2[i] == r);
                    if (lane == 0) runs->longs[r >> 5] = b;
                    shorts |= some && len2[i] < LORA_SHORT;
                }
                // (a named barrier that also tells whether any thread saw a short run)
                {
                    int any;
                    asm volatile(
                        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\t"
                        "bar.red.or.pred q, 1, 128, p;\n\t"
                        "selp.s32 %0, 1, 0, q;\n\t}"
                        : "=r"(any)
                        : "r"((int)shorts)
                        : "memory");
                    shorts = any != 0;
                }
                int before[2] = {0, 0}, count = 0;
                for (int w = 0; w < 8; ++w) {
                    const uint32_t v = runs->longs[w];
                    for (int i = 0; i < 2; ++i) {
                        const int r = etid + 128 * i;
                        before[i] += w < (r >> 5) ? __popc(v) : w == (r >> 5) ? __popc(v & ((1u << (r & 31)) - 1u)) : 0;
                    }
                    count += __popc(v);
                }
                for (int i = 0; i < 2; ++i) {
                    const int r = etid + 128 * i;
                    if (id2[i] != 0xffff && len2[i] >= LORA_SHORT) {
                        if (begin2[i] == r && free) {
                            runs->begin[before[i]] = r;
                            runs->end[before[i]] = min(r + len2[i], t.n);
                            runs->id[before[i]] = id2[i];
                        }
                        row_ids[r] = 0xffff;            // its term is a matrix step's
                    }
                }
                if (etid == 0) {
                    runs->count = free ? count : 0;                 // (a time-out leaves no list)
                    if (free) runs->broken = 0;
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (adapters) {
                    if (lane == 0) tc::mbar_arrive(lfull);
                    lphase ^= 1;
                }
            }
            float *dump = reinterpret_cast<float *>(epi);
            bool ok = true;
            if (split > 1) {
                // the partial sums of the tile before have been read (first tile: passes at once); the
                // rows that this block will write take their adapter terms while the products run
                ok = __all_sync(~0u, tc::mbar_wait_cluster(done, sum_phase ^ 1, abort));
                if (shorts && ok) {
                    for (int row = (int)rank; row < t.n; row += 4 * split) {
                        int id[4];
                        int64_t ts[4];
                        float add[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = row + i * split;
                            id[i] = r < t.n && ch < p.out && row_ids[r] != 0xffff ? (int)row_ids[r] : -1;
                            ts[i] = t.t0 + r;
                        }
                        lora_terms<T, DIR, 4>(m.lora, id, ts, ch, p.out, add);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (row + i * split < t.n) dump[(row + i * split) * MM_LANES + wq * 32 + lane] = add[i];
                    }
                }
            }
            ok = tc::mbar_wait(&tfull[acc], acc_phase, abort) && ok;
            ok = __all_sync(~0u, ok);
            tc::fence_after_sync();
            const uint32_t at = tmem + acc * p.acc_cols + ((uint32_t)(wq * 32) << 16);
            auto release = [&]() {
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR && rank != 0) tc::mbar_arrive_remote(tc::mapa_shared(tc::smem_u32(&tempty[acc]), 0));
                    else tc::mbar_arrive(&tempty[acc]);
                }
            };
            if (m.lora.R > 0 && ok && __any_sync(~0u, *(volatile int *)&runs->broken != 0))
                add_nonfinite<T, DIR>(m.lora, runs, t.t0, ch, p.out, at);
            if (split == 1) {
                if (shorts && ok) {
                    // their terms into the accumulators
                    for (int r = 0; r < t.n; r += 4) {
                        int id[4];
                        int64_t ts[4];
                        float add[4];
                        bool some = false;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            id[i] = r + i < t.n && row_ids[r + i] != 0xffff ? (int)row_ids[r + i] : -1;
                            some |= id[i] >= 0;
                            if (ch >= p.out) id[i] = -1;
                            ts[i] = t.t0 + r + i;
                        }
                        if (!some) continue;
                        lora_terms<T, DIR, 4>(m.lora, id, ts, ch, p.out, add);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t y = tc::tmem_ld_32x32b_x1(at + r + i);
                            tc::tmem_ld_wait();
                            tc::tmem_st_32x32b_x1(at + r + i, __float_as_uint(__uint_as_float(y) + add[i]));
                        }
                    }
                    tc::tmem_st_wait();
                }
                // through shared memory as [row][channel], `chunk` rows at a time
                const int chunk = p.epi / 256;
                T *stg = reinterpret_cast<T *>(epi);
                for (int r0 = 0; r0 < t.n; r0 += chunk) {
                    const int rows = min(chunk, t.n - r0);
                    if (ok) {
                        // `chunk` is a multiple of 32; the columns past the tile's rows are not written out
                        uint16_t *d = reinterpret_cast<uint16_t *>(epi) + wq * 32 + lane;
#pragma unroll 1
                        for (int r = 0; r < rows; r += 32, d += 32 * MM_LANES) {
                            uint32_t y[32];
                            tc::tmem_ld_32x32b_x32(at + r0 + r, y);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 32; j += 2) {
                                const uint32_t h = Half2<T>::pack(s * __uint_as_float(y[j]), s * __uint_as_float(y[j + 1]));
                                d[j * MM_LANES] = (uint16_t)h;
                                d[(j + 1) * MM_LANES] = (uint16_t)(h >> 16);
                            }
                        }
                    }
                    if (r0 + chunk >= t.n) release();
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                    if (ok) {
                        const int q = etid & 15, c = t.c0 + 8 * q;
                        for (int r = etid >> 4; r < rows; r += 8) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(stg + r * MM_LANES + 8 * q);
                            T *d = Y + (t.t0 + r0 + r) * m.ldy + c;
                            if (p.yvec && c + 8 <= p.out) {
                                *reinterpret_cast<uint4 *>(d) = x;
                            } else {
                                const uint32_t h[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    if (c + j < p.out)
                                        reinterpret_cast<uint16_t *>(d)[j] = (uint16_t)(h[j >> 1] >> (16 * (j & 1)));
                            }
                        }
                    }
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                }
            } else {
                // partial sums of the cluster's blocks as [row][channel], summed in rank order by
                // the block that writes the row
                if (ok) {
                    for (int r = 0; r < t.n16; r += 16) {
                        uint32_t y[16];
                        tc::tmem_ld_32x32b_x16(at + r, y);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float *d = dump + (r + j) * MM_LANES + wq * 32 + lane;
                            // (split is a power of two)
                            const bool mine = shorts && ((r + j) & (split - 1)) == (int)rank && r + j < t.n;
                            *d = mine ? *d + __uint_as_float(y[j]) : __uint_as_float(y[j]);
                        }
                    }
                }
                release();
                if (lane < split)
                    tc::mbar_arrive_cluster(tc::mapa_shared(tc::smem_u32(ready), lane));
                bool all = tc::mbar_wait_cluster(ready, sum_phase, abort);
                all = __all_sync(~0u, all) && ok;
                if (all) {
                    // a warp a row, four channels a lane; the blocks' sums are requested at once
                    const int c4 = t.c0 + 4 * lane;
                    float s4[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s4[j] = per_channel && c4 + j < p.out ? __ldg(m.w.scales + (int64_t)t.e * m.w.N + c4 + j) : 1.f;
#pragma unroll 2
                    for (int row = (int)rank + split * wq; row < t.n; row += 4 * split) {
                        const uint32_t from = tc::smem_u32(dump + row * MM_LANES + 4 * lane);
                        float4 v[8];
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            v[c] = c < split ? tc::ld_shared_cluster_f4(tc::mapa_shared(from, c)) : make_float4(0.f, 0.f, 0.f, 0.f);
                        float4 sum = v[0];
#pragma unroll
                        for (int c = 1; c < 8; ++c) {
                            sum.x += v[c].x; sum.y += v[c].y; sum.z += v[c].z; sum.w += v[c].w;
                        }
                        const uint32_t y0 = Half2<T>::pack(s4[0] * sum.x, s4[1] * sum.y);
                        const uint32_t y1 = Half2<T>::pack(s4[2] * sum.z, s4[3] * sum.w);
                        T *d = Y + (t.t0 + row) * m.ldy + c4;
                        if (p.yvec && c4 + 4 <= p.out) {
                            *reinterpret_cast<uint2 *>(d) = make_uint2(y0, y1);
                        } else {
                            uint16_t *e = reinterpret_cast<uint16_t *>(d);
                            if (c4 < p.out) e[0] = (uint16_t)y0;
                            if (c4 + 1 < p.out) e[1] = (uint16_t)(y0 >> 16);
                            if (c4 + 2 < p.out) e[2] = (uint16_t)y1;
                            if (c4 + 3 < p.out) e[3] = (uint16_t)(y1 >> 16);
                        }
                    }
                }
                // before the next tile's sums (the release waits for the outputs, too: not for nothing)
                __syncwarp();
                if (u + ngroups < tiles && lane < split)
                    tc::mbar_arrive_cluster(tc::mapa_shared(tc::smem_u32(done), lane));
                sum_phase ^= 1;
            }
            if (++acc == p.accs) { acc = 0; acc_phase ^= 1; }
        }
    } else if (warp == MM_WARP_X) {
        // the whole warp walks, one elected lane issues (as for the MMAs below)
        if (tiled) {
            RingPos pos{0, 0};
            bool ok = true;
            for (int u = group; u < tiles && ok; u += ngroups) {
                const MmTile t = mm_tile(p, table, tiles_out, u, WIDTH, first, GRAIN);
                const int rows = PAIR ? t.n16 / 2 : t.n16;
                const int row0 = (int)t.t0 + (PAIR ? (int)rank * rows : 0);
                const int boxes = (rows + p.box_rows - 1) / p.box_rows;
                const uint32_t bytes = boxes * p.box_rows * 256;
#pragma unroll 1
                for (int i = 0; i < nmain; ++i) {
                    ok = __all_sync(~0u, tc::mbar_wait(&empty[pos.stage], pos.phase ^ 1, abort));
                    if (!ok) break;
                    uint8_t *st = smem + pos.stage * stage_bytes;
                    const int x = (k0 + i) * MM_BK;
                    if (tc::elect_one()) {
                        if (!PAIR || rank == 0) tc::mbar_arrive_expect_tx(&full[pos.stage], PAIR ? 2 * bytes : bytes);
                        for (int b = 0; b < boxes; ++b) {
                            uint8_t *d = st + b * p.box_rows * 128;
                            const int y = row0 + b * p.box_rows;
                            if constexpr (PAIR) {
                                const uint32_t fb = tc::mapa_shared(tc::smem_u32(&full[pos.stage]), 0);
                                tc::tma_load_2d_pair(d, &xmap, fb, x, y);
                                tc::tma_load_2d_pair(d + MM_HALF, &xmap, fb, x + 64, y);
                            } else {
                                tc::tma_load_2d(d, &xmap, &full[pos.stage], x, y);
                                tc::tma_load_2d(d + MM_HALF, &xmap, &full[pos.stage], x + 64, y);
                            }
                        }
                    }
                    __syncwarp();
                    pos.advance(stages);
                }
                if (ok && adapters) {
                    const int count = runs_wait() ? runs->count : 0;
                    for (int run = 0; run < count && ok; ++run) {
                        for (int rs = 0; rs < rsteps; ++rs) {
                            ok = __all_sync(~0u, tc::mbar_wait(&empty[pos.stage], pos.phase ^ 1, abort));
                            if (!ok) break;
                            if (lane == 0 && (!PAIR || rank == 0)) tc::mbar_arrive(&full[pos.stage]);
                            pos.advance(stages);
                        }
                    }
                    runs_done();
                }
            }
            if (!ok) {
                // loads still in flight land before the block can exit
                const long long from = clock64();
                while (clock64() - from < 20000000ll) {
                }
            }
        }
    } else if (warp >= MM_WARP_WORDS) {
        // a stage: the block's channels x a step's columns (forward), or half a step's rows x the
        // block's columns
        constexpr int PER = 128 / Ring::ROWS;       // stages of a step
        RingPos pos{0, 0};
        bool ok = true;
        if (p.wtiled) {
            if (warp == MM_WARP_WORDS) {
                for (int u = group; u < tiles && ok; u += ngroups) {
                    const MmTile t = mm_tile(p, table, tiles_out, u, WIDTH, first, GRAIN);
                    const int erow = t.e * m.w.N;
#pragma unroll 1
                    for (int i = 0; i < PER * nmain; ++i) {
                        ok = __all_sync(~0u, tc::mbar_wait(&wempty[pos.stage], pos.phase ^ 1, abort));
                        if (!ok) break;
                        const int k = DIR == 0 ? (k0 + i) * MM_BK : t.c0;
                        const int n = DIR == 0 ? t.c0 : k0 * MM_BK + i * Ring::ROWS;
                        if (tc::elect_one()) {
                            tc::mbar_arrive_expect_tx(&wfull[pos.stage], Ring::STAGE);
                            tc::tma_load_2d(words + pos.stage * Ring::STAGE, &wmap, &wfull[pos.stage], (k >> 5) * B, erow + n);
                        }
                        __syncwarp();
                        pos.advance(Ring::STAGES);
                    }
                }
                if (!ok) {
                    const long long from = clock64();
                    while (clock64() - from < 20000000ll) {
                    }
                }
            }
        } else {
            // half of a stage's rows a warp
            const int nw = (int)(((int64_t)m.w.K * B + 31) / 32);
            for (int u = group; u < tiles && ok; u += ngroups) {
                const MmTile t = mm_tile(p, table, tiles_out, u, WIDTH, first, GRAIN);
                const int64_t erow = (int64_t)t.e * m.w.N;
                for (int i = 0; i < PER * nmain; ++i) {
                    ok = tc::mbar_wait(&wempty[pos.stage], pos.phase ^ 1, abort);
                    ok = __all_sync(~0u, ok);
                    if (!ok) break;
                    const int w0 = ((DIR == 0 ? (k0 + i) * MM_BK : t.c0) >> 5) * B;
                    const int n0 = DIR == 0 ? t.c0 : k0 * MM_BK + i * Ring::ROWS;
                    // lanes take neighbouring words of as many whole rows as fit a warp
                    constexpr int RW = 4 * B, PW = B == 3 ? 2 : 4, RL = 32 / RW;    // words of a row, of a piece; rows
                    const uint32_t dst = tc::smem_u32(words + pos.stage * Ring::STAGE);
                    const int sub = lane / RW, wd = lane - sub * RW;
                    if (sub < RL) {
                        const bool in = w0 + wd < nw;
                        const int row0 = (warp - MM_WARP_WORDS) * (Ring::ROWS / 2), left = m.w.N - n0;
                        const uint32_t *src = m.w.words + (erow + n0 + row0 + sub) * m.w.ldw + w0 + wd;
                        const int64_t by = RL * m.w.ldw;
#pragma unroll 8
                        for (int r = row0 + sub; r < row0 + Ring::ROWS / 2; r += RL, src += by)
                            copy_async<4>(dst + Ring::at(r, wd / PW) + (wd % PW) * 4, in && r < left ? src : nullptr,
                                          m.w.words);
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(&wfull[pos.stage]))
                                 : "memory");
                    pos.advance(Ring::STAGES);
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else {
        // the whole warp walks the steps, so that what an MMA takes stays in uniform registers (with
        // one lane walking, issuing an MMA took longer than the MMA); one elected lane issues
        if (!PAIR || rank == 0) {
            RingPos pos{0, 0};
            int acc = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            constexpr int MROWS = PAIR ? 2 * MM_LANES : MM_LANES;
            const uint32_t ring = tc::smem_u32(smem);
            const uint64_t bdesc0 = tc::desc_sw128(ring, 16, 1024);
            const uint64_t adesc0 = tc::desc_sw128(ring + MM_B_BYTES, MM_BOX, 1024);
            // the MMAs of one step: kks of 16, into columns from d on, and the stage's release
            auto issue = [&](uint32_t d, int stage, int kks, uint32_t id, uint32_t add) {
                const uint64_t bd = bdesc0 + (uint32_t)(stage * stage_bytes >> 4);
                const uint64_t ad = adesc0 + (uint32_t)(stage * stage_bytes >> 4);
                const uint32_t at = tmem + 256 + stage * 64;
                if (tc::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < MM_BK / 16; ++kk) {
                        if (kk >= kks) break;
                        const uint64_t bk = bd + ((kk >> 2) * MM_HALF + (kk & 3) * 32 >> 4);
                        const uint32_t on = kk > 0 ? 1u : add;
                        if constexpr (DIR == 0) {
                            if constexpr (PAIR) tc::mma_f16_ts_pair(d, at + kk * 8, bk, id, on);
                            else tc::mma_f16_ts(d, at + kk * 8, bk, id, on);
                        } else {
                            if constexpr (PAIR) tc::mma_bf16_pair(d, ad + kk * 128, bk, id, on);
                            else tc::mma_bf16(d, ad + kk * 128, bk, id, on);
                        }
                    }
                    if constexpr (PAIR) tc::mma_commit_both(&empty[stage]);
                    else tc::mma_commit(&empty[stage]);
                }
                __syncwarp();
            };
            for (int u = group; u < tiles && ok; u += ngroups) {
                const MmTile t = mm_tile(p, table, tiles_out, u, WIDTH, first, GRAIN);
                const uint32_t id = tc::idesc_f16_f32(Half2<T>::kType, MROWS, t.n16, DIR, 0);
                ok = __all_sync(~0u, tc::mbar_wait(&tempty[acc], acc_phase ^ 1, abort));
                if (!ok) break;
                tc::fence_after_sync();
                const uint32_t d = tmem + acc * p.acc_cols;
                for (int i = 0; i < nmain; ++i) {
                    ok = __all_sync(~0u, tc::mbar_wait(&full[pos.stage], pos.phase, abort));
                    if (!ok) break;
                    tc::fence_after_sync();
                    issue(d, pos.stage, MM_BK / 16, id, i > 0 ? 1u : 0u);
                    pos.advance(stages);
                }
                if (ok && adapters) {
                    const int count = runs_wait() ? runs->count : 0;
                    for (int run = 0; run < count && ok; ++run) {
                        const int b0 = runs->begin[run] & -GRAIN, b1 = (runs->end[run] + GRAIN - 1) & -GRAIN;
                        const uint32_t rid = tc::idesc_f16_f32(Half2<__nv_bfloat16>::kType, MROWS, b1 - b0, DIR, 0);
                        for (int rs = 0; rs < rsteps; ++rs) {
                            ok = __all_sync(~0u, tc::mbar_wait(&full[pos.stage], pos.phase, abort));
                            if (!ok) break;
                            tc::fence_after_sync();
                            issue(d + b0, pos.stage, (min(MM_BK, inner_r - rs * MM_BK) + 15) / 16, rid, 1u);
                            pos.advance(stages);
                        }
                    }
                    runs_done();
                }
                if (ok && tc::elect_one()) {
                    if constexpr (PAIR) tc::mma_commit_both(&tfull[acc]);
                    else tc::mma_commit(&tfull[acc]);
                }
                __syncwarp();
                if (++acc == p.accs) { acc = 0; acc_phase ^= 1; }
            }
            // every MMA issued completes before TMEM is released
            if (tc::elect_one()) {
                if constexpr (PAIR) tc::mma_commit_pair(tc::mapa_shared(tc::smem_u32(drain), 0));
                else tc::mma_commit(drain);
                volatile int never = 0;
                tc::mbar_wait(drain, 0, &never);
            }
        }
    }

    if (m.lora.R > 0) grid_wait();          // whatever came before is done before this kernel is
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (cluster > 1) tc::cluster_sync_relaxed();    // no block leaves while others use its memory
    if (*abort && threadIdx.x == 0) set_status(m.status, GPTQ_ERR_TIMEOUT);
    if (warp == MM_WARP_MMA) {
        tc::fence_after_sync();
        if constexpr (PAIR) tc::tmem_dealloc_pair(tmem, MM_TMEM);
        else tc::tmem_dealloc(tmem, MM_TMEM);
    }
}

template <typename T, int B, int DIR>
static gptq_status launch_tc(const CUtensorMap &map, const CUtensorMap &wmap, const MmTcArg &p, bool pair, int blocks, size_t smem,
                             cudaStream_t st) {
    const int cluster = pair ? 2 : p.split;
    if (p.m.w.g_idx)
        return pair ? launch_pdl(k_matmul_tc<T, B, DIR, true, true>, dim3(blocks), MM_THREADS, smem, SMEM_MOST, cluster, st, map, wmap, p)
                    : launch_pdl(k_matmul_tc<T, B, DIR, true, false>, dim3(blocks), MM_THREADS, smem, SMEM_MOST, cluster, st, map, wmap, p);
    return pair ? launch_pdl(k_matmul_tc<T, B, DIR, false, true>, dim3(blocks), MM_THREADS, smem, SMEM_MOST, cluster, st, map, wmap, p)
                : launch_pdl(k_matmul_tc<T, B, DIR, false, false>, dim3(blocks), MM_THREADS, smem, SMEM_MOST, cluster, st, map, wmap, p);
}

template <typename T, int DIR>
static gptq_status launch_tc_bits(const CUtensorMap &map, const CUtensorMap &wmap, const MmTcArg &p, int bits, bool pair, int blocks,
                                  size_t smem, cudaStream_t st) {
    switch (bits) {
        case 2: return launch_tc<T, 2, DIR>(map, wmap, p, pair, blocks, smem, st);
        case 3: return launch_tc<T, 3, DIR>(map, wmap, p, pair, blocks, smem, st);
        case 4: return launch_tc<T, 4, DIR>(map, wmap, p, pair, blocks, smem, st);
        default: return launch_tc<T, 8, DIR>(map, wmap, p, pair, blocks, smem, st);
    }
}

}  // namespace gptq
