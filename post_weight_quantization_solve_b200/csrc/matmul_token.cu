// Packed-weight products for a few rows: Y[t] = W^_e X[t] (+ adapters) when decoding.
//
// With a handful of rows the product is bound by reading the packed words once, so the kernel
// is laid out for that: a block takes 32 output channels of one range and up to 8 of
// its rows; its 8 warps split the contraction, and each lane reads whole chunks of 32 codes,
// several requests in flight. Four lanes of a quad hold four neighbouring chunks of one row,
// which is the m16n8k16 fragment layout with the contraction index permuted: a sum does not
// care, as long as the rows X are read in the same order. X is put into shared memory once a
// block, in the order in which codes leave a word, so a fragment is four 16-byte reads and the
// unpacking needs no permutes (read from global memory per fragment, with its bounds and
// permutes, X cost as many instructions as the codes: 5.2 a code against 3.9). The matrix
// instruction adds in fp32; the warps' partial sums meet in shared memory in warp order.
//
// Scales: one scale a channel enters in fp32 at the end (the codes are exact); with input
// groups each weight is rounded once to the rows' 16-bit type, as in the tiled kernel.
//
// One row, 4,096 -> 14,336, 3 bits: 16.7 us for 22 MB (1.3 TB/s). Four instructions a code keep the
// issue slots half busy (49 %, the integer pipe 44 %); the rest is latency, of the first words (all
// blocks run at once and read a step ahead only of their neighbours), of the block's barriers and of the
// launch. Eight of 64 experts of 2,048 -> 1,024: 10 us, one launch's latency. By g_idx every code
// gathers its scale: 4,096 -> 14,336, 4 bits, groups of 128: 156 us against 29.
#include <algorithm>
#include <type_traits>

#include "matmul.cuh"

namespace gptq {

namespace {
constexpr int TK_WARPS = 8;
constexpr int TK_CH = 32;                  // channels of a block (two 16-row fragments)
constexpr int TK_SPAN = TK_WARPS * 128;    // columns that the warps cover in one step each
constexpr int TK_SMEM = 64 * 1024;         // most of X that is staged at a time, without the rows' padding
constexpr int TK_PAD = 32;
}  // namespace

struct TokenArg {
    MatmulArg m;
    int fold, vec, xvec, E;
    int rows, span;       // rows of X that a block stages at most, columns at a time (multiple of TK_SPAN)
};

// 32 neighbouring values of a row in the pair order of unpack32<B, T, false>.
template <int B>
__device__ __forceinline__ void to_pair_order(uint32_t (&x)[16]) {
    if constexpr (B == 3 || B == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a = x[4 * i], b = x[4 * i + 1], c = x[4 * i + 2], d = x[4 * i + 3];
            x[4 * i] = __byte_perm(a, c, 0x5410);
            x[4 * i + 1] = __byte_perm(a, c, 0x7632);
            x[4 * i + 2] = __byte_perm(b, d, 0x5410);
            x[4 * i + 3] = __byte_perm(b, d, 0x7632);
        }
    } else if constexpr (B == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = x[8 * i + j];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[8 * i + 2 * j] = __byte_perm(y[j], y[j + 4], 0x5410);
                x[8 * i + 2 * j + 1] = __byte_perm(y[j], y[j + 4], 0x7632);
            }
        }
    }
}

// IDX: groups by g_idx.
template <typename T, int B, bool IDX>
__global__ void __launch_bounds__(TK_WARPS * 32, !IDX && B <= 4 ? (B == 4 ? 3 : 4) : 2)
    k_matmul_token(const __grid_constant__ TokenArg p) {
    constexpr int ROWS = 8, NR = 4;
    extern __shared__ uint8_t xs[];                     // [row][chunk of 64 bytes], padded rows
    __shared__ float part[TK_WARPS][ROWS][TK_CH + 1];
    __shared__ int found[4];
    const MatmulArg &m = p.m;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = lane & 3, g = lane >> 2;
    // With adapters the kernel before this one is the one that makes T; all that is read up to the
    // sums was there before that one began, so only the sums wait for it.
    if (m.lora.R == 0) grid_wait();
    grid_release();

    // which range, and which of its rows
    int e = 0;
    int64_t t0;
    int n;
    if (m.offsets == nullptr) {
        t0 = (int64_t)blockIdx.y * ROWS;
        n = (int)min((int64_t)ROWS, m.M - t0);
        if (failed(m.status)) return;
    } else {
        if (threadIdx.x < 4) found[threadIdx.x] = 0;
        __syncthreads();
        const int nr = m.lora.R > 0 ? m.lora.R : p.E;
        bool bad = offsets_bad(m.offsets, nr, m.M, threadIdx.x, TK_WARPS * 32);
        if (m.lora.R > 0) bad |= ids_bad(m.lora.ids, m.lora.R, m.lora.L, threadIdx.x, TK_WARPS * 32);
        if (bad) found[3] = 1;
        __syncthreads();
        if (found[3]) {
            if (threadIdx.x == 0) set_status(m.status, GPTQ_ERR_ARG);
            grid_wait();
            return;
        }
        if (failed(m.status)) {
            grid_wait();
            return;
        }
        if (m.lora.R > 0) {
            const int begin = __ldg(m.offsets), end = __ldg(m.offsets + m.lora.R);
            t0 = begin + (int64_t)blockIdx.y * ROWS;
            n = (int)min((int64_t)ROWS, end - t0);
        } else {
            // the blockIdx.y-th group of ROWS rows, ranges in order
            if (warp == 0) {
                int base = 0;
                for (int e0 = 0; e0 < p.E; e0 += 32) {
                    const int x = e0 + lane;
                    int begin = 0, cnt = 0;
                    if (x < p.E) {
                        begin = __ldg(m.offsets + x);
                        cnt = __ldg(m.offsets + x + 1) - begin;
                    }
                    const int nt = (cnt + ROWS - 1) / ROWS;
                    int sum = nt;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const int v = __shfl_up_sync(~0u, sum, d);
                        if (lane >= d) sum += v;
                    }
                    const int j = (int)blockIdx.y - (base + sum - nt);
                    if (nt > 0 && j >= 0 && j < nt) {
                        found[0] = x;
                        found[1] = begin + j * ROWS;
                        found[2] = min(ROWS, cnt - j * ROWS);
                    }
                    base += __shfl_sync(~0u, sum, 31);
                    if (base > (int)blockIdx.y) break;
                }
            }
            __syncthreads();
            e = found[0];
            t0 = found[1];
            n = found[2];
        }
    }
    if (n <= 0) {
        grid_wait();
        return;
    }

    const int c0 = blockIdx.x * TK_CH;
    const int64_t erow = (int64_t)e * m.w.N;
    const int nw = (int)(((int64_t)m.w.K * B + 31) / 32);
    const int K = m.w.K;
    const T *X = static_cast<const T *>(m.X);
    const int32_t *gi = IDX ? m.w.g_idx + (int64_t)e * K : nullptr;
    // channels g, g + 8, ... of the block (past the last channel the last one again: its sums are
    // not written)
    const uint32_t *row[NR];
    int last[NR];                                       // their scales' rows
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        last[i] = min(c0 + g + 8 * i, m.w.N - 1);
        row[i] = m.w.words + (erow + last[i]) * m.w.ldw + (warp * 4 + quad) * B;
    }
    float acc[2][4];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[a][i] = 0.f;

    // a step: the warp's quads cover 4 chunks of 32 columns; the warps take steps in turn. Words and
    // scales are requested a step ahead only by the next block on the SM: four of them fit, and all
    // blocks of a layer run at once (with words held a step ahead three fitted, and the few blocks
    // over took as long again).
    const int steps = (K + 127) / 128, mine = (steps - warp + TK_WARPS - 1) / TK_WARPS;
    uint32_t w[NR][B];
    float sc[NR];
    auto fetch = [&](int j) {
        if (j >= mine) return;
        const int chunk = (warp + j * TK_WARPS) * 4 + quad, by = j * (TK_WARPS * 4 * B);
        if ((chunk + 1) * B <= nw) {
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const uint32_t *r = row[i] + by;
                if (B == 3 || !p.vec) {
#pragma unroll
                    for (int e = 0; e < B; ++e) w[i][e] = __ldg(r + e);
                } else if constexpr (B == 2) {
                    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(r));
                    w[i][0] = v.x; w[i][1] = v.y;
                } else if constexpr (B != 3) {
#pragma unroll
                    for (int e = 0; e < B; e += 4) {
                        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(r + e));
                        w[i][e] = v.x; w[i][e + 1] = v.y; w[i][e + 2] = v.z; w[i][e + 3] = v.w;
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < NR; ++i)
#pragma unroll
                for (int e = 0; e < B; ++e) w[i][e] = chunk * B + e < nw ? __ldg(row[i] + by + e) : 0u;
        }
        if (!IDX && p.fold) {
#pragma unroll
            for (int i = 0; i < NR; ++i)
                sc[i] = chunk * 32 < K ? __ldg(m.w.scales + (erow + last[i]) * m.w.groups + ((chunk * 32) >> m.w.gshift))
                                       : 0.f;
        }
    };
    fetch(0);

    // X by spans of columns. Piece q of chunk c stands at q ^ (c >> 1 & 1), rows 32 bytes apart
    // modulo 128: the eight lanes that read together then meet eight different 16-byte banks.
    const int pitch = p.span * 2 + TK_PAD;
    const int rounds = (steps + TK_WARPS - 1) / TK_WARPS, per_span = p.span / TK_SPAN;
    auto stage = [&](int round) {
        const int k0 = round * TK_SPAN, chunks = min(p.span, (K - k0 + 127) & ~127) / 32;
        if (round > 0) __syncthreads();                 // everyone is done with the span before
        for (int r = 0; r < n; ++r)
        for (int c = threadIdx.x; c < chunks; c += TK_WARPS * 32) {
            const int k = k0 + c * 32;
            const T *src = X + (t0 + r) * m.ldx + k;
            uint32_t x[16];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t v[4] = {0u, 0u, 0u, 0u};
                const int left = K - k - 8 * q;
                if (left >= 8 && p.xvec) {
                    const uint4 y = __ldg(reinterpret_cast<const uint4 *>(src + 8 * q));
                    v[0] = y.x; v[1] = y.y; v[2] = y.z; v[3] = y.w;
                } else {
                    const unsigned short *s = reinterpret_cast<const unsigned short *>(src + 8 * q);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < left) v[e >> 1] |= (uint32_t)__ldg(s + e) << (16 * (e & 1));
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * q + e] = v[e];
            }
            to_pair_order<B>(x);
            uint8_t *d = xs + r * pitch + c * 64;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint4 *>(d + ((q ^ ((c >> 1) & 1)) << 4)) =
                    make_uint4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
        }
        __syncthreads();
    };
#pragma unroll 1
    for (int round = 0; round < rounds; ++round) {
        if (round % per_span == 0) stage(round);
        if (round >= mine) continue;
        const uint8_t *xr = xs + g * pitch + (((round % per_span) * TK_WARPS + warp) * 4 + quad) * 64;
        const int k0 = ((warp + round * TK_WARPS) * 4 + quad) * 32;
        uint32_t all[IDX ? NR : 1][16];                 // by g_idx a chunk is scaled as a whole
        if constexpr (IDX) {
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                unpack32<B, T, false>(w[i], all[i]);
                if (k0 < K)
                    scale32_by_index<T, B, false>(all[i], m.w.scales + (erow + last[i]) * m.w.groups, gi, k0, K,
                                                  m.w.groups, m.status);
            }
        }
        // eight columns a lane at a time: the pairs of four channels, then their MMAs
        auto eight = [&](auto I) {
            constexpr int i8 = decltype(I)::value;
            uint32_t v[NR][4];
            uint4 y = make_uint4(0u, 0u, 0u, 0u);
            if (g < n) y = *reinterpret_cast<const uint4 *>(xr + ((i8 ^ (quad >> 1)) << 4));
            const uint32_t x[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                if constexpr (IDX) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i][j] = all[i][4 * i8 + j];
                } else {
                    unpack8<B, T, i8>(w[i], v[i]);
                    if (p.fold) scale8<T>(v[i], sc[i]);
                }
            }
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    mma_16816<T>(acc[a], v[2 * a][2 * j], v[2 * a + 1][2 * j], v[2 * a][2 * j + 1],
                                 v[2 * a + 1][2 * j + 1], x[2 * j], x[2 * j + 1]);
        };
        eight(std::integral_constant<int, 0>{});
        eight(std::integral_constant<int, 1>{});
        eight(std::integral_constant<int, 2>{});
        eight(std::integral_constant<int, 3>{});
        fetch(round + 1);
    }
    // fragment (16 channels x 8 rows): channel g (+ 8), rows 2 quad, 2 quad + 1
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            part[warp][2 * quad + (i & 1)][a * 16 + g + 8 * (i >> 1)] = acc[a][i];
    __syncthreads();
    if (m.lora.R > 0) grid_wait();
    T *Y = static_cast<T *>(m.Y);
    for (int i = threadIdx.x; i < ROWS * TK_CH; i += TK_WARPS * 32) {
        const int row = i / TK_CH, c = i % TK_CH, ch = c0 + c;
        if (row >= n || ch >= m.w.N) continue;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < TK_WARPS; ++w) sum += part[w][row][c];
        if (!p.fold) sum *= __ldg(m.w.scales + erow + ch);
        if (m.lora.R > 0) {
            const int t = (int)t0 + row;
            const int s = request_of(m.offsets, m.lora.R, t);
            const int id = __ldg(m.lora.ids + s);
            if (id >= 0) {
                const int ids[1] = {id};
                const int64_t ts[1] = {t};
                float add[1];
                lora_terms<T, 0, 1>(m.lora, ids, ts, ch, m.w.N, add);
                sum += add[0];
            }
        }
        Y[(t0 + row) * m.ldy + ch] = from_f32<T>(sum);
    }
}

template <typename T, bool IDX>
static gptq_status launch_token(const TokenArg &p, int bits, dim3 grid, cudaStream_t st) {
    const size_t smem = (size_t)p.rows * (p.span * 2 + TK_PAD);
    switch (bits) {
        case 2: return launch_pdl(k_matmul_token<T, 2, IDX>, grid, TK_WARPS * 32, smem, TK_SMEM + 8 * TK_PAD, 1, st, p);
        case 3: return launch_pdl(k_matmul_token<T, 3, IDX>, grid, TK_WARPS * 32, smem, TK_SMEM + 8 * TK_PAD, 1, st, p);
        case 4: return launch_pdl(k_matmul_token<T, 4, IDX>, grid, TK_WARPS * 32, smem, TK_SMEM + 8 * TK_PAD, 1, st, p);
        default: return launch_pdl(k_matmul_token<T, 8, IDX>, grid, TK_WARPS * 32, smem, TK_SMEM + 8 * TK_PAD, 1, st, p);
    }
}

gptq_status matmul_token(const MatmulArg &m, int dtype, int bits, cudaStream_t st) {
    constexpr int rows = 8;
    TokenArg p{};
    p.m = m;
    p.E = m.lora.R > 0 ? 1 : m.w.E;
    p.fold = m.w.groups > 0 ? 1 : 0;
    p.vec = aligned(m.w.words, 16) && m.w.ldw % 4 == 0;
    p.xvec = aligned(m.X, 16) && m.ldx % 8 == 0;
    p.rows = (int)std::min<int64_t>(rows, m.M);
    p.span = std::min((m.w.K + TK_SPAN - 1) / TK_SPAN, std::max(1, TK_SMEM / (p.rows * 2 * TK_SPAN))) * TK_SPAN;
    // groups of rows there can be, at most: one of each range that has a row, and the full ones
    const int64_t items = p.E == 1 ? (m.M + rows - 1) / rows : std::min<int64_t>(p.E, m.M) + m.M / rows;
    const dim3 grid((m.w.N + TK_CH - 1) / TK_CH, (unsigned)items);
    const bool indexed = m.w.g_idx != nullptr;
    if (dtype == GPTQ_BF16)
        return indexed ? launch_token<__nv_bfloat16, true>(p, bits, grid, st)
                       : launch_token<__nv_bfloat16, false>(p, bits, grid, st);
    return indexed ? launch_token<__half, true>(p, bits, grid, st) : launch_token<__half, false>(p, bits, grid, st);
}

}  // namespace gptq
