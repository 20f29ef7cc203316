// Packed-weight products for a few rows: Y[t] = W^_e X[t] (+ adapters) when decoding.
//
// With a handful of rows the product is bound by reading the packed words once, so the kernel
// is laid out for that: a block takes 32 output channels of one range and up to 8 (or 16) of
// its rows; its 8 warps split the contraction, and each lane reads whole chunks of 32 codes,
// several requests in flight. Four lanes of a quad hold four neighbouring chunks of one row,
// which is the m16n8k16 fragment layout with the contraction index permuted: a sum does not
// care, as long as the rows X are read in the same order, and they are (a lane reads the 32
// values of its own chunk). The matrix instruction adds in fp32; the warps' partial sums meet
// in shared memory in warp order.
//
// Scales: one scale a channel enters in fp32 at the end (the codes are exact); with input
// groups each weight is rounded once to the rows' 16-bit type, as in the tiled kernel.
#include <algorithm>

#include "matmul.cuh"

namespace gptq {

namespace {
constexpr int TK_WARPS = 8;
}  // namespace

struct TokenArg {
    MatmulArg m;
    int fold, vec, xvec, E;
};

template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (Half2<T>::kType == 1)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// U chunks (32 U codes) of a row in whole 16-byte pieces, or word by word.
template <int B, int U>
__device__ __forceinline__ void load_unit(const uint32_t *row, int chunk, int nw, bool vec,
                                          uint32_t (&w)[U * B]) {
    const int at = chunk * B;
    if (row != nullptr && vec && at + U * B <= nw) {
#pragma unroll
        for (int j = 0; j < U * B; j += 4) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(row + at + j));
            w[j] = v.x; w[j + 1] = v.y; w[j + 2] = v.z; w[j + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < U * B; ++j) w[j] = row != nullptr && at + j < nw ? __ldg(row + at + j) : 0u;
    }
}

// Eight neighbouring values of a row in the pair order of unpack32<B, T, false>.
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

// MT fragments of 16 channels, NT of 8 rows.
template <typename T, int B, int NT, int MT>
__global__ void __launch_bounds__(TK_WARPS * 32, MT == 1 ? 2 : 1)
    k_matmul_token(const __grid_constant__ TokenArg p) {
    constexpr int U = B == 3 ? 4 : B == 2 ? 2 : 1;      // chunks that fill 16-byte pieces
    constexpr int ROWS = 8 * NT, TK_CH = 16 * MT, NR = 2 * MT;
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
    const int32_t *gi = m.w.g_idx ? m.w.g_idx + (int64_t)e * K : nullptr;
    const uint32_t *rows[NR];
    const float *srow[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int ch = c0 + g + 8 * i;
        const bool in = ch < m.w.N;
        rows[i] = in ? m.w.words + (erow + ch) * m.w.ldw : nullptr;
        srow[i] = in && p.fold ? m.w.scales + (erow + ch) * m.w.groups : nullptr;
    }
    float acc[MT][NT][4];
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[a][b][i] = 0.f;

    // a step: the warp's quads cover 4 U chunks of 32 columns. Words and scales of the next step
    // are requested before this one's are used.
    const int steps = (K + 128 * U - 1) / (128 * U);
    uint32_t cur[NR][U * B], nxt[NR][U * B];
    float sc[NR][U], sn[NR][U];
    auto fetch = [&](int step, uint32_t (&w)[NR][U * B], float (&s)[NR][U]) {
        const int chunk = (step * 4 + quad) * U;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            load_unit<B, U>(step < steps ? rows[i] : nullptr, chunk, nw, p.vec, w[i]);
            if (p.fold && !gi) {
#pragma unroll
                for (int c = 0; c < U; ++c)
                    s[i][c] = srow[i] && (chunk + c) * 32 < K ? __ldg(srow[i] + (((chunk + c) * 32) >> m.w.gshift)) : 0.f;
            }
        }
    };
    fetch(warp, cur, sc);
#pragma unroll 1
    for (int step = warp; step < steps; step += TK_WARPS) {
        if (step + TK_WARPS < steps) fetch(step + TK_WARPS, nxt, sn);
#pragma unroll
        for (int c = 0; c < U; ++c) {
            const int k0 = ((step * 4 + quad) * U + c) * 32;
            uint32_t x[NT][16];
#pragma unroll
            for (int b = 0; b < NT; ++b) {
                const int row = b * 8 + g;
                const T *src = X + (t0 + row) * m.ldx + k0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t v[4] = {0u, 0u, 0u, 0u};
                    const int left = row < n ? K - k0 - 8 * q : 0;
                    if (left >= 8 && p.xvec) {
                        const uint4 y = __ldg(reinterpret_cast<const uint4 *>(src + 8 * q));
                        v[0] = y.x; v[1] = y.y; v[2] = y.z; v[3] = y.w;
                    } else if (left > 0) {
                        const unsigned short *s = reinterpret_cast<const unsigned short *>(src + 8 * q);
#pragma unroll 1
                        for (int i = 0; i < 8 && i < left; ++i) {
                            const uint32_t h = (uint32_t)__ldg(s + i) << (16 * (i & 1));
                            v[0] |= i >> 1 == 0 ? h : 0u;
                            v[1] |= i >> 1 == 1 ? h : 0u;
                            v[2] |= i >> 1 == 2 ? h : 0u;
                            v[3] |= i >> 1 == 3 ? h : 0u;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[b][4 * q + i] = v[i];
                }
                to_pair_order<B>(x[b]);
            }
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                uint32_t v[2][16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int i = 2 * a + h;
                    uint32_t w[B];
#pragma unroll
                    for (int j = 0; j < B; ++j) w[j] = cur[i][c * B + j];
                    unpack32<B, T, false>(w, v[h]);
                    if (p.fold) {
                        if (gi) {
                            if (srow[i] && k0 < K)
                                scale32_by_index<T, B, false>(v[h], srow[i], gi, k0, K, m.w.groups, m.status);
                        } else {
                            scale32<T>(v[h], sc[i][c]);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int b = 0; b < NT; ++b)
                        mma_16816<T>(acc[a][b], v[0][2 * j], v[1][2 * j], v[0][2 * j + 1], v[1][2 * j + 1],
                                     x[b][2 * j], x[b][2 * j + 1]);
            }
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
#pragma unroll
            for (int j = 0; j < U * B; ++j) cur[i][j] = nxt[i][j];
#pragma unroll
            for (int c = 0; c < U; ++c) sc[i][c] = sn[i][c];
        }
    }
    // fragment (16 channels x 8 rows): channel g (+ 8), rows 2 quad, 2 quad + 1
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part[warp][b * 8 + 2 * quad + (i & 1)][a * 16 + g + 8 * (i >> 1)] = acc[a][b][i];
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

template <typename T, int NT, int MT>
static gptq_status launch_token(const TokenArg &p, int bits, dim3 grid, cudaStream_t st) {
    switch (bits) {
        case 2: return launch_pdl(k_matmul_token<T, 2, NT, MT>, grid, TK_WARPS * 32, 0, 1, st, p);
        case 3: return launch_pdl(k_matmul_token<T, 3, NT, MT>, grid, TK_WARPS * 32, 0, 1, st, p);
        case 4: return launch_pdl(k_matmul_token<T, 4, NT, MT>, grid, TK_WARPS * 32, 0, 1, st, p);
        default: return launch_pdl(k_matmul_token<T, 8, NT, MT>, grid, TK_WARPS * 32, 0, 1, st, p);
    }
}

gptq_status matmul_token(const MatmulArg &m, int dtype, int bits, cudaStream_t st) {
    TokenArg p{};
    p.m = m;
    p.E = m.lora.R > 0 ? 1 : m.w.E;
    p.fold = m.w.groups > 0 ? 1 : 0;
    p.vec = aligned(m.w.words, 16) && m.w.ldw % 4 == 0;
    p.xvec = aligned(m.X, 16) && m.ldx % 8 == 0;
    // one range: up to 16 rows at once, which share the reading of X between 32 channels;
    // several ranges: most have a few rows
    const bool wide = p.E == 1 && m.M > 8;
    const int rows = wide ? 16 : 8, channels = wide ? 32 : 16;
    const int64_t items = p.E == 1 ? (m.M + rows - 1) / rows : std::min<int64_t>(p.E, m.M) + m.M / rows;
    const dim3 grid((m.w.N + channels - 1) / channels, (unsigned)items);
    if (dtype == GPTQ_BF16)
        return wide ? launch_token<__nv_bfloat16, 2, 2>(p, bits, grid, st)
                    : launch_token<__nv_bfloat16, 1, 1>(p, bits, grid, st);
    return wide ? launch_token<__half, 2, 2>(p, bits, grid, st)
                : launch_token<__half, 1, 1>(p, bits, grid, st);
}

}  // namespace gptq
