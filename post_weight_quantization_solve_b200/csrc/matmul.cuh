// Shared parts of the packed-weight products (matmul_tc.cu, matmul_token.cu, matmul_dw.cu,
// lora.cu): the packed layer as kernels see it, unpacking of 32 codes into 16-bit pairs, the
// table of ragged row ranges, and the tiled-copy descriptors.
//
// A packed row is a little-endian bit stream (gptq_pack_codes), so 32 codes fill exactly
// `bits` words and one thread turns those words into 16 registers of two values each. The
// values c - z are integers of at most 8 bits, exact in bf16 and fp16.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "gptq_matmul.h"
#include "tc_ptx.cuh"

namespace gptq {

// ---- arguments as kernels see them ---------------------------------------------------------

struct PackedArg {
    const uint32_t *words;    // [E][N][ldw]
    int64_t ldw;
    const float *scales;      // [E][N] (groups == 0) or [E][N][groups]
    const int32_t *g_idx;     // [E][K] or NULL (column k in group k >> gshift)
    int E, N, K;
    int groups, gshift;
};

// Adapters beside a product, and the rows that use them.
struct LoraArg {
    const void *P;            // forward: B [L][N][rank]; input gradient: A [L][rank][K]
    const __nv_bfloat16 *T3;  // [M][LORA_PARTS rank]: the rank-space rows as parts
    const int32_t *ids;       // [R] adapter of each request, -1 none
    int R, L, rank;
};

// A rank-space value is kept as three bf16 parts that add up to it (24 bits, the range of fp32: it is
// no row of the model, and fp16 would lose small gradients and overflow on large ones). Outputs of 16
// bits take the first two (16 bits, bf16) or all of them (fp16; two where they are matrix operands).
// The adapters' gradients, fp32 sums, take all of them, fp16 rows a scaled pair (lora.cu).
constexpr int LORA_PARTS = 3;

struct MatmulArg {
    PackedArg w;
    const void *X;            // [M][ldx]: tokens (forward) or output gradients (input gradient)
    int64_t ldx;
    void *Y;                  // [M][ldy]
    int64_t ldy;
    const int32_t *offsets;   // [E + 1], or [R + 1] with adapters, or NULL (all M rows)
    int64_t M;
    LoraArg lora;             // R == 0: none
    int32_t *status;
};

// One gradient of the adapters: P [M][ldp] against the rank-space rows Q [M][ldq], `halves` parts of
// them side by side, each adapter's times 2^(141 - e) where `most` holds its largest value with the
// exponent field e; parts: room for the sums of adapter_parts() parts where there is more than one.
struct AdapterGrad {
    const void *P;
    int64_t ldp;
    int np;
    const void *Q;
    int ldq, halves;
    const uint32_t *most;
    float *out, *parts;
    int transposed;
};

constexpr int MATMUL_MAX_EXPERTS = 512;

// ---- 16-bit types --------------------------------------------------------------------------

// The bits of -v (an integer of at most mantissa + 1 bits) in a 16-bit floating type.
__host__ __device__ constexpr uint32_t negative_bits(int v, int mantissa, int bias) {
    int e = 0;
    while ((v >> e) > 1) ++e;
    return 0x8000u | (uint32_t)((bias + e) << mantissa) | ((((uint32_t)v << mantissa) >> e) & ((1u << mantissa) - 1u));
}

template <typename T>
struct Half2;
template <>
struct Half2<__nv_bfloat16> {
    static constexpr uint32_t kMagic = 0x43004300u;     // 128 + c for c < 128
    static constexpr uint32_t kType = 1;                // instruction-descriptor type code
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    // (128 + c 2^UP) / 2^UP - 128 / 2^UP - Z = c - Z, every step exact
    template <int UP, int Z>
    static __device__ __forceinline__ uint32_t scaled(uint32_t v) {
        constexpr uint32_t inv = (127u - UP) << 7;                     // 2^-UP
        constexpr uint32_t cc = negative_bits((128 >> UP) + Z, 7, 127) * 0x00010001u;
        uint32_t d;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(v), "r"(inv * 0x00010001u), "r"(cc));
        return d;
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t d;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
        return d;
    }
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
};
template <>
struct Half2<__half> {
    static constexpr uint32_t kMagic = 0x64006400u;     // 1024 + c for c < 1024
    static constexpr uint32_t kType = 0;
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    // (1024 + c 2^UP) / 2^UP - 1024 / 2^UP - Z = c - Z, every step exact
    template <int UP, int Z>
    static __device__ __forceinline__ uint32_t scaled(uint32_t v) {
        constexpr uint32_t inv = (15u - UP) << 10;
        constexpr uint32_t cc = negative_bits((1024 >> UP) + Z, 10, 15) * 0x00010001u;
        uint32_t d;
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(v), "r"(inv * 0x00010001u), "r"(cc));
        return d;
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t d;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
        return d;
    }
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    }
};
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// ---- unpacking -----------------------------------------------------------------------------

template <uint32_t MASK, uint32_t OR>
__device__ __forceinline__ uint32_t and_or(uint32_t a) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "n"(MASK), "n"(OR));
    return d;
}

// 32 codes (B words) -> c - z as 16 pairs. Each code is placed under the exponent bits of 128
// (bf16) or 1024 (fp16), where its value is the number's low mantissa; one packed operation then
// gives c - z exactly: a subtraction, or, for a code masked in place a few bits up in the
// mantissa (128 + 8 c), a multiply-add by the power of two, which saves the shift.
// Codes come out of a word two 16-bit lanes at a time (code i with code i + 4, or i + 8 for 2
// bits). NATURAL: byte permutes put neighbouring columns together; otherwise the pairs stay as
// they come, in the order of pair_column, for a reader whose rows are in that order too.
template <int B, bool NATURAL>
__host__ __device__ constexpr int pair_column(int i, int h) {
    return NATURAL || B == 8 ? 2 * i + h
           : B == 2          ? (i / 8) * 16 + i % 8 + 8 * h
                             : (i / 4) * 8 + i % 4 + 4 * h;
}

// q[J..]: codes J.. of both lanes of a field as c - z. Code J sits at bit B (J mod PER) of the
// field shifted by whole runs of PER codes.
template <int B, typename T, int J, int LANE, int PER, uint32_t MASK, int Z>
__device__ __forceinline__ void pair_fields(uint32_t f, uint32_t (&q)[LANE]) {
    if constexpr (J < LANE) {
        constexpr int UP = B * (J % PER);
        const uint32_t v = and_or<(MASK << UP), Half2<T>::kMagic>(f >> (B * (J - J % PER)));
        if constexpr (UP == 0) q[J] = Half2<T>::sub(v, Half2<T>::kMagic + Z * 0x00010001u);
        else q[J] = Half2<T>::template scaled<UP, Z>(v);
        pair_fields<B, T, J + 1, LANE, PER, MASK, Z>(f, q);
    }
}

template <int B, typename T, bool NATURAL = true>
__device__ __forceinline__ void unpack32(const uint32_t (&w)[B], uint32_t (&out)[16]) {
    using H = Half2<T>;
    constexpr uint32_t M = H::kMagic;
    if constexpr (B == 8) {
        constexpr uint32_t hi = M >> 24;     // the exponent byte
        constexpr uint32_t hi4 = hi * 0x01010101u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t p = __byte_perm(w[i], hi4, h ? 0x4342 : 0x4140);
                if constexpr (H::kType == 1) {
                    // 128 + (c & 127) less 128 where c >= 128 and 256 elsewhere
                    const uint32_t x = p & 0xff7fff7fu;
                    const uint32_t y = (p & 0x43804380u) ^ 0x00800080u;
                    out[2 * i + h] = H::sub(x, y);
                } else {
                    out[2 * i + h] = H::sub(p, M + 0x00800080u);
                }
            }
        }
    } else {
        // fields of four (2 bits: eight) codes in each 16-bit lane, and a word's worth of them
        constexpr int LANE = B == 2 ? 8 : 4, FIELDS = 16 / LANE;
        constexpr uint32_t MASK = ((1u << B) - 1u) * 0x00010001u;
        constexpr int z = 1 << (B - 1);
        constexpr int MANT = H::kType == 1 ? 7 : 10;         // mantissa bits that hold codes
        constexpr int PER = MANT / B;                        // codes read without a shift
#pragma unroll
        for (int i = 0; i < FIELDS; ++i) {
            uint32_t f;
            if constexpr (B == 3) {
                const uint32_t g = i == 0 ? w[0]
                                   : i == 1 ? __funnelshift_r(w[0], w[1], 24)
                                   : i == 2 ? __funnelshift_r(w[1], w[2], 16)
                                            : (w[2] >> 8);
                f = (g & 0xfffu) | ((g << 4) & 0x0fff0000u);
            } else {
                f = w[i];
            }
            uint32_t q[LANE];
            pair_fields<B, T, 0, LANE, PER, MASK, z>(f, q);
            if constexpr (NATURAL) {
#pragma unroll
                for (int j = 0; j < LANE / 2; ++j) {
                    out[LANE * i + j] = __byte_perm(q[2 * j], q[2 * j + 1], 0x5410);
                    out[LANE * i + LANE / 2 + j] = __byte_perm(q[2 * j], q[2 * j + 1], 0x7632);
                }
            } else {
#pragma unroll
                for (int j = 0; j < LANE; ++j) out[LANE * i + j] = q[j];
            }
        }
    }
}

// Eight of the codes (the I-th of four groups) as 4 pairs, in the order of unpack32<B, T, false>.
template <int B, typename T, int I>
__device__ __forceinline__ void unpack8(const uint32_t (&w)[B], uint32_t (&q)[4]) {
    if constexpr (B == 8) {
        uint32_t all[16], two[8] = {w[2 * I], w[2 * I + 1], 0u, 0u, 0u, 0u, 0u, 0u};
        unpack32<8, T, false>(two, all);
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = all[j];
    } else {
        constexpr uint32_t MASK = ((1u << B) - 1u) * 0x00010001u;
        constexpr int PER = (Half2<T>::kType == 1 ? 7 : 10) / B;
        uint32_t f;
        if constexpr (B == 3) {
            const uint32_t g = I == 0 ? w[0]
                               : I == 1 ? __funnelshift_r(w[0], w[1], 24)
                               : I == 2 ? __funnelshift_r(w[1], w[2], 16)
                                        : (w[2] >> 8);
            f = (g & 0xfffu) | ((g << 4) & 0x0fff0000u);
        } else if constexpr (B == 2) {
            f = w[I >> 1] >> (8 * (I & 1));
        } else {
            f = w[I];
        }
        pair_fields<B, T, 0, 4, PER, MASK, 1 << (B - 1)>(f, q);
    }
}

// What bf16 leaves of a scale, as a pair; nothing of an infinite one.
__device__ __forceinline__ uint32_t rest_of_scale(float s, uint32_t hi) {
    const float rest = s - __uint_as_float(hi & 0xffff0000u);
    const float v = isfinite(rest) ? rest : 0.f;
    return Half2<__nv_bfloat16>::pack(v, v);
}

// Four values' pairs times one scale (as scale32).
template <typename T>
__device__ __forceinline__ void scale8(uint32_t (&v)[4], float s) {
    if constexpr (Half2<T>::kType == 1) {
        const uint32_t hi = Half2<T>::pack(s, s);
        const uint32_t lo = rest_of_scale(s, hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t t;
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(t) : "r"(v[i]), "r"(lo));
            asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v[i]) : "r"(v[i]), "r"(hi), "r"(t));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = Half2<T>::unpack(v[i]);
            v[i] = Half2<T>::pack(f.x * s, f.y * s);
        }
    }
}

// The 32 values times one scale, each product rounded once to the 16-bit type. bf16: the
// scale as a pair of bf16 (16 significant bits), v s_lo + v s_hi in one packed multiply-add.
// fp16 scales can lie below fp16's normal range, so there the products are formed in fp32.
template <typename T>
__device__ __forceinline__ void scale32(uint32_t (&v)[16], float s) {
    if constexpr (Half2<T>::kType == 1) {
        const uint32_t hi = Half2<T>::pack(s, s);
        const uint32_t lo = rest_of_scale(s, hi);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            uint32_t t;
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(t) : "r"(v[i]), "r"(lo));
            asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v[i]) : "r"(v[i]), "r"(hi), "r"(t));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 f = Half2<T>::unpack(v[i]);
            v[i] = Half2<T>::pack(f.x * s, f.y * s);
        }
    }
}

// The 32 values of columns k0 .. k0 + 31, each times the scale of its column's group. Out of
// line: 64 dependent reads a chunk, whatever the registers around it.
template <typename T, int B, bool NATURAL>
__device__ __noinline__ void scale32_indexed(uint32_t *v, const float *row_scales, const int32_t *g_idx,
                                             int k0, int K, int groups, int32_t *status) {
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
        float s[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = k0 + pair_column<B, NATURAL>(i, h);
            int g = k < K ? __ldg(g_idx + k) : 0;
            if ((unsigned)g >= (unsigned)groups) {
                set_status(status, GPTQ_ERR_ARG);
                g = 0;
            }
            s[h] = __ldg(row_scales + g);
        }
        const float2 f = Half2<T>::unpack(v[i]);
        v[i] = Half2<T>::pack(f.x * s[0], f.y * s[1]);
    }
}

template <typename T, int B, bool NATURAL>
__device__ __forceinline__ void scale32_by_index(uint32_t (&v)[16], const float *row_scales,
                                                 const int32_t *g_idx, int k0, int K, int groups,
                                                 int32_t *status) {
    uint32_t t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = v[i];
    scale32_indexed<T, B, NATURAL>(t, row_scales, g_idx, k0, K, groups, status);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = t[i];
}

// Where a lane's column k has its scale in a table of `stride` floats a group (columns past the last
// one: group 0).
__device__ __forceinline__ int group_place(const int32_t *g_idx, int k, int K, int groups, int stride, int32_t *status) {
    int g = k < K ? __ldg(g_idx + k) : 0;
    if ((unsigned)g >= (unsigned)groups) {
        set_status(status, GPTQ_ERR_ARG);
        g = 0;
    }
    return g * stride;
}

// The 32 values of neighbouring columns, each times the scale of its column's group; lane i's `place`
// is column i's in this thread's table. The columns are the same for the whole warp, so their groups
// are read and checked once a lane, not once a code (57 -> 41 us for the input gradient of 666 rows over
// five layers of 1,416 x 1,000).
template <typename T>
__device__ __forceinline__ void scale32_by_table(uint32_t (&v)[16], const float *scales, int place) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float s0 = scales[__shfl_sync(~0u, place, 2 * i)], s1 = scales[__shfl_sync(~0u, place, 2 * i + 1)];
        const float2 f = Half2<T>::unpack(v[i]);
        v[i] = Half2<T>::pack(f.x * s0, f.y * s1);
    }
}

// One fragment of legacy matrix work, for products too small for tiles: D (16 x 8) += A (16 x 16) B (16 x 8).
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

// ---- ragged ranges -------------------------------------------------------------------------

// Row ranges are refused as a whole when an offset is negative, above M or below the one
// before it: then no row is read or written through them. Every block checks all of them.
__device__ __forceinline__ bool offsets_bad(const int32_t *off, int n, int64_t M, int tid,
                                            int nthreads) {
    bool bad = false;
    for (int i = tid; i <= n; i += nthreads) {
        const int v = __ldg(off + i);
        bad |= v < 0 || (int64_t)v > M || (i > 0 && v < __ldg(off + i - 1));
    }
    return bad;
}

__device__ __forceinline__ bool ids_bad(const int32_t *ids, int R, int L, int tid, int nthreads) {
    bool bad = false;
    for (int i = tid; i < R; i += nthreads) {
        const int v = __ldg(ids + i);
        bad |= v < -1 || v >= L;
    }
    return bad;
}

// First request whose end lies behind row t (off[s + 1] > t), by bisection.
__device__ __forceinline__ int request_of(const int32_t *off, int R, int t) {
    int lo = 0, hi = R;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(off + mid + 1) > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// A run is neighbouring rows of one adapter inside a tile. Runs shorter than this are added by the
// outputs' threads, row by row; longer ones are matrix operands of their own (an MMA takes 16
// columns at least, and a round of barriers).
constexpr int LORA_SHORT = 16;

// The adapter terms of one output channel for NROW rows t[i] with adapters id[i] (negative:
// zero): sum_j P_a[ch][j] T[t][j] (forward, P = B) or sum_j P_a[j][ch] T[t][j] (input gradient,
// P = A), fp32. The rows' reads are independent, so they overlap.
template <typename T, int DIR, int NROW>
__device__ __forceinline__ void lora_terms(const LoraArg &l, const int (&id)[NROW], const int64_t (&t)[NROW], int ch,
                                           int channels, float (&add)[NROW]) {
    const int r = l.rank;
#pragma unroll
    for (int i = 0; i < NROW; ++i) add[i] = 0.f;
#pragma unroll 1
    for (int j = 0; j < r; j += 8) {
        constexpr int USED = Half2<T>::kType == 1 ? 2 : 3;
        uint4 tv[USED][NROW], pv[NROW];
#pragma unroll
        for (int i = 0; i < NROW; ++i) {
            pv[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int h = 0; h < USED; ++h) tv[h][i] = make_uint4(0u, 0u, 0u, 0u);
            if (id[i] < 0) continue;
            const __nv_bfloat16 *h0 = l.T3 + t[i] * LORA_PARTS * r + j;
#pragma unroll
            for (int h = 0; h < USED; ++h) tv[h][i] = __ldcg(reinterpret_cast<const uint4 *>(h0 + h * r));
            if constexpr (DIR == 0) {
                pv[i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(l.P) +
                                                              ((int64_t)id[i] * channels + ch) * r + j));
            } else {
                const unsigned short *a = reinterpret_cast<const unsigned short *>(l.P) +
                                          ((int64_t)id[i] * r + j) * channels + ch;
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    w[q] = __ldg(a + (int64_t)(2 * q) * channels) | ((uint32_t)__ldg(a + (int64_t)(2 * q + 1) * channels) << 16);
                pv[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
#pragma unroll
        for (int i = 0; i < NROW; ++i) {
            const uint32_t pp[4] = {pv[i].x, pv[i].y, pv[i].z, pv[i].w};
            float2 sum[4] = {};
#pragma unroll
            for (int h = USED - 1; h >= 0; --h) {
                const uint32_t tt[4] = {tv[h][i].x, tv[h][i].y, tv[h][i].z, tv[h][i].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 f = Half2<__nv_bfloat16>::unpack(tt[q]);
                    sum[q].x += f.x;
                    sum[q].y += f.y;
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 fp = Half2<T>::unpack(pp[q]);
                add[i] = fmaf(fp.x, sum[q].x, add[i]);
                add[i] = fmaf(fp.y, sum[q].y, add[i]);
            }
        }
    }
}

// ---- host ----------------------------------------------------------------------------------

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            ptr = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(ptr);
    }();
    return fn;
}

// A row-major [rows][cols] matrix of a 16-bit type as boxes of 64 columns x box_rows rows in the
// 128-byte swizzle. False when its layout does not allow tiled copies (then plain loads serve).
inline bool rows_map(CUtensorMap *map, const void *ptr, int dtype, int64_t rows, int64_t cols,
                     int64_t ld, int box_rows) {
    EncodeTiled enc = encode_tiled();
    if (!enc || !aligned(ptr, 16) || (ld * 2) % 16 != 0 || rows < 1) return false;
    const cuuint64_t dim[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t stride[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    const cuuint32_t step[2] = {1, 1};
    return enc(map,
               dtype == GPTQ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
               2, const_cast<void *>(ptr), dim, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int device_sms() {
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 148;
}

constexpr size_t SMEM_MOST = 227 * 1024;                // dynamic shared memory of a block without static

// One launch as a programmatic dependent of the previous kernel on the stream, in clusters of
// `cluster` blocks along x, with `smem` bytes of dynamic shared memory; no launch of the kernel takes
// more than `most`. The limit belongs to the kernel and the device, and another host thread's call may
// come between setting it and the launch, so every call sets the same one.
template <typename... KArgs, typename... Args>
inline gptq_status launch_pdl(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, size_t most,
                              int cluster, cudaStream_t st, Args... args) {
    if (smem > most) return GPTQ_ERR_CUDA;
    // (kernels with dynamic shared memory have less than 24 KB of static)
    if (most > 24 * 1024 &&
        cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) != cudaSuccess) {
        cudaGetLastError();
        return GPTQ_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    cudaLaunchKernelEx(&cfg, kernel, KArgs(args)...);
    return launch_status();
}

// Wait for the previous kernel of the stream, then let the next one set up.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void grid_dependency() {
    grid_wait();
    grid_release();
}

}  // namespace gptq
