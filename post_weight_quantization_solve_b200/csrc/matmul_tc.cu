// Which tiles a packed-weight product on the tensor cores takes (the kernel is in matmul_tc.cuh).
#include <atomic>

#include "matmul_tc.cuh"

namespace gptq {

static size_t ring_bytes(int bits, int dir) {
    switch (bits) {
        case 2: return dir == 0 ? MmRing<2, 0>::BYTES : MmRing<2, 1>::BYTES;
        case 3: return dir == 0 ? MmRing<3, 0>::BYTES : MmRing<3, 1>::BYTES;
        case 4: return dir == 0 ? MmRing<4, 0>::BYTES : MmRing<4, 1>::BYTES;
        default: return dir == 0 ? MmRing<8, 0>::BYTES : MmRing<8, 1>::BYTES;
    }
}

// The packed rows of all experts as boxes of `rows` rows x 128 codes. False when the rows do not
// start on 16-byte boundaries.
static bool words_map(CUtensorMap *map, const PackedArg &w, int bits, int rows) {
    EncodeTiled enc = encode_tiled();
    if (!enc || !aligned(w.words, 16) || w.ldw % 4 != 0) return false;
    const cuuint64_t dim[2] = {(cuuint64_t)(((int64_t)w.K * bits + 31) / 32), (cuuint64_t)w.E * w.N};
    const cuuint64_t stride[1] = {(cuuint64_t)w.ldw * 4};
    const cuuint32_t box[2] = {(cuuint32_t)(4 * bits), (cuuint32_t)rows};
    const cuuint32_t step[2] = {1, 1};
    const CUtensorMapSwizzle swizzle = bits == 2   ? CU_TENSOR_MAP_SWIZZLE_32B
                                       : bits == 3 ? CU_TENSOR_MAP_SWIZZLE_NONE
                                       : bits == 4 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                   : CU_TENSOR_MAP_SWIZZLE_128B;
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint32_t *>(w.words), dim, stride, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of `size` blocks that run at once, one block an SM: SMs that a processing cluster has left
// over stay idle (33 of 4 and 15 of 8 on the 148 SMs of a B200), and a cluster that waits for others
// to end would double the time. Asked once a device.
static int matmul_tc_clusters(int size) {
    static std::atomic<int> known[64][9];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 || size < 1 || size > 8) return 1;
    int n = known[dev][size].load(std::memory_order_relaxed);
    if (n > 0) return n;
    n = size == 1 ? device_sms() : matmul_tc_occupancy(size);
    if (n < 1) n = std::max(1, device_sms() / size);
    known[dev][size].store(n, std::memory_order_relaxed);
    return n;
}

// dir 0: Y = X W^T, 1: dX = dY W.
gptq_status matmul_tc(const MatmulArg &m, int dir, int dtype, int bits, cudaStream_t st) {
    MmTcArg p{};
    p.m = m;
    p.out = dir == 0 ? m.w.N : m.w.K;
    p.inner = dir == 0 ? m.w.K : m.w.N;
    p.E = m.lora.R > 0 ? 1 : m.w.E;
    p.fold = (dir == 1 || m.w.groups > 0 || m.lora.R > 0) ? 1 : 0;
    p.yvec = aligned(m.Y, 16) && m.ldy % 8 == 0;
    const int sms = device_sms();
    const int steps = (p.inner + MM_BK - 1) / MM_BK;
    // tiles of `cols` rows there can be, at most: one of each range that has a row, and the full ones
    auto tiles = [&](int width, int cols) {
        return (int64_t)((p.out + width - 1) / width) * (std::min<int64_t>(p.E, m.M) + m.M / cols);
    };
    // Pairs of blocks on tiles of 256 rows where the ranges fill such tiles and there are enough of
    // them; single blocks on 128 rows elsewhere, their contraction split over a cluster while that
    // leaves machine idle.
    const int64_t mean = m.M / p.E;
    const bool pair = mean > 128 && p.out > MM_LANES && 2 * tiles(2 * MM_LANES, 256) >= sms;
    // (beside the words of 8 bits, the partial sums of 128 rows would leave the input gradient one
    // operand stage: its split tiles have 64 rows)
    p.cols = pair ? 256 : 128;
    p.split = 1;
    const int split_cols = dir == 1 && bits == 8 ? 64 : 128;
    if (!pair)
        while (p.split < 8 && tiles(MM_LANES, split_cols) <= matmul_tc_clusters(2 * p.split) && steps >= 4 * p.split)
            p.split *= 2;
    if (p.split > 1) p.cols = split_cols;
    // large boxes of X (few copies to issue), smaller ones where most ranges have a few rows
    p.box_rows = mean <= 32 ? 32 : mean <= 64 ? 64 : MM_ROWS;
    CUtensorMap map{};
    if (!rows_map(&map, m.X, dtype, m.M, p.inner, m.ldx, p.box_rows)) p.box_rows = 0;
    CUtensorMap wmap{};
    p.wtiled = words_map(&wmap, m.w, bits, dir == 0 ? MmRing<4, 0>::ROWS : MmRing<4, 1>::ROWS);
    // two accumulators where they fit beside the forward product's A stages
    p.accs = dir == 1 || !pair ? 2 : 1;
    p.acc_cols = p.cols;
    // staging: a whole tall tile where it holds the only accumulator, partial sums in fp32 when split
    p.epi = p.split > 1 ? p.cols * MM_LANES * 4 : p.accs == 1 ? p.cols * MM_LANES * 2 : 32 * MM_LANES * 2;
    const int stage = MM_B_BYTES + (dir == 1 ? MM_A_BYTES : 0);
    size_t fixed = ring_bytes(bits, dir) + p.epi + MM_TABLE + 1024 + 320;
    // by g_idx: each unpacking thread keeps its row's scales in shared memory, 1,536 bytes a group, where
    // they leave two operand stages (gathered from global memory for each code, they cost 13,000 clocks
    // a step). Groups that fit, by bits 2, 3, 4, 8: forward 83, 75, 67, 67 with single blocks, 46, 38,
    // 30, 30 with pairs and split tiles; input gradient 49, 45, 49, 41, split 11, 7, 11, 25. Neither
    // pairs nor the split are given up for a table.
    const size_t table = (size_t)m.w.groups * MM_WARP_OUT * 32 * 4;
    if (m.w.g_idx && fixed + table + 2 * stage <= SMEM_MOST) {
        p.idx_table = 1;
        fixed += table;
    }
    p.stages = (int)std::min<size_t>(MM_MAX_STAGES, (SMEM_MOST - fixed) / stage);
    const size_t smem = fixed + (size_t)p.stages * stage;
    const int cluster = pair ? 2 : p.split;
    const int64_t groups = std::min<int64_t>(tiles(pair ? 2 * MM_LANES : MM_LANES, p.cols), matmul_tc_clusters(cluster));
    const int blocks = (int)std::max<int64_t>(1, groups) * cluster;
    return dtype == GPTQ_BF16 ? matmul_tc_bf16(map, wmap, p, dir, bits, pair, blocks, smem, st)
                              : matmul_tc_fp16(map, wmap, p, dir, bits, pair, blocks, smem, st);
}

}  // namespace gptq
