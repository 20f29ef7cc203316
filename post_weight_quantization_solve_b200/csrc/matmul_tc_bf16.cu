// The tiled packed-weight products for bf16 rows (one translation unit a type, so that they
// compile side by side).
#include "matmul_tc.cuh"

namespace gptq {
gptq_status matmul_tc_bf16(const CUtensorMap &map, const CUtensorMap &wmap, const MmTcArg &p, int dir, int bits, bool pair, int blocks,
                         size_t smem, cudaStream_t st) {
    return dir == 0 ? launch_tc_bits<__nv_bfloat16, 0>(map, wmap, p, bits, pair, blocks, smem, st)
                    : launch_tc_bits<__nv_bfloat16, 1>(map, wmap, p, bits, pair, blocks, smem, st);
}
}  // namespace gptq
