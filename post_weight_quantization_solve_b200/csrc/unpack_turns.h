// Which set of unpacking warps takes which half of a step (plain C++ beside CUDA, so that a CPU test
// can run it).
//
// The sets wait for a stage of a ring by the parity of its uses. A parity tells two neighbouring uses
// apart and no more: a set that waits for use n of a stage must know that use n - 1 is over, and it
// must have a part in use n, or the ring may be a whole turn further on when it looks. A set takes
// two steps of three, so neither comes by itself.
//
// Operand stages (two at least) are freed by products, which complete in order. Any two steps in
// a row hold a half of every set. So a set that waits at step s for the product of step s - n (n
// stages) has waited at step s - 1 or s - 2 before, for the product of step s - 2 - n or a later
// one, and the use before, of step s - 2 n, is over.
//
// The words' stages are filled by copies, which land in any order. Their halves go to the sets in turn
// over all tiles, so with a multiple of three stages (of a step, or of half a step) every use of a
// stage is read by the same sets: they wait for each of them, one after the other.
#pragma once

#ifdef __CUDACC__
#define GPTQ_TURNS_FN __host__ __device__ __forceinline__
#else
#define GPTQ_TURNS_FN inline
#endif

namespace gptq {

constexpr int UNPACK_SETS = 3;

// A tile's halves 0, 1, ... go to the sets in turn, from the tile's first set `turn` on; this is the
// first one of `set`, and it takes every third from there. The next tile's turn follows.
GPTQ_TURNS_FN int unpack_first_half(int set, int turn) { return (set - turn + UNPACK_SETS) % UNPACK_SETS; }
GPTQ_TURNS_FN int unpack_next_turn(int turn, int halves) { return (turn + halves) % UNPACK_SETS; }

// The set of half i of the n (an even number) of the adapters' steps between two tiles; `turn` is the
// next tile's. They go on in turn. Only where one step is over would the last step's sets be those of
// the next tile's first step: its second half goes to the third set.
GPTQ_TURNS_FN int unpack_adapter_set(int turn, int i, int n) {
    const int by = i == n - 1 && n % UNPACK_SETS == 2 ? 2 : i;
    return (turn + by) % UNPACK_SETS;
}

}  // namespace gptq

#undef GPTQ_TURNS_FN
