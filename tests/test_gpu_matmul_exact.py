"""Products of packed layers whose results are known to the last bit: rows of -1, 0 and 1 and scales
that are powers of two make every product and every sum of them exact in fp32, so an output is one
rounding to the rows' type and any wrong, lost or doubled piece of a contraction shows."""

import numpy as np
import pytest
import torch

import matmul_util as ref
import post_weight_quantization_solve_b200 as gq

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def off(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def signs(rng, rows, cols, t):
    return torch.from_numpy(rng.integers(-1, 2, (rows, cols)).astype(np.float32)).to(t).cuda()


def layer(rng, E, N, K, bits, groupsize, indexed=False, pitch=0):
    """Words, scales, g_idx, and the weights in 64 bits on the GPU. The largest sum of K products is
    below 2^24 times the smallest scale: codes of up to 8 bits, scales from 1/8 to 1."""
    codes = rng.integers(0, 2 ** bits, (E, N, K)).astype(np.uint8)
    shape = (E, N, -(-K // groupsize)) if groupsize else (E, N)
    scales = np.exp2(rng.integers(-3, 1, shape)).astype(np.float32)
    g = np.stack([rng.permutation(np.arange(K) // groupsize) for _ in range(E)]).astype(np.int32) if indexed else None
    words = torch.from_numpy(ref.pack(codes, bits).view(np.int32)).cuda()
    if pitch:
        words = torch.nn.functional.pad(words, (0, pitch))[:, :, :words.shape[2]]
    return (words, torch.from_numpy(scales).cuda(), None if g is None else torch.from_numpy(g).cuda(),
            torch.from_numpy(ref.weights(codes, bits, scales, groupsize, g)).cuda())


def by_range(X, W, counts):
    return torch.cat([x.double() @ w for x, w in zip(X.split(counts), W)]).to(X.dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("K,counts,indexed", [(12032, [40, 300], True), (4096, [300, 700], True), (12032, [40, 300], False)])
def test_words_hold_while_they_are_read(dtype, bits, K, counts, indexed):
    # scales gathered from global memory keep the reads of the words waiting while the copies of
    # later words run ahead; each call many times
    t, rng = TYPES[dtype], np.random.default_rng(K + bits)
    words, s, g, W = layer(rng, 2, 200, K, bits, 32, indexed)
    X, dY = signs(rng, sum(counts), K, t), signs(rng, sum(counts), 200, t)
    o = off(counts)
    y, dx = by_range(X, W.transpose(1, 2), counts), by_range(dY, W, counts)
    flush = torch.empty(1 << 26, device="cuda")
    for i in range(25):
        if i % 2:
            flush.add_(1)
        assert torch.equal(gq.gptq_matmul_grouped(X, words, s, bits, o, 32, g), y), i
        assert torch.equal(gq.gptq_matmul_grouped_dx(dY, words, s, bits, K, o, 32, g), dx), i
