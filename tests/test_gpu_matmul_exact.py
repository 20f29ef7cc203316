"""Products of packed layers whose results are known to the last bit: rows of -1, 0 and 1 and scales
that are powers of two make every product and every sum of them exact in fp32, so an output is one
rounding to the rows' type and any wrong, lost or doubled piece of a contraction shows. A worst-case
bound grows with the length of the contraction, a lost piece with its square root: beside these, a
bound on the mean square of ordinary values' errors."""

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


SHAPES = [  # counts, N, K: contractions split over clusters, pairs of blocks, several tiles a block, odd sizes
    ([1], 96, 14336), ([8], 300, 4096), ([24], 64, 14336), ([40], 200, 6000), ([100, 0, 1, 300], 136, 2100),
    ([700, 300], 2571, 520), ([3, 2, 0, 7], 77, 1001), ([130], 7, 4097), ([1500, 0, 2500], 1100, 256),
]


@pytest.mark.parametrize("counts,N,K", SHAPES)
@pytest.mark.parametrize("dtype,bits,groupsize,indexed,pitch", [
    ("bf16", 4, 128, False, 0), ("bf16", 3, 0, False, 0), ("fp16", 8, 64, False, 0), ("fp16", 2, 32, True, 0),
    ("bf16", 8, 128, True, 0), ("bf16", 4, 64, False, 1), ("fp16", 3, 128, True, 3), ("bf16", 2, 0, False, 1)])
def test_rows(dtype, bits, groupsize, indexed, pitch, counts, N, K):
    t, rng = TYPES[dtype], np.random.default_rng(K + N + bits)
    words, s, g, W = layer(rng, len(counts), N, K, bits, groupsize, indexed, pitch)
    M, o = sum(counts), off(counts)
    for xpad in (0, 3):                     # (rows that tiled copies take, and rows that they refuse)
        X, dY = signs(rng, M, K + xpad, t)[:, :K], signs(rng, M, N + xpad, t)[:, :N]
        status = gq.new_status()
        y = gq.gptq_matmul_grouped(X, words, s, bits, o, groupsize, g, status=status)
        assert torch.equal(y, by_range(X, W.transpose(1, 2), counts))
        dx = gq.gptq_matmul_grouped_dx(dY, words, s, bits, K, o, groupsize, g, status=status)
        assert torch.equal(dx, by_range(dY, W, counts))
        gq.raise_on_status(status)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("counts,N,K", [([4200], 128, 72), ([0, 65, 1, 130], 200, 264), ([2100, 140], 1200, 2200),
                                        ([600, 90, 33], 1201, 2203), ([1] * 300, 40, 72)])
def test_weight_gradients(dtype, counts, N, K):
    t, rng = TYPES[dtype], np.random.default_rng(K)
    X, dY = signs(rng, sum(counts), K, t), signs(rng, sum(counts), N, t)
    G = gq.gptq_matmul_grouped_dw(dY, X, off(counts))
    want = torch.stack([d.double().t() @ x.double() for d, x in zip(dY.split(counts), X.split(counts))])
    assert torch.equal(G.double(), want)
    again = gq.gptq_matmul_grouped_dw(dY, X, off(counts), out=G.clone(), accumulate=True)
    assert torch.equal(again.double(), 2 * want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("counts,ids,rank,N,K", [
    ([1] * 6, [0, 1, 2, 0, -1, 2], 16, 200, 520), ([0, 300, 1, 1, 0, 20, 5], [0, 1, 1, -1, 2, 2, 0], 40, 200, 264),
    ([700, 1300], [2, 0], 128, 77, 101), ([37, 70, 21, 100] * 12, [0, 1, 2, 1] * 12, 72, 1300, 136),
    ([1] * 50, [i % 3 for i in range(50)], 8, 264, 4096)])
def test_adapters(dtype, counts, ids, rank, N, K):
    # A and B of -1, 0 and 1 with one entry in 16, factors 1, 1/2 and 2: T and U stay below 2^10, every
    # sum below 2^22
    t, rng = TYPES[dtype], np.random.default_rng(rank + K)
    words, s, _, W = layer(rng, 1, N, K, 4, 64)
    M, o = sum(counts), off(counts)

    def sparse(*shape):
        v = rng.integers(-1, 2, shape) * (rng.random(shape) < 1 / 16)
        return torch.from_numpy(v.astype(np.float32)).to(t).cuda()

    A, B = sparse(3, rank, K), sparse(3, N, rank)
    alpha = torch.tensor([1.0, 0.5, 2.0], device="cuda")
    X, dY = signs(rng, M, K, t), signs(rng, M, N, t)
    args = (words[0], s[0], 4, A, B, alpha, o, torch.tensor(ids, dtype=torch.int32, device="cuda"), 64)
    y, dx = X.double() @ W[0].t(), dY.double() @ W[0]
    dA, dB = torch.zeros(A.shape, dtype=torch.float64, device="cuda"), torch.zeros(B.shape, dtype=torch.float64, device="cuda")
    at = 0
    for n, a in zip(counts, ids):
        p = slice(at, at + n)
        at += n
        if a < 0:
            continue
        a64, b64, f = A[a].double(), B[a].double(), float(alpha[a])
        T, U = f * (X[p].double() @ a64.t()), f * (dY[p].double() @ b64)
        y[p] += T @ b64.t()
        dx[p] += U @ a64
        dA[a] += U.t() @ X[p].double()
        dB[a] += dY[p].double().t() @ T
    assert torch.equal(gq.gptq_matmul_lora(X, *args), y.to(t))
    got = gq.gptq_matmul_lora_backward(dY, X, *args)
    assert torch.equal(got[0], dx.to(t))
    assert torch.equal(got[1].double(), dA) and torch.equal(got[2].double(), dB)


@pytest.mark.parametrize("counts,N,K,bits,groupsize,indexed", [
    ([24], 64, 14336, 4, 128, False), ([5], 64, 14336, 4, 128, False), ([40, 300], 200, 12032, 4, 32, True),
    ([300, 700], 640, 4096, 8, 128, False)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_mean_square_error(dtype, counts, N, K, bits, groupsize, indexed):
    """Each weight is rounded once, by at most eps of itself and independently, so the mean square of
    an output's error is at most eps^2 sum (x w)^2, beside eps |y| for the output's own rounding and
    n 2^-24 |y| for sums of n steps of 16 that are cut off. A lost piece of 1/n of the contraction
    adds sum (x w)^2 / n: 1/112 for a step of the longest here, 600 times the bound."""
    t, rng = TYPES[dtype], np.random.default_rng(K)
    codes = rng.integers(0, 2 ** bits, (len(counts), N, K)).astype(np.uint8)
    scales = (0.01 + 0.02 * rng.random((len(counts), N, -(-K // groupsize)))).astype(np.float32)
    g = np.stack([rng.permutation(np.arange(K) // groupsize) for _ in counts]).astype(np.int32) if indexed else None
    W = torch.from_numpy(ref.weights(codes, bits, scales, groupsize, g)).cuda()
    words, s = torch.from_numpy(ref.pack(codes, bits).view(np.int32)).cuda(), torch.from_numpy(scales).cuda()
    gi = None if g is None else torch.from_numpy(g).cuda()
    M, o, eps = sum(counts), off(counts), torch.finfo(t).eps / 2

    def mean_square(got, x, w, n):
        want = torch.cat([a.double() @ b for a, b in zip(x.split(counts), w)])
        parts = torch.cat([a.double().square() @ b.square() for a, b in zip(x.split(counts), w)]).mean()
        y2 = want.square().mean()
        assert (got.double() - want).square().mean() <= eps ** 2 * (parts + y2) + (n / 16 * 2.0 ** -24) ** 2 * y2

    X = torch.from_numpy(rng.standard_normal((M, K))).to(t).cuda()
    mean_square(gq.gptq_matmul_grouped(X, words, s, bits, o, groupsize, gi), X, W.transpose(1, 2), K)
    dY = torch.from_numpy(rng.standard_normal((M, N)) * 0.1).to(t).cuda()
    mean_square(gq.gptq_matmul_grouped_dx(dY, words, s, bits, K, o, groupsize, gi), dY, W, N)
