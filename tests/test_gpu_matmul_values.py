"""Products of packed layers at the ends of their value ranges."""

import numpy as np
import pytest
import torch

import matmul_util as ref
import post_weight_quantization_solve_b200 as gq
from test_gpu_matmul import TYPES, check, dev, f64, gen, layer, limit, lora_case, off, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,K,N", [([64, 32], 264, 200), ([37, 70, 5], 264, 200), ([512, 256], 136, 2568)])
@pytest.mark.parametrize("dtype,rank", [("bf16", 16), ("fp16", 72)])
def test_an_infinite_adapter_gives_infinities(counts, K, N, dtype, rank):
    # rows that share no matrix step with others, rows that do, rows of a short run: an infinity of
    # the adapter times a finite T is an infinity of that sign
    ids = [0, 1, 0][:len(counts)]
    c = lora_case(17, dtype, 4, 32, counts, ids, 2, rank, N, K)
    c["B"][0, 5, 3] = float("inf")
    c["B"][0, 150, rank - 1] = float("-inf")
    al = c["alpha"].astype(np.float64)
    y = f64(gq.gptq_matmul_lora(c["X"], *c["args"]))
    want = ref.lora(f64(c["X"]), c["L"]["W"][0], f64(c["A"]), f64(c["B"]), al, c["o"], c["ids"], np.zeros((c["M"], N)))
    own = np.repeat(np.array(ids) == 0, counts)
    assert np.isinf(want[own][:, [5, 150]]).all() and np.array_equal(np.isfinite(y), np.isfinite(want))
    assert np.array_equal(y[own][:, [5, 150]], want[own][:, [5, 150]])
    c = lora_case(18, dtype, 4, 32, counts, ids, 2, rank, K, N)
    c["A"][0, 3, 5] = float("inf")
    c["A"][0, rank - 1, 150] = float("-inf")
    dX = f64(gq.gptq_matmul_lora_backward(c["dY"], c["X"], *c["args"], want=(True, False, False))[0])
    want = ref.lora_backward(f64(c["dY"]), f64(c["X"]), c["L"]["W"][0], f64(c["A"]), f64(c["B"]), al, c["o"], c["ids"],
                             np.zeros((c["M"], N)))[0]
    assert np.isinf(want[own][:, [5, 150]]).all() and np.array_equal(np.isfinite(dX), np.isfinite(want))
    assert np.array_equal(dX[own][:, [5, 150]], want[own][:, [5, 150]])


# (X, dY, A, B) of an fp16 layer whose weights are zero, so that the adapters' terms stand alone, and
# rank-space rows far below fp16's smallest step, and above its largest value
RANK_SPACE = {"small": (1.0, 1e-5, 3000.0, 1e-4), "large": (60.0, 30.0, 40.0, 60.0)}


@pytest.mark.parametrize("size", list(RANK_SPACE))
@pytest.mark.parametrize("counts,ids,rank,N,K", [([1] * 6, [0, 1, 2, 0, -1, 2], 16, 200, 264),
                                                 ([0, 300, 1, 1, 0, 20, 5], [0, 1, 1, -1, 2, 2, 0], 48, 200, 264),
                                                 ([700, 1300], [2, 0], 16, 200, 264), ([40, 300], [1, 0], 128, 77, 101)])
def test_rank_space_rows_of_fp16_have_the_range_of_fp32(size, counts, ids, rank, N, K):
    c = lora_case(21, "fp16", 4, 64, counts, ids, 3, rank, N, K, first=1, pad=2)
    rng, t, o = gen(22), torch.float16, c["o"]
    for name, scale in zip(("X", "dY", "A", "B"), RANK_SPACE[size]):
        c[name].copy_(rows_of(rng, tuple(c[name].shape), t, scale).cuda())
    c["args"][1].zero_()
    if size == "large":                     # (the outputs have to stay below 65,504)
        c["A"].div_(2000.0)
    x, d, A, B = f64(c["X"]), f64(c["dY"]), f64(c["A"]), f64(c["B"])
    al, W = c["alpha"].astype(np.float64), np.zeros((N, K))
    eps, n = torch.finfo(t).eps / 2, max(N, K) + 3 * rank + 20

    dX, dA, dB = gq.gptq_matmul_lora_backward(c["dY"], c["X"], *c["args"], dX=torch.zeros(c["M"], K, dtype=t, device="cuda"))
    want = ref.lora_backward(d, x, W, A, B, al, o, c["ids"], np.zeros((c["M"], K)))
    S = ref.lora_backward(*map(np.abs, (d, x, W, A, B)), al, o, c["ids"], np.zeros((c["M"], K)))
    rows = np.repeat(np.array(ids), counts)
    U = np.abs(np.concatenate([al[a] * d[1 + i:2 + i] @ B[a] for i, a in enumerate(rows) if a >= 0]))
    if size == "large":
        assert U.max() > 65504
    else:
        assert U.max() < 2.0 ** -22
    # two bf16 parts of U, of A one or two: 2^-17 + 2^-18 of each product; half of fp16's smallest step
    check(f64(dX), want[0], eps * np.abs(want[0]) + (n * 2.0 ** -23 + 2.0 ** -16) * S[0] * (1 + eps) + 2.0 ** -25)
    # 22 bits of U and T, or 2^-39 of the adapter's largest
    m = len(rows)
    for got, w, s, other, big in ((dA, want[1], S[1], x, U.max()),
                                  (dB, want[2], S[2], d, np.abs(al.max() * x @ A.reshape(-1, K).T).max())):
        check(f64(got), w, ((n + min(m, 512) + m // 512) * 2.0 ** -23 + 2.0 ** -21) * s
              + 2.0 ** -39 * big * np.abs(other).sum(0).max() + 1e-37)

    if size == "large":
        c["A"].mul_(2000.0)
        c["B"].div_(20000.0)
    A, B = f64(c["A"]), f64(c["B"])
    T = np.abs(np.concatenate([al[a] * x[1 + i:2 + i] @ A[a].T for i, a in enumerate(rows) if a >= 0]))
    assert size == "small" or T.max() > 65504
    y = gq.gptq_matmul_lora(c["X"], *c["args"], out=torch.zeros(c["M"], N, dtype=t, device="cuda"))
    want = ref.lora(x, W, A, B, al, o, c["ids"], np.zeros((c["M"], N)))
    S = ref.lora(*map(np.abs, (x, W, A, B)), al, o, c["ids"], np.zeros((c["M"], N)))
    check(f64(y), want, eps * np.abs(want) + (n * 2.0 ** -23 + 2.0 ** -16) * S * (1 + eps) + 2.0 ** -25)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("bits,rows", [(2, 5), (3, 40), (4, 5), (8, 300)])
def test_an_infinite_scale_gives_infinities(dtype, bits, rows):
    rng, t, N, K = gen(bits), TYPES[dtype], 140, 256
    codes = rng.integers(0, 2 ** bits, (1, N, K)).astype(np.uint8)
    codes[0, 3, 64:128] = 2 ** bits - 1                     # positive weights
    scales = (0.01 + 0.02 * rng.random((1, N, 4))).astype(np.float32)
    scales[0, 3, 1] = np.inf
    words = torch.from_numpy(ref.pack(codes, bits).view(np.int32)).cuda()
    x = torch.rand(rows, K).add_(0.5).to(t)
    d = torch.rand(rows, N).add_(0.5).to(t)
    args = (words, dev(scales), bits)
    y = f64(gq.gptq_matmul_grouped(x.cuda(), *args, dev(off([rows])), 64))
    dx = f64(gq.gptq_matmul_grouped_dx(d.cuda(), *args, K, dev(off([rows])), 64))
    W = ref.weights(codes, bits, scales, 64)[0]
    for got, want in ((y, f64(x) @ W.T), (dx, f64(d) @ W)):
        bad = np.isinf(want)
        assert bad.any() and np.array_equal(got[bad], want[bad]) and np.isfinite(got[~bad]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("counts,rank,N,K,chain", [([7] * 60, 128, 13656, 264, 16), ([22], 64, 9408, 960, 16),
                                                   ([300], 16, 264, 65528, 32), ([1000, 200], 64, 30000, 136, 32)])
def test_rank_space_sums_do_not_drift(dtype, counts, rank, N, K, chain):
    """The matrix units cut each step of a sum off, by half of 2^-23 of it in the mean and always towards
    zero, so a chain of n steps is n / 2 such halves off; chains, and the parts that are added to
    nearest, count 4 more, as do the gradients' own sums of at most 32 steps of these few rows (16)."""
    ids = [i % 2 for i in range(len(counts))]
    c = lora_case(31, dtype, 4, 0, counts, ids, 2, rank, N, K)
    _, dA, dB = gq.gptq_matmul_lora_backward(c["dY"], c["X"], *c["args"], want=(False, True, True))
    x, d, A, B = (c[n].double() for n in ("X", "dY", "A", "B"))
    wA, wB = torch.zeros_like(A), torch.zeros_like(B)
    for r, a in enumerate(ids):
        p, f = slice(int(c["o"][r]), int(c["o"][r + 1])), float(c["alpha"][a])
        wA[a] += f * (d[p] @ B[a]).t() @ x[p]
        wB[a] += f * d[p].t() @ (x[p] @ A[a].t())
    own = min(32, max(counts) / 16 if len(counts) < 3 else 4)
    for got, want in ((dA, wA), (dB, wB)):
        assert (got.double() - want).norm() <= (chain / 2 + 4 + own / 2) * 2.0 ** -23 * want.norm()
