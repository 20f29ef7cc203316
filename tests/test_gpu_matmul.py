"""Products of packed layers (gptq_matmul_*) on the GPU against a plain 64-bit statement:
types, bits, input groups and g_idx, ragged and empty ranges, pitches and alignments, rows
outside the ranges, refusals that only the device sees, streams and captured graphs.

Tolerances. eps is half a step of the 16-bit type, torch.finfo(t).eps / 2 (bf16 2^-8, fp16 2^-11). An output is one rounding of a sum, |error| <= eps |y|, plus the sum's
own error: each product x w carries the rounding of w to the type where the scale is folded
(eps |x w|), and fp32 accumulation of n terms adds at most n 2^-23 sum |x w| (two half steps:
the matrix unit truncates). With S = sum |x w| elementwise:
    |y_gpu - y| <= eps |y| + (fold eps + n 2^-23) S (1 + eps) + tiny.
"""

import numpy as np
import pytest
import torch

import matmul_util as ref
import post_weight_quantization_solve_b200 as gq

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def gen(seed):
    return np.random.default_rng(seed)


def rows_of(rng, shape, dtype, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(dtype)


def layer(rng, E, N, K, bits, groupsize, indexed=False):
    codes = rng.integers(0, 2 ** bits, (E, N, K)).astype(np.uint8)
    G = -(-K // groupsize) if groupsize else 0
    scales = (0.01 + 0.02 * rng.random((E, N, G) if G else (E, N))).astype(np.float32)
    g_idx = None
    if indexed:
        g_idx = np.stack([rng.permutation(np.arange(K) // groupsize) for _ in range(E)]).astype(np.int32)
    return {"codes": codes, "scales": scales, "g_idx": g_idx, "bits": bits, "groupsize": groupsize,
            "W": ref.weights(codes, bits, scales, groupsize, g_idx),
            "words": torch.from_numpy(ref.pack(codes, bits).view(np.int32)).cuda(),
            "s": torch.from_numpy(scales).cuda(),
            "g": None if g_idx is None else torch.from_numpy(g_idx).cuda()}


def off(counts, first=0):
    return np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def limit(y, S, n, dtype, fold):
    eps = torch.finfo(dtype).eps / 2
    return eps * np.abs(y) + (fold * eps + n * 2.0 ** -23) * S * (1 + eps) + 1e-7


def check(got, want, bound):
    d = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (d <= bound).all(), (d / np.maximum(bound, 1e-300)).max()


def forward_case(dtype, bits, groupsize, indexed, counts, N, K, seed=0, pad=0, first=0, xpad=0):
    rng, t = gen(seed), TYPES[dtype]
    E = len(counts)
    L = layer(rng, E, N, K, bits, groupsize, indexed)
    o = off(counts, first)
    M = int(o[-1]) + pad
    X = rows_of(rng, (M, K + xpad), t).cuda()[:, :K]
    out = torch.full((M, N), 7.0, dtype=t, device="cuda")
    status = gq.new_status()
    y = gq.gptq_matmul_grouped(X, L["words"], L["s"], bits, dev(o), groupsize, L["g"], out=out, status=status)
    assert y is out
    gq.raise_on_status(status)
    x = f64(X)
    want = ref.grouped(x, L["W"], o, np.full((M, N), 7.0))
    S = ref.grouped(np.abs(x), np.abs(L["W"]), o, np.zeros((M, N)))
    check(f64(y), want, limit(want, S, K, t, 1 if groupsize else 0))
    assert (f64(y)[:first] == 7.0).all() and (f64(y)[int(o[-1]):] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("groupsize,indexed", [(0, False), (64, False), (32, True)])
@pytest.mark.parametrize("rows", [1, 12, 70])
def test_forward_one_layer(dtype, bits, groupsize, indexed, rows):
    forward_case(dtype, bits, groupsize, indexed, [rows], 136, 520, seed=bits + rows)


@pytest.mark.parametrize("counts", [[0, 3, 0, 1, 5, 0], [0, 0, 40, 0], [300, 1, 0, 17, 256, 257], [16, 16]])
@pytest.mark.parametrize("bits,groupsize", [(4, 128), (3, 0)])
def test_forward_ragged_ranges(counts, bits, groupsize):
    forward_case("bf16", bits, groupsize, False, counts, 200, 256, pad=5, first=3)


@pytest.mark.parametrize("K,N", [(1, 1), (31, 129), (33, 7), (127, 128), (1001, 65)])
@pytest.mark.parametrize("rows", [4, 37])
def test_forward_odd_sizes(K, N, rows):
    for bits in (3, 4):
        forward_case("fp16", bits, 0, False, [rows], N, K)
        forward_case("bf16", bits, 32, False, [rows, 2], N, K)


@pytest.mark.parametrize("rows", [5, 100])
@pytest.mark.parametrize("xpad", [1, 8])
def test_forward_row_pitch(rows, xpad):
    forward_case("bf16", 4, 64, False, [rows], 96, 128, xpad=xpad)


@pytest.mark.parametrize("K", [1600, 4200, 9000, 12032])
@pytest.mark.parametrize("dtype,bits", [("bf16", 4), ("fp16", 8), ("fp16", 3)])
def test_many_groups_by_index(K, dtype, bits):
    # with and without room for tables of scales, words by tiled copies and by plain ones
    forward_case(dtype, bits, 32, True, [40, 300], 200, K)
    rng, t, counts = gen(K), TYPES[dtype], [130, 0, 21]
    L = layer(rng, 3, 200, K, bits, 32, True)
    o = off(counts)
    dY = rows_of(rng, (151, 200), t).cuda()
    dX = gq.gptq_matmul_grouped_dx(dY, L["words"], L["s"], bits, K, dev(o), 32, L["g"])
    d, Wt, z = f64(dY), L["W"].transpose(0, 2, 1), np.zeros((151, K))
    want, S = ref.grouped(d, Wt, o, z), ref.grouped(np.abs(d), np.abs(Wt), o, z)
    check(f64(dX), want, limit(want, S, 200, t, 1))


@pytest.mark.parametrize("experts", [257, 512])
@pytest.mark.parametrize("most", [3, 12])
def test_many_experts(experts, most):
    # a few rows each, with ranges of several fragments (most 3), and enough rows for tiles
    rng = gen(experts + most)
    counts = [int(v) for v in rng.integers(0, most, experts)]
    counts[0], counts[experts // 2], counts[-1] = 20, 8, 9
    forward_case("bf16", 4, 32, False, counts, 40, 72, pad=1)
    forward_case("fp16", 3, 0, False, counts, 33, 130, first=1)
    forward_case("bf16", 2, 32, True, counts, 40, 72)
    o = off(counts)
    dY, X = rows_of(rng, (int(o[-1]), 40), torch.bfloat16).cuda(), rows_of(rng, (int(o[-1]), 72), torch.bfloat16).cuda()
    G = gq.gptq_matmul_grouped_dw(dY, X, dev(o))
    d, x = f64(dY), f64(X)
    check(f64(G), ref.grouped_dw(d, x, o), 30 * 2.0 ** -23 * ref.grouped_dw(np.abs(d), np.abs(x), o) + 1e-30)
    L = layer(rng, experts, 40, 72, 4, 32, False)
    dX = gq.gptq_matmul_grouped_dx(dY, L["words"], L["s"], 4, 72, dev(o), 32)
    Wt = L["W"].transpose(0, 2, 1)
    z = np.zeros((int(o[-1]), 72))
    want, S = ref.grouped(d, Wt, o, z), ref.grouped(np.abs(d), np.abs(Wt), o, z)
    check(f64(dX), want, limit(want, S, 40, torch.bfloat16, 1))


def test_offsets_past_32_bits():
    # rows that begin 2.4e9 values into their tensors
    M, K, N, n = 300000, 8192, 40, 150
    rng, t = gen(1), torch.bfloat16
    L = layer(rng, 2, N, K, 4, 128, False)
    o = np.array([0, M - n, M], dtype=np.int32)
    X = torch.zeros(M, K, dtype=t, device="cuda")
    X[-n:] = rows_of(rng, (n, K), t).cuda()
    dY = torch.zeros(M, N, dtype=t, device="cuda")
    dY[-n:] = rows_of(rng, (n, N), t).cuda()
    x, d, W = f64(X[-n:]), f64(dY[-n:]), L["W"][1]
    y = gq.gptq_matmul_grouped(X, L["words"], L["s"], 4, dev(o), 128)
    want, S = x @ W.T, np.abs(x) @ np.abs(W).T
    check(f64(y[-n:]), want, limit(want, S, K, t, 1))
    dX = gq.gptq_matmul_grouped_dx(dY, L["words"], L["s"], 4, K, dev(o), 128)
    want, S = d @ W, np.abs(d) @ np.abs(W)
    check(f64(dX[-n:]), want, limit(want, S, N, t, 1))
    assert not dX[:-n].any() and not y[:-n].any()
    del dX
    G = gq.gptq_matmul_grouped_dw(dY, X, dev(o))
    check(f64(G[1]), d.T @ x, (n + 4) * 2.0 ** -23 * (np.abs(d).T @ np.abs(x)) + 1e-30)
    assert not G[0].any()
    A, B = rows_of(rng, (1, 8, K), t, K ** -0.5).cuda(), rows_of(rng, (1, N, 8), t, 0.1).cuda()
    alpha, ids = torch.ones(1, device="cuda"), dev(np.array([-1, 0], dtype=np.int32))
    args = (L["words"][1], L["s"][1], 4, A, B, alpha, dev(o), ids, 128)
    y = gq.gptq_matmul_lora(X, *args)
    arrays = [x, W, f64(A), f64(B)]
    tail, z = [0, n], np.zeros((n, N))
    want = ref.lora(*arrays, [1.0], tail, [0], z)
    S = ref.lora(*map(np.abs, arrays), [1.0], tail, [0], z)
    check(f64(y[-n:]), want, limit(want, S, K + 16, t, 1) + 2 * pair_eps(t) * S)
    dX, dA, dB = gq.gptq_matmul_lora_backward(dY, X, *args)
    want = ref.lora_backward(d, *arrays, [1.0], tail, [0], np.zeros((n, K)))
    S = ref.lora_backward(*map(np.abs, [d, *arrays]), [1.0], tail, [0], np.zeros((n, K)))
    check(f64(dX[-n:]), want[0], limit(want[0], S[0], N + 16, t, 1) + 2 * pair_eps(t) * S[0])
    for got, w, s in ((dA, want[1], S[1]), (dB, want[2], S[2])):
        check(f64(got), w, ((K + n + 20) * 2.0 ** -23 + 2 * part_eps(t)) * s + 1e-30)


@pytest.mark.parametrize("K,N", [(256, 2560), (201, 2571)])
@pytest.mark.parametrize("counts", [[1500, 0, 2500], [200] * 20, [60] * 20])
def test_forward_many_tiles_a_block(K, N, counts):
    forward_case("bf16", 4, 64, False, counts, N, K, pad=3)
    forward_case("fp16", 3, 0, False, counts, N, K, first=2)


def test_forward_long_contraction_and_wide_layer():
    forward_case("bf16", 4, 128, False, [24], 64, 14336)     # clusters share the contraction
    forward_case("bf16", 2, 0, False, [2], 5000, 640)


@pytest.mark.parametrize("rows", [3, 90])
def test_padded_words_and_strided_output(rows):
    # words rows with a pitch, output rows inside a wider buffer
    rng = gen(5)
    L = layer(rng, 2, 40, 100, 3, 0)
    nw = L["words"].shape[-1]
    words = torch.zeros(2, 40, nw + 3, dtype=torch.int32, device="cuda")
    words[:, :, :nw] = L["words"]
    o = off([rows, 2])
    X = rows_of(rng, (rows + 2, 100), torch.bfloat16).cuda()
    wide = torch.zeros(rows + 2, 50, dtype=torch.bfloat16, device="cuda")
    gq.gptq_matmul_grouped(X, words[:, :, :nw], L["s"], 3, dev(o), out=wide[:, 3:43])
    want = ref.grouped(f64(X), L["W"], o, np.zeros((rows + 2, 40)))
    S = ref.grouped(np.abs(f64(X)), np.abs(L["W"]), o, np.zeros((rows + 2, 40)))
    check(f64(wide[:, 3:43]), want, limit(want, S, 100, torch.bfloat16, 0))
    assert (wide[:, :3] == 0).all() and (wide[:, 43:] == 0).all()


@pytest.mark.parametrize("rows", [4, 64])
def test_rows_of_others_do_not_leak(rows):
    # infinities and NaN in rows of another range, or outside all of them, stay there
    rng = gen(6)
    L = layer(rng, 2, 64, 128, 4, 64)
    o = off([rows, rows])
    X = rows_of(rng, (2 * rows + 9, 128), torch.bfloat16)
    X[rows:2 * rows] = float("nan")
    X[2 * rows:] = float("inf")
    Xd = X.cuda()
    y = gq.gptq_matmul_grouped(Xd, L["words"], L["s"], 4, dev(o), 64)
    assert torch.isfinite(y[:rows]).all() and torch.isnan(y[rows:2 * rows]).all()
    X[rows:] = 0
    z = gq.gptq_matmul_grouped(X.cuda(), L["words"], L["s"], 4, dev(o), 64)
    assert torch.equal(y[:rows], z[:rows])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("bits,groupsize,indexed", [(2, 64, True), (3, 0, False), (4, 128, False), (8, 32, False)])
@pytest.mark.parametrize("counts,N,K", [([70], 200, 264), ([0, 1, 33, 300, 0], 136, 300), ([5, 2], 77, 33)])
def test_input_gradient(dtype, bits, groupsize, indexed, counts, N, K):
    rng, t = gen(bits + K), TYPES[dtype]
    L = layer(rng, len(counts), N, K, bits, groupsize, indexed)
    o = off(counts, 2)
    M = int(o[-1]) + 3
    dY = rows_of(rng, (M, N), t, 0.1).cuda()
    out = torch.full((M, K), 7.0, dtype=t, device="cuda")
    status = gq.new_status()
    gq.gptq_matmul_grouped_dx(dY, L["words"], L["s"], bits, K, dev(o), groupsize, L["g"], out=out, status=status)
    gq.raise_on_status(status)
    WT = L["W"].transpose(0, 2, 1)
    want = ref.grouped(f64(dY), WT, o, np.full((M, K), 7.0))
    S = ref.grouped(np.abs(f64(dY)), np.abs(WT), o, np.zeros((M, K)))
    check(f64(out), want, limit(want, S, N, t, 1))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("counts,N,K", [([1], 8, 8), ([0, 65, 1, 130], 200, 264), ([4200], 128, 64),
                                        ([31, 47], 77, 301), ([2048, 2049], 64, 320),
                                        ([130, 0, 300, 17, 64, 128, 255, 1, 16], 1100, 1000), ([2100, 140], 1200, 2200),
                                        ([90, 33], 1201, 2203)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradient(dtype, counts, N, K, accumulate):
    rng, t = gen(K), TYPES[dtype]
    o = off(counts, 1)
    M = int(o[-1]) + 2
    dY, X = rows_of(rng, (M, N), t).cuda(), rows_of(rng, (M, K), t).cuda()
    dY[:1] = float("nan")
    X[int(o[-1]):] = float("inf")
    start = rng.standard_normal((len(counts), N, K)).astype(np.float32)
    out = dev(start) if accumulate else torch.full(start.shape, float("nan"), device="cuda")
    status = gq.new_status()
    gq.gptq_matmul_grouped_dw(dY, X, dev(o), out=out, accumulate=accumulate, status=status)
    gq.raise_on_status(status)
    d, x = np.nan_to_num(f64(dY)), np.nan_to_num(f64(X), posinf=0)
    want = ref.grouped_dw(d, x, o) + (start if accumulate else 0)
    S = ref.grouped_dw(np.abs(d), np.abs(x), o) + np.abs(start)
    # fp32: products are exact, a truncating sum of up to 512 terms and the chains' sums
    n = max(counts)
    check(f64(out), want, (min(n, 512) + n // 512 + 4) * 2.0 ** -23 * S + 1e-30)
    again = dev(start) if accumulate else torch.empty_like(out)
    gq.gptq_matmul_grouped_dw(dY, X, dev(o), out=again, accumulate=accumulate)
    assert torch.equal(again, out)


def lora_case(seed, dtype, bits, groupsize, counts, ids, adapters, rank, N, K, first=0, pad=0):
    rng, t = gen(seed), TYPES[dtype]
    L = layer(rng, 1, N, K, bits, groupsize)
    o = off(counts, first)
    M = int(o[-1]) + pad
    c = {"L": L, "o": o, "M": M, "t": t, "ids": np.array(ids, dtype=np.int32),
         "X": rows_of(rng, (M, K), t).cuda(), "dY": rows_of(rng, (M, N), t, 0.1).cuda(),
         "A": rows_of(rng, (adapters, rank, K), t, K ** -0.5).cuda(),
         "B": rows_of(rng, (adapters, N, rank), t, 0.1).cuda(),
         "alpha": (0.5 + rng.random(adapters)).astype(np.float32), "bits": bits, "groupsize": groupsize,
         "N": N, "K": K, "rank": rank}
    c["args"] = (L["words"][0], L["s"][0], bits, c["A"], c["B"], dev(c["alpha"]), dev(o), dev(c["ids"]), groupsize)
    return c


def pair_eps(t):
    """A rank-space row enters 16-bit outputs as two parts: half a step of the second one."""
    return (torch.finfo(t).eps / 2) ** 2


def part_eps(t):
    """It enters the fp32 gradients as all its parts, three of bf16 and two of fp16."""
    return (torch.finfo(t).eps / 2) ** (3 if t == torch.bfloat16 else 2)


def check_lora(c, y, start):
    x, A, B = f64(c["X"]), f64(c["A"]), f64(c["B"])
    W = c["L"]["W"][0]
    want = ref.lora(x, W, A, B, c["alpha"].astype(np.float64), c["o"], c["ids"], np.full((c["M"], c["N"]), start))
    S = ref.lora(np.abs(x), np.abs(W), np.abs(A), np.abs(B), c["alpha"], c["o"], c["ids"], np.zeros((c["M"], c["N"])))
    fold = 1 if c["groupsize"] or c["M"] > 8 else 0     # (the tiled kernel folds the scales)
    b = limit(want, S, c["K"] + 2 * c["rank"], c["t"], fold) + 2 * pair_eps(c["t"]) * S
    check(f64(y), want, b)


LORA = [  # counts, ids
    ([1] * 6, [0, 1, 2, 0, -1, 2]),                       # decode, few rows
    ([1] * 50, [i % 3 for i in range(50)]),               # decode, tiled kernel
    ([0, 300, 1, 1, 0, 20, 5], [0, 1, 1, -1, 2, 2, 0]),   # prompts and decoding, one run of two requests
    ([40, 3], [-1, -1]),                                  # no adapter at all
    ([700], [2]),
]


@pytest.mark.parametrize("counts,ids", LORA)
@pytest.mark.parametrize("dtype,bits,groupsize,rank", [("bf16", 4, 128, 16), ("fp16", 3, 0, 8), ("bf16", 8, 32, 40),
                                                       ("fp16", 2, 64, 128)])
def test_lora_forward(counts, ids, dtype, bits, groupsize, rank):
    c = lora_case(1, dtype, bits, groupsize, counts, ids, 3, rank, 200, 264, first=2, pad=3)
    out = torch.full((c["M"], c["N"]), 7.0, dtype=c["t"], device="cuda")
    status = gq.new_status()
    gq.gptq_matmul_lora(c["X"], *c["args"], out=out, status=status)
    gq.raise_on_status(status)
    check_lora(c, out, 7.0)


@pytest.mark.parametrize("counts,ids", LORA)
@pytest.mark.parametrize("dtype,bits,groupsize,rank,N,K", [("bf16", 4, 128, 16, 200, 264), ("fp16", 3, 0, 8, 77, 101),
                                                           ("bf16", 2, 64, 128, 264, 136)])
def test_lora_backward(counts, ids, dtype, bits, groupsize, rank, N, K):
    c = lora_case(2, dtype, bits, groupsize, counts, ids, 4, rank, N, K, first=2, pad=3)
    t, o = c["t"], c["o"]
    dX = torch.full((c["M"], K), 7.0, dtype=t, device="cuda")
    status = gq.new_status()
    _, dA, dB = gq.gptq_matmul_lora_backward(c["dY"], c["X"], *c["args"], dX=dX, status=status)
    gq.raise_on_status(status)
    arrays = [f64(c["dY"]), f64(c["X"]), c["L"]["W"][0], f64(c["A"]), f64(c["B"])]
    al = c["alpha"].astype(np.float64)
    want = ref.lora_backward(*arrays, al, o, c["ids"], np.full((c["M"], K), 7.0))
    S = ref.lora_backward(*map(np.abs, arrays), al, o, c["ids"], np.zeros((c["M"], K)))
    pe, ge = 2 * pair_eps(t), 2 * part_eps(t)
    # fp16's second part has a fixed smallest step: 2^-25 a value of T or U
    floor = 2.0 ** -24 if t == torch.float16 else 0.0
    check(f64(dX), want[0], limit(want[0], S[0], N + 2 * rank, t, 1) + pe * S[0] + floor * rank * np.abs(arrays[3]).max())
    m = int(o[-1] - o[0])
    for got, w, s, other in ((dA, want[1], S[1], arrays[1]), (dB, want[2], S[2], arrays[0])):
        check(f64(got), w, ((max(N, K) + min(m, 512) + m // 512 + 20) * 2.0 ** -23 + ge) * s
              + floor * m * np.abs(other).max() + 1e-30)
    # each gradient alone, and again: the same bits
    only = gq.gptq_matmul_lora_backward(c["dY"], c["X"], *c["args"], want=(False, True, False))
    assert only[0] is None and only[2] is None and torch.equal(only[1], dA)
    only = gq.gptq_matmul_lora_backward(c["dY"], c["X"], *c["args"], want=(False, False, True))
    assert torch.equal(only[2], dB)


@pytest.mark.parametrize("dtype,K,N,rank", [("bf16", 256, 2560, 64), ("fp16", 200, 2568, 16), ("bf16", 129, 2571, 8)])
def test_many_tiles_a_block(dtype, K, N, rank):
    # pairs of blocks that walk several tiles each, tiles with several long and short runs, and
    # layouts with and without tiled copies
    rng = gen(K)
    counts, ids = [], []
    while sum(counts) < 4000:
        counts.append(int(rng.choice([0, 1, 3, 15, 16, 17, 60, 300])))
        ids.append(int(rng.integers(-1, 4)))
    c = lora_case(5, dtype, 4, 32, counts, ids, 4, rank, N, K, first=1, pad=2)
    out = torch.full((c["M"], N), 7.0, dtype=c["t"], device="cuda")
    status = gq.new_status()
    gq.gptq_matmul_lora(c["X"], *c["args"], out=out, status=status)
    gq.raise_on_status(status)
    check_lora(c, out, 7.0)
    # the input gradient of a layer as wide (its channels are K there)
    c = lora_case(6, dtype, 4, 32, counts, ids, 4, rank, K, N, first=1, pad=2)
    dX = torch.full((c["M"], N), 7.0, dtype=c["t"], device="cuda")
    status = gq.new_status()
    gq.gptq_matmul_lora_backward(c["dY"], c["X"], *c["args"], dX=dX, want=(True, False, False), status=status)
    gq.raise_on_status(status)
    arrays = [f64(c["dY"]), f64(c["X"]), c["L"]["W"][0], f64(c["A"]), f64(c["B"])]
    al = c["alpha"].astype(np.float64)
    want = ref.lora_backward(*arrays, al, c["o"], c["ids"], np.full((c["M"], N), 7.0))[0]
    S = ref.lora_backward(*map(np.abs, arrays), al, c["o"], c["ids"], np.zeros((c["M"], N)))[0]
    floor = 2.0 ** -24 if c["t"] == torch.float16 else 0.0
    check(f64(dX), want, limit(want, S, K + 2 * rank, c["t"], 1) + 2 * pair_eps(c["t"]) * S
          + floor * rank * np.abs(arrays[3]).max())


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("counts,K,N", [([37, 70, 21, 100], 264, 200), ([37, 70, 21, 100] * 12, 136, 2568)])
@pytest.mark.parametrize("dtype,rank", [("bf16", 16), ("fp16", 72)])
def test_a_broken_adapter_stays_with_its_rows(value, counts, K, N, dtype, rank):
    # runs end between the columns that a matrix step takes, so a step holds rows of neighbours
    ids = [0, 1, 2, 1] * (len(counts) // 4)
    c = lora_case(7, dtype, 4, 32, counts, ids, 3, rank, N, K, pad=3)
    own = torch.zeros(c["M"], dtype=torch.bool, device="cuda")
    for r, a in enumerate(ids):
        own[int(c["o"][r]):int(c["o"][r + 1])] = a == 0
    clean = gq.gptq_matmul_lora(c["X"], *c["args"], out=torch.zeros(c["M"], N, dtype=c["t"], device="cuda"))
    c["B"][0, 5, 3] = value
    c["B"][0, 150, rank - 1] = -value
    out = gq.gptq_matmul_lora(c["X"], *c["args"], out=torch.zeros(c["M"], N, dtype=c["t"], device="cuda"))
    assert torch.equal(out[~own], clean[~own])
    want = ref.lora(f64(c["X"]), c["L"]["W"][0], f64(c["A"]), f64(c["B"]), c["alpha"].astype(np.float64), c["o"],
                    c["ids"], np.zeros((c["M"], N)))
    got = f64(out)
    bad = ~np.isfinite(want)
    assert bad[own.cpu().numpy()][:, [5, 150]].all() and (np.isfinite(got) == ~bad).all()
    assert np.array_equal(got[bad], want[bad], equal_nan=True)
    # the input gradient of a layer as wide; a gradient of one adapter from rows of its own alone
    c = lora_case(8, dtype, 4, 32, counts, ids, 3, rank, K, N, pad=3)
    fresh = lambda: torch.zeros(c["M"], N, dtype=c["t"], device="cuda")
    clean = gq.gptq_matmul_lora_backward(c["dY"], c["X"], *c["args"], dX=fresh())
    c["A"][0, 3, 5] = value
    c["A"][0, rank - 1, 150] = -value
    dX, dA, dB = gq.gptq_matmul_lora_backward(c["dY"], c["X"], *c["args"], dX=fresh())
    assert torch.equal(dX[~own], clean[0][~own])
    want = ref.lora_backward(f64(c["dY"]), f64(c["X"]), c["L"]["W"][0], f64(c["A"]), f64(c["B"]),
                             c["alpha"].astype(np.float64), c["o"], c["ids"], np.zeros((c["M"], N)))
    got, bad = f64(dX), ~np.isfinite(want[0])
    assert bad[own.cpu().numpy()][:, [5, 150]].all() and (np.isfinite(got) == ~bad).all()
    assert np.array_equal(got[bad], want[0][bad], equal_nan=True)
    assert torch.equal(dA, clean[1]) and torch.equal(dB[1:], clean[2][1:]) and not torch.isfinite(dB[0]).all()
    # non-finite rows of one request (its neighbours', in T, U, dX and the other adapters' gradients)
    c["A"][0, 3, 5] = c["A"][0, rank - 1, 150] = 0
    clean = gq.gptq_matmul_lora_backward(c["dY"], c["X"], *c["args"], dX=fresh())
    c["X"][own], c["dY"][own] = value, -value
    dX, dA, dB = gq.gptq_matmul_lora_backward(c["dY"], c["X"], *c["args"], dX=fresh())
    assert torch.equal(dX[~own], clean[0][~own]) and not torch.isfinite(dX[own]).any()
    assert torch.equal(dA[1:], clean[1][1:]) and torch.equal(dB[1:], clean[2][1:])


@pytest.mark.parametrize("requests,adapters", [(1200, 300), (33, 257), (1, 1)])
def test_lora_gradients_of_many_requests(requests, adapters):
    rng = gen(requests)
    counts = [int(v) for v in rng.integers(0, 4, requests)]
    ids = [int(v) for v in rng.integers(-1, adapters, requests)]
    c = lora_case(11, "bf16", 4, 0, counts, ids, adapters, 8, 40, 72, pad=1)
    _, dA, dB = gq.gptq_matmul_lora_backward(c["dY"], c["X"], *c["args"], want=(False, True, True))
    arrays = [f64(c["dY"]), f64(c["X"]), c["L"]["W"][0], f64(c["A"]), f64(c["B"])]
    al, z = c["alpha"].astype(np.float64), np.zeros((c["M"], 72))
    want = ref.lora_backward(*arrays, al, c["o"], c["ids"], z)
    S = ref.lora_backward(*map(np.abs, arrays), al, c["o"], c["ids"], z)
    for got, w, s in ((dA, want[1], S[1]), (dB, want[2], S[2])):
        check(f64(got), w, ((72 + min(c["M"], 512) + c["M"] // 512 + 20) * 2.0 ** -23 + 2 * part_eps(c["t"])) * s + 1e-30)


def test_lora_gradients_against_differences():
    # the loss sum(G * Y) is linear in each of X, A and B: a difference along a direction is exact
    c = lora_case(3, "bf16", 4, 0, [9, 30, 2], [0, 1, 0], 2, 8, 64, 96)
    o, ids, al = c["o"], c["ids"], c["alpha"].astype(np.float64)
    G, x, W, A, B = f64(c["dY"]), f64(c["X"]), c["L"]["W"][0], f64(c["A"]), f64(c["B"])
    dX, dA, dB = gq.gptq_matmul_lora_backward(c["dY"], c["X"], *c["args"])
    rng = gen(9)
    z = np.zeros((c["M"], 64))

    def loss(x, A, B):
        return (G * ref.lora(x, W, A, B, al, o, ids, z)).sum()

    base = loss(x, A, B)
    for got, v, at in ((dX, x, 0), (dA, A, 1), (dB, B, 2)):
        d = rng.standard_normal(v.shape)
        args = [x, A, B]
        args[at] = v + d
        diff, dot = loss(*args) - base, (f64(got) * d).sum()
        # rounding of each gradient entry (bf16 entries and bf16 weights for dX), independent
        # directions: the sum's error is at most eps sum |g d|, far below it in the mean
        eps = 2.0 ** -7 if at == 0 else 2.0 ** -14
        assert abs(diff - dot) <= eps * np.abs(f64(got) * d).sum() + 1e-6


def test_empty_calls():
    rng = gen(7)
    L = layer(rng, 2, 16, 32, 4, 0)
    X = torch.zeros(0, 32, dtype=torch.bfloat16, device="cuda")
    o = dev(off([0, 0]))
    assert gq.gptq_matmul_grouped(X, L["words"], L["s"], 4, o).shape == (0, 16)
    dw = gq.gptq_matmul_grouped_dw(torch.zeros(0, 16, dtype=torch.bfloat16, device="cuda"), X, o)
    assert dw.shape == (2, 16, 32) and (dw == 0).all()
    c = lora_case(3, "bf16", 4, 0, [0, 0], [0, 1], 2, 8, 64, 96)
    assert gq.gptq_matmul_lora(c["X"], *c["args"]).shape == (0, 64)
    dX, dA, dB = gq.gptq_matmul_lora_backward(c["dY"], c["X"], *c["args"])
    assert dX.shape == (0, 96) and (dA == 0).all() and (dB == 0).all()


BAD_OFFSETS = [[0, 5, 4, 40], [-1, 5, 20, 40], [0, 5, 20, 41], [3, 2, 1, 0], [0, 2 ** 31 - 1, 20, 40]]


@pytest.mark.parametrize("bad", BAD_OFFSETS)
@pytest.mark.parametrize("rows", [40, 400])
def test_bad_offsets_are_refused_on_the_device(bad, rows):
    rng = gen(8)
    bad = [v if v in (-1, 0, 1, 2, 3) or v > 2 ** 30 else v * rows // 40 for v in bad]
    bad = np.array(bad, dtype=np.int32)
    if bad[-1] == rows and (np.diff(bad.astype(np.int64)) >= 0).all() and bad[0] >= 0:
        pytest.skip("in order at this size")
    L = layer(rng, 3, 48, 64, 4, 0)
    X = rows_of(rng, (rows, 64), torch.bfloat16).cuda()
    dY = rows_of(rng, (rows, 48), torch.bfloat16).cuda()

    def refused(call, *outs):
        status = gq.new_status()
        call(status)
        assert int(status.item()) == gq.GPTQ_ERR_ARG
        for o in outs:
            assert (o == 7).all()

    y = torch.full((rows, 48), 7.0, dtype=torch.bfloat16, device="cuda")
    refused(lambda st: gq.gptq_matmul_grouped(X, L["words"], L["s"], 4, dev(bad), out=y, status=st), y)
    refused(lambda st: gq.gptq_matmul_grouped(X[:8], L["words"], L["s"], 4, dev(bad), out=y[:8], status=st), y)
    x = torch.full((rows, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    refused(lambda st: gq.gptq_matmul_grouped_dx(dY, L["words"], L["s"], 4, 64, dev(bad), out=x, status=st), x)
    g = torch.full((3, 48, 64), 7.0, device="cuda")
    refused(lambda st: gq.gptq_matmul_grouped_dw(dY, X, dev(bad), out=g, status=st), g)
    c = lora_case(3, "bf16", 4, 0, [rows - 2, 1, 1], [0, 1, 0], 2, 8, 48, 64)
    args = list(c["args"])
    args[6] = dev(bad)
    for n in (rows, 8):
        refused(lambda st: gq.gptq_matmul_lora(c["X"][:n], *args, out=y[:n], status=st), y)
    ga, gb = torch.full((2, 8, 64), 7.0, device="cuda"), torch.full((2, 48, 8), 7.0, device="cuda")
    refused(lambda st: gq.gptq_matmul_lora_backward(c["dY"], c["X"], *args, dX=x, dA=ga, dB=gb, status=st), x, ga, gb)


@pytest.mark.parametrize("n", [8, 60])
def test_bad_adapter_ids_and_groups_are_refused(n):
    c = lora_case(3, "bf16", 4, 0, [n - 1, 1], [0, 1], 2, 8, 48, 64)
    for bad in (2, -2):
        args = list(c["args"])
        args[7] = dev(np.array([0, bad], dtype=np.int32))
        y = torch.full((n, 48), 7.0, dtype=torch.bfloat16, device="cuda")
        status = gq.new_status()
        gq.gptq_matmul_lora(c["X"], *args, out=y, status=status)
        assert int(status.item()) == gq.GPTQ_ERR_ARG and (y == 7).all()
        ga = torch.full((2, 8, 64), 7.0, device="cuda")
        gb = torch.full((2, 48, 8), 7.0, device="cuda")
        status = gq.new_status()
        gq.gptq_matmul_lora_backward(c["dY"], c["X"], *args, dA=ga, dB=gb, status=status)
        assert int(status.item()) == gq.GPTQ_ERR_ARG and (ga == 7).all() and (gb == 7).all()
    L = layer(gen(4), 1, 48, 64, 4, 32, indexed=True)
    g = L["g"].clone()
    g[0, 5] = 2                                            # two groups: 0 and 1
    status = gq.new_status()
    gq.gptq_matmul_grouped(c["X"], L["words"], L["s"], 4, None, 32, g, status=status)
    assert int(status.item()) == gq.GPTQ_ERR_ARG


def test_refusals_without_a_status_write_nothing():
    # rows enough for the adapters' gradients to be summed from parts
    c = lora_case(3, "bf16", 4, 0, [2000, 1], [0, 1], 2, 8, 48, 64)
    for at, bad in ((6, [0, 2000, 1999]), (7, [0, 5])):
        args = list(c["args"])
        args[at] = dev(np.array(bad, dtype=np.int32))
        x = torch.full((2001, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        ga, gb = torch.full((2, 8, 64), 7.0, device="cuda"), torch.full((2, 48, 8), 7.0, device="cuda")
        gq.gptq_matmul_lora_backward(c["dY"], c["X"], *args, dX=x, dA=ga, dB=gb)
        for o in (x, ga, gb):
            assert (o == 7).all()


def test_a_failed_status_skips_the_call():
    c = lora_case(3, "bf16", 4, 0, [30, 1], [0, 1], 2, 8, 48, 64)
    status = torch.full((1,), gq.GPTQ_ERR_NOT_PD, dtype=torch.int32, device="cuda")
    y = torch.full((31, 48), 7.0, dtype=torch.bfloat16, device="cuda")
    gq.gptq_matmul_lora(c["X"], *c["args"], out=y, status=status)
    gq.gptq_matmul_grouped(c["X"][:4], c["args"][0], c["args"][1], 4, out=y[:4], status=status)
    x = torch.full((31, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    _, ga, gb = gq.gptq_matmul_lora_backward(c["dY"], c["X"], *c["args"], dX=x, dA=torch.full((2, 8, 64), 7.0, device="cuda"),
                                             dB=torch.full((2, 48, 8), 7.0, device="cuda"), status=status)
    assert int(status.item()) == gq.GPTQ_ERR_NOT_PD
    for o in (y, x, ga, gb):
        assert (o == 7).all()


def test_streams_and_graphs():
    # the same calls on another stream, from two streams at once, and captured and replayed on
    # new inputs; two graphs that share one workspace, replayed one after the other
    c = lora_case(4, "bf16", 4, 64, [40, 1, 7], [0, 1, 0], 2, 16, 96, 128)
    o = dev(off([48]))
    words, s = c["args"][0], c["args"][1]
    want = gq.gptq_matmul_lora(c["X"], *c["args"])
    plain = gq.gptq_matmul_grouped(c["X"], words, s, 4, o, 64)
    grads = gq.gptq_matmul_lora_backward(c["dY"], c["X"], *c["args"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for st in streams:
            got.append(gq.gptq_matmul_lora(c["X"], *c["args"], stream=st))
            got.append(gq.gptq_matmul_grouped(c["X"], words, s, 4, o, 64, stream=st))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, plain if i % 2 else want)

    ws = torch.empty(gq.gptq_lora_workspace_size(1, 48, 96, 128, 3, 2, 16), dtype=torch.uint8, device="cuda")
    X, dY = torch.zeros_like(c["X"]), torch.zeros_like(c["dY"])
    graphs, outs = [], []
    for kind in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            if kind == 0:
                outs.append(gq.gptq_matmul_lora(X, *c["args"], workspace=ws))
            else:
                outs.append(gq.gptq_matmul_lora_backward(dY, X, *c["args"], workspace=ws))
        graphs.append(g)
    X.copy_(c["X"])
    dY.copy_(c["dY"])
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want)
    for a, b in zip(outs[1], grads):
        assert torch.equal(a, b)


def test_new_outputs_on_another_stream():
    # the current stream is still writing memory that it has freed: a new output of a call on
    # another stream is not that memory
    M, K, N = 64, 256, 4096
    rng = gen(12)
    L = layer(rng, 1, N, K, 4, 0)
    X = rows_of(rng, (M, K), torch.bfloat16).cuda()
    want = gq.gptq_matmul_grouped(X, L["words"], L["s"], 4)
    big = torch.ones(1 << 28, device="cuda")
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        for _ in range(4):
            big.mul_(1.0)
        old = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        old.fill_(3.0)
        del old
        y = gq.gptq_matmul_grouped(X, L["words"], L["s"], 4, stream=other)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        del y


def test_together():
    # a layer as a user has it: quantised with input groups and act-order, packed, multiplied by
    # experts' rows, gradients back through it, the gradient into the first-order start
    from post_weight_quantization_solve_b200 import synth

    wl = synth.WORKLOADS["mlp_up"].scaled(K=256, N=192, M=2048, bits=4, chunk=2048)
    X = synth.tokens_chunk(wl, 0).cuda()
    W = synth.weights(wl).cuda()
    H = torch.zeros(256, 256, device="cuda")
    gq.gptq_accumulate_hessian(H, X)
    perm = gq.gptq_act_order(H)
    Hp = gq.gptq_permute_hessian(H, perm)
    status = gq.gptq_prepare(Hp)
    Wq = W.float()
    codes, scales, g_idx, status = gq.gptq_quantize_layer_grouped(Wq, Hp, 4, 64, 64, perm=perm, write_back=True,
                                                                  status=status)
    words = gq.gptq_pack_codes(codes, 4)
    x = X[:100].contiguous()
    y = gq.gptq_matmul_grouped(x, words, scales, 4, None, 64, g_idx, status=status)
    gq.raise_on_status(status)
    want, S = f64(x) @ f64(Wq).T, np.abs(f64(x)) @ np.abs(f64(Wq)).T
    check(f64(y), want, limit(want, S, 256, torch.bfloat16, 1) + 2.0 ** -22 * S)
    one = gq.gptq_matmul_grouped(x[:1], words, scales, 4, None, 64, g_idx)
    check(f64(one), want[:1], (limit(want, S, 256, torch.bfloat16, 1) + 2.0 ** -22 * S)[:1])
    dY = (y - x[:, :192]).contiguous()
    dX = gq.gptq_matmul_grouped_dx(dY, words, scales, 4, 256, None, 64, g_idx)
    wx, Sx = f64(dY) @ f64(Wq), np.abs(f64(dY)) @ np.abs(f64(Wq))
    check(f64(dX), wx, limit(wx, Sx, 192, torch.bfloat16, 1) + 2.0 ** -22 * Sx)
    G = gq.gptq_matmul_grouped_dw(dY, x)
    check(f64(G[0]), f64(dY).T @ f64(x), 104 * 2.0 ** -23 * (np.abs(f64(dY)).T @ np.abs(f64(x))) + 1e-30)
    H2 = H.clone()
    status = gq.gptq_prepare(H2)
    start = W.float()
    gq.gptq_first_order_shift(start, H2, G[0], 0.5, status=status)
    gq.raise_on_status(status)
    assert torch.isfinite(start).all() and not torch.equal(start, W.float())
