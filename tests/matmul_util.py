"""Plain 64-bit statements of the packed-layer products, for the tests of gptq_matmul_*."""

import numpy as np


def pack(codes, bits):
    """uint8 [..., K] -> uint32 [..., ceil(K bits / 32)], code k at bits [b k, b k + b)."""
    K = codes.shape[-1]
    stream = ((codes[..., None] >> np.arange(bits)) & 1).reshape(*codes.shape[:-1], K * bits)
    pad = -(K * bits) % 32
    stream = np.pad(stream, [(0, 0)] * (codes.ndim - 1) + [(0, pad)]).astype(np.uint64)
    words = stream.reshape(*codes.shape[:-1], -1, 32) << np.arange(32, dtype=np.uint64)
    return words.sum(-1).astype(np.uint32)


def weights(codes, bits, scales, groupsize, g_idx=None):
    """float64 [E][N][K]: scales[e][n][group(k)] (code - 2^(bits-1))."""
    E, N, K = codes.shape
    v = codes.astype(np.float64) - 2.0 ** (bits - 1)
    s = scales.astype(np.float64)
    if not groupsize:
        return v * s[:, :, None]
    g = g_idx if g_idx is not None else np.broadcast_to(np.arange(K) // groupsize, (E, K))
    return v * np.stack([s[e][:, g[e]] for e in range(E)])


def grouped(X, W, offsets, Y):
    """Y with the rows of each range replaced by X W_e^T."""
    Y = Y.copy()
    for e in range(W.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        Y[a:b] = X[a:b] @ W[e].T
    return Y


def grouped_dw(dY, X, offsets):
    return np.stack([dY[a:b].T @ X[a:b] for a, b in zip(offsets[:-1], offsets[1:])])


def lora(X, W, A, B, alpha, offsets, ids, Y):
    Y = grouped(X, W[None], [offsets[0], offsets[-1]], Y)
    for r, a in enumerate(ids):
        p = slice(int(offsets[r]), int(offsets[r + 1]))
        if a >= 0:
            Y[p] += alpha[a] * (X[p] @ A[a].T) @ B[a].T
    return Y


def lora_backward(dY, X, W, A, B, alpha, offsets, ids, dX):
    dX = dX.copy()
    s = slice(int(offsets[0]), int(offsets[-1]))
    dX[s] = dY[s] @ W
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    for r, a in enumerate(ids):
        p = slice(int(offsets[r]), int(offsets[r + 1]))
        if a < 0:
            continue
        U = alpha[a] * dY[p] @ B[a]
        dX[p] += U @ A[a]
        dA[a] += U.T @ X[p]
        dB[a] += alpha[a] * dY[p].T @ (X[p] @ A[a].T)
    return dX, dA, dB
