"""Workspace of the adapters' backward pass: room for what is written there and no more."""

import post_weight_quantization_solve_b200 as gq
from post_weight_quantization_solve_b200.build import build


def test_no_room_for_parts_of_gradients_that_have_one():
    build()
    # 32 adapters of rank 64 beside a layer of 14,336 x 4,096: tiles enough, so each gradient is one part
    M, N, K, R, L, r = 8192, 14336, 4096, 64, 32, 64
    size = gq.gptq_lora_workspace_size(1, M, N, K, R, L, r)
    rows, transposed = 2 * M * (3 + 2) * r * 2, L * N * r * 2        # T and U; B as [rank][N]
    assert rows + transposed <= size <= rows + transposed + 4 * (3 * L + R) + 16 * 1024


def test_room_for_the_parts_of_few_adapters():
    build()
    M, N, K, R, L, r = 8192, 1024, 1024, 8, 1, 16
    size = gq.gptq_lora_workspace_size(1, M, N, K, R, L, r)
    rows, transposed = 2 * M * (3 + 2) * r * 2, L * N * r * 2
    assert size >= rows + transposed + 2 * 2 * L * (N + K) * r * 4   # more than one part each
