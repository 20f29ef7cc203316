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
