"""Products of packed layers called from two host threads at once, each on a stream of its own and
with sizes that take different amounts of shared memory in the same kernel."""

import ctypes
import threading

import numpy as np
import pytest
import torch

import post_weight_quantization_solve_b200 as gq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,sizes", [("token", [(8, 4096), (8, 2048)]), ("tiled", [(40, 4096), (200, 256)]),
                                        ("gradient", [(40, 4096), (200, 256)]), ("sums", [(40, 1024), (40, 64)])])
def test_two_host_threads(kind, sizes):
    rng, errors, lib = np.random.default_rng(0), [], gq.load_library()
    ready = threading.Barrier(len(sizes))

    def work(M, K):
        try:
            # the C entry points, with little else in the threads' loops
            N, stream = 256, torch.cuda.Stream()
            words = torch.from_numpy(rng.integers(0, 2 ** 31, (N, K // 8), dtype=np.int32)).cuda()
            s = torch.ones(N, device="cuda")
            x = torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
            d = torch.ones(M, N, dtype=torch.bfloat16, device="cuda")
            W = ctypes.byref(gq.GPTQPacked(words.data_ptr(), K // 8, s.data_ptr(), None, 1, N, K, 4, 0))
            y, p, st = torch.empty(N * max(K, M), device="cuda"), ctypes.c_void_p, ctypes.c_void_p(stream.cuda_stream)
            y, px, pd = p(y.data_ptr()), p(x.data_ptr()), p(d.data_ptr())
            if kind == "sums":
                fn, args = lib.gptq_matmul_grouped_dw, (y, pd, N, px, K, 0, M, N, K, 1, None, 0, None, st)
            elif kind == "gradient":
                fn, args = lib.gptq_matmul_grouped_dx, (y, K, pd, N, 0, M, W, None, None, st)
            else:
                fn, args = lib.gptq_matmul_grouped, (y, N, px, K, 0, M, W, None, None, st)
            torch.cuda.synchronize()
            ready.wait(60)
            for i in range(20000):
                code = fn(*args)
                assert code == gq.GPTQ_OK, (code, i)
            stream.synchronize()
        except Exception as e:      # (a thread's failure does not end the test by itself)
            errors.append(e)

    threads = [threading.Thread(target=work, args=size) for size in sizes]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
