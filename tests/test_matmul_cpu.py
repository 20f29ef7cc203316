"""Products of packed layers: exports, host-side refusals of the C ABI and of the binding, and the
plain 64-bit statement the GPU tests compare with. No GPU call is made here."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import matmul_util as ref
import oracle as O
import post_weight_quantization_solve_b200 as gq
from post_weight_quantization_solve_b200.build import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
FAKE = 1 << 20          # never dereferenced: every call below fails its host checks


@pytest.fixture(scope="module")
def lib():
    build()
    return gq.load_library()


def test_exports_every_declared_symbol(lib):
    text = open(os.path.join(ROOT, "include", "gptq_matmul.h"), encoding="utf-8").read()
    names = re.findall(r"GPTQ_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)
    assert set(names) == set(gq.MATMUL_EXPORTS)
    for name in names:
        assert hasattr(lib, name) and hasattr(gq, name)


def packed(**kw):
    W = gq.GPTQPacked()
    v = dict(words=FAKE, ld_words=8, scales=FAKE, g_idx=None, experts=1, N=16, K=64, bits=4, groupsize=0)
    v.update(kw)
    for k, x in v.items():
        setattr(W, k, x)
    return W


BAD_LAYERS = [dict(words=None), dict(scales=None), dict(words=FAKE + 2), dict(bits=5), dict(N=0), dict(K=0),
              dict(N=65536), dict(K=65536, ld_words=1 << 20), dict(experts=0), dict(experts=513), dict(groupsize=16),
              dict(ld_words=7), dict(g_idx=FAKE), dict(g_idx=FAKE + 1, groupsize=32), dict(experts=2)]


@pytest.mark.parametrize("bad", BAD_LAYERS)
def test_layer_checks(lib, bad):
    W = packed(**bad)
    f = P(FAKE)
    for fn in (lib.gptq_matmul_grouped, lib.gptq_matmul_grouped_dx):
        assert fn(f, 99999, f, 99999, 0, 4, ctypes.byref(W), None, None, None) == gq.GPTQ_ERR_ARG
    assert lib.gptq_matmul_lora(f, 99999, f, 99999, 0, 4, ctypes.byref(W), f, f, f, 1, 8, f, f, 1, f, 1 << 30, None,
                                None) == gq.GPTQ_ERR_ARG


def test_row_checks(lib):
    W, f = packed(), P(FAKE)
    w = ctypes.byref(W)
    bad = [(None, 16, f, 64, 0, 4), (f, 16, None, 64, 0, 4), (f, 15, f, 64, 0, 4), (f, 16, f, 63, 0, 4),
           (f, 16, f, 64, gq.GPTQ_F32, 4), (f, 16, f, 64, 3, 4), (f, 16, f, 64, 0, -1), (f, 16, f, 64, 0, (1 << 30) + 1),
           (P(FAKE + 1), 16, f, 64, 0, 4), (f, 16, P(FAKE + 1), 64, 0, 4)]
    for y, ldy, x, ldx, dt, M in bad:
        assert lib.gptq_matmul_grouped(y, ldy, x, ldx, dt, M, w, None, None, None) == gq.GPTQ_ERR_ARG
        assert lib.gptq_matmul_grouped_dx(x, ldx, y, ldy, dt, M, w, None, None, None) == gq.GPTQ_ERR_ARG
    assert lib.gptq_matmul_grouped(f, 16, f, 64, 0, 4, w, P(FAKE + 2), None, None) == gq.GPTQ_ERR_ARG
    assert lib.gptq_matmul_grouped(None, 0, None, 0, 0, 0, w, None, None, None) == gq.GPTQ_OK     # no rows
    dw = lib.gptq_matmul_grouped_dw
    ok = [f, f, 16, f, 64, 0, 4, 16, 64, 1, None, 0, None, None]
    for at, v in ((0, None), (1, None), (2, 15), (4, 63), (5, 1), (6, -1), (7, 0), (8, 65536), (9, 0), (9, 513), (9, 2),
                  (11, 2), (10, P(FAKE + 1)), (0, P(FAKE + 2))):
        args = list(ok)
        args[at] = v
        assert dw(*args) == gq.GPTQ_ERR_ARG, at


def test_adapter_checks(lib):
    W, f = packed(), P(FAKE)
    ok = [f, 16, f, 64, 0, 4, ctypes.byref(W), f, f, f, 2, 16, f, f, 3, f, 1 << 30, None, None]
    for at, v in ((7, None), (8, None), (9, None), (12, None), (13, None), (7, P(FAKE + 8)), (8, P(FAKE + 2)), (10, 0),
                  (10, 65536), (11, 0), (11, 12), (11, 136), (14, 0), (14, 65536), (0, None), (1, 15), (4, 1)):
        args = list(ok)
        args[at] = v
        assert lib.gptq_matmul_lora(*args) == gq.GPTQ_ERR_ARG, at
    for at, v in ((15, None), (15, P(FAKE + 8)), (16, 64)):
        args = list(ok)
        args[at] = v
        assert lib.gptq_matmul_lora(*args) == gq.GPTQ_ERR_WORKSPACE
    back = [f, 64, f, f, f, 16, f, 64, 0, 4, ctypes.byref(W), f, f, f, 2, 16, f, f, 3, f, 64, None, None]
    assert lib.gptq_matmul_lora_backward(*back) == gq.GPTQ_ERR_WORKSPACE
    for at, v in ((4, None), (5, 15), (6, None), (1, 63), (2, P(FAKE + 2)), (3, P(FAKE + 1)), (8, 1)):
        args = list(back)
        args[at] = v
        assert lib.gptq_matmul_lora_backward(*args) == gq.GPTQ_ERR_ARG, at
    for at in (0, 2, 3):
        back[at] = None
    assert lib.gptq_matmul_lora_backward(*back) == gq.GPTQ_OK      # nothing wanted


def test_workspace_sizes(lib):
    size = gq.gptq_lora_workspace_size
    assert size(0, 100, 256, 512, 3, 2, 16) >= 100 * 32 * 2
    assert size(1, 100, 256, 512, 3, 2, 16) > size(0, 100, 256, 512, 3, 2, 16)
    assert size(0, 0, 256, 512, 3, 2, 16) % 256 == 0 and size(1, 1 << 20, 65535, 65535, 65535, 64, 128) % 256 == 0
    for bad in ((2, 1, 1, 1, 1, 1, 8), (0, -1, 1, 1, 1, 1, 8), (0, 1, 0, 1, 1, 1, 8), (0, 1, 1, 65536, 1, 1, 8),
                (0, 1, 1, 1, 0, 1, 8), (0, 1, 1, 1, 1, 0, 8), (0, 1, 1, 1, 1, 1, 4), (0, 1, 1, 1, 1, 1, 9)):
        assert size(*bad) == 0


def test_binding_refuses_host_tensors(lib):
    X = torch.zeros(4, 64, dtype=torch.bfloat16)
    dY = torch.zeros(4, 16, dtype=torch.bfloat16)
    words, s = torch.zeros(16, 8, dtype=torch.int32), torch.zeros(16)
    A, B = torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 16, 8, dtype=torch.bfloat16)
    al, o, ids = torch.zeros(2), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: gq.gptq_matmul_grouped(X, words, s, 4), lambda: gq.gptq_matmul_grouped_dx(dY, words, s, 4, 64),
                 lambda: gq.gptq_matmul_grouped_dw(dY, X), lambda: gq.gptq_matmul_lora(X, words, s, 4, A, B, al, o, ids),
                 lambda: gq.gptq_matmul_lora_backward(dY, X, words, s, 4, A, B, al, o, ids)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()


@pytest.fixture
def host_calls(lib, monkeypatch):
    """The wrappers on host tensors with a library that only checks argument types."""
    import contextlib

    calls = {}

    class FakeLib:
        def __getattr__(self, name):
            real = getattr(lib, name)
            if name == "gptq_lora_workspace_size":
                return real

            def fn(*args):
                assert len(args) == len(real.argtypes), (name, len(args), len(real.argtypes))
                for a, t in zip(args, real.argtypes):
                    t.from_param(a)
                calls[name] = args
                return 0
            return fn

    monkeypatch.setattr(gq, "_lib", FakeLib())
    monkeypatch.setattr(gq, "_device", lambda t, name: t.device)
    monkeypatch.setattr(gq, "_stream", lambda stream, dev=None: P(0))
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    return calls


def operands(t=torch.bfloat16):
    return dict(X=torch.zeros(4, 64, dtype=t), dY=torch.zeros(4, 16, dtype=t), words=torch.zeros(3, 16, 8, dtype=torch.int32),
                s=torch.zeros(3, 16), o=torch.zeros(4, dtype=torch.int32), A=torch.zeros(2, 8, 64, dtype=t),
                B=torch.zeros(2, 16, 8, dtype=t), al=torch.zeros(2), ids=torch.zeros(3, dtype=torch.int32))


def test_wrappers_match_their_c_signatures(host_calls):
    v = operands()
    assert gq.gptq_matmul_grouped(v["X"], v["words"], v["s"], 4, v["o"]).shape == (4, 16)
    assert gq.gptq_matmul_grouped_dx(v["dY"], v["words"], v["s"], 4, 64, v["o"]).shape == (4, 64)
    assert gq.gptq_matmul_grouped_dw(v["dY"], v["X"], v["o"]).shape == (3, 16, 64)
    w, s = v["words"][0], v["s"][0]
    rest = (v["A"], v["B"], v["al"], v["o"], v["ids"])
    assert gq.gptq_matmul_lora(v["X"], w, s, 4, *rest).shape == (4, 16)
    dX, dA, dB = gq.gptq_matmul_lora_backward(v["dY"], v["X"], w, s, 4, *rest)
    assert dX.shape == (4, 64) and dA.shape == (2, 8, 64) and dB.shape == (2, 16, 8)
    assert set(host_calls) == set(gq.MATMUL_EXPORTS) - {"gptq_lora_workspace_size"}


def test_binding_refuses_what_the_abi_cannot_see(host_calls):
    v = operands()
    X, words, s, o = v["X"], v["words"], v["s"], v["o"]
    f = gq.gptq_matmul_grouped
    rest = (v["A"], v["B"], v["al"], o, v["ids"])
    w1, s1 = words[0], s[0]
    for call in (lambda: f(X.float(), words, s, 4, o), lambda: f(X, words.long(), s, 4, o),
                 lambda: f(X, words, s.double(), 4, o), lambda: f(X, words, s, 4, o.long()),
                 lambda: f(X, words, s, 4, o, out=torch.zeros(4, 16)),
                 lambda: gq.gptq_matmul_grouped_dw(v["dY"], X.half(), o),
                 lambda: gq.gptq_matmul_lora(X, w1, s1, 4, v["A"].half(), *rest[1:])):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: f(X[0], words, s, 4, o), lambda: f(X, words, s[:2], 4, o), lambda: f(X, words, s, 4, o[:3]),
                 lambda: f(X, words[:, :, :7], s, 4, o), lambda: f(X, words, s, 4, o, 32),
                 lambda: f(X, words, s, 4, o, g_idx=torch.zeros(3, 64, dtype=torch.int32)),
                 lambda: f(X.t(), words, s, 4, o), lambda: f(X, words.transpose(1, 2), s, 4, o),
                 lambda: f(X, words, s, 4, o, out=torch.zeros(5, 16, dtype=torch.bfloat16)),
                 lambda: f(X, words[:, 1:], s[:, 1:].contiguous(), 4, o),
                 lambda: gq.gptq_matmul_grouped_dx(X, words, s, 4, 64, o),
                 lambda: gq.gptq_matmul_grouped_dw(v["dY"], X[:3], o),
                 lambda: gq.gptq_matmul_grouped_dw(v["dY"], X, o, accumulate=True),
                 lambda: gq.gptq_matmul_lora(X, w1, s1, 4, v["A"], v["B"][:, :15], *rest[2:]),
                 lambda: gq.gptq_matmul_lora(X, w1, s1, 4, v["A"], v["B"], v["al"], o[:3], v["ids"]),
                 lambda: gq.gptq_matmul_lora_backward(X, X, w1, s1, 4, *rest)):
        with pytest.raises(ValueError):
            call()


def test_the_plain_statement_packs_as_the_oracle_does():
    rng = np.random.default_rng(0)
    for bits in (2, 3, 4, 8):
        for K in (1, 31, 33, 100):
            c = rng.integers(0, 2 ** bits, (5, K)).astype(np.uint8)
            assert np.array_equal(ref.pack(c, bits), O.pack_codes(c, bits))


def test_the_plain_gradients_are_the_products_derivatives():
    rng = np.random.default_rng(1)
    o, ids = [1, 3, 3, 6], [1, 0, -1]
    X, W = rng.standard_normal((7, 5)), rng.standard_normal((4, 5))
    A, B, al = rng.standard_normal((2, 3, 5)), rng.standard_normal((2, 4, 3)), np.array([0.5, 2.0])
    G, z = rng.standard_normal((7, 4)), np.zeros((7, 4))
    G[0] = G[6] = 0
    dX, dA, dB = ref.lora_backward(G, X, W, A, B, al, o, ids, np.zeros((7, 5)))

    def loss(X, A, B):
        return (G * ref.lora(X, W, A, B, al, o, ids, z)).sum()

    for grad, at in ((dX, 0), (dA, 1), (dB, 2)):
        args = [X, A, B]
        d = rng.standard_normal(args[at].shape)
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + d, args[at] - d
        assert abs((loss(*up) - loss(*down)) / 2 - (grad * d).sum()) < 1e-10
