"""Workloads of the packed-weight products: products grouped by expert and low-rank adapters
beside a packed projection.

`listed()` and `draw()` give cases, `prepare()` makes a case's tensors on the GPU, `run()` is
one pass through an operator: the library's calls where `own` is true, elementary torch
operations in 32 bits where it is not. `exact()` states the same results in 64 bits.
"""

import math

import numpy as np
import torch

if __name__ == "__main__":
    raise SystemExit("this file is imported")

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEVICE = "cuda"
SIGMA = 0.02          # weights' standard deviation, as in the synthetic layers
MAX_FLOPS = 2.0e12    # no drawn case costs more than the largest listed one
MAX_WEIGHTS = 480e6   # E N K of a case


def _case(name, op, dtype, bits, group, experts, tokens, topk, K, N, **more):
    c = {"name": name, "op": op, "dtype": dtype, "bits": bits, "group": group, "g_idx": False,
         "experts": experts, "tokens": tokens, "topk": topk, "K": K, "N": N, "pad": 0,
         "requests": 0, "lengths": "", "adapters": 0, "rank": 0}
    c.update(more)
    return c


def listed():
    return [
        # one token through the up projection of the headline layer (3 bits): decoding alone
        _case("token_dense", "forward", "bf16", 3, 0, 1, 1, 1, 4096, 14336),
        # one token, eight of 64 experts, input groups: the smallest call of a mixture layer
        _case("token_experts", "forward", "bf16", 4, 128, 64, 1, 8, 2048, 1024),
        # 128 requests decode together over 32 experts: a few dozen rows an expert
        _case("batch_experts", "forward", "bf16", 4, 128, 32, 128, 4, 2048, 2816),
        # a prompt batch over eight experts at the headline layer's size
        _case("prompt_experts", "forward", "bf16", 4, 0, 8, 8192, 2, 4096, 14336),
        # the gradient of the inputs through the experts' down projection
        _case("dx_experts", "dx", "bf16", 4, 128, 8, 4096, 2, 4096, 4096),
        # the same through a small act-order layer of odd sizes: re-estimated groups, so g_idx
        # is scattered over the columns
        _case("dx_ragged", "dx", "fp16", 2, 64, 5, 333, 2, 1000, 1416, g_idx=True, pad=7),
        # the experts' weight gradients, which the first-order start takes
        _case("dw_experts", "dw", "bf16", 4, 0, 8, 4096, 2, 4096, 4096),
        # a short calibration batch over many experts, fp16, sizes that end inside a tile
        _case("dw_ragged", "dw", "fp16", 4, 0, 16, 500, 3, 1000, 1320, pad=3),
        # 48 requests decode, each with one of 32 adapters, beside a 4-bit projection
        _case("lora_tokens", "lora", "bf16", 4, 128, 1, 48, 1, 4096, 4096, requests=48,
              lengths="one", adapters=32, rank=16),
        # prompts and decoding requests in one batch beside the headline layer
        _case("lora_prompt", "lora", "bf16", 3, 0, 1, 8192, 1, 4096, 14336, requests=24,
              lengths="mixed", adapters=8, rank=64),
        # training four adapters on a packed projection
        _case("lora_training", "lora_backward", "bf16", 4, 128, 1, 8192, 1, 4096, 4096,
              requests=8, lengths="mixed", adapters=4, rank=16),
        # a short training batch of many requests, fp16, 8 bits a channel
        _case("lora_ragged", "lora_backward", "fp16", 8, 0, 1, 700, 1, 1000, 1320, requests=24,
              lengths="mixed", adapters=6, rank=32, pad=5),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["forward", "forward", "dx", "dw", "lora", "lora", "lora_backward"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    bits = rng.choice([2, 3, 4, 4, 8])
    group = rng.choice([0, 0, 32, 64, 128, 128])
    g_idx = bool(group) and rng.random() < 0.2
    lora = op.startswith("lora")
    experts = 1 if lora else rng.choice([1, 2, 4, 8, 16, 32, 64])
    topk = 1 if experts == 1 else rng.randint(1, min(8, experts))
    while True:
        K, N = log(128, 14336), log(128, 14336)
        if rng.random() < 0.9:     # rows of whole 16-byte pieces, as nearly every layer has
            K, N = (K + 7) // 8 * 8, (N + 7) // 8 * 8
        tokens = log(1, 16384) if op in ("forward", "lora") else log(16, 16384)
        if experts * N * K <= MAX_WEIGHTS and 2.0 * tokens * topk * N * K <= MAX_FLOPS / 2:
            break
    c = _case("", op, dtype, bits, group, experts, tokens, topk, K, N, g_idx=g_idx,
              pad=rng.choice([0, 0, 0, 1, 5, 64]))
    if lora:
        lengths = rng.choice(["one", "mixed", "even"]) if tokens <= 256 else rng.choice(["mixed", "even"])
        c.update(lengths=lengths, adapters=log(1, 32), rank=rng.choice([8, 16, 16, 32, 64, 128]),
                 requests=tokens if lengths == "one" else min(tokens, log(1, 64)))
    del c["name"]
    return c


def _rows_of_experts(case, seed):
    """How many rows each expert gets: every token takes its topk experts by a score with a
    popularity of the expert's own, so the sizes are ragged."""
    rng = np.random.default_rng(seed)
    E, k = case["experts"], case["topk"]
    score = rng.standard_normal((case["tokens"], E)) + 0.7 * rng.standard_normal(E)
    picks = np.argpartition(-score, k - 1, axis=1)[:, :k] if k < E else np.tile(np.arange(E), (case["tokens"], 1))
    return np.bincount(picks.reshape(-1), minlength=E).tolist()


def _rows_of_requests(case, seed):
    """Lengths of the requests and their adapters (-1: none)."""
    rng = np.random.default_rng(seed)
    M, R = case["tokens"], case["requests"]
    if case["lengths"] == "mixed":     # half of the requests decode, the others share the rest
        w = np.where(rng.random(R) < 0.5, 0.0, rng.exponential(size=R) + 0.1)
        w[int(rng.integers(R))] += 1.0
        n = 1 + np.floor((M - R) * w / w.sum()).astype(np.int64)
        n[int(np.argmax(n))] += M - int(n.sum())
    else:
        n = np.full(R, M // R) + (np.arange(R) < M % R)
    ids = rng.integers(0, case["adapters"], R)
    if R > 2:
        ids[rng.random(R) < 0.1] = -1
    return n.tolist(), ids.tolist()


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    dtype, bits, E, K, N = TYPES[case["dtype"]], case["bits"], case["experts"], case["K"], case["N"]
    rows = case["tokens"] * case["topk"]
    M = rows + case["pad"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE)

    s = {"case": case, "rows": rows}
    # tokens of heavy tails (Student t of four degrees), gradients of small normal ones
    if case["op"] != "dx":
        s["X"] = torch.empty(M, K, dtype=dtype, device=DEVICE)
        for x in s["X"].split(8192):
            t = normal(*x.shape)
            chi = sum(normal(*x.shape).square() for _ in range(4)) * 0.25
            x.copy_(t / chi.sqrt().clamp_min(0.05) * 0.7071)
    if case["op"] in ("dx", "dw", "lora_backward"):
        s["dY"] = (normal(M, N) * 0.05).to(dtype)
    if case["op"] != "dw":
        G = -(-K // case["group"]) if case["group"] else 0
        shape = (E, N, G) if G else (E, N)
        s["scales"] = SIGMA * (6 + 2 * torch.rand(shape, generator=g, device=DEVICE)) / (2 ** bits - 1)
        words = []
        for e in range(E):     # codes around the zero point, as a bit stream of 32-bit words
            z = 2 ** (bits - 1)
            c = (normal(N, K) * ((2 ** bits - 1) / 7.0) + z).round().clamp(0, 2 ** bits - 1).to(torch.int64)
            c = torch.nn.functional.pad(c, (0, -K % 32)).view(N, -1, 32)
            w = torch.zeros(N, c.shape[1], bits, dtype=torch.int64, device=DEVICE)
            for i in range(32):
                j, at = i * bits // 32, i * bits % 32
                w[:, :, j] |= (c[:, :, i] << at) & 0xFFFFFFFF
                if at + bits > 32:
                    w[:, :, j + 1] |= c[:, :, i] >> (32 - at)
            w = w.view(N, -1)[:, :(K * bits + 31) // 32]
            words.append(torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32))
        s["words"] = torch.stack(words)
        if G:
            k = torch.arange(K, device=DEVICE)
            if case["g_idx"]:   # groups of an act-order layer: runs of a processing order
                order = torch.rand(E, K, generator=g, device=DEVICE).argsort(1)
                s["g_idx"] = torch.empty(E, K, dtype=torch.int32, device=DEVICE)
                s["g_idx"].scatter_(1, order, (k // case["group"]).to(torch.int32).expand(E, K))
    if case["op"] in ("forward", "dx", "dw"):
        s["counts"] = _rows_of_experts(case, seed)
        s["offsets"] = torch.tensor([0] + np.cumsum(s["counts"]).tolist(), dtype=torch.int32, device=DEVICE)
    else:
        L, r = case["adapters"], case["rank"]
        n, ids = _rows_of_requests(case, seed)
        s["offsets"] = torch.tensor([0] + np.cumsum(n).tolist(), dtype=torch.int32, device=DEVICE)
        s["ids"] = torch.tensor(ids, dtype=torch.int32, device=DEVICE)
        s["A"] = (normal(L, r, K) / math.sqrt(K)).to(dtype)
        s["B"] = (normal(L, N, r) * 0.02).to(dtype)
        s["alpha"] = 0.5 + torch.rand(L, generator=g, device=DEVICE)
    if case["op"] in ("forward", "lora"):
        s["out"] = torch.zeros(M, N, dtype=dtype, device=DEVICE)
    if case["op"] in ("dx", "lora_backward"):
        s["out"] = torch.zeros(M, K, dtype=dtype, device=DEVICE)
    return s


# ---- the plain forms -----------------------------------------------------------------------

def _weights(s, e):
    """Expert e's weights from its words, in 32 bits."""
    c = s["case"]
    bits, K = c["bits"], c["K"]
    w = torch.nn.functional.pad(s["words"][e].to(torch.int64) & 0xFFFFFFFF, (0, 1))
    at = torch.arange(K, device=w.device) * bits
    code = (w[:, at // 32] | (w[:, at // 32 + 1] << 32)) >> (at % 32) & (2 ** bits - 1)
    code = (code - 2 ** (bits - 1)).float()
    scale = s["scales"][e]
    if c["g_idx"]:
        return code * scale[:, s["g_idx"][e].long()]
    if c["group"]:
        return code * scale[:, torch.arange(K, device=w.device) // c["group"]]
    return code * scale[:, None]


def _adapter_of_rows(s, like, L):
    """One column for each adapter, alpha where the row's request has it and 0 elsewhere."""
    row = torch.arange(like.shape[0], device=like.device)
    seg = (row[:, None] >= s["offsets"][None, 1:]).sum(1)
    ids = torch.nn.functional.pad(s["ids"], (0, 1), value=-1)[seg]
    return (ids[:, None] == torch.arange(L, device=like.device)[None]).float() * s["alpha"]


def _plain(s):
    c = s["case"]
    op, E, rows, dtype = c["op"], c["experts"], s["rows"], TYPES[c["dtype"]]
    if op in ("forward", "dx"):
        x = s["X" if op == "forward" else "dY"][:rows].float().split(s["counts"])
        y = [x[e] @ (_weights(s, e).T if op == "forward" else _weights(s, e))
             for e in range(E) if s["counts"][e]]
        s["out"][:rows] = torch.cat(y).to(dtype)
        return s["out"]
    if op == "dw":
        x, d = s["X"][:rows].float().split(s["counts"]), s["dY"][:rows].float().split(s["counts"])
        return torch.stack([d[e].T @ x[e] for e in range(E)])
    L, r = c["adapters"], c["rank"]
    x, A, B = s["X"][:rows].float(), s["A"].float(), s["B"].float()
    W = _weights(s, 0)
    which = _adapter_of_rows(s, x, L)[:, :, None]                        # [rows][L][1]
    T = ((x @ A.reshape(L * r, -1).T).view(rows, L, r) * which).view(rows, L * r)
    flat = B.permute(0, 2, 1).reshape(L * r, -1)                         # [L r][N]
    if op == "lora":
        s["out"][:rows] = (x @ W.T + T @ flat).to(dtype)
        return s["out"]
    d = s["dY"][:rows].float()
    U = ((d @ flat.T).view(rows, L, r) * which).view(rows, L * r)
    s["out"][:rows] = (d @ W + U @ A.reshape(L * r, -1)).to(dtype)
    dA = (U.T @ x).view(L, r, -1)
    dB = (d.T @ T).view(-1, L, r).permute(1, 0, 2).contiguous()
    return s["out"], dA, dB


def run(s):
    if not own:
        return _plain(s)
    import post_weight_quantization_solve_b200 as gq
    c = s["case"]
    layer = dict(groupsize=c["group"], g_idx=s.get("g_idx"))
    if c["op"] == "forward":
        return gq.gptq_matmul_grouped(s["X"], s["words"], s["scales"], c["bits"], s["offsets"],
                                      out=s["out"], **layer)
    if c["op"] == "dx":
        return gq.gptq_matmul_grouped_dx(s["dY"], s["words"], s["scales"], c["bits"], c["K"],
                                         s["offsets"], out=s["out"], **layer)
    if c["op"] == "dw":
        return gq.gptq_matmul_grouped_dw(s["dY"], s["X"], s["offsets"])
    adapters = (s["A"], s["B"], s["alpha"], s["offsets"], s["ids"])
    if c["op"] == "lora":
        return gq.gptq_matmul_lora(s["X"], s["words"], s["scales"], c["bits"], *adapters,
                                   out=s["out"], **layer)
    return gq.gptq_matmul_lora_backward(s["dY"], s["X"], s["words"], s["scales"], c["bits"],
                                        *adapters, dX=s["out"], **layer)


def work(case):
    E, K, N, b = case["experts"], case["K"], case["N"], case["bits"]
    rows = case["tokens"] * case["topk"]
    G = -(-K // case["group"]) if case["group"] else 1
    # experts that get a row: all of them, but for the smallest batches
    used = min(E, rows) if case["tokens"] == 1 else E * (1 - (1 - case["topk"] / E) ** case["tokens"])
    weights = used * N * (K * b / 8 + 4 * G) + (4 * K * used if case["g_idx"] else 0)
    product = 2.0 * rows * N * K
    if case["op"] in ("forward", "dx"):
        return {"bytes": weights + 2 * rows * (K + N), "flops": product}
    if case["op"] == "dw":
        return {"bytes": 2 * rows * (K + N) + 4.0 * E * N * K, "flops": product}
    L, r = case["adapters"], case["rank"]
    used = L * (1 - (1 - 1 / L) ** case["requests"])
    pair = used * r * (K + N)
    if case["op"] == "lora":
        return {"bytes": weights + 2 * rows * (K + N) + 2 * pair,
                "flops": product + 2.0 * rows * r * (K + N)}
    return {"bytes": weights + 2 * rows * (2 * K + N) + 2 * pair + 4.0 * L * r * (K + N),
            "flops": product + 2.0 * rows * r * 3 * (K + N)}


# ---- 64 bits -------------------------------------------------------------------------------

def exact(case, seed):
    """From the definition: each code is bits [b k, b k + b) of its row's bit stream."""
    s = prepare(case, seed)
    b, K, N, E, rows = case["bits"], case["K"], case["N"], case["experts"], s["rows"]

    def layer(e):
        octets = s["words"][e].contiguous().view(torch.uint8)            # little-endian bytes
        stream = torch.stack([(octets >> i) & 1 for i in range(8)], 2).view(N, -1)
        digits = stream[:, :K * b].reshape(N, K, b).double()
        value = digits @ (2.0 ** torch.arange(b, device=digits.device, dtype=torch.float64)) - 2.0 ** (b - 1)
        sc = s["scales"][e].double()
        if case["group"] == 0:
            return value * sc.view(N, 1)
        group = s["g_idx"][e].long() if case["g_idx"] else torch.div(
            torch.arange(K, device=sc.device), case["group"], rounding_mode="floor")
        return value * torch.gather(sc, 1, group.expand(N, K))

    ends = s["offsets"].tolist()
    if case["op"] in ("forward", "dx"):
        a = s["X" if case["op"] == "forward" else "dY"].double()
        y = torch.zeros_like(s["out"], dtype=torch.float64)
        for e in range(E):
            if ends[e + 1] > ends[e]:
                w = layer(e)
                part = a[ends[e]:ends[e + 1]]
                y[ends[e]:ends[e + 1]] = part @ w.t() if case["op"] == "forward" else part @ w
        return y
    if case["op"] == "dw":
        y = torch.zeros(E, N, K, dtype=torch.float64, device=DEVICE)
        for e in range(E):
            part = slice(ends[e], ends[e + 1])
            y[e] = s["dY"][part].double().t() @ s["X"][part].double()
        return y
    w = layer(0)
    x = s["X"].double()
    y = torch.zeros_like(s["out"], dtype=torch.float64)
    if case["op"] == "lora_backward":
        d = s["dY"].double()
        dA, dB = torch.zeros_like(s["A"], dtype=torch.float64), torch.zeros_like(s["B"], dtype=torch.float64)
        y[:rows] = d[:rows] @ w
    else:
        y[:rows] = x[:rows] @ w.t()
    for i, a in enumerate(s["ids"].tolist()):
        if a < 0 or ends[i + 1] == ends[i]:
            continue
        part = slice(ends[i], ends[i + 1])
        A, B, alpha = s["A"][a].double(), s["B"][a].double(), float(s["alpha"][a])
        if case["op"] == "lora":
            y[part] += alpha * (x[part] @ A.t()) @ B.t()
        else:
            y[part] += alpha * (d[part] @ B) @ A
            dA[a] += alpha * (d[part] @ B).t() @ x[part]
            dB[a] += alpha * d[part].t() @ (x[part] @ A.t())
    return (y, dA, dB) if case["op"] == "lora_backward" else y
