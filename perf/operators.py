"""The operators on packed 4- and 6-bit weight tables, as cases to be measured.

Weight-only linear layers on 4-bit weights with group scales (flexq.linear4,
flexq.linear4_group), and the lookup of rows of a packed table with its
gradient (flexq.embedding, flexq.embedding_backward).  A case's `run` is one
pass: in plain torch operations, or, where `own` is true, the library's calls.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
QMAX = {4: 7, 6: 31}


# ------------------------------------------------------------------- cases --
def _linear(name, M, N, K, gs, dtype="fp16"):
    """N: the layers' widths as a text; several layers read the same x."""
    return {"name": name, "op": "linear", "M": M, "N": N, "K": K, "gs": gs, "dtype": dtype}


def _embedding(name, B, S, pad, V, K, gs, bits, scale, dtype="fp16"):
    """B sequences of S tokens; sequence b ends in pad * S * 2b/B padding ids."""
    return {"name": name, "op": "embedding", "B": B, "S": S, "pad": pad, "V": V, "K": K,
            "gs": gs, "bits": bits, "scale": scale, "dtype": dtype}


def _backward(name, B, S, pad, V, K, gs, bits, scale, dtype="fp16", table="none"):
    """table: the type of the table's row gradient, or none of it."""
    c = _embedding(name, B, S, pad, V, K, gs, bits, scale, dtype)
    c.update(op="backward", table=table)
    return c


def listed():
    return [
        # decoding one token: the 7B block's square layers, where latency counts
        _linear("linear4 1 token 4096x4096", 1, "4096", 4096, 128),
        # ... and the 70B block's gate layer, a pure stream of weights
        _linear("linear4 1 token 28672x8192", 1, "28672", 8192, 128),
        # 70B q, k and v of one token: three layers that read the same input
        _linear("linear4 1 token q/k/v", 1, "8192,1024,1024", 8192, 128),
        # a few drafted tokens through an output head with an odd number of rows
        _linear("linear4 5 tokens 32003x4096 g64", 5, "32003", 4096, 64),
        # a decoding batch through the 70B down layer, bfloat16 activations
        _linear("linear4 16 tokens 8192x28672 bf16", 16, "8192", 28672, 128, "bf16"),
        # a short prompt, and a long one, through the 7B gate layer
        _linear("linear4 256 tokens 11008x4096 bf16", 256, "11008", 4096, 128, "bf16"),
        _linear("linear4 2048 tokens 11008x4096", 2048, "11008", 4096, 128),
        # the next token's row while decoding
        _embedding("embedding 1 token", 1, 1, 0.0, 32000, 8192, 128, 4, 1.0),
        # prompts: a full batch on an odd table, and a padded one on a 6-bit table
        _embedding("embedding 16x1024 tokens", 16, 1024, 0.0, 32003, 8192, 128, 4, 90.5),
        _embedding("embedding 8x512 padded 6-bit bf16", 8, 512, 0.25, 32000, 4096, 128, 6, 1.0, "bf16"),
        # tuning the scales of a frozen table on one short sequence
        _backward("backward 37 tokens scales 6-bit g64", 1, 37, 0.0, 32000, 4096, 64, 6, 1.0),
        # a training batch: the scales' gradient and the rows' one
        _backward("backward 8x1024 padded rows and scales", 8, 1024, 0.125, 32000, 4096, 128, 4, 64.0,
                  "bf16", "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    gs = rng.choice([32, 64, 128, 256])
    dtype = rng.choice(["fp16", "bf16"])
    if rng.random() < 0.5:
        layers = rng.choice([1, 1, 1, 2, 3, 4])
        K = gs * max(1, _log(rng, 256, 28672) // gs)
        most = 28672 * 8192 // K
        N = [_log(rng, 48, max(49, min(32768, most) // layers)) for _ in range(layers)]
        M = _log(rng, 1, min(2048, max(1, 2048 * 11008 * 4096 // (sum(N) * K))))
        return _drawn(_linear("", M, ",".join(str(n) for n in N), K, gs, dtype))
    bits = rng.choice([4, 4, 6])
    if bits == 6:
        K, V = 256 * _log(rng, 1, 32), 128 * _log(rng, 4, 250)
    else:
        K, V = gs * max(1, _log(rng, 256, 8192) // gs), _log(rng, 500, 32000)
    S = _log(rng, 1, 1024)
    B = _log(rng, 1, max(1, min(16, 4 * 8192 * 1024 // (S * K))))
    case = _embedding("", B, S, rng.choice([0.0, 0.0, 0.1, 0.4]), V, K, gs, bits,
                      rng.choice([1.0, math.sqrt(K)]), dtype)
    if rng.random() < 0.5:
        return _drawn(case)
    case.update(op="backward", table=rng.choice(["none", dtype, "fp32"]))
    if case["table"] != "none":                # the rows' gradient is written whole
        most = 250_000_000 // (K * DTYPES[case["table"]].itemsize)
        case["V"] = min(V, most // 128 * 128)
    return _drawn(case)


def _drawn(case):
    del case["name"]
    return case


def _widths(case):
    return [int(n) for n in case["N"].split(",")]


def _lengths(case):
    """Tokens of each sequence before its padding."""
    B, S = case["B"], case["S"]
    return [S - int(case["pad"] * S * 2 * b / B) for b in range(B)]


def _zipf(V):
    """The probability of the r-th most frequent token."""
    p = 1.0 / (np.arange(V, dtype=np.float64) + 3.0)
    return p / p.sum()


def _distinct(case):
    """How many rows of the table the tokens of a batch touch, on average."""
    return float((1.0 - (1.0 - _zipf(case["V"])) ** sum(_lengths(case))).sum())


def work(case):
    K, G = case["K"], case["K"] // case["gs"]
    if case["op"] == "linear":
        M, N = case["M"], sum(_widths(case))
        return {"bytes": N * K // 2 + 2 * N * G + 2 * M * K + 2 * M * N, "flops": 2 * M * N * K}
    T, U = sum(_lengths(case)), _distinct(case)
    row = K * case["bits"] // 8
    if case["op"] == "embedding":
        return {"bytes": int(8 * case["B"] * case["S"] + U * (row + 2 * G) + 2 * case["B"] * case["S"] * K),
                "flops": 2 * T * K}
    size = {"none": 0, "fp16": 2, "bf16": 2, "fp32": 4}[case["table"]]
    return {"bytes": int(8 * case["B"] * case["S"] + 2 * T * K + U * row + case["V"] * (K * size + 4 * G)),
            "flops": int(T * K + 2 * U * K)}


# ------------------------------------------------------------------ inputs --
def _weights(N, K, gen):
    return (torch.randn(N, K, generator=gen, dtype=torch.float32, device="cuda") * 0.02).half()


def _inputs(case, seed):
    """The tensors a case starts from: FP16 weights, and activations with a
    few channels of outliers, or tokens by Zipf's law and their gradients."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    K, dtype = case["K"], DTYPES[case["dtype"]]
    if case["op"] == "linear":
        w = [_weights(n, K, gen) for n in _widths(case)]
        x = torch.randn(case["M"], K, generator=gen, device="cuda")
        x[:, torch.randperm(K, generator=gen, device="cuda")[:max(1, K // 100)]] *= 20
        return {"w": w, "x": x.to(dtype)}
    B, S, V = case["B"], case["S"], case["V"]
    rank = torch.searchsorted(torch.from_numpy(np.cumsum(_zipf(V))).cuda(),
                              torch.rand(B, S, generator=gen, dtype=torch.float64, device="cuda"))
    ids = torch.randperm(V, generator=gen, device="cuda")[rank.clamp_(max=V - 1)]
    ends = torch.tensor(_lengths(case), device="cuda")[:, None]
    ids = torch.where(torch.arange(S, device="cuda") < ends, ids, -1).reshape(-1)
    made = {"w": [_weights(V, K, gen)], "ids": ids}
    if case["op"] == "backward":
        made["dy"] = torch.randn(B * S, K, generator=gen, device="cuda").to(dtype)
    return made


def _quantize(w, gs, qmax):
    """The codes [N, G, gs] and FP16 scales [N, G] of FP16 weights."""
    g = w.float().view(w.shape[0], -1, gs)
    s = (g.abs().amax(-1) / qmax).half()
    q = torch.round(g / s.float()[..., None]).clamp_(-qmax, qmax)
    return torch.where(s[..., None] > 0, q, 0.0).to(torch.int8), s


def prepare(case, seed):
    """The case with its inputs and its weights as the program keeps them."""
    state = dict(case)
    state.update(_inputs(case, seed))
    bits = case.get("bits", 4)
    w = state.pop("w")
    if own:
        from bit_group_quantized_flexq_b200 import flexq
        pack = flexq.quantize_weight4 if bits == 4 else flexq.quantize_weight
        state["packed"] = [pack(m, case["gs"]) + (m.shape[0],) for m in w]
    else:
        state["packed"] = [_quantize(m, case["gs"], QMAX[bits]) for m in w]
    return state


# --------------------------------------------------------------- one pass ----
def _dequantized(q, s):
    return (q.float() * s.float()[..., None]).flatten(1)


def _plain(st):
    dtype = DTYPES[st["dtype"]]
    if st["op"] == "linear":
        x = st["x"].float()
        return [(x @ _dequantized(q, s).t()).to(dtype) for q, s in st["packed"]]
    q, s = st["packed"][0]
    here = (st["ids"] >= 0) & (st["ids"] < st["V"])
    row = torch.where(here, st["ids"], 0)
    if st["op"] == "embedding":
        y = _dequantized(q[row], s[row]) * st["scale"]
        return torch.where(here[:, None], y, 0.0).to(dtype)
    d = torch.zeros(st["V"], st["K"], device="cuda")
    d.index_add_(0, row, torch.where(here[:, None], st["dy"].float(), 0.0) * st["scale"])
    out = {"scales": (d.view_as(q) * q.float()).sum(-1)}
    if st["table"] != "none":
        out["table"] = d.to(DTYPES[st["table"]])
    return out


def _own(st):
    from bit_group_quantized_flexq_b200 import flexq
    if st["op"] == "linear":
        if len(st["packed"]) > 1:
            return flexq.linear4_group(st["x"], st["packed"], st["gs"])
        wp, ws, N = st["packed"][0]
        return [flexq.linear4(st["x"], wp, ws, N, st["gs"])]
    wp, ws, V = st["packed"][0]
    if st["op"] == "embedding":
        return flexq.embedding(st["ids"], wp, ws, V, st["gs"], scale=st["scale"],
                               weight_bits=st["bits"], dtype=DTYPES[st["dtype"]])
    table, scales = flexq.embedding_backward(
        st["dy"], st["ids"], wp, V, st["gs"], scale=st["scale"], weight_bits=st["bits"],
        table_dtype=None if st["table"] == "none" else DTYPES[st["table"]])
    # 6-bit tables keep their scales, and so the scales' gradient, group-major
    out = {"scales": scales if st["bits"] == 4 else scales.t()}
    if table is not None:
        out["table"] = table
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits ----
def _rows64(w, gs, qmax):
    """Codes and dequantized rows of FP16 weights by the definition."""
    blocks = w.double().unflatten(1, (-1, gs))
    scale = (blocks.abs().max(dim=2, keepdim=True).values / qmax).half().double()
    ratio = torch.where(scale > 0, blocks / scale.clamp(min=1e-30), 0.0)
    codes = torch.round(ratio).clamp(-qmax, qmax)
    return codes, codes * scale


def exact(case, seed):
    made = _inputs(case, seed)
    gs, qmax = case["gs"], QMAX[case.get("bits", 4)]
    if case["op"] == "linear":
        x = made["x"].double()
        outs = []
        for w in made["w"]:
            parts = [torch.einsum("mk,nk->mn", x, _rows64(part, gs, qmax)[1].flatten(1))
                     for part in w.split(4096)]
            outs.append(torch.cat(parts, dim=1))
        return outs
    w, ids = made["w"][0], made["ids"]
    inside = ids.ge(0).logical_and(ids.lt(case["V"])).nonzero()[:, 0]
    if case["op"] == "embedding":
        y = torch.zeros(ids.numel(), case["K"], dtype=torch.float64, device="cuda")
        for part in inside.split(4096):
            y[part] = _rows64(w[ids[part]], gs, qmax)[1].flatten(1) * case["scale"]
        return y
    # the tokens of each row one after the other in their sorted order
    order = inside[torch.sort(ids[inside], stable=True).indices]
    found, counts = torch.unique_consecutive(ids[order], return_counts=True)
    total = torch.zeros(counts.numel(), case["K"], dtype=torch.float64, device="cuda")
    owner = torch.repeat_interleave(torch.arange(counts.numel(), device="cuda"), counts)
    for o, t in zip(owner.split(4096), order.split(4096)):
        total.index_add_(0, o, made["dy"][t].double() * case["scale"])
    scales = torch.zeros(case["V"], case["K"] // gs, dtype=torch.float64, device="cuda")
    for i in torch.arange(counts.numel(), device="cuda").split(4096):
        codes = _rows64(w[found[i]], gs, qmax)[0]
        scales[found[i]] = (codes * total[i].unflatten(1, (-1, gs))).sum(2)
    out = {"scales": scales}
    if case["table"] != "none":
        out["table"] = torch.zeros(case["V"], case["K"], dtype=torch.float64, device="cuda")
        out["table"][found] = total
    return out
