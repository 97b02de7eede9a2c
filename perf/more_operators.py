"""Measured cases of the operators a serving step takes for a few tokens of many requests: a whole
mixture-of-experts layer in one call, and a projection with a low-rank adapter for each row.

The layer: logits = x w_router^T + bias; the k largest, ties to the lower expert; gates = softmax over
the chosen; y = sum of gate * expert(x) over the chosen (+ the shared expert), expert(x) =
(silu(x Wg^T) * (x Wu^T)) Wd^T.  Between the two products h is held in the activations' type, which is
part of the definition; with 8-bit weights the rows of x and of h are quantised instead (e4m3, one
scale s = max(|v|) / 448 per row and 128 columns, values e4m3(v * (1 / s)), m / 448, 1 / s and the
product each rounded to binary32).  Weights: binary32, bf16, 4-bit integers with a bf16 scale per 128
inputs of a row, or e4m3 with a binary32 scale per 128 x 128 block.

The projection: y = x W^T (or rows that another product left) + scale_a * (x A_a^T) B_a^T, where a is
the adapter of the row's request, or none; adapters have ranks of their own up to a common one.

With `own` false, run() computes each operator from elementary torch operations in 32 bits (the
router's logits and gates in 64: the choice lies at a border); with `own` true it calls the framework.
"""
import math
import random

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TOP = 448.0
LEAST = 2.0 ** -126


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one decoded token of the smaller layer: the weights of 8 experts read once
        {"name": "layer 1 token", "op": "layer", "w": "bf16", "T": 1, "d": 2048, "f": 768, "E": 128, "k": 8,
         "shared": False},
        # a small decode batch of it: experts chosen by one to many of the tokens
        {"name": "layer 16 tokens", "op": "layer", "w": "bf16", "T": 16, "d": 2048, "f": 768, "E": 128, "k": 8,
         "shared": False},
        # one decoded token of the larger layer, 4-bit weights, with its shared expert
        {"name": "layer 1 token, 4 bits", "op": "layer", "w": "int4", "T": 1, "d": 4096, "f": 2048, "E": 256, "k": 6,
         "shared": True},
        # a small decode batch of it
        {"name": "layer 16 tokens, 4 bits", "op": "layer", "w": "int4", "T": 16, "d": 4096, "f": 2048, "E": 256, "k": 6,
         "shared": True},
        # the smallest layer, binary32: the latency of the call
        {"name": "layer 16 tokens, 32 bits", "op": "layer", "w": "f32", "T": 16, "d": 64, "f": 128, "E": 8, "k": 2,
         "shared": False},
        # 8-bit weights, sizes that are no powers of two, a few speculative tokens
        {"name": "layer 5 tokens, 8 bits", "op": "layer", "w": "fp8", "T": 5, "d": 1152, "f": 640, "E": 60, "k": 4,
         "shared": True},
        # a projection of one decoded token with its request's adapter
        {"name": "projection 1 row", "op": "lora", "M": 1, "N": 4096, "K": 2048, "r": 16, "n": 8, "w": True,
         "base": "none", "out": "bf16", "ranks": False, "runs": False},
        # a decode batch, every request with one of 16 adapters or none, result in binary32
        {"name": "projection 37 rows", "op": "lora", "M": 37, "N": 2048, "K": 4096, "r": 64, "n": 16, "w": True,
         "base": "none", "out": "f32", "ranks": True, "runs": False},
        # the adapters alone, added to the binary32 rows that an 8-bit projection left; 64 loaded adapters
        {"name": "adapters 64 rows", "op": "lora", "M": 64, "N": 2048, "K": 2048, "r": 32, "n": 64, "w": False,
         "base": "f32", "out": "bf16", "ranks": False, "runs": False},
        # nothing a multiple of a tile: a few prompts in one chunk, odd output width, ranks of their own
        {"name": "projection 1000 odd rows", "op": "lora", "M": 1000, "N": 1001, "K": 2000, "r": 24, "n": 5, "w": True,
         "base": "none", "out": "bf16", "ranks": True, "runs": True},
        # a prefill chunk of several requests: bound by the matrix cores
        {"name": "projection 8192 rows", "op": "lora", "M": 8192, "N": 4096, "K": 4096, "r": 32, "n": 12, "w": True,
         "base": "none", "out": "bf16", "ranks": False, "runs": True},
        # the adapters of a prefill chunk added to another product's rows: bound by memory
        {"name": "adapters 8192 rows", "op": "lora", "M": 8192, "N": 4096, "K": 4096, "r": 64, "n": 12, "w": False,
         "base": "bf16", "out": "bf16", "ranks": False, "runs": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        w = rng.choice(["bf16", "bf16", "int4", "int4", "fp8", "f32"])
        E = _log(rng, 4, 256)
        c = {"op": "layer", "w": w, "T": rng.choice([1, 2, 3, _log(rng, 1, 16), rng.randint(1, 16)]), "E": E,
             "k": rng.randint(1, min(8, E)), "shared": rng.random() < 0.5}
        if w == "f32":
            c["d"], c["f"] = 64 * _log(rng, 1, 16), 32 * _log(rng, 2, 32)
        elif w == "bf16":
            c["d"], c["f"] = 64 * _log(rng, 2, 64), 32 * _log(rng, 2, 40)
        else:
            c["d"], c["f"] = 128 * _log(rng, 1, 32), 128 * _log(rng, 1, 16)
        most = max(work(l)["bytes"] for l in listed() if l["op"] == "layer")
        while work(c)["bytes"] > most:  # a drawn layer reads no more than the largest listed one
            c["f"] = max(128, c["f"] // 2 // 128 * 128)
            c["E"] = max(c["k"], c["E"] * 3 // 4)
        return c
    c = {"op": "lora", "M": _log(rng, 1, 8192), "N": _log(rng, 64, 4096), "K": 8 * _log(rng, 16, 512),
         "r": 8 * _log(rng, 1, 16), "n": _log(rng, 1, 64), "w": rng.random() < 0.7,
         "base": rng.choice(["none", "bf16", "f32"]), "out": rng.choice(["bf16", "bf16", "f32"]),
         "ranks": rng.random() < 0.5}
    if rng.random() < 0.6:  # widths of models are multiples of 128
        c["N"], c["K"] = max(128, c["N"] // 128 * 128), max(128, c["K"] // 128 * 128)
    c["runs"] = c["M"] > 128 or rng.random() < 0.3  # longer calls hold whole prompts one after the other
    if not c["w"] and c["base"] == "none":
        c["base"] = "bf16"
    most = max(work(l)["flops"] for l in listed())
    while work(c)["flops"] > most:
        c["M"] = c["M"] * 7 // 8
    return c


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rows(g, T, d):
    """Activation rows: unit variance, a few columns some ten times larger, as hidden states have."""
    column = torch.ones(d, device="cuda")
    column[torch.randint(0, d, (max(1, d // 200),), generator=g, device="cuda")] = 12.0
    return _rand(g, T, d) * column


def _matrices(g, w, n, R, K):
    """n weight matrices [R, K] as a checkpoint holds them -> (values, scales or None): binary32, bf16,
    nibbles 1 .. 15 (the integer plus 8) with a bf16 scale per 128 inputs, or e4m3 with block scales."""
    if w == "f32":
        return 0.02 * _rand(g, n, R, K), None
    v = torch.empty(n, R, K, dtype={"bf16": torch.bfloat16, "int4": torch.uint8, "fp8": E4M3}[w], device="cuda")
    for i in range(0, n, 16):
        part = torch.randn(min(16, n - i), R, K, generator=g, device="cuda", dtype=torch.bfloat16)
        if w == "bf16":
            v[i:i + 16] = part * 0.02
        elif w == "int4":
            v[i:i + 16] = (part * 2.4).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
        else:
            v[i:i + 16] = (part * 105).clamp_(-TOP, TOP).to(E4M3)
    if w == "bf16":
        return v, None
    if w == "int4":
        return v, (0.02 / 2.4 * torch.exp(0.2 * _rand(g, n, R, K // 128))).to(torch.bfloat16)
    return v, 0.02 / 105 * torch.exp(0.2 * _rand(g, n, -(-R // 128), -(-K // 128)))


def _blocks(w, v, s):
    """Matrices [n, R, K] as the 16-row blocks of a slot image, [n, R/16, bytes]: fragments of 16 rows x 32
    (or 128) inputs in the order of a wave's lanes, then the block's scales."""
    n, R, K = v.shape
    if w in ("bf16", "f32"):  # lane l: row l % 16, inputs 8 (l / 16) .. + 7 of the fragment
        frag = v.view(n, R // 16, 16, K // 32, 4, 8).permute(0, 1, 3, 4, 2, 5).contiguous()
        return frag.view(torch.uint8).view(n, R // 16, -1)
    if w == "int4":  # lane l: row l % 16, word s: inputs 32 s + 8 (l / 16) + 0 .. 7, even ones in the low half
        f = v.view(n, R // 16, 16, K // 128, 4, 4, 4, 2).permute(0, 1, 3, 5, 2, 4, 6, 7)
        word = torch.zeros(f.shape[:-2], dtype=torch.int32, device="cuda")
        for p in range(4):
            word |= f[..., p, 0].int() << (4 * p) | f[..., p, 1].int() << (16 + 4 * p)
        frag = word.view(torch.uint8).view(n, R // 16, -1)
        return torch.cat([frag, s.contiguous().view(torch.uint8).view(n, R // 16, -1)], 2)
    # e4m3: halves of 64 inputs, lane l: row l % 16, inputs 16 (l / 16) .. + 15 of the half
    frag = v.view(torch.uint8).view(n, R // 16, 16, K // 128, 2, 4, 16).permute(0, 1, 3, 4, 5, 2, 6)
    tail = torch.zeros(n, R // 16, -(-(K // 128) // 16) * 16, dtype=torch.float32, device="cuda")
    tail[:, :, :K // 128] = s.repeat_interleave(8, 1)
    return torch.cat([frag.reshape(n, R // 16, 16 * K), tail.view(torch.uint8)], 2)


def _images(w, m, i, j):
    """Slot images [j - i, bytes] of experts i .. j-1: gate and up blocks in turn, then the down blocks,
    padded to 256 bytes."""
    b = [_blocks(w, v[i:j], None if s is None else s[i:j]) for v, s in m]
    gu, dn = torch.stack(b[:2], 2).flatten(1), b[2].flatten(1)
    return torch.nn.functional.pad(torch.cat([gu, dn], 1), (0, -(gu.shape[1] + dn.shape[1]) % 256))


def _prepare_layer(s, g, case):
    T, E, k, d, f, w = (case[n] for n in ("T", "E", "k", "d", "f", "w"))
    act = TYPES["f32" if w == "f32" else "bf16"]
    n = E + int(case["shared"])
    m = s["m"] = [_matrices(g, w, n, f, d), _matrices(g, w, n, f, d), _matrices(g, w, n, d, f)]
    # expert e lives in slot order[e]; the shared expert's image stands by itself
    order = torch.randperm(E, generator=g, device="cuda")
    s["stride"] = _images(w, m, 0, 1).shape[1]
    s["pool"] = torch.empty(E, s["stride"], dtype=torch.uint8, device="cuda")
    for i in range(0, E, 8):
        s["pool"][order[i:i + 8]] = _images(w, m, i, min(i + 8, E))
    s["shared"] = _images(w, m, E, E + 1)[0] if case["shared"] else None
    s["slots"] = order.to(torch.int32)
    s["router"] = (0.02 * _rand(g, E, d)).to(act)
    # popularity falls as 1 / rank^1.1
    s["bias"] = -1.1 * torch.log(1.0 + torch.randperm(E, generator=g, device="cuda"))
    # a token two of whose best logits lie within binary32's rounding of each other has no one answer:
    # of more tokens than needed, those are left out
    x = _rows(g, 4 * T + 16, d).to(act)
    best = (x.double() @ s["router"].double().T + s["bias"].double()).topk(min(k + 1, E), dim=1).values
    gap = (best[:, :-1] - best[:, 1:]).amin(1) if best.shape[1] > 1 else torch.ones(x.shape[0], device="cuda")
    s["x"] = x[(gap < 1e-4).to(torch.int32).argsort(stable=True)[:T]].contiguous()
    s["out"] = (torch.empty(T, d, dtype=act, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda"),
                torch.empty(T, k, device="cuda"))
    # the call's zero-filled workspace: logits and a header, rows of h, of x in 8 bits, partial rows of y
    s["ws"] = torch.zeros((1 << 18) + T * (k + 1) * f * 4 + T * d * 72 + 4 * T * E, dtype=torch.uint8, device="cuda")


def _prepare_lora(s, g, case):
    M, N, K, r, n = (case[c] for c in ("M", "N", "K", "r", "n"))
    s["x"] = _rows(g, M, K).to(torch.bfloat16)
    s["w"] = (0.02 * _rand(g, N, K)).to(torch.bfloat16) if case["w"] else None
    s["base"] = _rand(g, M, N).to(TYPES[case["base"]]) if case["base"] != "none" else None
    s["a"] = (_rand(g, n, r, K) / math.sqrt(K)).to(torch.bfloat16)
    s["b"] = (0.03 * _rand(g, n, N, r)).to(torch.bfloat16)
    s["scale"] = 2.0 / torch.randint(1, 5, (n,), generator=g, device="cuda").float()
    s["rank"] = torch.randint(max(1, r // 4), r + 1, (n,), generator=g, device="cuda").to(torch.int32) if case["ranks"] else None
    # one request in eight has no adapter; in longer calls a request holds a run of rows
    if case["runs"]:
        cuts = torch.randint(0, M + 1, (n,), generator=g, device="cuda")
        who = (torch.arange(M, device="cuda")[:, None] >= cuts[None, :]).sum(1)
        name = torch.randint(0, n, (n + 1,), generator=g, device="cuda")
        name[torch.rand(n + 1, generator=g, device="cuda") < 0.125] = -1
        s["adapter"] = name[who].to(torch.int32)
    else:
        name = torch.randint(0, n, (M,), generator=g, device="cuda")
        name[torch.rand(M, generator=g, device="cuda") < 0.125] = -1
        s["adapter"] = name.to(torch.int32)
    s["out"] = torch.empty(M, N, dtype=TYPES[case["out"]], device="cuda")
    s["ws"] = torch.zeros((1 << 20) + 8 * M * r * 4, dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    (_prepare_layer if case["op"] == "layer" else _prepare_lora)(s, g, case)
    return s


# ---------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------
def _quantise(v):
    """binary32 rows -> the values their e4m3 rows and scales stand for."""
    T, d = v.shape
    p = v.view(T, -1, 128)
    s = (p.abs().amax(2, keepdim=True).double() / TOP).float().clamp_min(LEAST)  # a quotient rounded once
    return ((p * s.double().reciprocal().float()).to(E4M3).float() * s).view(T, d)


def _matrix32(w, m, e):
    v, s = m[0][e], None if m[1] is None else m[1][e].float()
    if w == "int4":
        return (v.float() - 8) * s.repeat_interleave(128, 1)
    if w == "fp8":
        return v.float() * s.repeat_interleave(128, 0).repeat_interleave(128, 1)
    return v.float()


def _layer(s):
    case, x = s["case"], s["x"]
    w, k = case["w"], case["k"]
    # stable: equal logits keep the lower expert first
    logits = x.double() @ s["router"].double().T + s["bias"].double()
    top, idx = logits.sort(dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    gate = torch.exp(top - top[:, :1])
    gate = (gate / gate.sum(1, keepdim=True)).float()
    rows = _quantise(x.float()) if w == "fp8" else x.float()

    def expert(e, r):
        a = r @ _matrix32(w, s["m"][0], e).T
        h = a / (1 + torch.exp(-a)) * (r @ _matrix32(w, s["m"][1], e).T)
        h = _quantise(h) if w == "fp8" else h.to(x.dtype).float()
        return h @ _matrix32(w, s["m"][2], e).T

    y = torch.zeros(x.shape, device="cuda")
    for e in sorted(set(idx.flatten().tolist())):  # each chosen expert runs once on its tokens
        t, j = (idx == e).nonzero(as_tuple=True)
        y[t] += gate[t, j].unsqueeze(1) * expert(e, rows[t])
    if case["shared"]:
        y += expert(case["E"], rows)
    return {"y": y.to(x.dtype), "topk_idx": idx.to(torch.int32), "topk_w": gate}


def _lora(s):
    case, x = s["case"], s["x"].float()
    y = x @ s["w"].float().T if case["w"] else torch.zeros(s["out"].shape, device="cuda")
    if s["base"] is not None:
        y += s["base"].float()
    for a in range(case["n"]):
        t = (s["adapter"] == a).nonzero().flatten()
        r = case["r"] if s["rank"] is None else int(s["rank"][a])
        y[t] += s["scale"][a] * ((x[t] @ s["a"][a, :r].float().T) @ s["b"][a, :, :r].float().T)
    return {"y": y.to(s["out"].dtype)}


def run(state):
    s, case = state, state["case"]
    if not own:
        return _layer(s) if case["op"] == "layer" else _lora(s)
    import expert_offload_cache_amd as moe

    if case["op"] == "layer":
        y, idx, gate = moe.layer_few(s["x"], s["router"], s["bias"], case["k"], s["slots"], s["pool"], case["E"],
                                     s["stride"], case["w"], case["f"], shared_w=s["shared"], out=s["out"], ws=s["ws"])
        return {"y": y, "topk_idx": idx, "topk_w": gate}
    return {"y": moe.lora_linear(s["x"], s["a"], s["b"], s["scale"], s["adapter"], w=s["w"], base=s["base"],
                                 rank=s["rank"], out=s["out"], ws=s["ws"])}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def _touched(T, E, k, d):
    """Experts that some token chooses under the routing of prepare(), in the mean over a few trials."""
    rng = np.random.default_rng(1)
    sd = 0.02 * math.sqrt(d + 143 * max(1, d // 200))
    bias = -1.1 * np.log(1.0 + np.arange(E))
    seen = [np.unique(np.argpartition(-(sd * rng.standard_normal((T, E)) + bias), k - 1, axis=1)[:, :k]).size
            for _ in range(16)]
    return sum(seen) / len(seen)


def work(case):
    if case["op"] == "layer":
        T, E, k, d, f, w = (case[n] for n in ("T", "E", "k", "d", "f", "w"))
        size = {"f32": 4, "bf16": 2, "int4": 0.5 + 2 / 128, "fp8": 1 + 4 / 16384}[w]
        act = 4 if w == "f32" else 2
        experts = _touched(T, E, k, d) + int(case["shared"])
        return {"bytes": int(experts * 3 * d * f * size + E * d * act + 4 * E + 2 * T * d * act + 8 * T * k),
                "flops": 6 * T * (k + int(case["shared"])) * d * f + 2 * T * E * d}
    M, N, K, r, n = (case[c] for c in ("M", "N", "K", "r", "n"))
    rank = 0.625 * r if case["ranks"] else r
    draws = n + 1 if case["runs"] else M  # requests, each with one of n adapters or, one in eight, none
    touched = n * (1 - (1 - 0.875 / n) ** min(draws, M))
    size = {"none": 0, "bf16": 2, "f32": 4}
    return {"bytes": int(2 * M * K + (2 * N * K if case["w"] else 0) + 2 * touched * rank * (K + N) + 4 * M
                         + M * N * (size[case["base"]] + size[case["out"]])),
            "flops": int((2 * M * N * K if case["w"] else 0) + 0.875 * 2 * M * rank * (K + N))}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _nearest_e4m3(v):
    """binary64 values of magnitude up to 448 (a little over it rounds to it) -> nearest e4m3 value,
    ties to even: steps of 2^(e-3) in the binade [2^e, 2^(e+1)), of 2^-9 below 2^-6."""
    _, e = torch.frexp(v)
    step = torch.exp2((e.to(torch.float64) - 1).clamp_min(-6) - 3)
    return torch.round(v / step) * step


def _quantise64(v):
    out = []
    for c in range(0, v.shape[1], 128):
        p = v[:, c:c + 128]
        s = torch.clamp_min((p.abs().max(1, keepdim=True).values / TOP).float().double(), LEAST)
        out.append(_nearest_e4m3((p * s.reciprocal().float()).float().double()) * s)
    return torch.cat(out, 1)


def _matrix64(w, v, s, e):
    v = v[e].double()
    if s is None:
        return v
    rows, cols = torch.arange(v.shape[0], device="cuda"), torch.arange(v.shape[1], device="cuda") // 128
    if w == "int4":
        return (v - 8.0) * s[e].double()[rows[:, None], cols[None, :]]
    return v * s[e].double()[(rows // 128)[:, None], cols[None, :]]


def _exact_layer(s, case):
    T, E, k, w = (case[n] for n in ("T", "E", "k", "w"))
    x = s["x"].double()
    logits = x @ s["router"].double().t() + s["bias"].double()
    idx = torch.empty(T, k, dtype=torch.int64, device="cuda")
    left = logits.clone()
    for j in range(k):  # the first of the largest that are left
        best = left == left.max(1, keepdim=True).values
        idx[:, j] = best.to(torch.int8).argmax(1)
        left[torch.arange(T, device="cuda"), idx[:, j]] = -torch.inf
    gate = torch.softmax(logits.gather(1, idx), 1)
    if w == "fp8":
        x = _quantise64(x)
    y = torch.zeros(T, case["d"], dtype=torch.float64, device="cuda")
    share = torch.zeros(T, E + 1, dtype=torch.float64, device="cuda")
    share.scatter_(1, idx, gate)
    if case["shared"]:
        share[:, E] = 1.0
    for e in (share != 0).any(0).nonzero().flatten().tolist():
        mg, mu, md = (_matrix64(w, v, sc, e) for v, sc in s["m"])
        t = (share[:, e] != 0).nonzero().flatten()
        a = x[t] @ mg.t()
        h = a * torch.sigmoid(a) * (x[t] @ mu.t())
        h = _quantise64(h) if w == "fp8" else h.to(s["x"].dtype).double()
        y[t] += share[t, e, None] * (h @ md.t())
    return {"y": y, "topk_idx": idx.to(torch.int32), "topk_w": gate}


def _exact_lora(s, case):
    y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
    for i in range(0, case["M"], 1024):  # every row's own adapter, row by row of the definition
        x = s["x"][i:i + 1024].double()
        if case["w"]:
            y[i:i + 1024] = x @ s["w"].double().t()
        if s["base"] is not None:
            y[i:i + 1024] += s["base"][i:i + 1024].double()
        who = s["adapter"][i:i + 1024].long()
        for a in torch.unique(who[who >= 0]).tolist():
            keep = torch.arange(case["r"], device="cuda") < (case["r"] if s["rank"] is None else s["rank"][a])
            v = (x @ s["a"][a].double().t()) * keep * (who == a)[:, None]
            y[i:i + 1024] += s["scale"][a].double() * (v @ s["b"][a].double().t())
    return {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_layer if case["op"] == "layer" else _exact_lora)(s, case)


if __name__ == "__main__":
    rng = random.Random(0)
    for c in listed() + [draw(rng) for _ in range(12)]:
        n = work(c)
        print(f"{n['bytes'] / 1e6:10.2f} MB {n['flops'] / 1e9:10.3f} GFLOP  {c}")
