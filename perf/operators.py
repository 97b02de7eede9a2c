"""Measured cases of the block-scaled 8-bit operators: the norm before a layer with its residual's
addition, the quantisation of activation rows, the matrix product of quantised operands, and the
routed experts with 8-bit weights behind the slot table.

8-bit values are e4m3 (4 exponent bits, 3 mantissa bits, largest finite value 448, no infinities).
Activations carry one binary32 scale per row and 128 consecutive columns, weights one per 128 x 128
block; the last group or block of a row or matrix may be shorter.  A group's scale s is its largest
magnitude over 448 in binary32, never below 2^-126, and its values are v (1 / s), the reciprocal and
the product each rounded to binary32, then to the nearest e4m3.  Those two roundings are part of the
definition: v / s of two bf16 values often lies at a border between two e4m3 values to within them.

With `own` false, run() computes each operator from elementary torch operations in 32 bits; with
`own` true it calls the framework.
"""
import math

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
        # a decode step of one token enters a layer: residual added, the norm for the router and, in
        # 8 bits, for the experts; the call is one launch's latency
        {"name": "norm 1 token", "op": "norm", "T": 1, "d": 4096, "act": "bf16", "residual": True, "emit": "both"},
        # a prefill chunk enters a layer, same outputs: bound by memory
        {"name": "norm 8192 tokens", "op": "norm", "T": 8192, "d": 4096, "act": "bf16", "residual": True, "emit": "both"},
        # binary32 rows of a width that is no multiple of 128, a few dozen of them
        {"name": "quantise 48 odd rows", "op": "quant", "T": 48, "d": 2000, "act": "f32"},
        # activations of a prefill chunk that no norm precedes
        {"name": "quantise 8192 rows", "op": "quant", "T": 8192, "d": 2048, "act": "bf16"},
        # a projection of one decoded token: bound by reading the weights once
        {"name": "product 1 row", "op": "gemm", "M": 1, "N": 4096, "K": 2048, "out": "bf16"},
        # a projection of a decode batch, result in binary32
        {"name": "product 37 rows", "op": "gemm", "M": 37, "N": 2048, "K": 4096, "out": "f32"},
        # nothing a multiple of a tile: a short chunk, odd output width, last block of 80 columns
        {"name": "product 1000 odd rows", "op": "gemm", "M": 1000, "N": 1001, "K": 2000, "out": "bf16"},
        # a projection of a prefill chunk: bound by the matrix cores
        {"name": "product 8192 rows", "op": "gemm", "M": 8192, "N": 4096, "K": 4096, "out": "bf16"},
        # decode of one token through 6 of 256 experts and the shared expert, rows still in bf16
        {"name": "experts 1 token", "op": "experts", "T": 1, "E": 256, "k": 6, "d": 4096, "f": 2048, "shared": True,
         "x": "bf16"},
        # a decode batch of 64 tokens, 8 of 128 experts, nearly every expert touched by a few tokens
        {"name": "experts 64 tokens", "op": "experts", "T": 64, "E": 128, "k": 8, "d": 2048, "f": 768, "shared": False,
         "x": "fp8"},
        # a short prefill with ragged groups
        {"name": "experts 517 tokens", "op": "experts", "T": 517, "E": 128, "k": 8, "d": 2048, "f": 768,
         "shared": False, "x": "fp8"},
        # a prefill chunk of the larger layer
        {"name": "experts 8192 tokens", "op": "experts", "T": 8192, "E": 256, "k": 6, "d": 4096, "f": 2048,
         "shared": True, "x": "fp8"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quant", "gemm", "experts"])
    if op in ("norm", "quant"):
        c = {"op": op, "T": _log(rng, 1, 8192), "d": _log(rng, 64, 8192), "act": rng.choice(["bf16", "bf16", "f32"])}
        if rng.random() < 0.6:  # widths of models are multiples of 128
            c["d"] = max(128, c["d"] // 128 * 128)
        if op == "norm":
            c["residual"] = rng.random() < 0.75
            c["emit"] = rng.choice(["y", "fp8", "both"])
        return c
    if op == "gemm":
        c = {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 4096), "K": _log(rng, 256, 4096) // 16 * 16,
             "out": rng.choice(["bf16", "bf16", "f32"])}
        if rng.random() < 0.6:
            c["N"], c["K"] = max(128, c["N"] // 128 * 128), max(128, c["K"] // 128 * 128)
        return c
    E = _log(rng, 4, 256)
    return {"op": op, "T": _log(rng, 1, 4096), "E": E, "k": rng.randint(1, min(8, E)),
            "d": 128 * _log(rng, 2, 32), "f": 128 * _log(rng, 1, 16), "shared": rng.random() < 0.5,
            "x": rng.choice(["fp8", "fp8", "bf16"])}


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


def _weights(g, n, rows, cols):
    """n quantised matrices as a checkpoint holds them: bell-shaped e4m3 values that reach the type's
    top in a block, scales around those of weights with a deviation of 0.02."""
    q = torch.empty(n, rows, cols, dtype=E4M3, device="cuda")
    for i in range(0, n, 16):
        part = torch.randn(min(16, n - i), rows, cols, generator=g, device="cuda", dtype=torch.bfloat16)
        q[i:i + 16] = (part * 105).clamp_(-TOP, TOP).to(E4M3)
    s = 0.02 / 105 * torch.exp(0.2 * _rand(g, n, -(-rows // 128), -(-cols // 128)))
    return q, s


def _blocks(q, s):
    """Matrices [n, R, K] and their scales as the 16-row blocks of a slot image [n, R/16, bytes]: K/128
    fragments of two halves (64 inputs each) x 64 lanes x 16 bytes, lane l holding row l % 16, inputs
    16 (l / 16) .. + 15 of the half; then the block's K/128 scales, padded to 64 bytes."""
    n, R, K = q.shape
    frag = q.view(torch.uint8).view(n, R // 16, 16, K // 128, 2, 4, 16).permute(0, 1, 3, 4, 5, 2, 6)
    frag = frag.reshape(n, R // 16, 16 * K)
    tail = torch.zeros(n, R // 16, -(-(K // 128) // 16) * 16, dtype=torch.float32, device="cuda")
    tail[:, :, :K // 128] = s.repeat_interleave(8, 1)
    return torch.cat([frag, tail.view(torch.uint8)], 2)


def _images(wg, sg, wu, su, wd, sd):
    """Slot images [n, bytes]: gate and up blocks in turn, then the down blocks, padded to 256 bytes."""
    n = wg.shape[0]
    gu = torch.stack([_blocks(wg, sg), _blocks(wu, su)], 2).flatten(1)
    dn = _blocks(wd, sd).flatten(1)
    out = torch.zeros(n, -(-(gu.shape[1] + dn.shape[1]) // 256) * 256, dtype=torch.uint8, device="cuda")
    out[:, :gu.shape[1]] = gu
    out[:, gu.shape[1]:gu.shape[1] + dn.shape[1]] = dn
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("norm", "quant"):
        T, d, act = case["T"], case["d"], TYPES[case["act"]]
        s["x"] = _rows(g, T, d).to(act)
        q = (torch.empty(T, d, dtype=E4M3, device="cuda"), torch.empty(T, -(-d // 128), device="cuda"))
        if op == "quant":
            s["out"] = q
            return s
        s["residual"] = (3 * _rows(g, T, d)).to(act) if case["residual"] else None
        s["weight"] = (1 + 0.2 * _rand(g, d)).to(act)
        s["out"] = (torch.empty_like(s["x"]) if case["emit"] != "fp8" else None,
                    torch.empty_like(s["x"]) if case["residual"] else None) + (q if case["emit"] != "y" else (None, None))
    elif op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"], s["a_scale"] = _quantise(_rows(g, M, K))
        w, ws = _weights(g, 1, N, K)
        s["w"], s["w_scale"] = w[0], ws[0]
        s["out"] = torch.empty(M, N, dtype=TYPES[case["out"]], device="cuda")
    else:
        T, E, k, d, f = (case[n] for n in ("T", "E", "k", "d", "f"))
        n = E + int(case["shared"])
        s["wg"], s["sg"] = _weights(g, n, f, d)
        s["wu"], s["su"] = _weights(g, n, f, d)
        s["wd"], s["sd"] = _weights(g, n, d, f)
        # expert e lives in slot order[e]; the shared expert's image stands by itself
        order = torch.randperm(E, generator=g, device="cuda")
        names = ("wg", "sg", "wu", "su", "wd", "sd")
        s["stride"] = _images(*[s[m][:1] for m in names]).shape[1]
        s["pool"] = torch.empty(E, s["stride"], dtype=torch.uint8, device="cuda")
        for i in range(0, E, 16):
            s["pool"][order[i:i + 16]] = _images(*[s[m][i:min(i + 16, E)] for m in names])
        s["shared"] = _images(*[s[m][E:] for m in names])[0] if case["shared"] else None
        s["slots"] = order.to(torch.int32)
        # a router's choice with popularity falling as 1 / rank^1.1, distinct experts for a token
        popular = -1.1 * torch.log(1.0 + torch.randperm(E, generator=g, device="cuda"))
        u = torch.rand(T, E, generator=g, device="cuda").clamp_min_(1e-9)
        ids = (popular - torch.log(-torch.log(u).clamp_min_(1e-30))).topk(k, dim=1).indices.flatten()
        s["counts"] = torch.bincount(ids, minlength=E).to(torch.int32)
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        s["offsets"][1:] = s["counts"].cumsum(0)
        s["perm"] = ids.argsort(stable=True).to(torch.int32)
        s["bounds"] = s["offsets"].tolist()
        x = _rows(g, T, d)
        if case["x"] == "bf16":
            s["x"], s["x_scale"] = x.to(torch.bfloat16), None
        else:
            s["x"], s["x_scale"] = _quantise(x)
        s["out"] = torch.empty(T * k + (T if case["shared"] else 0), d, dtype=torch.bfloat16, device="cuda")
        # the call's zero-filled workspace: a header, the rows of h in binary32 at most, the rows of x in 8 bits
        rows = s["out"].shape[0]
        s["ws"] = torch.zeros((1 << 17) + 4096 + rows * f * 4 + T * d * 2, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------------
def _quantise(v):
    """binary32 rows -> e4m3 rows and their scales."""
    T, d = v.shape
    p = torch.nn.functional.pad(v, (0, -d % 128)).view(T, -1, 128)
    s = (p.abs().amax(2).double() / TOP).float().clamp_min(LEAST)  # a quotient rounded once
    return (p * s.double().reciprocal().float()[:, :, None]).view(T, -1)[:, :d].to(E4M3).contiguous(), s


def _rows32(q, s):
    return q.float() * s.repeat_interleave(128, 1)[:, :q.shape[1]]


def _matrix32(q, s):
    return q.float() * s.repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]


def _norm(s):
    case, x = s["case"], s["x"].float()
    h = None
    if case["residual"]:
        h = (x + s["residual"].float()).to(s["x"].dtype)
        x = h.float()
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * s["weight"].float()
    q, scale = _quantise(y) if case["emit"] != "y" else (None, None)
    return {"y": y.to(s["x"].dtype) if case["emit"] != "fp8" else None, "residual": h, "q": q, "scale": scale}


def _product(s):
    return (_rows32(s["a"], s["a_scale"]) @ _matrix32(s["w"], s["w_scale"]).T).to(s["out"].dtype)


def _experts(s):
    case = s["case"]
    x = _rows32(*_quantise(s["x"].float()) if case["x"] == "bf16" else (s["x"], s["x_scale"]))
    token = s["perm"].long() // case["k"]
    y = torch.empty_like(s["out"])

    def expert(e, rows):
        g = rows @ _matrix32(s["wg"][e], s["sg"][e]).T
        u = rows @ _matrix32(s["wu"][e], s["su"][e]).T
        h = _rows32(*_quantise(g / (1 + torch.exp(-g)) * u))
        return (h @ _matrix32(s["wd"][e], s["sd"][e]).T).to(y.dtype)

    for e in range(case["E"]):  # each expert that has tokens runs once on them
        lo, hi = s["bounds"][e], s["bounds"][e + 1]
        if hi > lo:
            y[lo:hi] = expert(e, x[token[lo:hi]])
    if case["shared"]:
        y[case["T"] * case["k"]:] = expert(case["E"], x)
    return y


def run(state):
    s, case = state, state["case"]
    if not own:
        if case["op"] == "norm":
            return _norm(s)
        if case["op"] == "quant":
            q, scale = _quantise(s["x"].float())
            return {"q": q, "scale": scale}
        return _product(s) if case["op"] == "gemm" else _experts(s)
    import expert_offload_cache_amd as moe

    if case["op"] == "norm":
        y, h, q, scale = moe.add_rmsnorm(s["x"], s["weight"], 1e-6, residual=s["residual"], emit=case["emit"],
                                         out=s["out"])
        return {"y": y, "residual": h, "q": q, "scale": scale}
    if case["op"] == "quant":
        q, scale = moe.quant_fp8(s["x"], out=s["out"])
        return {"q": q, "scale": scale}
    if case["op"] == "gemm":
        return moe.gemm_fp8(s["a"], s["a_scale"], s["w"], s["w_scale"], out=s["out"])
    if case["x"] == "bf16":
        return moe.expert_ffn_grouped(s["x"], s["perm"], s["offsets"], s["counts"], s["slots"], s["pool"], case["E"],
                                      s["stride"], "fp8", case["f"], case["k"], shared_w=s["shared"], y_perm=s["out"],
                                      ws=s["ws"])[0]
    return moe.expert_ffn_fp8(s["x"], s["x_scale"], s["perm"], s["offsets"], s["counts"], s["slots"], s["pool"],
                              case["E"], s["stride"], case["f"], case["k"], shared_w=s["shared"], y_perm=s["out"],
                              ws=s["ws"])[0]


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    if case["op"] in ("norm", "quant"):
        T, d, size = case["T"], case["d"], 2 if case["act"] == "bf16" else 4
        quantised = T * (d + 4 * -(-d // 128))
        if case["op"] == "quant":
            return {"bytes": T * d * size + quantised, "flops": 3 * T * d}
        n = T * d * size
        return {"bytes": n + d * size + (2 * n if case["residual"] else 0) + (n if case["emit"] != "fp8" else 0)
                + (quantised if case["emit"] != "y" else 0),
                "flops": T * d * (4 + int(case["residual"]) + (3 if case["emit"] != "y" else 0))}
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        G = -(-K // 128)
        return {"bytes": M * K + 4 * M * G + N * K + 4 * -(-N // 128) * G + M * N * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * M * N * K}
    T, E, k, d, f = (case[n] for n in ("T", "E", "k", "d", "f"))
    rows = T * k + (T if case["shared"] else 0)
    # experts that some token is expected to choose under the routing of prepare(): each token picks k of
    # them by popularity without replacement, taken here as k independent picks
    p = [(1.0 + r) ** -1.1 for r in range(E)]
    total = sum(p)
    touched = min(float(E), max(float(min(k, E)), sum(1 - (1 - v / total) ** (T * k) for v in p)))
    touched += int(case["shared"])
    x = T * d * 2 if case["x"] == "bf16" else T * (d + d // 32)
    return {"bytes": int(touched * 3 * d * f + x + rows * d * 2 + 8 * T * k), "flops": 6 * rows * d * f}


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
    parts = [v[:, c:c + 128] for c in range(0, v.shape[1], 128)]
    scale = [torch.clamp_min((p.abs().max(1).values / TOP).float().double(), LEAST) for p in parts]
    q = [_nearest_e4m3((p * s.reciprocal().float().unsqueeze(1)).float().double()) for p, s in zip(parts, scale)]
    return torch.cat(q, 1), torch.stack(scale, 1)


def _scaled64(q, scale, by_rows):
    rows = torch.arange(q.shape[0], device=q.device)
    cols = torch.arange(q.shape[1], device=q.device) // 128
    return q.double() * scale.double()[(rows if by_rows else rows // 128)[:, None], cols[None, :]]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        q, scale = _quantise64(s["x"].double())
        return {"q": q, "scale": scale}
    if case["op"] == "norm":
        x, h = s["x"].double(), None
        if case["residual"]:
            x = (x + s["residual"].double()).to(s["x"].dtype).double()  # the sum is kept in the rows' type
            h = x
        y = x / torch.sqrt((x * x).sum(1, keepdim=True) / x.shape[1] + 1e-6) * s["weight"].double()
        q, scale = _quantise64(y) if case["emit"] != "y" else (None, None)
        return {"y": y if case["emit"] != "fp8" else None, "residual": h, "q": q, "scale": scale}
    if case["op"] == "gemm":
        return _scaled64(s["a"], s["a_scale"], True) @ _scaled64(s["w"], s["w_scale"], False).t()
    T, k, E = case["T"], case["k"], case["E"]
    q, scale = _quantise64(s["x"].double()) if case["x"] == "bf16" else (s["x"], s["x_scale"])
    x = _scaled64(q, scale, True)
    groups = [(e, (s["perm"][s["bounds"][e]:s["bounds"][e + 1]].long()).div(k, rounding_mode="floor"))
              for e in range(E) if s["bounds"][e + 1] > s["bounds"][e]]
    if case["shared"]:
        groups.append((E, torch.arange(T, device="cuda")))
    out = []
    for e, tokens in groups:
        up = x[tokens] @ _scaled64(s["wu"][e], s["su"][e], False).t()
        gate = x[tokens] @ _scaled64(s["wg"][e], s["sg"][e], False).t()
        h = _scaled64(*_quantise64(up * gate * torch.sigmoid(gate)), True)
        out.append(h @ _scaled64(s["wd"][e], s["sd"][e], False).t())
    return torch.cat(out, 0)
