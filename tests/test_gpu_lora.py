"""moe_lora_linear against its definition in 64 bits: with and without a projection and a base, one row to thousands,
odd widths and ranks, adapters mixed in a tile or in runs, strides, infinities, captured and repeated calls.

The tolerance of an element is a bound, derived here and not fitted: a binary32 sum of n terms, added in any order,
is off by at most n 2^-24 of the sum of its terms' magnitudes; v = scale (A x) carries the bound of its own sum
through B; v enters the second product in bf16 parts that leave 2^-16 of it (BF16 results: two parts, each
rounding by half a step of 2^-8) or 2^-24 (F32); the result is rounded once, by half a step at most."""
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def make(M, N, K, r, n, w=True, base=None, out="bf16", ranks=False, runs=False, seed=0, none=0.125):
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    s = dict(x=rnd(M, K).bfloat16(), a=(rnd(n, r, K) / K ** 0.5).bfloat16(), b=(0.05 * rnd(n, N, r)).bfloat16(),
             scale=0.5 + torch.rand(n, generator=g, device="cuda"),
             w=(0.02 * rnd(N, K)).bfloat16() if w else None, base=rnd(M, N).to(dt[base]) if base else None,
             rank=torch.randint(0, r + 1, (n,), generator=g, device="cuda").int() if ranks else None)
    if runs:
        cut = torch.randint(0, M + 1, (max(1, n),), generator=g, device="cuda")
        who = (torch.arange(M, device="cuda")[:, None] >= cut).sum(1)
        ids = torch.randint(0, n, (n + 1,), generator=g, device="cuda")[who]
    else:
        ids = torch.randint(0, n, (M,), generator=g, device="cuda")
    ids[torch.rand(M, generator=g, device="cuda") < none] = -1
    s["adapter"] = ids.int()
    return s, dt[out]


def definition(s, out_dtype, rows=None):
    """-> (y, bound) float64 of the given rows (all by default)."""
    import torch

    x, ids = s["x"], s["adapter"].long()
    base = s["base"]
    if rows is not None:
        x, ids, base = x[rows], ids[rows], None if base is None else base[rows]
    x = x.double()
    M, K = x.shape
    n, N, r = s["b"].shape
    y = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    mag, late = torch.zeros_like(y), torch.zeros_like(y)
    if s["w"] is not None:
        w = s["w"].double()
        y += x @ w.T
        late += K * U * (x.abs() @ w.abs().T)
        mag += y.abs()
    if base is not None:
        y += base.double()
        mag += base.double().abs()
    part = 2.0 ** -16 if out_dtype == torch.bfloat16 else 2 * U
    for a in range(n):
        t = (ids == a).nonzero().flatten()
        rank = r if s["rank"] is None else int(s["rank"][a])
        if len(t) == 0 or rank == 0:
            continue
        A, B, sc = s["a"][a, :rank].double(), s["b"][a, :, :rank].double(), float(s["scale"][a])
        v = sc * (x[t] @ A.T)
        ev = sc * K * U * (x[t].abs() @ A.abs().T) + 2 * U * v.abs() + part * v.abs()
        y[t] += v @ B.T
        late[t] += ev @ B.abs().T + 3 * r * U * (v.abs() @ B.abs().T)
        mag[t] += (v @ B.T).abs()
    late += 4 * U * mag
    half = 2.0 ** -8 if out_dtype == torch.bfloat16 else U
    return y, late + half * (y.abs() + late)


def check(got, ref, bound, what):
    assert bool(got.isfinite().all()), what
    worst = float(((got.double() - ref).abs() / bound.clamp_min(1e-300)).max())
    print(f"{what}: worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0, what


CASES = [  # M, N, K, r, n, options
    (1, 64, 64, 8, 1, dict(none=0.0)),
    (1, 4096, 2048, 16, 8, dict(none=0.0)),
    (1, 33, 4096, 64, 4, dict(out="f32", none=0.0)),
    (3, 1001, 200, 24, 5, dict(ranks=True)),
    (16, 256, 1024, 40, 16, dict(base="f32")),
    (17, 130, 72, 128, 3, dict(out="f32", base="bf16", ranks=True)),
    (37, 640, 4096, 64, 16, dict(out="f32", ranks=True)),
    (64, 2048, 2048, 32, 64, dict(w=False, base="f32")),
    (64, 512, 512, 256, 2, dict(w=False)),
    (65, 96, 264, 72, 9, dict(base="bf16", out="f32")),
    (128, 1001, 2000, 24, 5, dict(ranks=True, runs=True)),
    (300, 515, 1032, 512, 4, dict(ranks=True)),
    (512, 512, 512, 16, 7, dict(runs=True, base="bf16")),
    (1000, 1001, 2000, 24, 5, dict(ranks=True, runs=True)),
    (1537, 777, 136, 8, 40, dict()),
    (2048, 1024, 1024, 64, 6, dict(runs=True, out="f32")),
    (700, 2000, 64, 96, 3, dict(w=False, base="bf16", runs=True)),
    (4100, 320, 4096, 128, 12, dict(w=False, base="f32", out="f32", runs=True)),
]


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c[:5])) + "".join(f"-{k}{v}" for k, v in c[5].items()) for c in CASES])
def test_against_definition(case):
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    M, N, K, r, n, kw = case
    s, dt = make(M, N, K, r, n, **kw)
    print(f"lora {case}", flush=True)
    ws = torch.empty(moe.lora_workspace_bytes(M, r), dtype=torch.uint8, device="cuda")
    ws.fill_(255)  # NaN wherever the call reads what it has not written
    out = torch.full((M, N), float("nan"), dtype=dt, device="cuda")
    moe.lora_linear(**s, out=out, ws=ws)
    torch.cuda.synchronize()
    check(out, *definition(s, dt), "y")
    again = moe.lora_linear(**s, out_dtype=dt)
    assert torch.equal(again, out)
