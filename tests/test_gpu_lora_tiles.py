"""moe_lora_linear: every form of its launches, named by the profile, at sizes with remainders: the three tiles with whole and
ended steps, mixed adapters (more of them in a tile than a wave has lanes), ranks beyond 64, and NaN in one adapter or row.
Definition and bounds: test_gpu_lora.py."""
import pytest

from gpu_util import need_gpu
from test_gpu_lora import check, definition, make

pytestmark = pytest.mark.gpu

BIG, MIDDLE, SMALL = "lora_tile_256x256_2", "lora_tile_128x128_3", "lora_tile_64x64_6"


def profiled(call):
    """-> (the call's result, the names of its launches)."""
    import torch

    import expert_offload_cache_amd as moe

    moe.profile_reset()
    moe.profile_enable(True)
    try:
        out = call()
        torch.cuda.synchronize()
        moe.profile_collect()
        return out, set(moe.profile_results())
    finally:
        moe.profile_enable(False)
        moe.profile_reset()


CASES = [  # M, N, K, r, n, options of the inputs, launches
    (1, 300, 520, 16, 3, dict(none=0.0), {"lora_alone"}),
    (1, 300, 520, 24, 3, dict(none=0.0), {"lora_both", "lora_stream"}),
    (1, 300, 520, 8, 3, dict(w=False, base="f32", none=0.0), {"lora_alone"}),
    (1, 4096, 264, 16, 3, dict(none=0.0), {"lora_alone"}),
    (1, 4097, 264, 16, 3, dict(none=0.0), {"lora_both", "lora_stream"}),      # more workgroups than compute units
    (1, 4097, 264, 16, 3, dict(w=False, base="bf16", none=0.0), {"lora_shrink", "lora_stream"}),
    (1, 130, 1032, 16, 3, dict(none=0.0), {"lora_both", "lora_stream"}),      # long rows of a narrow matrix
    (1, 130, 1032, 16, 3, dict(w=False, base="f32", none=0.0), {"lora_alone"}),
    (64, 4100, 264, 16, 3, dict(), {"lora_shrink", "lora_stream"}),  # more sums than launch 1's place holds
    (64, 1000, 2056, 72, 30, dict(), {"lora_both", "lora_stream"}),
    (64, 1000, 520, 72, 30, dict(w=False, base="bf16"), {"lora_shrink", "lora_stream"}),
    (65, 1000, 520, 72, 30, dict(w=False, base="bf16"), {"lora_shrink", "lora_add"}),
    (65, 130, 72, 72, 5, dict(ranks=True), {"lora_shrink", SMALL}),
    (2100, 1610, 136, 72, 9, dict(ranks=True), {"lora_shrink", MIDDLE}),
    (2100, 1610, 136, 136, 9, dict(ranks=True, base="bf16", out="f32"), {"lora_shrink", MIDDLE}),
    (2049, 1537, 64, 16, 300, dict(base="f32"), {"lora_shrink", MIDDLE}),     # some 90 adapters a tile, one step
    (1921, 1664, 1000, 40, 4, dict(runs=True), {"lora_shrink", MIDDLE}),
    (3590, 3350, 72, 72, 9, dict(ranks=True), {"lora_shrink", BIG}),
    (3590, 3350, 72, 136, 9, dict(ranks=True, base="f32", out="f32"), {"lora_shrink", BIG}),
    (3329, 3585, 64, 16, 300, dict(base="bf16"), {"lora_shrink", BIG}),       # some 150 adapters a tile, one step
    (3900, 3328, 1032, 64, 6, dict(runs=True, out="f32"), {"lora_shrink", BIG}),
]


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c[:5])) + "".join(f"-{k}{v}" for k, v in c[5].items()) for c in CASES])
def test_every_form(case):
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    M, N, K, r, n, kw, launches = case
    s, dt = make(M, N, K, r, n, seed=M + N, **kw)
    print(f"lora {case}", flush=True)
    ws = torch.empty(moe.lora_workspace_bytes(M, r), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    out = torch.full((M, N), float("nan"), dtype=dt, device="cuda")
    _, names = profiled(lambda: moe.lora_linear(**s, out=out, ws=ws))
    assert names == launches
    check(out, *definition(s, dt), "y")
    assert torch.equal(moe.lora_linear(**s, out_dtype=dt), out)


@pytest.mark.parametrize("M,N,K,tile", [(65, 130, 136, SMALL), (2100, 1610, 136, MIDDLE), (3590, 3350, 72, BIG)])
def test_bad_rows_and_adapters_keep_to_themselves_in_every_tile(M, N, K, tile):
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    s, dt = make(M, N, K, 72, 7, seed=3, none=0.1)
    s["rank"] = torch.tensor([72, 65, 0, 8, 64, 33, 71], dtype=torch.int32, device="cuda")
    clean, names = profiled(lambda: moe.lora_linear(**s))
    assert names == {"lora_shrink", tile}
    check(clean, *definition(s, dt), "clean")
    for value in (float("nan"), float("inf")):
        for what in ("a", "b", "scale"):
            t = {**s, what: s[what].clone()}
            t[what][3] = value
            print(f"{what} {value} {tile}", flush=True)
            got = moe.lora_linear(**t)
            own = t["adapter"] == 3
            assert torch.equal(got[~own], clean[~own]) and not bool(got[own].isfinite().any())
        x = s["x"].clone()
        x[M // 2, 3] = value
        got = moe.lora_linear(**{**s, "x": x})
        rest = torch.arange(M, device="cuda") != M // 2
        assert torch.equal(got[rest], clean[rest]) and not bool(got[M // 2].isfinite().any())
