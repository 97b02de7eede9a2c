"""moe_lora_linear where the adapters' sum and the rows it is added to nearly cancel, so that the result shows how many bits of
v = scale (A x) enter the second product: all 24 for any number of rows and either type of result.

Every sum is exact in binary32, so there is one right answer: a row of A has one entry, which makes v a product of three
numbers, rounded once; a row of B has one entry, a power of two; W is zero or absent; base takes v's upper 12 bits
away, and what is left has 12 bits at most (rounded once more to a BF16 result)."""
import pytest

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("w", [False, True])
@pytest.mark.parametrize("M,N,K,r,n", [
    (1, 96, 64, 16, 2), (1, 96, 64, 64, 2), (20, 130, 64, 32, 4), (64, 256, 128, 64, 8), (65, 256, 128, 64, 8),
    (200, 520, 64, 72, 5), (777, 333, 64, 128, 6), (2100, 1610, 72, 40, 9)])
def test_bits_of_v(M, N, K, r, n, w, out):
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[out]
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    a = torch.zeros(n, r, K, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(n, N, r, dtype=torch.bfloat16, device="cuda")
    j = torch.arange(r, device="cuda")
    of = (torch.arange(n, device="cuda")[:, None] + j) % K      # the input that rank j of an adapter takes
    a.scatter_(2, of[:, :, None], torch.randn(n, r, 1, generator=g, device="cuda").bfloat16())
    col = torch.arange(N, device="cuda") % r                    # the rank that a column takes
    b.scatter_(2, col[None, :, None].expand(n, N, 1), torch.exp2(torch.randint(-3, 3, (n, N, 1), generator=g, device="cuda").float()).bfloat16())
    scale = 0.5 + torch.rand(n, generator=g, device="cuda")
    ids = torch.randint(0, n, (M,), generator=g, device="cuda")
    v = scale[ids][:, None] * (a.float().sum(2)[ids] * x.float().gather(1, of[ids]))  # [M, r], one rounding (the last)
    whole = v[:, col] * b.float().sum(2)[ids]                   # exact
    base = -(whole.view(torch.int32) & ~0xFFF).view(torch.float32)
    left = whole.double() + base.double()
    want = left.float().to(dt)                                  # left is exact in binary32
    assert bool((left == left.float().double()).all()) and bool((left != 0).any())
    print(f"bits M={M} N={N} K={K} r={r} w={w} {out}", flush=True)
    got = moe.lora_linear(x, a, b, scale, ids.int(), base=base, out_dtype=dt,
                          w=torch.zeros(N, K, dtype=torch.bfloat16, device="cuda") if w else None)
    wrong = got != want
    print(f"{int(wrong.sum())} of {wrong.numel()} differ, by {float(((got.double() - left).abs() / left.abs().clamp_min(1e-30)).max()):.2e} of the value at most", flush=True)
    assert not bool(wrong.any())
