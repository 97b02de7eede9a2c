"""moe_layer_few and moe_lora_linear at the ends of their ranges, and called from two threads at once.  Definitions and bounds are
those of the two operators' own test files."""
import threading

import numpy as np
import pytest

from gpu_util import need_gpu
from test_gpu_few import check_y, layer_bound, make as make_layer
from test_gpu_lora import check, definition, make as make_lora

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,wdt,d,f,E,k,shared,T", [
    ("bf16", "bf16", 16384, 64, 3, 2, True, 16), ("bf16", "bf16", 16384, 96, 2, 1, False, 1),
    ("bf16", "int4", 16384, 128, 3, 2, True, 16), ("bf16", "int4", 16384, 256, 2, 2, False, 1),
    ("bf16", "fp8", 16384, 128, 3, 2, True, 16), ("f32", "f32", 16384, 64, 2, 2, False, 13),
    ("bf16", "bf16", 64, 16384, 3, 2, True, 16), ("bf16", "int4", 128, 16384, 3, 2, True, 16),
    ("bf16", "fp8", 128, 16384, 3, 2, True, 16), ("f32", "f32", 64, 16384, 2, 2, False, 16),
    ("bf16", "bf16", 64, 64, 1, 1, True, 16), ("bf16", "int4", 128, 128, 1, 1, False, 1),
])
def test_few_largest_and_smallest(act, wdt, d, f, E, k, shared, T):
    need_gpu()
    import torch

    li, layer = make_layer(act, wdt, d, f, E, k, shared, T)
    print(f"few {act} {wdt} d={d} f={f} E={E} k={k} T={T}", flush=True)
    bufs = layer.buffers_few(T)
    out = layer.forward_few(layer.x_to_device(li.x), bufs=bufs)
    torch.cuda.synchronize()
    ref, bound, idx, _ = layer_bound(li, li.x)
    assert np.array_equal(out["topk_idx"].cpu().numpy(), idx)
    check_y(out["y"], ref, bound, wdt)
    assert int(bufs["ws"][:4].view(torch.int32)) == 0


@pytest.mark.parametrize("T", range(1, 17))
def test_few_every_number_of_tokens(T):
    need_gpu()
    import torch

    for act, wdt in (("bf16", "bf16"), ("bf16", "int4"), ("bf16", "fp8"), ("f32", "f32")):
        li, layer = make_layer(act, wdt, 384, 384, 11, 5, True, T, seed=T)
        print(f"few {wdt} T={T}", flush=True)
        out = layer.forward_few(layer.x_to_device(li.x))
        ref, bound, idx, _ = layer_bound(li, li.x)
        assert np.array_equal(out["topk_idx"].cpu().numpy(), idx) and int(out["ws"][:4].view(torch.int32)) == 0
        check_y(out["y"], ref, bound, wdt)


@pytest.mark.parametrize("M", [1, 2, 16, 64, 65, 300])
@pytest.mark.parametrize("w,base,out", [(True, None, "bf16"), (False, "bf16", "f32"), (True, "f32", "bf16")])
def test_lora_smallest(M, w, base, out):
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    for N in (1, 2, 17):
        s, dt = make_lora(M, N, 8, 8, 1, w=w, base=base, out=out, seed=M, none=0.3 if M > 1 else 0.0)
        print(f"lora M={M} N={N} w={w} {base} {out}", flush=True)
        got = moe.lora_linear(**s, out_dtype=dt)
        check(got, *definition(s, dt), "y")


def test_lora_longest_rows():
    need_gpu()
    import expert_offload_cache_amd as moe

    for M in (1, 3, 70):
        s, dt = make_lora(M, 24, 1 << 20, 8, 2, out="f32", none=0.0)
        print(f"lora K=2^20 M={M}", flush=True)
        check(moe.lora_linear(**s, out_dtype=dt), *definition(s, dt), "y")


@pytest.mark.parametrize("M", [1, 64, 70])
@pytest.mark.parametrize("w", [True, False])
def test_lora_widest(M, w):
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    N = 1 << 22
    s, dt = make_lora(M, N, 8, 8, 2, w=w, none=0.0 if M == 1 else 0.1)
    print(f"lora N=2^22 M={M} w={w}", flush=True)
    got = moe.lora_linear(**s, out_dtype=dt)
    for cols in (slice(0, 300), slice(N // 2 - 100, N // 2 + 100), slice(N - 300, N)):
        part = dict(s, b=s["b"][:, cols], w=None if s["w"] is None else s["w"][cols])
        check(got[:, cols], *definition(part, dt), f"{cols}")


@pytest.mark.parametrize("w,base", [(True, None), (False, "bf16")])
def test_lora_most_rows(w, base):
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    M = 1 << 21
    s, dt = make_lora(M, 24, 8, 8, 3, w=w, base=base, runs=True)
    print(f"lora M=2^21 w={w}", flush=True)
    check(moe.lora_linear(**s, out_dtype=dt), *definition(s, dt), "y")


@pytest.mark.parametrize("M", [2, 64, 400])
def test_lora_most_adapters(M):
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    n, N, K, r = 1 << 20, 40, 16, 8
    g = torch.Generator(device="cuda").manual_seed(M)
    s, dt = make_lora(M, N, K, r, 1, out="f32")
    s["a"] = torch.randn(n, r, K, generator=g, device="cuda").bfloat16()
    s["b"] = torch.randn(n, N, r, generator=g, device="cuda").bfloat16()
    s["scale"] = 0.5 + torch.rand(n, generator=g, device="cuda")
    s["adapter"] = torch.randint(0, n, (M,), generator=g, device="cuda").int()
    s["adapter"][0], s["adapter"][M - 1] = n - 1, 0
    print(f"lora 2^20 adapters M={M}", flush=True)
    got = moe.lora_linear(**s, out_dtype=dt)
    ids = s["adapter"].long()
    few = dict(s, a=s["a"][ids], b=s["b"][ids], scale=s["scale"][ids], adapter=torch.arange(M, device="cuda").int())
    check(got, *definition(few, dt), "y")


def test_two_threads_at_once():
    """Each with a stream of its own, different sizes of the same forms: what a call sets on the host is its own."""
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    work = []
    for T, f in ((2, 768), (16, 416)):
        li, layer = make_layer("bf16", "bf16", 320, f, 9, 4, True, T, seed=T)
        x = layer.x_to_device(li.x)
        s, dt = make_lora(70 * T, 264, 512, 32, 4, seed=T)
        work.append((layer, x, layer.forward_few(x)["y"].clone(), s, moe.lora_linear(**s).clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    wrong = []

    def run(layer, x, y, s, z, stream):
        try:
            with torch.cuda.stream(stream):
                for _ in range(100):
                    a, b = layer.forward_few(x), moe.lora_linear(**s)
                    if not torch.equal(a["y"], y) or not torch.equal(b, z) or int(a["ws"][:4].view(torch.int32)):
                        wrong.append(x.shape)
        except Exception as e:  # noqa: BLE001 -- reported by the main thread
            wrong.append(e)

    print("threads", flush=True)
    threads = [threading.Thread(target=run, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
