"""moe_layer_few and moe_lora_linear without a GPU: workspaces, empty calls and every refusal (all of them checked on
the host before any launch)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def moe():
    import os

    import expert_offload_cache_amd as m
    from expert_offload_cache_amd import _lib

    if not os.path.exists(_lib.LIB_PATH):
        from expert_offload_cache_amd import build as b

        b.build()
    return m


@pytest.mark.parametrize("wdt,d,f,E,k,shared", [("f32", 64, 96, 8, 2, False), ("bf16", 2048, 768, 128, 8, False),
                                                ("int4", 4096, 2048, 256, 6, True), ("fp8", 1152, 640, 60, 4, True),
                                                ("bf16", 320, 33 * 32, 1024, 32, True)])
def test_few_workspace_of_more_tokens_serves_fewer(moe, wdt, d, f, E, k, shared):
    sizes = [moe.layer_few_workspace_bytes(T, d, f, E, k, shared, wdt) for T in range(1, 17)]
    assert sizes == sorted(sizes) and 0 < sizes[0] < sizes[-1]
    assert moe.layer_few_workspace_bytes(17, d, f, E, k, shared, wdt) == 0
    # the same whether the layer has a shared expert or more experts: never less
    assert moe.layer_few_workspace_bytes(16, d, f, E, k, True, wdt) >= moe.layer_few_workspace_bytes(16, d, f, E, k, False, wdt)


def test_lora_workspace(moe):
    sizes = [moe.lora_workspace_bytes(M, 64) for M in range(0, 300)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    sizes = [moe.lora_workspace_bytes(200, r) for r in range(8, 513, 8)]
    assert sizes == sorted(sizes)
    assert moe.lora_workspace_bytes(1 << 21, 512) > 1 << 32
    for M, r in ((-1, 8), (4, 0), (4, 12), (4, 520), (4, -8)):
        assert moe.lora_workspace_bytes(M, r) == 0


def test_few_refusals(moe):
    L, e = moe.lib(), moe._lib
    p, odd = ctypes.c_void_p(256), lambda n: ctypes.c_void_p(256 + n)
    base = dict(x=p, act=1, T=4, d=256, f=128, E=8, k=2, router=p, bias=p, forced=None, slot=p, n=8, pool=p, stride=None,
                w=1, shared=None, idx=p, gate=p, y=p, ws=p, wsb=None)

    def few(**kw):
        a = {**base, **kw}
        wdt = {0: "f32", 1: "bf16", 2: "int4", 3: "fp8"}.get(a["w"], "bf16")
        stride = a["stride"] if a["stride"] is not None else max(256, moe.slot_bytes(a["d"], a["f"], wdt))
        wsb = a["wsb"] if a["wsb"] is not None else 1 << 30
        return L.moe_layer_few(a["x"], a["act"], a["T"], a["d"], a["f"], a["E"], a["k"], a["router"], a["bias"], a["forced"],
                               a["slot"], a["n"], a["pool"], stride, a["w"], a["shared"], a["idx"], a["gate"], a["y"], a["ws"],
                               wsb, None)

    assert few(T=0) == e.MOE_OK and few(T=0, x=None, y=None, ws=None) == e.MOE_OK
    need = moe.layer_few_workspace_bytes(4, 256, 128, 8, 2, False, "bf16")
    bad = [(dict(T=-1), e.MOE_ESHAPE), (dict(T=17), e.MOE_ESHAPE), (dict(d=0), e.MOE_ESHAPE), (dict(d=-64), e.MOE_ESHAPE),
           (dict(d=288), e.MOE_ESHAPE), (dict(d=250), e.MOE_ESHAPE), (dict(f=0), e.MOE_ESHAPE), (dict(f=100), e.MOE_ESHAPE),
           (dict(E=0), e.MOE_ESHAPE), (dict(E=1025), e.MOE_ESHAPE), (dict(k=0), e.MOE_ESHAPE), (dict(k=9), e.MOE_ESHAPE),
           (dict(E=64, k=33), e.MOE_ESHAPE), (dict(act=2), e.MOE_EDTYPE), (dict(act=3), e.MOE_EDTYPE), (dict(w=4), e.MOE_EDTYPE),
           (dict(w=-1), e.MOE_EDTYPE), (dict(act=0, w=1), e.MOE_EDTYPE), (dict(act=1, w=0), e.MOE_EDTYPE), (dict(act=0, w=2), e.MOE_EDTYPE),
           (dict(act=0, w=3), e.MOE_EDTYPE), (dict(w=2, d=192), e.MOE_ESHAPE), (dict(w=3, f=64), e.MOE_ESHAPE),
           (dict(n=0), e.MOE_EINVAL), (dict(stride=256), e.MOE_EINVAL), (dict(stride=moe.slot_bytes(256, 128, "bf16") + 128), e.MOE_EINVAL),
           (dict(pool=odd(128)), e.MOE_EINVAL), (dict(shared=odd(64)), e.MOE_EINVAL), (dict(wsb=need - 1), e.MOE_ENOMEM),
           (dict(wsb=0), e.MOE_ENOMEM), (dict(bias=odd(2)), e.MOE_EINVAL), (dict(forced=odd(1)), e.MOE_EINVAL),
           (dict(slot=odd(2)), e.MOE_EINVAL), (dict(idx=odd(2)), e.MOE_EINVAL), (dict(gate=odd(2)), e.MOE_EINVAL)]
    bad += [(({n: None}), e.MOE_EINVAL) for n in ("x", "router", "slot", "pool", "idx", "gate", "y", "ws")]
    bad += [(({n: odd(8)}), e.MOE_EINVAL) for n in ("x", "router", "y", "ws")]
    for kw, code in bad:
        assert few(**kw) == code, kw
        assert b"moe_layer_few" in L.moe_last_error()


def test_lora_refusals(moe):
    L, e = moe.lib(), moe._lib
    p, odd = ctypes.c_void_p(256), lambda n: ctypes.c_void_p(256 + n)
    base = dict(x=p, ldx=64, M=4, K=64, w=p, ldw=64, N=32, base=None, ldb=0, bt=1, a=p, b=p, r=16, n=3, scale=p, rank=None,
                adapter=p, y=p, ldy=32, out=1, ws=p, wsb=1 << 30)

    def lora(**kw):
        a = {**base, **kw}
        return L.moe_lora_linear(a["x"], a["ldx"], a["M"], a["K"], a["w"], a["ldw"], a["N"], a["base"], a["ldb"], a["bt"], a["a"],
                                 a["b"], a["r"], a["n"], a["scale"], a["rank"], a["adapter"], a["y"], a["ldy"], a["out"], a["ws"],
                                 a["wsb"], None)

    assert lora(M=0) == e.MOE_OK and lora(M=0, x=None, y=None, ws=None) == e.MOE_OK
    far = ctypes.c_void_p(4096)
    bad = [(dict(M=-1), e.MOE_ESHAPE), (dict(M=(1 << 21) + 1), e.MOE_ESHAPE), (dict(K=0), e.MOE_ESHAPE), (dict(K=60), e.MOE_ESHAPE),
           (dict(K=(1 << 20) + 8, ldx=1 << 21, ldw=1 << 21), e.MOE_ESHAPE), (dict(N=0), e.MOE_ESHAPE),
           (dict(N=(1 << 22) + 1, ldy=1 << 23), e.MOE_ESHAPE), (dict(r=0), e.MOE_ESHAPE), (dict(r=12), e.MOE_ESHAPE),
           (dict(r=520), e.MOE_ESHAPE), (dict(n=0), e.MOE_ESHAPE), (dict(n=(1 << 20) + 1), e.MOE_ESHAPE), (dict(out=2), e.MOE_EDTYPE),
           (dict(out=-1), e.MOE_EDTYPE), (dict(base=far, ldb=32, bt=2), e.MOE_EDTYPE), (dict(ldx=56), e.MOE_EINVAL),
           (dict(ldx=68), e.MOE_EINVAL), (dict(ldw=56), e.MOE_EINVAL), (dict(ldw=68), e.MOE_EINVAL), (dict(ldy=31), e.MOE_EINVAL),
           (dict(base=far, ldb=31), e.MOE_EINVAL), (dict(base=p, ldb=40), e.MOE_EINVAL), (dict(base=p, ldb=32, bt=0), e.MOE_EINVAL),
           (dict(y=odd(1)), e.MOE_EINVAL), (dict(y=odd(2), out=0), e.MOE_EINVAL), (dict(base=odd(3), ldb=32), e.MOE_EINVAL),
           (dict(base=odd(2), ldb=32, bt=0), e.MOE_EINVAL), (dict(scale=odd(2)), e.MOE_EINVAL), (dict(rank=odd(2)), e.MOE_EINVAL),
           (dict(adapter=odd(1)), e.MOE_EINVAL), (dict(wsb=moe.lora_workspace_bytes(4, 16) - 1), e.MOE_ENOMEM)]
    bad += [(({n: None}), e.MOE_EINVAL) for n in ("x", "a", "b", "scale", "adapter", "y", "ws")]
    bad += [(({n: odd(8)}), e.MOE_EINVAL) for n in ("x", "w", "a", "b", "ws")]
    for kw, code in bad:
        assert lora(**kw) == code, kw
        assert b"moe_lora_linear" in L.moe_last_error()


def test_binding_refusals(moe):
    """The binding checks shapes, types and where tensors live before it calls the library."""
    import torch

    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    x, a, b = torch.zeros(4, 64, dtype=bf), torch.zeros(3, 16, 64, dtype=bf), torch.zeros(3, 32, 16, dtype=bf)
    scale, ids, w = torch.ones(3), torch.zeros(4, dtype=i32), torch.zeros(32, 64, dtype=bf)
    good = dict(x=x, a=a, b=b, scale=scale, adapter=ids, w=w)
    for kw in (dict(x=x.float()), dict(x=x[:, :32]), dict(a=a.float()), dict(a=a[:, :, :32]), dict(a=a[:2]), dict(b=b[:, :, :8]),
               dict(scale=scale.double()), dict(scale=scale[:2]), dict(adapter=ids.long()), dict(adapter=ids[:3]),
               dict(w=w.float()), dict(w=w[:, :32]), dict(w=w[:16]), dict(base=torch.zeros(4, 16)), dict(base=torch.zeros(4, 32).double()),
               dict(rank=torch.zeros(2, dtype=i32)), dict(rank=torch.zeros(3)), dict(out=torch.zeros(4, 31, dtype=bf)),
               dict(out=torch.zeros(4, 32, dtype=torch.float16)), dict(x=torch.zeros(64, 4, dtype=bf).T)):
        with pytest.raises((ValueError, TypeError)):
            moe.lora_linear(**{**good, **kw})
    n = moe.slot_bytes(64, 64, "bf16")
    few = dict(x=x, w_router=torch.zeros(8, 64, dtype=bf), bias=torch.zeros(8), k=2, slot_of_expert=torch.zeros(8, dtype=i32),
               slot_pool=torch.zeros(8 * n, dtype=torch.uint8), n_slots=8, slot_stride=n, wdt="bf16", f=64)
    for kw in (dict(w_router=torch.zeros(8, 64)), dict(w_router=torch.zeros(8, 32, dtype=bf)), dict(bias=torch.zeros(7)),
               dict(forced_idx=torch.zeros(4, 3, dtype=i32)), dict(forced_idx=torch.zeros(4, 2)), dict(slot_of_expert=torch.zeros(7, dtype=i32)),
               dict(slot_of_expert=torch.zeros(8)), dict(slot_pool=torch.zeros(8 * n - 1, dtype=torch.uint8)),
               dict(shared_w=torch.zeros(n - 1, dtype=torch.uint8)), dict(x=torch.zeros(64, 4, dtype=bf).T),
               dict(out=(torch.zeros(4, 64), torch.zeros(4, 2, dtype=i32), torch.zeros(4, 2)))):
        with pytest.raises((ValueError, TypeError)):
            moe.layer_few(**{**few, **kw})
