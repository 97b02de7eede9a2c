"""moe_layer_few and moe_lora_linear where they can go wrong: absent and masked experts, forced and repeated ids, NaN and
infinities in one row or one adapter, wide and long shapes, strides, aliases, offsets beyond 32 bits, other streams, two
calls at once, captured and replayed graphs, and both of them in a run with the norm between.  Definitions and bounds
are those of the two operators' own test files."""
import numpy as np
import pytest

from gpu_util import need_gpu, rel_err_per_token, to_dev, y_to_f64
from test_gpu_few import check_y, layer_bound, make as make_layer
from test_gpu_lora import check, definition, make as make_lora

pytestmark = pytest.mark.gpu

ELSEWHERE = -2  # MOE_SLOT_ELSEWHERE


def _clone(out):
    return {k: v.clone() for k, v in out.items() if v is not None}


# ---- moe_layer_few ------------------------------------------------------------------------------------
@pytest.mark.parametrize("act,wdt,shared", [("f32", "f32", True), ("bf16", "bf16", False), ("bf16", "int4", True), ("bf16", "fp8", False)])
@pytest.mark.parametrize("T", [1, 6])
def test_few_absent_and_elsewhere(act, wdt, shared, T):
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    d, f, E, k = 256, 128, 6, 3
    li, layer = make_layer(act, wdt, d, f, E, k, shared, T)
    x = layer.x_to_device(li.x)
    home = layer.slot_of_expert.clone()
    for name, gone, value, status in (("none", [], -1, 0), ("elsewhere", [0, 4], ELSEWHERE, 0), ("absent", [1], -1, 1),
                                      ("past the pool", [2, 3], layer.n_slots, 1), ("all absent", list(range(E)), -1, 1),
                                      ("all elsewhere", list(range(E)), ELSEWHERE, 0)):
        print(f"slots: {wdt} T={T} {name}", flush=True)
        slot = home.clone()
        slot[gone] = value
        bufs = layer.buffers_few(T)
        out = layer.forward_few(x, slot_of_expert=slot, bufs=bufs)
        torch.cuda.synchronize()
        ref, bound, idx, _ = layer_bound(li, li.x, skip=gone)
        assert np.array_equal(out["topk_idx"].cpu().numpy(), idx)
        check_y(out["y"], ref, bound + 1e-300, name)
        used = set(idx.ravel().tolist()) & set(gone)
        assert int(bufs["ws"][:4].view(torch.int32)) == (status if used else 0)
        # the word stays, the results do not depend on it
        again = layer.forward_few(x, bufs=bufs)["y"].clone()
        assert torch.equal(again, layer.forward_few(x)["y"])
        assert int(bufs["ws"][:4].view(torch.int32)) == (status if used else 0)


@pytest.mark.parametrize("act,wdt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "int4"), ("bf16", "fp8")])
def test_few_forced_and_repeated_ids(act, wdt):
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    d, f, E, k, T = 128, 256, 9, 4, 7
    li, layer = make_layer(act, wdt, d, f, E, k, True, T)
    x = layer.x_to_device(li.x)
    rng = np.random.default_rng(3)
    forced = rng.integers(0, E, (T, k)).astype(np.int32)
    forced[0] = [5, 5, 5, 5]  # one expert four times
    forced[1] = [2, 7, 2, 0]
    forced[2:5] = [[8, 1, 3, 4]] * 3  # the same experts for several tokens
    print(f"forced {wdt}", flush=True)
    ids = to_dev(forced, "i32")
    out = layer.forward_few(x, forced_idx=ids)
    ref, bound, idx, gates = layer_bound(li, li.x, forced=forced)
    assert np.array_equal(out["topk_idx"].cpu().numpy(), forced)
    assert torch.equal(out["topk_w"], moe.route(x, layer.w_router, layer.bias, k, forced_idx=ids)[1])
    check_y(out["y"], ref, bound, wdt)
    far = forced.copy()
    far[3, 1], far[6, 0] = 10 ** 6, -5  # read as the nearest id; the other rows are what they were
    got = layer.forward_few(x, forced_idx=to_dev(far, "i32"))["y"]
    rest = [0, 1, 2, 4, 5]
    assert torch.equal(got[rest], out["y"][rest]) and bool(got.isfinite().all())


@pytest.mark.parametrize("act,wdt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "int4"), ("bf16", "fp8")])
def test_few_masked_experts_and_bad_rows(act, wdt):
    """Experts masked by a bias of minus infinity or of the type's lowest value; a row of NaN, one with an infinity."""
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    d, f, E, k, T = 256, 128, 12, 4, 8
    li, layer = make_layer(act, wdt, d, f, E, k, False, T)
    x = layer.x_to_device(li.x)
    for low in (-float("inf"), torch.finfo(torch.float32).min):
        bias = torch.full((E,), low, device="cuda")
        bias[[1, 3, 6, 7, 10]] = layer.bias[[1, 3, 6, 7, 10]]
        print(f"masked {wdt} {low}", flush=True)
        y, idx, w = moe.layer_few(x, layer.w_router, bias, k, layer.slot_of_expert, layer.pool, layer.n_slots, layer.stride, wdt, f)
        ids, gates, _ = moe.route(x, layer.w_router, bias, k)
        assert torch.equal(idx, ids) and torch.equal(w, gates)
        assert set(idx.unique().tolist()) <= {1, 3, 6, 7, 10} and bool(y.isfinite().all())
    clean = _clone(layer.forward_few(x))
    ref, bound, _, _ = layer_bound(li, li.x)
    for value in (float("nan"), float("inf"), -float("inf")):
        bad = x.clone()
        bad[2, 5] = value
        bad[5] = value
        print(f"bad rows {wdt} {value}", flush=True)
        out = layer.forward_few(bad)
        rest = [0, 1, 3, 4, 6, 7]
        for n in ("topk_idx", "topk_w"):
            assert torch.equal(out[n][rest], clean[n][rest]), n
        check_y(out["y"][rest], ref[rest], bound[rest], "the other rows")  # (their sums may be cut elsewhere)
    # nothing of it stays in the workspace
    bufs = layer.buffers_few(T)
    layer.forward_few(bad, bufs=bufs)
    assert torch.equal(layer.forward_few(x, bufs=bufs)["y"], clean["y"])


@pytest.mark.parametrize("act,wdt,d,f,E,k,shared,T", [
    ("bf16", "bf16", 64, 64, 1024, 32, False, 16),    # the most experts and choices
    ("f32", "f32", 128, 64, 600, 32, True, 16),
    ("bf16", "bf16", 4160, 64, 5, 2, True, 3),        # rows beyond what a wave holds
    ("bf16", "bf16", 8256, 96, 3, 1, False, 16),
    ("f32", "f32", 4224, 64, 4, 2, False, 2),
    ("bf16", "int4", 4224, 128, 4, 2, False, 16),
    ("bf16", "fp8", 8320, 128, 3, 2, True, 4),
    ("bf16", "bf16", 64, 6176, 3, 2, False, 16),      # long rows of h
    ("bf16", "int4", 128, 4992, 3, 2, True, 16),
    ("bf16", "fp8", 128, 5120, 4, 3, False, 2),
    ("f32", "f32", 64, 2080, 4, 4, True, 16),
    ("bf16", "bf16", 192, 64, 1, 1, False, 1),        # one expert
])
def test_few_wide_and_long(act, wdt, d, f, E, k, shared, T):
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


@pytest.mark.parametrize("T", [1, 4, 16])
def test_few_int4_rows_beside_their_norm(T):
    """The elements' bound of int4 counts the nibbles' offset and is wide; a row as a whole is nearer: each h and each y is off by
    half a step (2^-8 of the row's norm together, twice), the sums' errors are far below (n 2^-24 * 280 / sqrt(n)
    of it, n = 1408: 2^-11), and flips of h's rounding count once more: 2^-6 at most."""
    need_gpu()
    li, layer = make_layer("bf16", "int4", 1408, 384, 16, 4, True, T)
    ref, _, _, _ = layer_bound(li, li.x)
    y = y_to_f64(layer.forward_few(layer.x_to_device(li.x))["y"])
    assert rel_err_per_token(y, ref).max() <= 2.0 ** -6


@pytest.mark.parametrize("act,wdt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "int4"), ("bf16", "fp8")])
def test_few_one_workspace_for_many_calls_and_y_in_place(act, wdt):
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    li, layer = make_layer(act, wdt, 256, 384, 10, 3, True, 16)
    x = layer.x_to_device(li.x)
    ws = layer.buffers_few(16)["ws"]
    call = lambda x, out=None, ws=None: moe.layer_few(x, layer.w_router, layer.bias, 3, layer.slot_of_expert, layer.pool, layer.n_slots,
                                                     layer.stride, wdt, 384, shared_w=layer.shared, out=out, ws=ws)
    want = {T: call(x[:T].clone())[0] for T in (1, 2, 3, 5, 9, 16)}
    for T in (16, 1, 9, 3, 16, 2, 5, 1, 16):
        y, idx, w = call(x[:T].clone(), ws=ws)
        assert torch.equal(y, want[T]), T
        rows = x[:T].clone()
        call(rows, out=(rows, idx, w), ws=ws)
        assert torch.equal(rows, want[T]), T
    empty = torch.empty(0, 256, dtype=x.dtype, device="cuda")
    assert call(empty)[0].shape == (0, 256)


def test_few_streams_graphs_and_two_at_once():
    need_gpu()
    import torch

    layers = [make_layer("bf16", "bf16", 320, 160, 12, 4, True, 16, seed=1), make_layer("bf16", "int4", 256, 256, 9, 3, False, 16, seed=2),
              make_layer("bf16", "fp8", 384, 128, 7, 2, True, 16, seed=3)]
    cases = []
    for li, layer in layers:
        for T in (1, 7, 16):
            x = layer.x_to_device(li.x[:T])
            cases.append((layer, x, _clone(layer.forward_few(x))))
    torch.cuda.synchronize()
    # each on a stream of its own, all at once, each with its own workspace
    streams = [torch.cuda.Stream() for _ in cases]
    bufs = [layer.buffers_few(x.shape[0]) for layer, x, _ in cases]
    torch.cuda.synchronize()
    print("streams", flush=True)
    for _ in range(5):
        for (layer, x, _), b, s in zip(cases, bufs, streams):
            with torch.cuda.stream(s):
                layer.forward_few(x, bufs=b, stream=s)
    torch.cuda.synchronize()
    for (_, _, want), b in zip(cases, bufs):
        assert torch.equal(b["few"][0], want["y"]) and torch.equal(b["few"][1], want["topk_idx"])
    # captured, replayed with new rows, eager calls in the same workspace between the replays
    print("graphs", flush=True)
    s = streams[0]
    for (layer, x, _), b in zip(cases, bufs):
        rows = x.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            layer.forward_few(rows, bufs=b)
        for i in range(4):
            rows.copy_(x.roll(i, 0) * (1 + i))
            g.replay()
            torch.cuda.synchronize()
            got = _clone(dict(y=b["few"][0], idx=b["few"][1]))
            eager = layer.forward_few(rows, bufs=b)
            assert torch.equal(got["y"], eager["y"]) and torch.equal(got["idx"], eager["topk_idx"])
            assert torch.equal(layer.forward_few(rows)["y"], got["y"])
    for b in bufs:
        assert int(b["ws"][:4].view(torch.int32)) == 0


# ---- moe_lora_linear ----------------------------------------------------------------------------------
@pytest.mark.parametrize("M", [1, 5, 33, 64, 65, 300])
@pytest.mark.parametrize("w,base", [(True, None), (True, "f32"), (False, "bf16")])
def test_lora_strides_and_columns_beside(M, w, base):
    """Rows apart from each other, results that start on any element: what lies beside them stays."""
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    N, K, r, n = 145, 136, 24, 4
    for dt, off in ((torch.bfloat16, 3), (torch.float32, 1), (torch.bfloat16, 8), (torch.float32, 4)):
        s, _ = make_lora(M, N, K, r, n, w=w, base=base, seed=M, ranks=True)
        xs = torch.full((M, K + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
        xs[:, :K] = s["x"]
        s["x"] = xs[:, :K]
        if w:
            wide = torch.full((N, K + 8), float("inf"), dtype=torch.bfloat16, device="cuda")
            wide[:, :K] = s["w"]
            s["w"] = wide[:, :K]
        if base:
            wide = torch.full((M, N + 7), float("nan"), dtype=s["base"].dtype, device="cuda")
            wide[:, 5:5 + N] = s["base"]
            s["base"] = wide[:, 5:5 + N]
        ld = (N + off + 9) // 8 * 8 + (0 if off % 4 == 0 else 1)
        buf = torch.full((M + 2, ld), 7.0, dtype=dt, device="cuda")
        print(f"strides M={M} w={w} base={base} {dt} {off}", flush=True)
        out = moe.lora_linear(**s, out=buf[1:M + 1, off:off + N])
        check(out, *definition(s, dt), "y")
        rest = buf.clone()
        rest[1:M + 1, off:off + N] = 7.0
        assert bool((rest == 7.0).all())


@pytest.mark.parametrize("M", [2, 40, 64, 200, 1100])
@pytest.mark.parametrize("base", ["bf16", "f32"])
def test_lora_in_place(M, base):
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    for w in (True, False):
        s, _ = make_lora(M, 520, 256, 32, 5, w=w, base=base, seed=M)
        want = moe.lora_linear(**s, out_dtype=s["base"].dtype)
        print(f"in place M={M} w={w} {base}", flush=True)
        got = moe.lora_linear(**s, out=s["base"])
        assert torch.equal(got, want)


@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (9, 96, 264), (37, 130, 512), (200, 200, 264), (2100, 1100, 128)])
@pytest.mark.parametrize("w", [True, False])
def test_lora_bad_rows_and_adapters_keep_to_themselves(M, N, K, w):
    """NaN and infinities in a row of x, in one adapter, beyond an adapter's rank; ids outside the list; rank 0."""
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    r, n = 40, 6
    s, dt = make_lora(M, N, K, r, n, w=w, base=None if w else "f32", seed=5, none=0.1)
    s["rank"] = torch.tensor([40, 33, 0, 8, 17, 39], dtype=torch.int32, device="cuda")
    clean = moe.lora_linear(**s)
    check(clean, *definition(s, dt), "clean")
    t = dict(s)
    for a in range(n):  # what lies beyond a rank is not used
        k = int(s["rank"][a])
        t["a"], t["b"] = t["a"].clone(), t["b"].clone()
        t["a"][a, k:] = float("nan")
        t["b"][a, :, k:] = float("inf")
    print(f"beyond the ranks M={M} w={w}", flush=True)
    assert torch.equal(moe.lora_linear(**t), clean)
    ids = s["adapter"].clone()
    ids[ids == 2] = torch.tensor([n, 2 ** 31 - 1, -2 ** 31, -7], dtype=torch.int32, device="cuda").repeat(M)[: int((ids == 2).sum())]
    assert torch.equal(moe.lora_linear(**{**s, "adapter": ids}), clean)  # rank 0 and no adapter are the same
    for value in (float("nan"), float("inf")):
        for what in ("a", "b", "scale"):
            t = {**s, what: s[what].clone()}
            t[what][3] = value
            if M == 1:
                t["adapter"] = torch.full_like(s["adapter"], 3)
            print(f"{what} {value} M={M} w={w}", flush=True)
            got = moe.lora_linear(**t)
            own = t["adapter"] == 3
            assert torch.equal(got[~own], clean[~own])
            assert not bool(got[own].isfinite().any())
        x = s["x"].clone()
        x[M // 2, 3] = value
        got = moe.lora_linear(**{**s, "x": x})
        rest = torch.arange(M, device="cuda") != M // 2
        assert torch.equal(got[rest], clean[rest])
        if w:
            assert not bool(got[M // 2].isfinite().any())


@pytest.mark.parametrize("M", [1, 20, 64, 130])
def test_lora_no_adapters_at_all(M):
    """Every row without one: the projection, the base, or zeros; what the workspace and the adapters hold is not used."""
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    for w, base in ((True, None), (False, "f32"), (False, None), (True, "bf16")):
        s, dt = make_lora(M, 100, 128, 16, 3, w=w, base=base, none=2.0)
        assert bool((s["adapter"] == -1).all())
        s["a"][:], s["b"][:] = float("nan"), float("inf")
        ws = torch.full((moe.lora_workspace_bytes(M, 16),), 255, dtype=torch.uint8, device="cuda")
        got = moe.lora_linear(**s, ws=ws)
        check(got, *definition(s, dt), f"w={w} base={base}")
        if not w and base:
            assert torch.equal(got, s["base"].bfloat16())
    empty = moe.lora_linear(s["x"][:0], s["a"], s["b"], s["scale"], s["adapter"][:0], w=s["w"])
    assert empty.shape == (0, 100)


def test_lora_offsets_beyond_32_bits():
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    # adapters that begin 4 GB and more into their arrays, rows of x, base and y more than 4 GB apart
    n, r, K, N = 68, 512, 64 * 1024, 136
    s, _ = make_lora(70, N, K, 8, 2, w=False)
    a = torch.zeros(n, r, K, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(n, N, r, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in (0, n - 1):
        a[i] = torch.randn(r, K, generator=g, device="cuda").bfloat16() / 256
        b[i] = torch.randn(N, r, generator=g, device="cuda").bfloat16() / 16
    assert a[n - 1].storage_offset() * 2 > 2 ** 32
    for M in (3, 70):
        ids = torch.full((M,), n - 1, dtype=torch.int32, device="cuda")
        ids[1] = 0
        t = dict(x=s["x"][:M], a=a, b=b, scale=torch.ones(n, device="cuda"), adapter=ids, w=None, base=None, rank=None)
        print(f"far adapters M={M}", flush=True)
        got = moe.lora_linear(**t, out_dtype=torch.float32)
        few = dict(t, a=a[[0, n - 1]], b=b[[0, n - 1]], scale=t["scale"][:2], adapter=(ids > 0).int())
        check(got, *definition(few, torch.float32), "y")
    del a, b, t, few
    ld = (1 << 31) + 64
    far = torch.zeros(2 * ld + 4096, dtype=torch.bfloat16, device="cuda")
    rows = lambda o, n: far.as_strided((3, n), (ld, 1), o)
    s, dt = make_lora(3, 136, 64, 16, 2, base="bf16")
    s["x"], s["base"] = rows(0, 64).copy_(s["x"]), rows(1024, 136).copy_(s["base"])
    print("far rows", flush=True)
    out = moe.lora_linear(**s, out=rows(2048, 136))
    check(out, *definition(s, dt), "far rows")


def test_lora_streams_graphs_and_two_at_once():
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    cases = []
    for M, w, base in ((1, True, None), (1, False, "f32"), (20, True, None), (64, False, "bf16"), (300, True, "bf16"), (1000, False, "f32")):
        s, dt = make_lora(M, 264, 512, 32, 4, w=w, base=base, seed=M)
        cases.append((s, moe.lora_linear(**s), torch.empty(M, 264, dtype=dt, device="cuda"),
                      torch.empty(moe.lora_workspace_bytes(M, 32), dtype=torch.uint8, device="cuda")))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    print("streams", flush=True)
    for _ in range(5):
        for (s, _, out, ws), st in zip(cases, streams):
            moe.lora_linear(**s, out=out, ws=ws, stream=st)
    torch.cuda.synchronize()
    for _, want, out, _ in cases:
        assert torch.equal(out, want)
    print("graphs", flush=True)
    for s, want, out, ws in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[0]):
            moe.lora_linear(**s, out=out, ws=ws)
        first = s["adapter"].clone()
        for i in range(4):
            s["adapter"].copy_((first + i) % 5 - 1)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, moe.lora_linear(**s)), i
            ws.fill_(255)


# ---- together -----------------------------------------------------------------------------------------
@pytest.mark.parametrize("wdt", ["bf16", "int4", "fp8"])
@pytest.mark.parametrize("T", [1, 6, 16])
def test_decode_step_of_adapters_norm_and_layer(wdt, T):
    """A decode step of a small batch: the projection before the layer with each request's adapter, the norm with the
    residual, the layer; eager against the definitions, then captured and replayed."""
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    from expert_offload_cache_amd.layer import DeviceLayer

    d, f, E, k, K, r, n = 384, 256, 10, 3, 256, 16, 5
    import synth
    from gpu_util import small_workload

    li = synth.layer_inputs(small_workload("bf16", wdt, d, f, E, k, shared=True), T, seed=T)
    weight = torch.from_numpy(1 + 0.1 * np.random.default_rng(1).normal(size=d)).bfloat16()
    layer = DeviceLayer.from_inputs(li, norm_weight=weight.view(torch.int16).numpy().view(np.uint16))
    s, dt = make_lora(T, d, K, r, n, seed=T, none=0.3)
    residual = torch.randn(T, d, device="cuda").bfloat16()
    bufs, rows = layer.buffers_few(T), torch.empty(T, d, dtype=dt, device="cuda")
    ws = torch.empty(moe.lora_workspace_bytes(T, r), dtype=torch.uint8, device="cuda")

    def step():
        moe.lora_linear(**s, out=rows, ws=ws)
        return layer.forward_few(rows, bufs=bufs, residual=residual)

    print(f"step {wdt} T={T}", flush=True)
    out = step()
    torch.cuda.synchronize()
    check(rows, *definition(s, dt), "projection")
    # the norm and the layer from the rows that the step before them left
    y, kept, _, _ = moe.add_rmsnorm(rows, layer.norm_weight, 1e-6, residual=residual)
    assert torch.equal(out["x"], y) and torch.equal(out["residual"], kept)
    x = out["x"].view(torch.int16).cpu().numpy().view(np.uint16)
    ref, bound, idx, _ = layer_bound(li, x)
    assert np.array_equal(out["topk_idx"].cpu().numpy(), idx)
    check_y(out["y"], ref, bound, "layer")
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for i in range(4):
        s["x"].copy_(s["x"].roll(1, 0) * 1.25)
        residual.mul_(0.5)
        g.replay()
        torch.cuda.synchronize()
        got = _clone(out)
        eager = step()
        for name in ("y", "x", "residual", "topk_idx", "topk_w"):
            assert torch.equal(got[name], eager[name]), name
