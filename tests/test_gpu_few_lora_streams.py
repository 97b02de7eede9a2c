"""Calls on another stream than the current one that make their own results and workspaces: what they make belongs to the stream
that they run on, whatever the current stream does before and after."""
import pytest

from gpu_util import need_gpu
from test_gpu_few import make as make_layer
from test_gpu_lora import make as make_lora

pytestmark = pytest.mark.gpu


class Watched:
    """The library, with the addresses that one entry point was given."""

    def __init__(self, lib, name):
        self._lib, self._name, self.given = lib, name, []

    def __getattr__(self, name):
        fn = getattr(self._lib, name)
        if name != self._name:
            return fn

        def call(*args):
            self.given.append(args)
            return fn(*args)

        return call


def busy():
    """Keeps the current stream busy for some time (40 ms or more) and the compute units free: what a call leaves to the current
    stream comes late (unless the streams happen to share a hardware queue)."""
    import torch

    torch.cuda._sleep(100_000_000)


def soiled(sizes):
    """Leaves blocks of these sizes, every byte set, to be given out again on the current stream."""
    import torch

    blocks = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    del blocks


def kept_from(address, nbytes, device="cuda"):
    """Whether the current stream's next allocations of that size leave the block alone."""
    import torch

    blocks = [torch.empty(nbytes, dtype=torch.uint8, device=device) for _ in range(8)]
    return all(b.data_ptr() + nbytes <= address or address + nbytes <= b.data_ptr() for b in blocks)


def streams():
    """A stream, and the two forms in which a call takes it."""
    import torch

    s = torch.cuda.Stream()
    return s, [("a Stream", s), ("its handle", s.cuda_stream)]


@pytest.mark.parametrize("wdt,T", [("bf16", 1), ("int4", 9), ("fp8", 16)])
def test_layer_few_makes_its_workspace_on_the_launch_stream(wdt, T, monkeypatch):
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    li, layer = make_layer("bf16", wdt, 256, 256, 9, 3, True, T)
    x = layer.x_to_device(li.x)
    call = lambda **kw: moe.layer_few(x, layer.w_router, layer.bias, 3, layer.slot_of_expert, layer.pool, layer.n_slots, layer.stride, wdt,
                                      256, shared_w=layer.shared, **kw)
    want = [t.clone() for t in call()]
    need = moe.layer_few_workspace_bytes(T, 256, 256, 9, 3, True, wdt)
    side, forms = streams()
    seen = Watched(moe.lib(), "moe_layer_few")
    for name, s in forms:
        soiled([need])
        monkeypatch.setattr(moe, "lib", lambda: seen)
        print(f"layer_few on {name}, {wdt} T={T}", flush=True)
        busy()
        got = call(stream=s)
        ws = seen.given[-1][-3]  # address, bytes, stream
        assert kept_from(ws, need)
        side.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g.cpu(), w.cpu())
        monkeypatch.undo()
        torch.cuda.synchronize()


@pytest.mark.parametrize("M,w,base", [(1, True, None), (20, True, "bf16"), (64, False, "f32"), (200, True, None), (300, False, "bf16")])
def test_lora_linear_makes_its_workspace_on_the_launch_stream(M, w, base, monkeypatch):
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    s, dt = make_lora(M, 264, 512, 32, 4, w=w, base=base, seed=M)
    want = moe.lora_linear(**s).cpu()
    need = moe.lora_workspace_bytes(M, 32)
    side, forms = streams()
    seen = Watched(moe.lib(), "moe_lora_linear")
    for name, st in forms:
        soiled([need])
        monkeypatch.setattr(moe, "lib", lambda: seen)
        print(f"lora_linear on {name}, M={M} w={w} base={base}", flush=True)
        busy()
        got = moe.lora_linear(**s, stream=st)
        assert kept_from(seen.given[-1][-3], need)
        side.synchronize()
        assert torch.equal(got.cpu(), want)
        monkeypatch.undo()
        torch.cuda.synchronize()


def separate_calls(moe, layer, x, residual):
    """The layer's separate calls and those beside them, each with the results and workspaces it makes for itself."""
    l = layer
    fp8 = l.wdt == "fp8"

    def run(s):
        out = {}
        y, h, q, qs = moe.add_rmsnorm(x, l.norm_weight, residual=residual, emit="both" if fp8 else "y", stream=s)
        out.update(norm=y, sum=h)
        rows, rs = moe.quant_fp8(y, stream=s)
        out.update(rows=rows, rows_scale=rs)
        out["product"] = moe.gemm_fp8(rows, rs, rows, run.wscale, stream=s)
        idx, w, logits = moe.route(y, l.w_router, l.bias, l.k, stream=s)
        counts, offsets, perm, inv = moe.permute(idx, l.E, stream=s)
        out.update(idx=idx, gate=w, logits=logits, counts=counts, offsets=offsets, perm=perm, inv=inv)
        if fp8:
            out["experts"], out["ws"] = moe.expert_ffn_fp8(q, qs, perm, offsets, counts, l.slot_of_expert, l.pool, l.n_slots, l.stride, l.f, l.k,
                                                            shared_w=l.shared, stream=s)
        else:
            out["experts"], out["ws"] = moe.expert_ffn_grouped(y, perm, offsets, counts, l.slot_of_expert, l.pool, l.n_slots, l.stride, l.wdt,
                                                                l.f, l.k, shared_w=l.shared, stream=s)
        out["y"] = moe.combine(out["experts"], w, inv, l.k, l.shared is not None, x.dtype, stream=s)
        return out

    run.wscale = None
    return run


@pytest.mark.parametrize("wdt,T", [("bf16", 3), ("int4", 40), ("fp8", 100)])
def test_separate_calls_make_their_results_on_the_launch_stream(wdt, T):
    need_gpu()
    import numpy as np
    import torch

    import expert_offload_cache_amd as moe
    import synth
    from expert_offload_cache_amd.layer import DeviceLayer
    from gpu_util import small_workload

    li = synth.layer_inputs(small_workload("bf16", wdt, 256, 128, 10, 3, shared=True), T, seed=T)
    weight = torch.from_numpy(1 + 0.1 * np.random.default_rng(1).normal(size=256)).bfloat16()
    layer = DeviceLayer.from_inputs(li, norm_weight=weight.view(torch.int16).numpy().view(np.uint16))
    x, residual = layer.x_to_device(li.x), torch.randn(T, 256, device="cuda").bfloat16()
    calls = separate_calls(moe, layer, x, residual)
    calls.wscale = torch.rand((T + 127) // 128, 2, device="cuda")
    whole = lambda s: layer.forward(x, residual=residual, stream=s)
    side, forms = streams()
    for what, run in (("separate", calls), ("forward", whole)):
        eager = torch.cuda.Stream()
        with torch.cuda.stream(eager):
            run(eager)
            torch.cuda.synchronize()
            want = {n: t.clone() for n, t in run(eager).items() if t is not None}
        torch.cuda.synchronize()
        sizes = [t.nbytes for t in want.values()]
        for name, s in forms:
            soiled(sizes)
            print(f"{what} on {name}, {wdt} T={T}", flush=True)
            busy()
            got = {n: t for n, t in run(s).items() if t is not None}
            with torch.cuda.stream(side):  # (ordered after the calls, not after the current stream)
                status = int(got["ws"][:4].view(torch.int32))
            same = {n: torch.equal(got[n].view(torch.uint8), want[n].view(torch.uint8)) for n in want if n not in ("ws", "residual", "x")}
            assert all(same.values()) and status == 0, (same, status)
            places = [(t.data_ptr(), t.nbytes) for t in got.values() if t.data_ptr() not in (x.data_ptr(), residual.data_ptr())]
            del got
            assert all(kept_from(*p) for p in places)
            torch.cuda.synchronize()
