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


def busy(ms=30):
    """Work that keeps the current stream busy for some time."""
    import torch

    a = torch.ones(4096, 4096, device="cuda")
    for _ in range(ms):  # a product of binary32 takes about a millisecond or more
        a = (a @ a) * 2.0 ** -12
    return a


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
        a = busy()
        got = call(stream=s)
        ws = seen.given[-1][-3]  # address, bytes, stream
        assert kept_from(ws, need)
        busy_still = not torch.cuda.current_stream().query()
        side.synchronize()
        assert busy_still, "the current stream was to be busy while the other one ran"
        for g, w in zip(got, want):
            assert torch.equal(g.cpu(), w.cpu())
        monkeypatch.undo()
        torch.cuda.synchronize()
        del a


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
        a = busy()
        got = moe.lora_linear(**s, stream=st)
        assert kept_from(seen.given[-1][-3], need)
        busy_still = not torch.cuda.current_stream().query()
        side.synchronize()
        assert busy_still, "the current stream was to be busy while the other one ran"
        assert torch.equal(got.cpu(), want)
        monkeypatch.undo()
        torch.cuda.synchronize()
        del a
