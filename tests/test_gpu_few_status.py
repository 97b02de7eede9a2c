"""The status word of moe_layer_few reaches callers who leave the workspace to the call."""
import pytest

from gpu_util import need_gpu
from test_gpu_few import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wdt", ["bf16", "int4", "fp8"])
@pytest.mark.parametrize("T", [1, 11])
def test_status_without_a_workspace(wdt, T):
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    li, layer = make("bf16", wdt, 128, 128, 4, 2, True, T)
    x = layer.x_to_device(li.x)
    for name, slots, want in (("all there", layer.slot_of_expert, 0), ("none there", torch.full_like(layer.slot_of_expert, -1), 1),
                              ("elsewhere", torch.full_like(layer.slot_of_expert, -2), 0)):
        print(f"{name} {wdt} T={T}", flush=True)
        few = moe.layer_few(x, layer.w_router, layer.bias, 2, slots, layer.pool, layer.n_slots, layer.stride, wdt, 128, shared_w=layer.shared)
        y, idx, w = few
        assert few.status.dtype == torch.int32 and few.status.tolist() == [want]
        out = layer.forward_few(x, slot_of_expert=slots)
        assert torch.equal(out["y"], y) and torch.equal(out["topk_idx"], idx) and torch.equal(out["topk_w"], w)
        assert int(out["ws"][:4].view(torch.int32)) == want
    # a workspace of the caller's, of any type: its own first word, which stays set
    words = torch.zeros(moe.layer_few_workspace_bytes(T, 128, 128, 4, 2, True, wdt) // 8, 2, dtype=torch.int32, device="cuda")
    call = lambda slots: moe.layer_few(x, layer.w_router, layer.bias, 2, slots, layer.pool, layer.n_slots, layer.stride, wdt, 128,
                                       shared_w=layer.shared, ws=words)
    assert call(layer.slot_of_expert).status.tolist() == [0]
    assert call(torch.full_like(layer.slot_of_expert, -1)).status.tolist() == [1]
    few = call(layer.slot_of_expert)
    assert few.status.tolist() == [1] and few.ws is words and few.status.data_ptr() == words.data_ptr()
