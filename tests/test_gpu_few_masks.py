"""moe_layer_few where a bias of minus infinity leaves a token fewer experts than it chooses, or none: ids and gates are those of
moe_route, masked experts that are chosen all the same count with a gate of zero, and a row without any is NaN as the separate
calls' is."""
import dataclasses

import numpy as np
import pytest

from gpu_util import need_gpu
from test_gpu_few import check_y, layer_bound, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,wdt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "int4"), ("bf16", "fp8")])
@pytest.mark.parametrize("T", [1, 9])
def test_fewer_experts_than_choices(act, wdt, T):
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    d, f, E, k = 256, 128, 10, 4
    li, layer = make(act, wdt, d, f, E, k, True, T)
    x = layer.x_to_device(li.x)
    for live in ([2, 7], [5], []):
        bias = np.full(E, -np.inf, np.float32)
        bias[live] = li.bias[live]
        db = torch.from_numpy(bias).cuda()
        print(f"masks {wdt} T={T} live {live}", flush=True)
        few = moe.layer_few(x, layer.w_router, db, k, layer.slot_of_expert, layer.pool, layer.n_slots, layer.stride, wdt, f, shared_w=layer.shared)
        y, idx, w = few
        ids, gates, _ = moe.route(x, layer.w_router, db, k)
        assert torch.equal(idx, ids) and torch.equal(w.view(torch.int32), gates.view(torch.int32)) and few.status.tolist() == [0]
        if live:
            assert set(live) == set(idx[0, :len(live)].tolist()) and bool((w[:, len(live):] == 0).all())
            ref, bound, _, _ = layer_bound(dataclasses.replace(li, bias=bias), li.x)
            check_y(y, ref, bound, f"live {live}")
        else:
            layer.bias = db
            assert bool(y.isnan().all()) and bool(layer.forward(x)["y"].isnan().all())
