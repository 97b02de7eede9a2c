"""moe_layer_few at widths whose row blocks of y are no multiple of the 8 lists of work items and whose sums are cut into several
runs, so that run 0 joins what workgroups of other lists' items leave.  Definition and bounds: test_gpu_few.py."""
import numpy as np
import pytest

from gpu_util import need_gpu
from test_gpu_few import check_y, layer_bound, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,wdt,d,f,E,k,shared,T", [
    # row blocks x runs:
    ("f32", "f32", 64, 128, 8, 2, False, 16),       # 4 x 2
    ("bf16", "bf16", 2880, 416, 12, 4, False, 16),  # 45 x 4
    ("bf16", "bf16", 2880, 2080, 5, 4, False, 3),   # 45 x 4
    ("bf16", "bf16", 2816, 416, 8, 4, True, 16),    # 44 x 4
    ("bf16", "bf16", 2304, 416, 9, 4, False, 16),   # 36 x 4
    ("bf16", "bf16", 1152, 448, 10, 4, False, 16),  # 18 x 8
    ("bf16", "bf16", 1472, 1216, 9, 2, True, 9),    # 23 x 8
    ("bf16", "int4", 640, 1024, 12, 3, True, 16),   # 10 x 4
    ("bf16", "fp8", 1152, 1152, 10, 2, False, 16),  # 18 x 4
])
def test_joined_runs_of_other_lists(act, wdt, d, f, E, k, shared, T):
    need_gpu()
    import torch

    li, layer = make(act, wdt, d, f, E, k, shared, T)
    x = layer.x_to_device(li.x)
    bufs = layer.buffers_few(T)
    print(f"few {wdt} d={d} f={f} E={E} k={k} T={T}", flush=True)
    out = layer.forward_few(x, bufs=bufs)
    torch.cuda.synchronize()
    assert int(bufs["ws"][:4].view(torch.int32)) == 0
    ref, bound, idx, _ = layer_bound(li, li.x)
    assert np.array_equal(out["topk_idx"].cpu().numpy(), idx)
    check_y(out["y"], ref, bound, wdt)
    first = out["y"].clone()
    for _ in range(20):
        assert torch.equal(layer.forward_few(x, bufs=bufs)["y"], first)
    assert int(bufs["ws"][:4].view(torch.int32)) == 0
