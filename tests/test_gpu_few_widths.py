"""moe_layer_few at widths that choose its forms: row blocks of y that are no multiple of the 8 lists of work items, their sums cut
into several runs; every form of launch 2, named by the profile.  Definition and bounds: test_gpu_few.py."""
import numpy as np
import pytest

from gpu_util import need_gpu, rel_err_per_token, y_to_f64
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


FORMS = [
    # act, weights, d, f, E, k, shared, tokens; steps of x held, steps a chunk, row blocks
    ("f32", "f32", 192, 96, 5, 3, True, 3, "0_1_1"),
    ("f32", "f32", 192, 416, 6, 4, False, 16, "0_1_4"),
    ("bf16", "bf16", 1024, 96, 6, 4, True, 1, "4_1_1"),
    ("bf16", "bf16", 960, 800, 6, 4, False, 16, "4_1_4"),
    ("bf16", "bf16", 1600, 64, 6, 4, False, 1, "8_1_1"),
    ("bf16", "bf16", 2048, 128, 6, 4, True, 5, "8_1_1"),
    ("bf16", "bf16", 1600, 800, 6, 4, True, 16, "8_1_4"),
    ("bf16", "bf16", 2048, 416, 8, 4, False, 15, "8_1_4"),
    ("bf16", "bf16", 2112, 64, 6, 4, True, 1, "16_1_1"),
    ("bf16", "bf16", 2112, 800, 6, 4, False, 16, "16_1_4"),
    ("bf16", "bf16", 4096, 416, 5, 4, True, 14, "16_1_4"),
    ("bf16", "bf16", 4160, 64, 6, 4, False, 4, "0_1_1"),
    ("bf16", "bf16", 4160, 800, 6, 4, True, 16, "0_1_4"),
    ("bf16", "int4", 1408, 256, 6, 4, False, 1, "2_2_1"),
    ("bf16", "int4", 1408, 768, 6, 4, True, 16, "2_2_4"),
    ("bf16", "int4", 2048, 1536, 6, 4, False, 9, "2_2_4"),
    ("bf16", "int4", 2176, 256, 6, 4, True, 1, "4_2_1"),
    ("bf16", "int4", 4096, 512, 5, 3, True, 3, "4_2_1"),
    ("bf16", "int4", 2176, 768, 6, 4, False, 16, "4_2_4"),
    ("bf16", "int4", 640, 384, 6, 4, False, 2, "0_1_1"),
    ("bf16", "int4", 4224, 256, 6, 4, True, 2, "0_1_1"),
    ("bf16", "int4", 640, 640, 6, 4, True, 16, "0_1_4"),
    ("bf16", "int4", 4224, 768, 6, 4, False, 13, "0_1_4"),
    ("bf16", "fp8", 1152, 128, 6, 4, True, 1, "2_1_1"),
    ("bf16", "fp8", 1152, 640, 6, 4, False, 16, "2_1_4"),
    ("bf16", "fp8", 2176, 128, 6, 4, False, 1, "4_1_1"),
    ("bf16", "fp8", 2176, 640, 6, 4, True, 16, "4_1_4"),
    ("bf16", "fp8", 4224, 128, 6, 4, True, 3, "0_1_1"),
    ("bf16", "fp8", 4224, 640, 6, 4, False, 16, "0_1_4"),
]


@pytest.mark.parametrize("act,wdt,d,f,E,k,shared,T,form", FORMS, ids=["-".join(map(str, c[1:])) for c in FORMS])
def test_every_form(act, wdt, d, f, E, k, shared, T, form):
    """int4: beside the elements' bound, which counts the nibbles' offset and is wide, a row as a whole: h and y off by half a
    step each (2^-8 of the row's norm), the sums' errors far below (sqrt(n) 2^-24 280, n = 4224: 2^-9.8), flips of h's
    rounding once more: 2^-6 at most."""
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    li, layer = make(act, wdt, d, f, E, k, shared, T, seed=d + T)
    x = layer.x_to_device(li.x)
    bufs = layer.buffers_few(T)
    print(f"few {wdt} d={d} f={f} T={T} {form}", flush=True)
    moe.profile_reset()
    moe.profile_enable(True)
    try:
        out = layer.forward_few(x, bufs=bufs)
        torch.cuda.synchronize()
        moe.profile_collect()
        names = set(moe.profile_results())
    finally:
        moe.profile_enable(False)
        moe.profile_reset()
    assert names == {"few_prepare", f"few_layer_{wdt}_{form}"}
    ref, bound, idx, _ = layer_bound(li, li.x)
    assert np.array_equal(out["topk_idx"].cpu().numpy(), idx)
    check_y(out["y"], ref, bound, wdt)
    if wdt == "int4":
        assert rel_err_per_token(y_to_f64(out["y"]), ref).max() <= 2.0 ** -6
    assert int(bufs["ws"][:4].view(torch.int32)) == 0
