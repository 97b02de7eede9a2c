"""moe_layer_few against the layer's definition in 64 bits: every weight type, 1 to 16 tokens, odd sizes, absent and
masked experts, forced ids, repeated and captured calls.

The tolerance of an element of y is a bound, derived here and not fitted: binary32 sums of n terms are off
by at most n 2^-24 of the sum of their magnitudes (n: the additions that follow one another); an element of h is
rounded (or quantised) from a value that is off by its sums' bound, so where that interval crosses a border of the
type the whole step counts; the result is rounded once more, by half a step at most."""
import numpy as np
import pytest

import synth
from gpu_util import need_gpu, small_workload, y_to_f64
from oracle import fp8
from oracle.numerics import act_to_f64, bf16_to_f64, expert_to_f64, round_to_bf16
from oracle.router import route

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _quant_as(rows, like):
    """rows quantised with the scales of `like` -> the values they stand for."""
    out = np.empty_like(rows)
    for c in range(0, rows.shape[1], 128):
        s = (np.abs(like[:, c:c + 128]).max(1) / 448.0).astype(np.float32)
        s = np.maximum(s, np.float32(2.0 ** -126)).astype(np.float64)
        r = (1.0 / s).astype(np.float32).astype(np.float64)
        out[:, c:c + 128] = fp8.round_e4m3(np.clip(rows[:, c:c + 128] * r[:, None], -463, 463)) * s[:, None]
    return out


def expert_bound(a, ew, act):
    """-> (y, bound): one expert on rows a [n, d] (float64), h held as the layer holds it."""
    wg, wu, wd = expert_to_f64(ew)
    d, f = a.shape[1], wd.shape[1]
    if ew.wdt == "fp8":
        a = fp8.rows_value(*fp8.quantise(a))
    g, u = a @ wg.T, a @ wu.T
    # a wave adds its share of the steps one after the other, each step's 32 products in an order of the
    # instruction's own; then 8 waves' sums; int4 sums hold nibbles as 128 + u and take 136 sum(x) off again
    n = d // 256 + 32 + 8 + 4

    def err(w, scales):
        m = np.abs(a) @ np.abs(w).T
        if ew.wdt == "int4":  # |128 + u| + 136 at most 280 times the scale
            m = 280.0 * np.abs(a) @ np.repeat(bf16_to_f64(scales), 128, axis=1).T
        return n * U * m

    eg, eu = err(wg, ew.sg), err(wu, ew.su)
    sg = 1.0 / (1.0 + np.exp(-g))
    h = g * sg * u
    # |d silu| <= 1.1; the product of the two errors and 8 roundings of the exponential and quotient on top
    eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(g * sg) * eu + 16 * U * np.abs(h)
    if ew.wdt == "fp8":
        hr = fp8.rows_value(*fp8.quantise(h))
        eh = eh + 4 * U * np.abs(h)
        # the group's scale moves with its largest value, by their relative error
        flip = np.abs(_quant_as(h + eh, h) - _quant_as(h - eh, h))
        for c in range(0, f, 128):
            m = np.abs(h[:, c:c + 128])
            rel = (eh[:, c:c + 128].max(1) / np.maximum(m.max(1), 1e-300))[:, None]
            wide = eh[:, c:c + 128] + rel * m
            flip[:, c:c + 128] = np.abs(_quant_as(h[:, c:c + 128] + wide, h[:, c:c + 128]) -
                                        _quant_as(h[:, c:c + 128] - wide, h[:, c:c + 128])) + rel * m
    elif act == "bf16":
        hr = round_to_bf16(h)
        flip = np.abs(round_to_bf16(h + eh) - round_to_bf16(h - eh))
    else:
        hr, flip = h, eh
    y = hr @ wd.T
    m = np.abs(hr) @ np.abs(wd).T
    if ew.wdt == "int4":
        m = 280.0 * np.abs(hr) @ np.repeat(bf16_to_f64(ew.sd), 128, axis=1).T
    return y, flip @ np.abs(wd).T + (f // 32 + 32 + 8 + 4) * U * m


def layer_bound(li, x, forced=None, skip=()):
    """-> (y, bound, idx, gates): the layer in 64 bits; experts in `skip` add nothing."""
    wl = li.wl
    _, idx, gates = route(x, li.w_router, li.bias, wl.act, wl.k, forced)
    a = act_to_f64(x, wl.act)
    y, b = np.zeros_like(a), np.zeros_like(a)
    mag = np.zeros_like(a)
    for e in range(wl.E):
        t, j = np.nonzero(idx == e)
        if len(t) == 0 or e in skip:
            continue
        rows = np.unique(t)
        ye, be = expert_bound(a[rows], li.experts[e], wl.act)
        share = np.array([gates[r][idx[r] == e].sum() for r in rows])[:, None]
        y[rows] += share * ye
        b[rows] += share * (be + 4 * U * np.abs(ye))
        mag[rows] += np.abs(share * ye)
    if li.shared is not None:
        ye, be = expert_bound(a, li.shared, wl.act)
        y += ye
        b += be
        mag += np.abs(ye)
    b += (wl.k + 8) * U * mag
    half = 2.0 ** -8 if wl.act == "bf16" else U
    return y, b + half * (np.abs(y) + b), idx, gates


def check_y(y, ref, bound, what):
    y = y_to_f64(y)
    assert np.isfinite(y).all(), what
    worst = (np.abs(y - ref) / bound).max()
    print(f"{what}: worst error / bound {worst:.3f}, bound / row norm {np.median(np.linalg.norm(bound, axis=1) / np.linalg.norm(ref, axis=1)):.2e}", flush=True)
    assert worst <= 1.0, what


def make(act, wdt, d, f, E, k, shared, T, seed=0, **kw):
    from expert_offload_cache_amd.layer import DeviceLayer

    wl = small_workload(act, wdt, d, f, E, k, shared=shared)
    li = synth.layer_inputs(wl, T, seed=seed)
    return li, DeviceLayer.from_inputs(li, **kw)


CASES = [
    # act, weights, d, f, E, k, shared, tokens
    ("f32", "f32", 64, 128, 8, 2, False, (1, 16, 5)),
    ("f32", "f32", 192, 96, 5, 5, True, (3, 16)),
    ("bf16", "bf16", 64, 64, 4, 1, False, (1, 2, 16)),
    ("bf16", "bf16", 320, 96, 9, 3, True, (1, 7, 16)),
    ("bf16", "bf16", 1024, 416, 70, 6, True, (1, 4, 11)),
    ("bf16", "bf16", 2112, 64, 3, 2, False, (1, 16)),
    ("bf16", "int4", 128, 128, 4, 2, False, (1, 16)),
    ("bf16", "int4", 640, 384, 17, 4, True, (1, 2, 9, 16)),
    ("bf16", "int4", 1408, 256, 6, 3, False, (6,)),
    ("bf16", "fp8", 128, 128, 4, 2, True, (1, 16)),
    ("bf16", "fp8", 1152, 640, 12, 4, True, (1, 5, 16)),
    ("bf16", "fp8", 256, 1152, 20, 8, False, (3,)),
]


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c[:7])) for c in CASES])
def test_against_definition(case):
    need_gpu()
    import torch

    import expert_offload_cache_amd as moe

    act, wdt, d, f, E, k, shared, Ts = case
    li, layer = make(act, wdt, d, f, E, k, shared, max(Ts))
    for T in Ts:
        x = li.x[:T]
        dx = layer.x_to_device(x)
        print(f"few {case[:7]} T={T}", flush=True)
        bufs = layer.buffers_few(T)
        out = layer.forward_few(dx, bufs=bufs)
        torch.cuda.synchronize()
        ref, bound, idx, gates = layer_bound(li, x)
        assert np.array_equal(out["topk_idx"].cpu().numpy(), idx)
        ids, w, _ = moe.route(dx, layer.w_router, layer.bias, k)
        assert torch.equal(out["topk_idx"], ids) and torch.equal(out["topk_w"], w)
        check_y(out["y"], ref, bound, f"{wdt} T={T}")
        assert int(bufs["ws"][:4].view(torch.int32)) == 0
        # the same bits again, from the same workspace
        first = out["y"].clone()
        for _ in range(3):
            again = layer.forward_few(dx, bufs=bufs)
            assert torch.equal(again["y"], first)
