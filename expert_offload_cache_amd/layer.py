"""Device-resident MoE layer: weights packed into an HBM slot pool, forward = the four libmoe calls.

Marshalling only: packing happens in libmoe (moe_pack_expert), compute in its kernels.
"""
from __future__ import annotations

from typing import Optional

import numpy as np

from . import (_new, add_rmsnorm, combine, expert_ffn_fp8, expert_ffn_grouped, layer_few, layer_few_workspace_bytes,
               pack_expert, permute_workspace, route_permute, slot_bytes, workspace_bytes, y_perm_dtype, WDT)
from ._lib import MOE_BF16, MOE_F32


def _to_device(a: np.ndarray, dtype: str, device):
    import torch

    if dtype == "bf16":
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(device).view(torch.bfloat16)
    if dtype == "f32":
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(device)
    raise ValueError(dtype)


def _expert_arrays(ew):
    return (ew.wg, ew.wu, ew.wd, getattr(ew, "sg", None), getattr(ew, "su", None), getattr(ew, "sd", None))


def pack_pool(experts, slot_of_expert, n_slots: int, d: int, f: int, wdt: str) -> np.ndarray:
    """Host image of a slot pool: expert e packed into slot slot_of_expert[e]."""
    stride = slot_bytes(d, f, wdt)
    pool = np.zeros((n_slots, stride), dtype=np.uint8)
    for e, ew in enumerate(experts):
        s = int(slot_of_expert[e])
        if s >= 0:
            pack_expert(wdt, d, f, *_expert_arrays(ew), out=pool[s])
    return pool


class DeviceLayer:
    """One MoE layer whose routed experts sit in HBM slots (all resident).  With `norm_weight` the
    layer begins with the norm (and, in forward, the residual's addition); experts with fp8 weights
    then take their rows in 8 bits from the norm itself."""

    def __init__(self, d, f, E, k, act: str, wdt: str, w_router, bias, experts, shared=None,
                 slot_of_expert=None, n_slots: Optional[int] = None, device="cuda", norm_weight=None,
                 norm_eps: float = 1e-6):
        import torch

        self.d, self.f, self.E, self.k, self.act, self.wdt = d, f, E, k, act, wdt
        self.device = device
        self.stride = slot_bytes(d, f, wdt)
        if slot_of_expert is None:
            slot_of_expert = np.arange(E, dtype=np.int32)
        self.n_slots = int(n_slots if n_slots is not None else max(int(np.max(slot_of_expert)) + 1, 1))
        host = pack_pool(experts, slot_of_expert, self.n_slots, d, f, wdt)
        self.pool = torch.from_numpy(host.reshape(-1)).to(device)
        del host
        self.slot_of_expert = torch.from_numpy(np.ascontiguousarray(slot_of_expert, dtype=np.int32)).to(device)
        self.w_router = _to_device(w_router, act, device)
        self.bias = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).to(device)
        self.shared = None
        if shared is not None:
            img = pack_expert(wdt, d, f, *_expert_arrays(shared))
            self.shared = torch.from_numpy(img).to(device)
        self.act_code = MOE_BF16 if act == "bf16" else MOE_F32
        self.norm_weight = None if norm_weight is None else _to_device(norm_weight, act, device)
        self.norm_eps = norm_eps

    @classmethod
    def from_inputs(cls, li, device="cuda", n_slots=None, norm_weight=None, norm_eps: float = 1e-6):
        wl = li.wl
        return cls(wl.d, wl.f, wl.E, wl.k, wl.act, wl.wdt, li.w_router, li.bias, li.experts, li.shared,
                   li.slot_of_expert, n_slots=n_slots, device=device, norm_weight=norm_weight, norm_eps=norm_eps)

    def x_to_device(self, x: np.ndarray):
        return _to_device(x, self.act, self.device)

    def workspace(self, T: int, stream=None):
        import torch

        n = workspace_bytes(T, self.d, self.f, self.E, self.k, self.shared is not None, self.act_code, WDT[self.wdt])
        return _new(stream, self.device, (n, torch.uint8), zero=True)[0]

    def buffers(self, T: int):
        """Outputs of a T-token forward allocated once (a serving loop's buffers), on the current stream: forward(...,
        bufs=...) writes into them, so each call overwrites the previous call's results."""
        import torch

        dev, k, E, d = self.device, self.k, self.E, self.d
        rows = T * k + (T if self.shared is not None else 0)
        act = torch.bfloat16 if self.act == "bf16" else torch.float32
        i32 = dict(dtype=torch.int32, device=dev)
        norm = {}
        if self.norm_weight is not None:
            q = self.wdt == "fp8"
            norm["norm"] = (torch.empty((T, d), dtype=act, device=dev), torch.empty((T, d), dtype=act, device=dev),
                            torch.empty((T, d), dtype=torch.float8_e4m3fn, device=dev) if q else None,
                            torch.empty((T, d // 128), dtype=torch.float32, device=dev) if q else None)
        return dict(
            **norm,
            route=(torch.empty((T, k), **i32), torch.empty((T, k), dtype=torch.float32, device=dev),
                   torch.empty((T, E), dtype=torch.float32, device=dev), torch.empty(E, **i32),
                   torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty(T * k, **i32)),
            y_perm=torch.empty((rows, d), dtype=y_perm_dtype(act, T), device=dev),
            y=torch.empty((T, d), dtype=act, device=dev),
            ws=self.workspace(T), pws=permute_workspace(T, k, E, dev))

    def buffers_few(self, T: int):
        """Outputs and workspace of a T-token forward_few (at most 16), allocated once, on the current stream: a call
        on another stream comes after it."""
        import torch

        act = torch.bfloat16 if self.act == "bf16" else torch.float32
        dev = self.device
        norm = {}
        if self.norm_weight is not None:
            norm["norm"] = tuple(torch.empty((T, self.d), dtype=act, device=dev) for _ in range(2)) + (None, None)
        n = layer_few_workspace_bytes(T, self.d, self.f, self.E, self.k, self.shared is not None, self.wdt)
        return dict(**norm, few=(torch.empty((T, self.d), dtype=act, device=dev),
                                 torch.empty((T, self.k), dtype=torch.int32, device=dev),
                                 torch.empty((T, self.k), dtype=torch.float32, device=dev)),
                    ws=torch.zeros(max(n, 1), dtype=torch.uint8, device=dev))

    def forward_few(self, x, forced_idx=None, stream=None, slot_of_expert=None, bufs=None, residual=None):
        """forward for at most 16 tokens through layer_few: two launches instead of six, no intermediate
        rows.  Returns a dict with y [T, d], topk_idx, topk_w and, as forward, x, residual and ws, whose first 4
        bytes are the status word (int32, to be looked at: see layer_few).  With `bufs` (from buffers_few(T)) the
        outputs are written there."""
        b = bufs or {}
        kept = None
        if self.norm_weight is not None:
            out = b.get("norm")
            if out is not None and residual is None:
                out = (out[0], None, None, None)
            x, kept, _, _ = add_rmsnorm(x, self.norm_weight, self.norm_eps, residual=residual, out=out, stream=stream)
        elif residual is not None:
            raise ValueError("a residual needs a layer with a norm weight")
        soe = self.slot_of_expert if slot_of_expert is None else slot_of_expert
        few = layer_few(x, self.w_router, self.bias, self.k, soe, self.pool, self.n_slots, self.stride, self.wdt, self.f,
                        shared_w=self.shared, forced_idx=forced_idx, out=b.get("few"), ws=b.get("ws"), stream=stream)
        y, idx, w = few
        return dict(y=y, topk_idx=idx, topk_w=w, ws=few.ws, x=x, residual=kept)

    def forward(self, x, forced_idx=None, ws=None, stream=None, slot_of_expert=None, bufs=None, residual=None):
        """x: device tensor [T, d].  Returns a dict of every intermediate and y [T, d].  With
        `bufs` (from buffers(T)) the outputs are written there instead of new tensors.  A layer with
        a norm weight takes `residual` [T, d] (or None) and also returns `residual`, the sum kept for
        the next layer, and `x`, the normed rows that the router saw."""
        T = x.shape[0]
        b = bufs or {}
        kept = x8 = x8_scale = None
        if self.norm_weight is not None:
            out = b.get("norm")
            if out is not None and residual is None:
                out = (out[0], None, out[2], out[3])
            x, kept, x8, x8_scale = add_rmsnorm(x, self.norm_weight, self.norm_eps, residual=residual,
                                                emit="both" if self.wdt == "fp8" else "y", out=out, stream=stream)
        elif residual is not None:
            raise ValueError("a residual needs a layer with a norm weight")
        pws = b["pws"] if "pws" in b else permute_workspace(T, self.k, self.E, x.device, stream)
        idx, w, logits, counts, offsets, perm, inv = route_permute(x, self.w_router, self.bias, self.k,
                                                                  forced_idx=forced_idx, out=b.get("route"),
                                                                  stream=stream, ws=pws)
        if ws is None:
            ws = b["ws"] if "ws" in b else self.workspace(T, stream)
        soe = self.slot_of_expert if slot_of_expert is None else slot_of_expert
        if x8 is not None:
            y_perm, ws = expert_ffn_fp8(x8, x8_scale, perm, offsets, counts, soe, self.pool, self.n_slots, self.stride,
                                        self.f, self.k, shared_w=self.shared, y_perm=b.get("y_perm"),
                                        y_dtype=y_perm_dtype(x.dtype, T), ws=ws, stream=stream)
        else:
            y_perm, ws = expert_ffn_grouped(x, perm, offsets, counts, soe, self.pool, self.n_slots, self.stride,
                                            self.wdt, self.f, self.k, shared_w=self.shared, y_perm=b.get("y_perm"),
                                            y_dtype=y_perm_dtype(x.dtype, T),
                                            ws=ws, stream=stream)
        y = combine(y_perm, w, inv, self.k, self.shared is not None, x.dtype, y=b.get("y"), stream=stream)
        return dict(y=y, topk_idx=idx, topk_w=w, logits=logits, counts=counts, offsets=offsets, perm=perm,
                    inv_perm=inv, y_perm=y_perm, ws=ws, x=x, residual=kept)
