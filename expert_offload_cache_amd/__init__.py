"""Routed-expert MoE layer behind an HBM expert-slot cache, on MI355X (gfx950).

Thin Python binding of libmoe (include/moe.h): argument marshalling only.  Every step
of the layer runs in the library's HIP kernels; device memory and streams come from
PyTorch.  There is no CPU fallback: calls fail when libmoe.so is missing.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import numpy as np

from ._lib import (MOE_BF16, MOE_F32, MOE_FP8_B128, MOE_INT4_G128, MoeError, check, lib)

__all__ = ["route", "permute", "permute_workspace", "permute_workspace_bytes", "route_permute", "expert_ffn_grouped", "expert_ffn_grouped_noalloc", "expert_ffn_fp8", "combine",
           "layer_few", "layer_few_workspace_bytes", "add_rmsnorm", "quant_fp8", "gemm_fp8", "lora_linear", "lora_workspace_bytes",
           "slot_bytes", "pack_expert", "workspace_bytes", "hybrid_split", "SlotCache", "pinned_alloc", "pinned_free", "profile_enable",
           "profile_collect", "profile_results", "profile_reset", "MoeError", "WDT", "lib"]

WDT = {"f32": MOE_F32, "bf16": MOE_BF16, "int4": MOE_INT4_G128, "fp8": MOE_FP8_B128}


def _torch():
    import torch

    return torch


def _act(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    raise TypeError(f"activations must be float32 or bfloat16, got {t.dtype}")


def _y_code(t) -> int:
    """Element type code of a y_perm tensor (float32 or bfloat16)."""
    torch = _torch()
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    raise TypeError(f"y_perm must be float32 or bfloat16, got {t.dtype}")


def y_perm_dtype(act_dtype, T: int):
    """The y_perm element type the layer orchestration uses: bfloat16 for bf16 prefill (more than 64
    tokens, the matrix-core path), where the intermediate rows may be bf16; float32 otherwise."""
    torch = _torch()
    return torch.bfloat16 if act_dtype == torch.bfloat16 and T > 64 else torch.float32


def _p(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _s(stream) -> Optional[int]:
    if stream is None:
        # the current device's current stream, as a handle: torch.cuda.current_stream() builds a Stream
        # object around it, 2.9 us of a call whose kernel may take 4
        C = _torch()._C
        return C._cuda_getCurrentRawStream(C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _new(stream, device, *specs, zero=False):
    """Tensors (shape, dtype) that a call makes for itself, uninitialised or zero-filled, on the stream that it launches on: a
    fill comes before the kernels, and the memory is neither in use by earlier work of the current stream nor given back to
    it while the kernels run.  On another stream than the current one they are marked as used by that one too: the caller
    may drop a result while its work there (after the launch stream's) is pending."""
    torch = _torch()
    make = torch.zeros if zero else torch.empty
    handle = None if stream is None else _s(stream)
    if handle is None or handle == _s(None):
        return [make(shape, dtype=dtype, device=device) for shape, dtype in specs]
    if handle == 0:
        side = torch.cuda.default_stream(device)
    else:
        side = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(handle, device=device)
    user = torch.cuda.current_stream(device)
    with torch.cuda.stream(side):
        ts = [make(shape, dtype=dtype, device=device) for shape, dtype in specs]
    for t in ts:
        t.record_stream(user)
    return ts


def _contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors passed to libmoe must be contiguous")


# ---------------------------------------------------------------------------------------------
# hot-path calls
# ---------------------------------------------------------------------------------------------
def route(x, w_router, bias, k: int, forced_idx=None, out=None, stream=None):
    """-> (topk_idx int32 [T,k], topk_w f32 [T,k], logits f32 [T,E])."""
    torch = _torch()
    _contig(x, w_router, bias, forced_idx)
    T, d = x.shape
    E = w_router.shape[0]
    if out is None:
        f32 = torch.float32
        out = tuple(_new(stream, x.device, ((T, k), torch.int32), ((T, k), f32), ((T, E), f32)))
    idx, w, logits = out
    check(lib().moe_route(_p(x), _act(x), T, d, _p(w_router), _p(bias), E, k, _p(forced_idx), _p(idx), _p(w),
                          _p(logits), _s(stream)))
    return idx, w, logits


def permute_workspace_bytes(T: int, k: int, E: int) -> int:
    return int(lib().moe_permute_workspace_bytes(T, k, E))


def permute_workspace(T: int, k: int, E: int, device, stream=None):
    """Device scratch for a split sort of T*k pairs (None when one workgroup sorts), made on `stream`."""
    n = permute_workspace_bytes(T, k, E)
    return _new(stream, device, (n, _torch().uint8))[0] if n else None


def permute(topk_idx, E: int, out=None, stream=None, ws=None):
    """-> (counts [E], offsets [E+1], perm [T*k], inv_perm [T*k]) int32.  ws: permute_workspace or None."""
    torch = _torch()
    _contig(topk_idx)
    T, k = topk_idx.shape
    if out is None:
        i32 = torch.int32
        out = tuple(_new(stream, topk_idx.device, (E, i32), (E + 1, i32), (T * k, i32), (T * k, i32)))
    c, o, p, ip = out
    check(lib().moe_permute(_p(topk_idx), T, k, E, _p(c), _p(o), _p(p), _p(ip), _p(ws),
                            0 if ws is None else ws.numel(), _s(stream)))
    return c, o, p, ip


def route_permute(x, w_router, bias, k: int, forced_idx=None, out=None, stream=None, ws=None):
    """route then permute as one call -> (topk_idx, topk_w, logits, counts, offsets, perm, inv_perm).
    ws: permute_workspace(T, k, E) or None (then a large batch sorts in one workgroup)."""
    torch = _torch()
    _contig(x, w_router, bias, forced_idx)
    T, d = x.shape
    E = w_router.shape[0]
    if out is None:
        i32, f32 = torch.int32, torch.float32
        out = tuple(_new(stream, x.device, ((T, k), i32), ((T, k), f32), ((T, E), f32), (E, i32), (E + 1, i32), (T * k, i32),
                         (T * k, i32)))
    idx, w, logits, c, o, p, ip = out
    check(lib().moe_route_permute(_p(x), _act(x), T, d, _p(w_router), _p(bias), E, k, _p(forced_idx), _p(idx),
                                  _p(w), _p(logits), _p(c), _p(o), _p(p), _p(ip), _p(ws),
                                  0 if ws is None else ws.numel(), _s(stream)))
    return out


def workspace_bytes(T, d, f, E, k, has_shared, act: int, wdt: int) -> int:
    return int(lib().moe_workspace_bytes(T, d, f, E, k, int(bool(has_shared)), act, wdt))


def _expert_tensors(T, d, f, E, k, wdt, perm, offsets, counts, slot_of_expert, slot_pool, n_slots, slot_stride, shared_w,
                    y_perm) -> None:
    """Checks that the kernels of a grouped expert call stay inside its tensors (the library has their addresses alone)."""
    i32 = _torch().int32
    if not (perm.dtype == offsets.dtype == counts.dtype == slot_of_expert.dtype == i32 and perm.numel() >= T * k
            and offsets.numel() > E and slot_of_expert.numel() >= E):
        for name, t, n in (("perm", perm, T * k), ("offsets", offsets, E + 1), ("counts", counts, E),
                           ("slot_of_expert", slot_of_expert, E)):
            if t.dtype != i32 or t.numel() < n:
                raise ValueError(f"{name} must be int32 of {n} elements at least, got {t.dtype} {list(t.shape)}")
    _contig(perm, offsets, counts, slot_of_expert, y_perm, slot_pool, shared_w)
    _y_code(y_perm)
    rows, slot = T * k, slot_bytes(d, f, wdt)
    if shared_w is not None:
        rows += T
        if shared_w.nbytes < slot:
            raise ValueError(f"shared_w must hold {slot} bytes, got {shared_w.nbytes}")
    if y_perm.numel() < rows * d:
        raise ValueError(f"y_perm must hold {rows} rows of {d}, got {list(y_perm.shape)}")
    if slot_pool.nbytes < (n_slots - 1) * slot_stride + slot:
        raise ValueError(f"slot_pool must hold {n_slots} slots of {slot_stride} bytes, got {slot_pool.nbytes} bytes")


def expert_ffn_grouped(x, perm, offsets, counts, slot_of_expert, slot_pool, n_slots: int, slot_stride: int,
                       wdt: str, f: int, k: int, shared_w=None, y_perm=None, ws=None, stream=None, y_dtype=None):
    """Grouped SwiGLU experts through the slot table. -> (y_perm [T*k (+T), d], ws).  y_perm's element
    type is that of the given tensor (float32, or bfloat16 with bf16 activations), else y_dtype
    (a torch dtype, default float32)."""
    torch = _torch()
    _contig(x)
    T, d = x.shape
    E = counts.shape[0]
    act = _act(x)
    rows = T * k + (T if shared_w is not None else 0)
    if y_perm is None:
        y_perm, = _new(stream, x.device, ((rows, d), y_dtype or torch.float32))
    _expert_tensors(T, d, f, E, k, wdt, perm, offsets, counts, slot_of_expert, slot_pool, n_slots, slot_stride, shared_w,
                    y_perm)
    if ws is None:
        need = workspace_bytes(T, d, f, E, k, shared_w is not None, act, WDT[wdt])
        ws, = _new(stream, x.device, (need, torch.uint8), zero=True)
    check(lib().moe_expert_ffn_grouped(_p(x), act, T, d, f, E, k, _p(perm), _p(offsets), _p(counts),
                                       _p(slot_of_expert), n_slots, _p(slot_pool), slot_stride, WDT[wdt],
                                       _p(shared_w), _p(y_perm), _y_code(y_perm), _p(ws), ws.numel(), _s(stream)))
    return y_perm, ws


def expert_ffn_grouped_noalloc(x, perm, offsets, counts, slot_of_expert, slot_pool, n_slots: int,
                               slot_stride: int, wdt: str, f: int, k: int, y_perm, shared_w=None, status=None,
                               stream=None):
    """expert_ffn_grouped through moe_expert_ffn_grouped_noalloc: no workspace, the library's
    per-GPU scratch instead; y_perm must be given.  status: device int32 tensor or None."""
    _contig(x)
    T, d = x.shape
    E = counts.shape[0]
    _expert_tensors(T, d, f, E, k, wdt, perm, offsets, counts, slot_of_expert, slot_pool, n_slots, slot_stride, shared_w,
                    y_perm)
    if status is not None and (status.dtype != _torch().int32 or status.numel() < 1):
        raise ValueError(f"status must be an int32 tensor, got {status.dtype} {list(status.shape)}")
    check(lib().moe_expert_ffn_grouped_noalloc(_p(x), _act(x), T, d, f, E, k, _p(perm), _p(offsets), _p(counts),
                                               _p(slot_of_expert), n_slots, _p(slot_pool), slot_stride, WDT[wdt],
                                               _p(shared_w), _p(y_perm), _y_code(y_perm), _p(status), _s(stream)))
    return y_perm


def _on_current_device(*ts) -> None:
    """The library launches on the current device: every tensor has to live there."""
    dev = -1
    for t in ts:
        if t is not None:
            if dev < 0 <= t.get_device():
                dev = _torch()._C._cuda_getDevice()
            if dev < 0 or t.get_device() != dev:
                raise ValueError(f"tensors must be on the current GPU, got {t.device}")


def _rows(name, t, shape, dtype) -> int:
    """Checks a [T, d] tensor of dense rows; -> elements from a row to the next."""
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    ld, inner = t.stride()
    if inner != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the elements of a row must lie next to each other")
    return ld if shape[0] > 1 else shape[1]


def _dense(name, t, shape, dtype) -> None:
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")


def _quantised_out(x, shape, q, scale, stream):
    """The given (or new) e4m3 rows and scales of `shape` -> (q, scale, elements from a row of q to the next)."""
    torch = _torch()
    groups = (shape[0], (shape[1] + 127) // 128)
    if q is None and scale is None:
        q, scale = _new(stream, x.device, (shape, torch.float8_e4m3fn), (groups, torch.float32))
    elif q is None or scale is None:
        raise ValueError("q and scale come together")
    ldq = _rows("q", q, shape, torch.float8_e4m3fn)
    _dense("scale", scale, groups, torch.float32)
    return q, scale, ldq


def add_rmsnorm(x, weight, eps: float = 1e-6, residual=None, emit: str = "y", out=None, stream=None):
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight, rows [T, d] (moe_add_rmsnorm).
    emit: "y" (rows in x's type), "fp8" (e4m3 rows and their scales) or "both".
    out: the returned tuple's tensors to write into (None where not emitted).
    -> (y, h, q, scale), None where there is none (h: without a residual)."""
    torch = _torch()
    act = _act(x)
    shape, dt = x.shape, x.dtype
    T, d = shape
    if emit not in ("y", "fp8", "both"):
        raise ValueError(f'emit must be "y", "fp8" or "both", got {emit!r}')
    if out is None:
        y = _new(stream, x.device, (shape, dt))[0] if emit != "fp8" else None
        h = _new(stream, x.device, (shape, dt))[0] if residual is not None else None
        q = scale = None
    else:
        y, h, q, scale = out
        if (y is None) != (emit == "fp8"):
            raise ValueError(f"emit {emit!r} and out's y do not agree")
        if emit == "y" and (q is not None or scale is not None):
            raise ValueError('out holds q or scale, but emit is "y"')
    if (residual is None) != (h is None):
        raise ValueError("a residual and its sum in out come together")
    ldr = ldh = ldy = ldq = 0
    if residual is not None:
        ldr, ldh = _rows("residual", residual, shape, dt), _rows("h", h, shape, dt)
    if y is not None:
        ldy = _rows("y", y, shape, dt)
    if emit != "y":
        q, scale, ldq = _quantised_out(x, shape, q, scale, stream)
    w_code = act if weight.dtype == dt else MOE_F32
    _dense("weight", weight, (d,), dt if w_code == act else torch.float32)
    _on_current_device(x, weight, residual, y, h, q, scale)
    check(lib().moe_add_rmsnorm(_p(x), act, T, d, _rows("x", x, shape, dt), _p(residual), ldr, _p(weight), w_code, eps,
                                _p(h), ldh, _p(y), ldy, _p(q), ldq, _p(scale), _s(stream)))
    return y, h, q, scale


def quant_fp8(x, out=None, stream=None):
    """Rows [T, d] -> (q e4m3 [T, d], scale f32 [T, ceil(d / 128)]) (moe_quant_fp8)."""
    act = _act(x)
    shape = x.shape
    T, d = shape
    q, scale, ldq = _quantised_out(x, shape, *(out if out is not None else (None, None)), stream)
    _on_current_device(x, q, scale)
    check(lib().moe_quant_fp8(_p(x), act, T, d, _rows("x", x, shape, x.dtype), _p(q), ldq, _p(scale), _s(stream)))
    return q, scale


def gemm_fp8(a, a_scale, w, w_scale, out_dtype=None, out=None, stream=None):
    """c [M, N] = rows a (e4m3 [M, K], scales [M, ceil(K/128)]) times w transposed (e4m3 [N, K],
    scales [ceil(N/128), ceil(K/128)]) (moe_gemm_fp8).  out_dtype: bfloat16 (default) or float32."""
    torch = _torch()
    M, K = a.shape
    N = w.shape[0]
    G = (K + 127) // 128
    if out is None:
        out, = _new(stream, a.device, ((M, N), out_dtype or torch.bfloat16))
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out is {out.dtype}, not {out_dtype}")
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"the result must be bfloat16 or float32, got {out.dtype}")
    e4m3 = torch.float8_e4m3fn
    lda, ldw, ldc = _rows("a", a, (M, K), e4m3), _rows("w", w, (N, K), e4m3), _rows("out", out, (M, N), out.dtype)
    _dense("a_scale", a_scale, (M, G), torch.float32)
    _dense("w_scale", w_scale, ((N + 127) // 128, G), torch.float32)
    _on_current_device(a, a_scale, w, w_scale, out)
    check(lib().moe_gemm_fp8(_p(a), lda, _p(a_scale), M, K, _p(w), ldw, _p(w_scale), N, _p(out), ldc,
                             MOE_BF16 if out.dtype == torch.bfloat16 else MOE_F32, _s(stream)))
    return out


def lora_workspace_bytes(M: int, r: int) -> int:
    return int(lib().moe_lora_workspace_bytes(M, r))


def lora_linear(x, a, b, scale, adapter, w=None, base=None, rank=None, out=None, out_dtype=None, ws=None, stream=None):
    """y [M, N] = x w^T + base + scale[i] * (x a[i]^T) b[i]^T, i = adapter[m], for each row m (moe_lora_linear).
    x bf16 [M, K]; a bf16 [n, r, K], b bf16 [n, N, r], scale f32 [n], rank int32 [n] (None: r for all);
    adapter int32 [M], a row's adapter or -1; w bf16 [N, K] (None: no projection); base [M, N] bfloat16 or float32
    rows to add to (None: none).  out_dtype: bfloat16 (default) or float32; out may be base."""
    torch = _torch()
    M, K = x.shape
    n, r = a.shape[:2]
    N = b.shape[1]
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    if out is None:
        out, = _new(stream, x.device, ((M, N), out_dtype or bf16))
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out is {out.dtype}, not {out_dtype}")
    for name, t in (("the result", out), ("base", base)):
        if t is not None and t.dtype not in (bf16, f32):
            raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    ldx, ldy = _rows("x", x, (M, K), bf16), _rows("out", out, (M, N), out.dtype)
    ldw = _rows("w", w, (N, K), bf16) if w is not None else 0
    ldb = _rows("base", base, (M, N), base.dtype) if base is not None else 0
    _dense("a", a, (n, r, K), bf16)
    _dense("b", b, (n, N, r), bf16)
    _dense("scale", scale, (n,), f32)
    _dense("adapter", adapter, (M,), i32)
    if rank is not None:
        _dense("rank", rank, (n,), i32)
    if ws is None:
        ws, = _new(stream, x.device, (lora_workspace_bytes(M, r) or 1, torch.uint8))
    else:
        _contig(ws)
    _on_current_device(x, a, b, scale, adapter, w, base, rank, out, ws)
    check(lib().moe_lora_linear(_p(x), ldx, M, K, _p(w), ldw, N, _p(base), ldb,
                                MOE_F32 if base is None or base.dtype == f32 else MOE_BF16, _p(a), _p(b), r, n, _p(scale),
                                _p(rank), _p(adapter), _p(out), ldy, MOE_BF16 if out.dtype == bf16 else MOE_F32, _p(ws),
                                ws.nbytes, _s(stream)))
    return out


def expert_ffn_fp8(x, x_scale, perm, offsets, counts, slot_of_expert, slot_pool, n_slots: int, slot_stride: int,
                   f: int, k: int, shared_w=None, y_perm=None, ws=None, stream=None, y_dtype=None):
    """expert_ffn_grouped with fp8 weights for quantised rows: x e4m3 [T, d], x_scale f32 [T, d/128]
    (moe_expert_ffn_fp8). -> (y_perm [T*k (+T), d], ws).  y_perm float32 (default) or bfloat16."""
    torch = _torch()
    T, d = x.shape
    E = counts.shape[0]
    _dense("x", x, (T, d), torch.float8_e4m3fn)
    _dense("x_scale", x_scale, (T, (d + 127) // 128), torch.float32)
    rows = T * k + (T if shared_w is not None else 0)
    if y_perm is None:
        y_perm, = _new(stream, x.device, ((rows, d), y_dtype or torch.float32))
    if ws is None:
        need = workspace_bytes(T, d, f, E, k, shared_w is not None, MOE_BF16, MOE_FP8_B128)
        ws, = _new(stream, x.device, (need, torch.uint8), zero=True)
    _expert_tensors(T, d, f, E, k, "fp8", perm, offsets, counts, slot_of_expert, slot_pool, n_slots, slot_stride, shared_w,
                    y_perm)
    _on_current_device(x, x_scale, perm, offsets, counts, slot_of_expert, slot_pool, shared_w, y_perm, ws)
    check(lib().moe_expert_ffn_fp8(_p(x), _p(x_scale), T, d, f, E, k, _p(perm), _p(offsets), _p(counts),
                                   _p(slot_of_expert), n_slots, _p(slot_pool), slot_stride, _p(shared_w), _p(y_perm),
                                   _y_code(y_perm), _p(ws), ws.numel(), _s(stream)))
    return y_perm, ws


def combine(y_perm, topk_w, inv_perm, k: int, has_shared: bool, out_dtype, y=None, stream=None):
    torch = _torch()
    _contig(y_perm, topk_w, inv_perm)
    T = topk_w.shape[0]
    d = y_perm.shape[1]
    if y is None:
        y, = _new(stream, y_perm.device, ((T, d), out_dtype))
    code = MOE_BF16 if y.dtype == torch.bfloat16 else MOE_F32
    check(lib().moe_combine(_p(y_perm), _y_code(y_perm), _p(topk_w), _p(inv_perm), T, k, d, int(bool(has_shared)),
                            _p(y), code, _s(stream)))
    return y


def layer_few_workspace_bytes(T: int, d: int, f: int, E: int, k: int, has_shared: bool, wdt: str) -> int:
    return int(lib().moe_layer_few_workspace_bytes(T, d, f, E, k, int(bool(has_shared)), WDT[wdt]))


class FewResult(tuple):
    """(y, topk_idx, topk_w) of layer_few, and the workspace of the call: `status`, its first word, is 0 when every chosen
    expert was there and every wait ended."""

    ws = None

    @property
    def status(self):
        """int32 [1] on the device, written by the call's kernels (sticky in a workspace that is used again)."""
        torch = _torch()
        return self.ws.flatten().view(torch.uint8)[:4].view(torch.int32)


def layer_few(x, w_router, bias, k: int, slot_of_expert, slot_pool, n_slots: int, slot_stride: int, wdt: str, f: int,
              shared_w=None, forced_idx=None, out=None, ws=None, stream=None):
    """The whole layer for at most 16 tokens (moe_layer_few): route, experts and combine in two launches.
    x [T, d], w_router [E, d] of x's type; bias f32 [E] or None; slots as expert_ffn_grouped takes them.
    out: (y, topk_idx, topk_w) to write into; ws: layer_few_workspace_bytes, zero-filled before its first use (on
    `stream`, or ordered before it) and used by one call at a time.
    -> (y [T, d], topk_idx int32 [T, k], topk_w f32 [T, k]), a tuple whose `.ws` is the workspace and `.status` its status
    word on the device, to be looked at once the call has run: 1: a chosen expert was in no slot and added nothing; 2: a
    second call used the workspace at the same time and y is wrong."""
    torch = _torch()
    act = _act(x)
    T, d = x.shape
    E = w_router.shape[0]
    dt, f32, i32 = x.dtype, torch.float32, torch.int32
    if out is None:
        out = tuple(_new(stream, x.device, ((T, d), dt), ((T, k), i32), ((T, k), f32)))
    y, idx, w = out
    for name, t, shape, dtype in (("x", x, (T, d), dt), ("w_router", w_router, (E, d), dt), ("y", y, (T, d), dt),
                                  ("topk_idx", idx, (T, k), i32), ("topk_w", w, (T, k), f32)):
        _dense(name, t, shape, dtype)
    if bias is not None:
        _dense("bias", bias, (E,), f32)
    if forced_idx is not None:
        _dense("forced_idx", forced_idx, (T, k), i32)
    if slot_of_expert.dtype != i32 or slot_of_expert.numel() < E:
        raise ValueError(f"slot_of_expert must be int32 of {E} elements at least, got {slot_of_expert.dtype} "
                         f"{list(slot_of_expert.shape)}")
    _contig(slot_of_expert, slot_pool, shared_w, ws)
    slot = slot_bytes(d, f, wdt)
    if shared_w is not None and shared_w.nbytes < slot:
        raise ValueError(f"shared_w must hold {slot} bytes, got {shared_w.nbytes}")
    if slot_pool.nbytes < (n_slots - 1) * slot_stride + slot:
        raise ValueError(f"slot_pool must hold {n_slots} slots of {slot_stride} bytes, got {slot_pool.nbytes} bytes")
    if ws is None:
        need = layer_few_workspace_bytes(T, d, f, E, k, shared_w is not None, wdt) or 1
        ws, = _new(stream, x.device, (need, torch.uint8), zero=True)
    _on_current_device(x, w_router, bias, forced_idx, slot_of_expert, slot_pool, shared_w, y, idx, w, ws)
    check(lib().moe_layer_few(_p(x), act, T, d, f, E, k, _p(w_router), _p(bias), _p(forced_idx), _p(slot_of_expert),
                              n_slots, _p(slot_pool), slot_stride, WDT[wdt], _p(shared_w), _p(idx), _p(w), _p(y),
                              _p(ws), ws.nbytes, _s(stream)))
    out = FewResult(out)
    out.ws = ws
    return out


# ---------------------------------------------------------------------------------------------
# slots
# ---------------------------------------------------------------------------------------------
def slot_bytes(d: int, f: int, wdt: str) -> int:
    return int(lib().moe_slot_bytes(d, f, WDT[wdt]))


def _np_ptr(a):
    return None if a is None else np.ascontiguousarray(a).ctypes.data


def pack_expert(wdt: str, d: int, f: int, wg, wu, wd, sg=None, su=None, sd=None, out=None) -> np.ndarray:
    """Canonical expert weights (numpy) -> slot image (numpy uint8, or written into ``out``)."""
    n = slot_bytes(d, f, wdt)
    if n == 0:
        raise MoeError(-2, f"unsupported slot shape d={d} f={f} {wdt}")
    if out is None:
        out = np.empty(n, dtype=np.uint8)
    arrs = [np.ascontiguousarray(a) if a is not None else None for a in (wg, wu, wd, sg, su, sd)]
    optr = out.ctypes.data if isinstance(out, np.ndarray) else int(out)
    check(lib().moe_pack_expert(WDT[wdt], d, f, *[_np_ptr(a) for a in arrs], optr))
    return out


def cpu_expert_ffn(slot_image, wdt: str, d: int, f: int, x_bf16: np.ndarray, y: Optional[np.ndarray] = None,
                   threads: int = 0) -> np.ndarray:
    """One expert on the host from its packed slot image (numpy uint8 array or a host address).
    x_bf16: bf16 bits (uint16) [n, d].  -> y float32 [n, d]."""
    x = np.ascontiguousarray(x_bf16, dtype=np.uint16)
    n = x.shape[0]
    if y is None:
        y = np.empty((n, d), dtype=np.float32)
    img = slot_image.ctypes.data if isinstance(slot_image, np.ndarray) else int(slot_image)
    check(lib().moe_cpu_expert_ffn(img, WDT[wdt], d, f, x.ctypes.data, n, y.ctypes.data, threads))
    return y


# moe_decode_layer (include/moe.h): six pointers, then layer and a reserved int32
DECODE_LAYER = np.dtype([("x", "<u8"), ("w_router", "<u8"), ("bias", "<u8"), ("forced", "<u8"),
                         ("shared_w", "<u8"), ("y", "<u8"), ("layer", "<i4"), ("reserved", "<i4")])


def _f32_rows(y_perm, fn: str):
    """The decode steps keep y_perm in binary32 (their C signature takes float rows)."""
    if _y_code(y_perm) != MOE_F32:
        raise TypeError(f"{fn}: y_perm must be float32, got {y_perm.dtype}")


def decode_step(cache, layers: np.ndarray, T: int, d: int, f: int, E: int, k: int, act: int, wdt: str, slot_pool,
                n_slots: int, slot_stride: int, slot_table, route_bufs, perm_bufs, y_perm, ws, host_idx, compute,
                copy):
    """One decode step of every layer in `layers` (a DECODE_LAYER array) through moe_decode_step."""
    _f32_rows(y_perm, "decode_step")
    idx, w, logits = route_bufs
    c, o, p, ip = perm_bufs
    check(lib().moe_decode_step(cache.h, len(layers), layers.ctypes.data, T, d, f, E, k, act, WDT[wdt],
                                _p(slot_pool), n_slots, slot_stride, _p(slot_table), _p(idx), _p(w), _p(logits),
                                _p(c), _p(o), _p(p), _p(ip), _p(y_perm), _p(ws), ws.numel(), host_idx.data_ptr(),
                                _s(compute), _s(copy)))



def decode_step_split(cache, layers: np.ndarray, T: int, d: int, f: int, E: int, k: int, act: int, wdt: str,
                      slot_pool, n_slots: int, slot_stride: int, slot_table, route_bufs, perm_bufs, y_perm, ws,
                      host_idx, host_tables, dev_tables, compute, copy):
    """One decode step of every layer in `layers` with split launches (moe_decode_step_split).
    host_tables: pinned int32 [2, E]; dev_tables: device int32 [2, E]."""
    _f32_rows(y_perm, "decode_step_split")
    idx, w, logits = route_bufs
    c, o, p, ip = perm_bufs
    check(lib().moe_decode_step_split(cache.h, len(layers), layers.ctypes.data, T, d, f, E, k, act, WDT[wdt],
                                      _p(slot_pool), n_slots, slot_stride, _p(slot_table), _p(idx), _p(w),
                                      _p(logits), _p(c), _p(o), _p(p), _p(ip), _p(y_perm), _p(ws), ws.numel(),
                                      host_idx.data_ptr(), host_tables.data_ptr(), _p(dev_tables), _s(compute),
                                      _s(copy)))

def decode_step_hybrid(cache, layers: np.ndarray, d: int, f: int, E: int, k: int, act: int, wdt: str, slot_pool,
                       n_slots: int, slot_stride: int, slot_table, route_bufs, perm_bufs, y_perm, ws, host_idx,
                       host_x, host_y, host_table, dev_table, cpu_rate: float, pcie_rate: float, copy_too: bool,
                       compute, copy, cpu_threads: int = 0, host_fixed_s: float = 0.0) -> int:
    """One batch-1 decode step of every layer in `layers` with hybrid miss handling
    (moe_decode_step_hybrid).  host_idx/host_x/host_y/host_table: pinned host tensors; dev_table:
    device int32 [E].  -> number of experts run on the host."""
    _f32_rows(y_perm, "decode_step_hybrid")
    idx, w, logits = route_bufs
    c, o, p, ip = perm_bufs
    n_cpu = ctypes.c_int64(0)
    check(lib().moe_decode_step_hybrid(cache.h, len(layers), layers.ctypes.data, d, f, E, k, act, WDT[wdt],
                                       _p(slot_pool), n_slots, slot_stride, _p(slot_table), _p(idx), _p(w),
                                       _p(logits), _p(c), _p(o), _p(p), _p(ip), _p(y_perm), _p(ws), ws.numel(),
                                       host_idx.data_ptr(), host_x.data_ptr(), host_y.data_ptr(),
                                       host_table.data_ptr(), _p(dev_table), float(cpu_rate), float(pcie_rate),
                                       float(host_fixed_s), int(bool(copy_too)), cpu_threads, ctypes.byref(n_cpu),
                                       _s(compute), _s(copy)))
    return n_cpu.value


def hybrid_split(m: int, cpu_rate: float, pcie_rate: float, host_fixed_s: float = 0.0) -> int:
    """Misses of a layer the host runs (moe_hybrid_split): of m misses, the n minimising
    max((m - n) / pcie_rate, host_fixed_s + n / cpu_rate) (m / pcie_rate for n = 0), ties to fewer."""
    n = ctypes.c_int32()
    check(lib().moe_hybrid_split(int(m), float(cpu_rate), float(pcie_rate), float(host_fixed_s), ctypes.byref(n)))
    return n.value

# ---------------------------------------------------------------------------------------------
# expert-slot cache
# ---------------------------------------------------------------------------------------------
class SlotCache:
    """LRU expert-slot cache shared by all layers (wraps moe_cache_*)."""

    def __init__(self, L: int, E: int, n_slots: int, slot_stride: int = 0, slot_pool=None, slot_table=None,
                 host_ptrs=None):
        self.L, self.E, self.C = L, E, n_slots
        self._host = None
        hp = None
        if host_ptrs is not None:
            self._host = (ctypes.c_void_p * (L * E))(*[int(p) for p in host_ptrs])
            hp = ctypes.cast(self._host, ctypes.c_void_p)
        h = ctypes.c_void_p()
        check(lib().moe_cache_create(L, E, n_slots, slot_stride, _p(slot_pool), _p(slot_table), hp,
                                     ctypes.byref(h)))
        self.h = h

    def lookup(self, layer: int, ids):
        ids = np.ascontiguousarray(np.asarray(ids, dtype=np.int32))
        slots = np.empty(len(ids), dtype=np.int32)
        nm = ctypes.c_int32()
        check(lib().moe_cache_lookup(self.h, layer, ids.ctypes.data, len(ids), slots.ctypes.data, ctypes.byref(nm)))
        return slots, nm.value

    def fill(self, copy_stream=None, compute_stream=None):
        check(lib().moe_cache_fill(self.h, _s(copy_stream), _s(compute_stream)))

    def fill_split(self, later, copy_stream=None, compute_stream=None):
        """fill(), with the copies of the experts in `later` deferred (compute does not wait)."""
        ids = np.ascontiguousarray(np.asarray(later, dtype=np.int32))
        check(lib().moe_cache_fill_split(self.h, ids.ctypes.data if len(ids) else None, len(ids),
                                         _s(copy_stream), _s(compute_stream)))

    def policy_fill_split(self, later):
        ids = np.ascontiguousarray(np.asarray(later, dtype=np.int32))
        check(lib().moe_cache_fill_split(self.h, ids.ctypes.data if len(ids) else None, len(ids), None, None))

    def prefetch_layer(self, layer: int, copy_stream=None, compute_stream=None):
        check(lib().moe_cache_prefetch_layer(self.h, layer, _s(copy_stream), _s(compute_stream)))

    def mark_read(self, layer: int, compute_stream=None):
        check(lib().moe_cache_mark_read(self.h, layer, _s(compute_stream)))

    def resize(self, n_slots: int, copy_stream=None, compute_stream=None):
        """Change the capacity at a safe point (every layer marked read, no fill pending)."""
        check(lib().moe_cache_resize(self.h, n_slots, _s(copy_stream), _s(compute_stream)))
        self.C = n_slots

    def policy_resize(self, n_slots: int):
        """resize() of a policy-only cache (no streams involved)."""
        check(lib().moe_cache_resize(self.h, n_slots, None, None))
        self.C = n_slots

    def policy_fill(self):
        """fill() of a policy-only cache (no streams involved)."""
        check(lib().moe_cache_fill(self.h, None, None))

    def policy_prefetch(self, layer: int):
        """prefetch_layer() of a policy-only cache (no streams involved)."""
        check(lib().moe_cache_prefetch_layer(self.h, layer, None, None))

    def policy_mark_read(self, layer: int):
        check(lib().moe_cache_mark_read(self.h, layer, None))

    def stats(self):
        out = np.zeros(6, dtype=np.int64)
        check(lib().moe_cache_stats(self.h, out.ctypes.data))
        keys = ("dec_acc", "dec_hit", "dec_miss", "pre_acc", "pre_miss", "bytes_h2d")
        return dict(zip(keys, (int(v) for v in out)))

    def trace(self):
        n = ctypes.c_int64()
        check(lib().moe_cache_trace(self.h, None, 0, ctypes.byref(n)))
        buf = np.empty(n.value, dtype=np.uint8)
        if n.value:
            check(lib().moe_cache_trace(self.h, buf.ctypes.data, n.value, ctypes.byref(n)))
        return buf

    def copy_log(self):
        n = ctypes.c_int64()
        check(lib().moe_cache_copy_log(self.h, None, 0, ctypes.byref(n)))
        buf = np.empty((n.value, 3), dtype=np.int64)
        if n.value:
            check(lib().moe_cache_copy_log(self.h, buf.ctypes.data, n.value, ctypes.byref(n)))
        return buf

    def inject_copy_failures(self, n: int):
        check(lib().moe_cache_inject_copy_failures(self.h, n))

    def slot_of(self, layer: int, expert: int) -> int:
        s = ctypes.c_int32()
        check(lib().moe_cache_slot_of(self.h, layer, expert, ctypes.byref(s)))
        return s.value

    def close(self):
        if self.h:
            lib().moe_cache_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def pinned_alloc(nbytes: int) -> int:
    p = ctypes.c_void_p()
    check(lib().moe_pinned_alloc(nbytes, ctypes.byref(p)))
    return p.value


def pinned_free(ptr: int):
    lib().moe_pinned_free(ptr)


# ---------------------------------------------------------------------------------------------
# kernel timing
# ---------------------------------------------------------------------------------------------
def profile_enable(on: bool = True):
    lib().moe_profile_enable(int(on))


def profile_collect():
    check(lib().moe_profile_collect())


def profile_results() -> dict:
    """{kernel name: (total ms, launches)} accumulated since the last reset."""
    out = {}
    i = 0
    name = ctypes.create_string_buffer(128)
    ms = ctypes.c_double()
    n = ctypes.c_int64()
    while lib().moe_profile_get(i, name, 128, ctypes.byref(ms), ctypes.byref(n)) == 0:
        out[name.value.decode()] = (ms.value, n.value)
        i += 1
    return out


def profile_reset():
    lib().moe_profile_reset()
