"""The 8-bit operators without a GPU: the oracle's number format against torch's e4m3 type and hand
cases, the slot layout of fp8 experts, and every refusal (checked on the host before any launch)."""
import ctypes

import numpy as np
import pytest

import synth
from oracle import fp8


@pytest.fixture(scope="module")
def moe():
    import os

    import expert_offload_cache_amd as m
    from expert_offload_cache_amd import _lib

    if not os.path.exists(_lib.LIB_PATH):
        from expert_offload_cache_amd import build as b

        b.build()
    return m


def test_e4m3_values_and_rounding_match_torch():
    import torch

    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp8.decode(codes), ref, equal_nan=True)
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.normal(size=50000) * 100, rng.normal(size=50000) * 2.0 ** -8, ref[~np.isnan(ref)],
                        [432.0, -432.0, 0.0, 2.0 ** -10, 3 * 2.0 ** -10, 459.9]])
    v = np.clip(v, -463, 463).astype(np.float32)
    t = torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp8.round_e4m3(v), t)
    assert np.array_equal(fp8.decode(synth.e4m3_bits(v.astype(np.float64))), t)


def test_quantise_definition_by_hand():
    # one group: the largest magnitude becomes 448 whatever it is; ties go to the even code
    x = np.zeros((1, 130))
    x[0, :4] = [7.0, -7.0, 6.75, 3.625]  # scale 1/64: 448, -448, 432 (between 416 and 448: 416 is odd), 232
    x[0, 129] = 14.0                      # the short second group has its own scale
    q, s = fp8.quantise(x)
    assert s.shape == (1, 2) and s[0, 0] == 7 / 448 and s[0, 1] == 14 / 448
    assert q[0, :4].tolist() == [448.0, -448.0, 448.0, 224.0]
    assert q[0, 128] == 0.0 and q[0, 129] == 448.0
    q, s = fp8.quantise(np.zeros((1, 16)))
    assert s[0, 0] == 2.0 ** -126 and not q.any()


def test_fp8_slot_layout(moe):
    d, f = 384, 256
    wl = synth.Workload("t", d=d, E=1, k=1, f=f, act="bf16", wdt="fp8", T_list=(1,))
    ew = synth.expert_weights(wl, 3, 0, 0)
    img = moe.pack_expert("fp8", d, f, ew.wg, ew.wu, ew.wd, ew.sg, ew.su, ew.sd)
    assert img.nbytes == moe.slot_bytes(d, f, "fp8")
    assert moe.slot_bytes(d, f, "fp8") == -(-((2 * f // 16) * (16 * d + 64) + (d // 16) * (16 * f + 64)) // 256) * 256
    assert moe.slot_bytes(4096, 2048, "fp8") == 256 * (65536 + 128) + 256 * (32768 + 64)
    assert moe.slot_bytes(64, 128, "fp8") == 0 and moe.slot_bytes(128, 192, "fp8") == 0

    def unpack(block0, stride, R, K, step):
        q, s = np.empty((R, K), np.uint8), np.empty((R // 16, K // 128), np.float32)
        for rb in range(R // 16):
            blk = img[block0 + rb * stride * step:][:stride]
            frag = blk[:16 * K].reshape(K // 128, 2, 64, 16)
            for l in range(64):
                for h in range(2):
                    for g in range(K // 128):
                        k0 = 128 * g + 64 * h + 16 * (l // 16)
                        q[rb * 16 + l % 16, k0:k0 + 16] = frag[g, h, l]
            s[rb] = blk[16 * K:16 * K + 4 * (K // 128)].view(np.float32)
        return q, s

    gu, dn = 16 * d + 64, 16 * f + 64
    for w, sc, (q, s) in ((ew.wg, ew.sg, unpack(0, gu, f, d, 2)), (ew.wu, ew.su, unpack(gu, gu, f, d, 2)),
                          (ew.wd, ew.sd, unpack(2 * (f // 16) * gu, dn, d, f, 1))):
        assert np.array_equal(q, w)
        assert np.array_equal(s, np.repeat(sc, 8, axis=0))
    with pytest.raises(moe.MoeError, match="scales"):
        moe.pack_expert("fp8", d, f, ew.wg, ew.wu, ew.wd)


@pytest.mark.parametrize("d,f,k,shared", [(128, 128, 1, False), (512, 2048, 8, True), (4096, 256, 2, False)])
def test_workspace_of_more_tokens_serves_fewer(moe, d, f, k, shared):
    sizes = [moe.workspace_bytes(T, d, f, 64, k, shared, moe._lib.MOE_BF16, moe._lib.MOE_FP8_B128) for T in range(1, 80)]
    assert sizes == sorted(sizes) and len(set(sizes)) > 20


def test_product_of_too_many_rows_is_refused(moe):
    L, p = moe.lib(), ctypes.c_void_p(256)
    for M in (2 ** 31 - 1, 2 ** 31 - 64, 65536 * 128):
        assert L.moe_gemm_fp8(p, 16, p, M, 16, p, 16, p, 64, p, 64, 1, None) == moe._lib.MOE_ESHAPE
        assert b"rows exceed" in L.moe_last_error()


def test_norm_and_quant_refusals(moe):
    L, e = moe.lib(), moe._lib
    p = ctypes.c_void_p(256)

    def norm(x=p, act=1, T=4, d=128, ldx=128, res=None, ldr=0, w=p, wd=1, eps=1e-6, ro=None, ldro=0, y=p, ldy=128,
             q=None, ldq=0, sc=None):
        return L.moe_add_rmsnorm(x, act, T, d, ldx, res, ldr, w, wd, eps, ro, ldro, y, ldy, q, ldq, sc, None)

    assert norm(T=0, x=None, w=None, y=None) == e.MOE_OK
    for bad, code in ((dict(T=-1), e.MOE_ESHAPE), (dict(d=0), e.MOE_ESHAPE), (dict(d=16385), e.MOE_ESHAPE),
                      (dict(act=2), e.MOE_EDTYPE), (dict(act=3), e.MOE_EDTYPE), (dict(wd=2), e.MOE_EDTYPE),
                      (dict(act=0, wd=1), e.MOE_EDTYPE), (dict(eps=-1.0), e.MOE_EINVAL),
                      (dict(eps=float("nan")), e.MOE_EINVAL), (dict(x=None), e.MOE_EINVAL),
                      (dict(w=None), e.MOE_EINVAL), (dict(y=None), e.MOE_EINVAL), (dict(q=p, ldq=128), e.MOE_EINVAL),
                      (dict(sc=p), e.MOE_EINVAL), (dict(res=p, ldr=128), e.MOE_EINVAL),
                      (dict(ro=p, ldro=128), e.MOE_EINVAL), (dict(ldx=127), e.MOE_EINVAL),
                      (dict(ldy=127), e.MOE_EINVAL), (dict(q=p, ldq=64, sc=p), e.MOE_EINVAL),
                      (dict(res=p, ldr=64, ro=p, ldro=128), e.MOE_EINVAL),
                      (dict(res=p, ldr=128, ro=p, ldro=64), e.MOE_EINVAL),
                      (dict(x=ctypes.c_void_p(257)), e.MOE_EINVAL), (dict(y=ctypes.c_void_p(257)), e.MOE_EINVAL),
                      (dict(q=p, ldq=128, sc=ctypes.c_void_p(258)), e.MOE_EINVAL)):
        assert norm(**bad) == code, bad
        assert b"moe_add_rmsnorm" in L.moe_last_error()

    def quant(x=p, act=1, T=4, d=128, ldx=128, q=p, ldq=128, sc=p):
        return L.moe_quant_fp8(x, act, T, d, ldx, q, ldq, sc, None)

    assert quant(T=0, x=None, q=None, sc=None) == e.MOE_OK
    for bad, code in ((dict(T=-1), e.MOE_ESHAPE), (dict(d=0), e.MOE_ESHAPE), (dict(d=20000), e.MOE_ESHAPE),
                      (dict(act=3), e.MOE_EDTYPE), (dict(x=None), e.MOE_EINVAL), (dict(q=None), e.MOE_EINVAL),
                      (dict(sc=None), e.MOE_EINVAL), (dict(ldx=100), e.MOE_EINVAL), (dict(ldq=100), e.MOE_EINVAL),
                      (dict(act=0, x=ctypes.c_void_p(258)), e.MOE_EINVAL)):
        assert quant(**bad) == code, bad


def test_gemm_refusals(moe):
    L, e = moe.lib(), moe._lib
    p = ctypes.c_void_p(256)

    def gemm(a=p, lda=128, asc=p, M=4, K=128, w=p, ldw=128, wsc=p, N=4, c=p, ldc=4, out=1):
        return L.moe_gemm_fp8(a, lda, asc, M, K, w, ldw, wsc, N, c, ldc, out, None)

    assert gemm(M=0, a=None, c=None) == e.MOE_OK
    for bad, code in ((dict(M=-1), e.MOE_ESHAPE), (dict(N=0), e.MOE_ESHAPE), (dict(K=0), e.MOE_ESHAPE),
                      (dict(K=120), e.MOE_ESHAPE), (dict(K=1 << 21, lda=1 << 21, ldw=1 << 21), e.MOE_ESHAPE),
                      (dict(out=2), e.MOE_EDTYPE), (dict(out=3), e.MOE_EDTYPE), (dict(a=None), e.MOE_EINVAL),
                      (dict(asc=None), e.MOE_EINVAL), (dict(w=None), e.MOE_EINVAL), (dict(wsc=None), e.MOE_EINVAL),
                      (dict(c=None), e.MOE_EINVAL), (dict(lda=112), e.MOE_EINVAL), (dict(ldw=112), e.MOE_EINVAL),
                      (dict(ldc=3), e.MOE_EINVAL), (dict(lda=136), e.MOE_EINVAL), (dict(ldw=136), e.MOE_EINVAL),
                      (dict(a=ctypes.c_void_p(264)), e.MOE_EINVAL), (dict(w=ctypes.c_void_p(264)), e.MOE_EINVAL),
                      (dict(c=ctypes.c_void_p(257)), e.MOE_EINVAL), (dict(asc=ctypes.c_void_p(258)), e.MOE_EINVAL)):
        assert gemm(**bad) == code, bad
        assert b"moe_gemm_fp8" in L.moe_last_error()


def test_expert_refusals(moe):
    L, e = moe.lib(), moe._lib
    p = ctypes.c_void_p(256)
    d, f, E, k, T = 256, 128, 8, 2, 4
    stride, ws = moe.slot_bytes(d, f, "fp8"), moe.workspace_bytes(T, d, f, E, k, False, 1, 3)
    assert ws > 0

    def ffn(x=p, xs=p, T=T, d=d, f=f, E=E, k=k, slots=8, pool=p, stride=stride, yd=1, w=p, wsb=ws, y=p):
        return L.moe_expert_ffn_fp8(x, xs, T, d, f, E, k, p, p, p, p, slots, pool, stride, None, y, yd, w, wsb, None)

    assert ffn(T=0) == e.MOE_OK
    for bad, code in ((dict(T=-1), e.MOE_ESHAPE), (dict(d=192), e.MOE_ESHAPE), (dict(f=64), e.MOE_ESHAPE),
                      (dict(E=1025), e.MOE_ESHAPE), (dict(k=9), e.MOE_ESHAPE), (dict(yd=2), e.MOE_EDTYPE),
                      (dict(yd=3), e.MOE_EDTYPE), (dict(x=None), e.MOE_EINVAL), (dict(xs=None), e.MOE_EINVAL),
                      (dict(xs=ctypes.c_void_p(258)), e.MOE_EINVAL), (dict(x=ctypes.c_void_p(264)), e.MOE_EINVAL),
                      (dict(slots=0), e.MOE_EINVAL), (dict(pool=ctypes.c_void_p(128)), e.MOE_EINVAL),
                      (dict(stride=stride - 256), e.MOE_EINVAL), (dict(y=None), e.MOE_EINVAL),
                      (dict(w=None), e.MOE_EINVAL), (dict(w=ctypes.c_void_p(128)), e.MOE_EINVAL),
                      (dict(wsb=ws - 1), e.MOE_ENOMEM)):
        assert ffn(**bad) == code, bad
    # the other entry points: fp8 weights with bf16 rows only, no fp8 rows, no host path
    def grouped(act, w):
        return L.moe_expert_ffn_grouped(p, act, T, d, f, E, k, p, p, p, p, 8, p, stride, w, None, p, 0, p, ws - 1, None)

    assert grouped(0, 3) == e.MOE_EDTYPE and grouped(3, 3) == e.MOE_EDTYPE and grouped(3, 1) == e.MOE_EDTYPE
    assert grouped(1, 3) == e.MOE_ENOMEM
    assert L.moe_route(p, 3, 4, 128, p, None, 8, 2, None, p, p, p, None) == e.MOE_EDTYPE
    assert L.moe_combine(p, 3, p, p, 4, 2, 8, 0, p, 1, None) == e.MOE_EDTYPE
    assert L.moe_cpu_expert_ffn(p, 3, d, f, p, 1, p, 0) == e.MOE_EDTYPE
    c = moe.SlotCache(2, 8, 4)
    try:
        layers = np.zeros(1, dtype=moe.DECODE_LAYER)
        assert L.moe_decode_step_hybrid(c.h, 1, layers.ctypes.data, d, f, E, k, 1, 3, p, 4, stride, p, *[None] * 9, 0, p,
                                        p, p, p, p, 1.0, 1.0, 0.0, 1, 0, None, None, None) == e.MOE_EDTYPE
    finally:
        c.close()


def test_binding_refusals(moe):
    """The binding checks shapes, types and where tensors live before it calls the library."""
    import torch

    e4 = torch.float8_e4m3fn
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    w = torch.zeros(128, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 128, dtype=e4), torch.zeros(4, 1)
    with pytest.raises(ValueError, match="emit"):
        moe.add_rmsnorm(x, w, emit="q")
    with pytest.raises(TypeError):
        moe.add_rmsnorm(x.half(), w)
    with pytest.raises(ValueError, match="agree"):
        moe.add_rmsnorm(x, w, emit="fp8", out=(x, None, q, s))
    with pytest.raises(ValueError, match="come together"):
        moe.add_rmsnorm(x, w, out=(x, x, None, None))
    with pytest.raises(ValueError, match="emit"):
        moe.add_rmsnorm(x, w, out=(x, None, q, s))
    with pytest.raises(ValueError, match="q must be"):
        moe.quant_fp8(x, out=(q[:3], s))
    with pytest.raises(ValueError, match="scale must be"):
        moe.quant_fp8(x, out=(q, torch.zeros(4, 2)))
    with pytest.raises(ValueError, match="next to each other"):
        moe.gemm_fp8(q.t().contiguous().t(), s, q, torch.zeros(1, 1))
    with pytest.raises(ValueError, match="a_scale"):
        moe.gemm_fp8(q, s.double(), q, torch.zeros(1, 1))
    with pytest.raises(ValueError, match="w_scale"):
        moe.gemm_fp8(q, s, q, torch.zeros(2, 1))
    with pytest.raises(ValueError, match="w must be"):
        moe.gemm_fp8(q, s, torch.zeros(4, 64, dtype=e4), torch.zeros(1, 1))
    with pytest.raises(TypeError):
        moe.gemm_fp8(q, s, q, torch.zeros(1, 1), out_dtype=torch.float16)
    with pytest.raises(ValueError, match="out is"):
        moe.gemm_fp8(q, s, q, torch.zeros(1, 1), out_dtype=torch.float32, out=torch.zeros(4, 4, dtype=torch.bfloat16))


def _grouped_tensors(moe, wdt, T=4, d=128, f=128, E=3, k=2):
    """Host tensors of the right types and sizes for a grouped expert call with a shared expert, no longer than needed."""
    import torch

    slot = moe.slot_bytes(d, f, wdt)
    i32 = dict(dtype=torch.int32)
    return dict(perm=torch.zeros(T * k, **i32), offsets=torch.zeros(E + 1, **i32), counts=torch.zeros(E, **i32),
                slot_of_expert=torch.zeros(E, **i32), slot_pool=torch.zeros(2 * slot + 256, dtype=torch.uint8), n_slots=2,
                slot_stride=slot + 256, f=f, k=k, shared_w=torch.zeros(slot, dtype=torch.uint8),
                y_perm=torch.zeros(T * k + T, d))


def _wrong_sizes(good):
    """(argument, tensor too short or of another type) for each tensor of a grouped expert call."""
    import torch

    for name in ("perm", "offsets", "counts", "slot_of_expert"):
        yield name, good[name].long()
    for name in ("perm", "offsets", "slot_of_expert", "slot_pool", "shared_w"):
        yield name, good[name][:-1]
    yield "y_perm", good["y_perm"][:-1]
    yield "y_perm", good["y_perm"][:, :-1].contiguous()


def test_expert_tensors_that_the_kernels_would_pass_the_end_of(moe):
    """The binding knows the tensors' sizes, the library only their addresses: what is too short is refused."""
    import torch

    x, xs = torch.zeros(4, 128, dtype=torch.float8_e4m3fn), torch.zeros(4, 1)
    good = _grouped_tensors(moe, "fp8")
    with pytest.raises(ValueError, match="current GPU"):  # nothing wrong but where they live
        moe.expert_ffn_fp8(x, xs, **good)
    for name, t in _wrong_sizes(good):
        with pytest.raises(ValueError, match=name):
            moe.expert_ffn_fp8(x, xs, **dict(good, **{name: t}))
    with pytest.raises(TypeError, match="y_perm"):
        moe.expert_ffn_fp8(x, xs, **dict(good, y_perm=good["y_perm"].half()))
    with pytest.raises(ValueError, match="contiguous"):
        moe.expert_ffn_fp8(x, xs, **dict(good, slot_pool=torch.zeros(2, 2 * good["slot_pool"].numel(), dtype=torch.uint8)[:, ::2]))


@pytest.mark.parametrize("wdt", ["bf16", "int4", "fp8"])
def test_grouped_tensors_that_the_kernels_would_pass_the_end_of(moe, wdt):
    """The same of the calls with bf16 rows (only calls that are refused: nothing is launched)."""
    import torch

    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    good = _grouped_tensors(moe, wdt)
    for name, t in _wrong_sizes(good):
        bad = dict(good, **{name: t})
        with pytest.raises(ValueError, match=name):
            moe.expert_ffn_grouped(x, wdt=wdt, **bad)
        with pytest.raises(ValueError, match=name):
            moe.expert_ffn_grouped_noalloc(x, wdt=wdt, **bad)
    for status in (torch.zeros(0, dtype=torch.int32), torch.zeros(1, dtype=torch.int16)):
        with pytest.raises(ValueError, match="status"):
            moe.expert_ffn_grouped_noalloc(x, wdt=wdt, status=status, **good)
