"""Refusals of the serving operators, before any launch (no GPU is touched)."""
import ctypes

import pytest
import torch

import mixture_experts_expert_histogram_amd as moe
from mixture_experts_expert_histogram_amd import _lib

P = ctypes.c_void_p(16)
BIG = 1 << 45


def few(d, ptr=P, ws_bytes=BIG, **null):
    a = {n: ptr for n in ("hidden", "ids", "w", "gu", "dn", "out", "ws")}
    a.update(null)
    return moe.library().moe_fwd_few(ctypes.byref(d), a["hidden"], a["ids"], a["w"], a["gu"], a["dn"], a["out"], a["ws"],
                                     ws_bytes, None)


def few_logits(d, ptr=P, ws_bytes=BIG, **null):
    a = {n: ptr for n in ("hidden", "logits", "gu", "dn", "out", "ids", "w", "ws")}
    a.update(null)
    return moe.library().moe_fwd_few_logits(ctypes.byref(d), a["hidden"], a["logits"], a["gu"], a["dn"], a["out"], a["ids"],
                                            a["w"], a["ws"], ws_bytes, None)


def mx(d, ptr=P, ws_bytes=BIG, **null):
    a = {n: ptr for n in ("hidden", "ids", "w", "gu", "gus", "dn", "dns", "out", "ws")}
    a.update(null)
    return moe.library().moe_mx_fwd(ctypes.byref(d), a["hidden"], a["ids"], a["w"], a["gu"], a["gus"], a["dn"], a["dns"],
                                    a["out"], a["ws"], ws_bytes, None)


def mx_logits(d, ptr=P, ws_bytes=BIG, **null):
    a = {n: ptr for n in ("hidden", "logits", "gu", "gus", "dn", "dns", "out", "ids", "w", "ws")}
    a.update(null)
    return moe.library().moe_mx_fwd_logits(ctypes.byref(d), a["hidden"], a["logits"], a["gu"], a["gus"], a["dn"], a["dns"],
                                           a["out"], a["ids"], a["w"], a["ws"], ws_bytes, None)


@pytest.mark.parametrize("call,names", [(few, "hidden ids w gu dn out ws"), (few_logits, "hidden logits gu dn out ids w ws"),
                                        (mx, "hidden ids w gu gus dn dns out ws"),
                                        (mx_logits, "hidden logits gu gus dn dns out ids w ws")])
def test_pointers(call, names):
    d = moe.make_desc(4, 64, 32, 8, 2)
    for n in names.split():
        assert call(d, **{n: None}) == _lib.MOE_ERR_INVALID_ARG, n
        assert call(d, **{n: ctypes.c_void_p(24)}) == _lib.MOE_ERR_INVALID_ARG, n
    assert call(d, ws_bytes=255) == _lib.MOE_ERR_WORKSPACE
    for bad in (moe.make_desc(-1, 64, 32, 8, 2), moe.make_desc(4, 64, 32, 0, 2), moe.make_desc(4, 64, 32, 8, 0)):
        assert call(bad) == _lib.MOE_ERR_INVALID_ARG
    assert call(moe.make_desc(4, 60, 32, 8, 2)) == _lib.MOE_ERR_UNSUPPORTED
    assert call(moe.make_desc(4, 64, 32, 2000, 2)) == _lib.MOE_ERR_UNSUPPORTED
    d.act = 9
    assert call(d) == _lib.MOE_ERR_INVALID_ARG


def test_logits_need_enough_experts():
    d = moe.make_desc(4, 64, 32, 2, 3)
    assert few_logits(d) == _lib.MOE_ERR_INVALID_ARG
    assert mx_logits(d) == _lib.MOE_ERR_INVALID_ARG


def test_few_tokens_limits():
    assert few(moe.make_desc(moe.FEW_MAX_TOKENS + 1, 64, 32, 8, 2)) == _lib.MOE_ERR_UNSUPPORTED
    assert few(moe.make_desc(128, 8, 1 << 24, 8, 64)) == _lib.MOE_ERR_UNSUPPORTED       # a past 2^31 bytes
    assert few(moe.make_desc(1, 1 << 24, 8, 1, 1, "fp32")) == _lib.MOE_ERR_UNSUPPORTED   # 64 weight rows past them
    with pytest.raises(moe.MoeError):
        moe.few_workspace_size(moe.make_desc(129, 64, 32, 8, 2))
    n = moe.few_workspace_size(moe.make_desc(16, 2880, 2880, 128, 4))
    assert n >= 64 * 2880 * 2 + 64 * 2880 * 4
    d = moe.make_desc(16, 2880, 2880, 128, 4)
    assert few(d, ws_bytes=n - 1) == _lib.MOE_ERR_WORKSPACE


def test_mx_limits():
    assert mx(moe.make_desc(4, 64, 32, 8, 2, "fp32")) == _lib.MOE_ERR_UNSUPPORTED
    assert mx(moe.make_desc(4, 72, 32, 8, 2)) == _lib.MOE_ERR_UNSUPPORTED
    assert mx(moe.make_desc(4, 64, 40, 8, 2)) == _lib.MOE_ERR_UNSUPPORTED
    with pytest.raises(moe.MoeError):
        moe.mx_workspace_size(moe.make_desc(4, 72, 32, 8, 2))
    for T in (1, 100, 1000, 5000):
        d = moe.make_desc(T, 2880, 2880, 128, 4)
        n = moe.mx_workspace_size(d)
        assert n >= T * 4 * 2880 * 6
        assert mx(d, ws_bytes=n - 1) == _lib.MOE_ERR_WORKSPACE


def test_quantize_arguments():
    lib = moe.library()
    for f, order in ((lib.moe_mx_quantize, "w t r c q s"), (lib.moe_mx_dequantize, "q s t r c w")):
        def call(**kw):
            a = dict(w=P, q=P, s=P, t=0, r=4, c=64)
            a.update(kw)
            return f(*[a[n] for n in order.split()], None)
        for n in ("w", "q", "s"):
            assert call(**{n: None}) == _lib.MOE_ERR_INVALID_ARG
            assert call(**{n: ctypes.c_void_p(8)}) == _lib.MOE_ERR_INVALID_ARG
        assert call(t=2) == _lib.MOE_ERR_INVALID_ARG
        assert call(r=-1) == _lib.MOE_ERR_INVALID_ARG
        assert call(c=0) == _lib.MOE_ERR_INVALID_ARG
        assert call(c=48) == _lib.MOE_ERR_UNSUPPORTED
        assert call(r=1 << 62, c=64) == _lib.MOE_ERR_UNSUPPORTED
        assert call(r=0) == _lib.MOE_OK   # nothing to do, nothing launched


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    ids, w = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, 1)
    gu, dn = torch.zeros(1, 64, 64, dtype=torch.bfloat16), torch.zeros(1, 64, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.fwd_few(x, ids, w, gu, dn)
    with pytest.raises(ValueError):
        moe.mx_quantize(gu)
    with pytest.raises(ValueError):
        moe.mx_dequantize(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8))
    q = (torch.zeros(1, 64, 32, dtype=torch.uint8), torch.zeros(1, 64, 2, dtype=torch.uint8))
    dq = (torch.zeros(1, 64, 16, dtype=torch.uint8), torch.zeros(1, 64, 1, dtype=torch.uint8))
    with pytest.raises(ValueError):
        moe.mx_fwd(x, ids, w, q, dq)
    # shapes and types, checked before the device is
    with pytest.raises(ValueError):
        moe.mx_fwd(x, ids, w, dq, q)
    with pytest.raises(ValueError):
        moe.fwd_few(x, ids, w, gu, gu)
    with pytest.raises(ValueError):
        moe.fwd_few(x.float(), ids, w, gu, dn)
