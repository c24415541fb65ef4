"""The balance-loss and 4-bit integer entry points reject bad arguments before
touching the GPU (no call here reaches a launch)."""
import ctypes

import numpy as np
import pytest
import torch

import combine_moe_route_topk_amd as moe
from combine_moe_route_topk_amd import _lib

lib = _lib.lib
ARG, UNSUP, WS = _lib.MOE_ERR_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
FAKE = ctypes.c_void_p(0x1000)      # never dereferenced
F32, BF16, F8 = 0, 1, 2


def _at(offset):
    return ctypes.c_void_p(0x1000 + offset)


def test_balance_errors():
    need = lib.moe_balance_loss_workspace_bytes(16, 8, 2)
    assert need > 0

    def call(**kw):
        a = dict(l=FAKE, i=FAKE, n=16, e=8, k=2, o=FAKE, b=2, m=None, lo=FAKE, z=FAKE, c=FAKE, p=FAKE, t=FAKE,
                 w=FAKE, wb=need)
        a.update(kw)
        return lib.moe_balance_loss(*[a[x] for x in ("l", "i", "n", "e", "k", "o", "b", "m", "lo", "z", "c", "p", "t",
                                                     "w", "wb")], None)
    assert call(n=-1) == ARG and call(e=0) == ARG and call(k=0) == ARG and call(k=9) == ARG and call(b=0) == ARG
    assert call(o=None) == ARG
    assert call(e=1025) == UNSUP and call(e=512, k=65) == UNSUP and call(n=2**31) == UNSUP
    assert call(n=2**30, k=2) == UNSUP and call(b=(1 << 20) + 1) == UNSUP
    for p in ("l", "i", "lo", "z", "c", "p", "t"):
        assert call(**{p: None}) == ARG, p
    for p in ("l", "i", "o", "lo", "z", "c", "p", "t"):
        assert call(**{p: _at(2)}) == ARG, p
    assert call(w=None) == WS and call(wb=need - 1) == WS and call(w=_at(128)) == WS
    # outputs are needed also without a token, whose sums are 0
    assert call(n=0, c=None) == ARG and call(n=0, l=None, i=None, w=None) == WS


def test_balance_backward_errors():
    def call(**kw):
        a = dict(l=FAKE, n=16, e=8, k=2, o=FAKE, b=2, m=None, c=FAKE, t=FAKE, dl=FAKE, dz=None, d=FAKE, acc=0)
        a.update(kw)
        return lib.moe_balance_loss_backward(*[a[x] for x in ("l", "n", "e", "k", "o", "b", "m", "c", "t", "dl", "dz",
                                                              "d", "acc")], None)
    assert call(n=-1) == ARG and call(e=0) == ARG and call(k=0) == ARG and call(k=9) == ARG and call(b=0) == ARG
    assert call(o=None) == ARG and call(e=1025) == UNSUP and call(b=(1 << 20) + 1) == UNSUP
    for p in ("l", "c", "t", "dl", "d"):
        assert call(**{p: None}) == ARG, p
    for p in ("l", "o", "c", "t", "dl", "dz", "d"):
        assert call(**{p: _at(2)}) == ARG, p
    assert call(n=0, l=None, c=None, t=None, dl=None, d=None) == 0


def test_balance_workspace_sizes():
    f = lib.moe_balance_loss_workspace_bytes
    assert f(0, 8, 1) > 0 and f(32768, 256, 37) >= 8 * 256 * (512 + 37)
    assert f(-1, 8, 1) == 0 and f(2**31, 8, 1) == 0 and f(8, 0, 1) == 0 and f(8, 1025, 1) == 0
    assert f(8, 8, 0) == 0 and f(8, 8, (1 << 20) + 1) == 0


@pytest.mark.parametrize("quantize", [True, False])
def test_int4_row_errors(quantize):
    def call(**kw):
        a = dict(x=FAKE, t=BF16, r=4, k=256, g=128, c=FAKE, s=FAKE, b=None, st=BF16)
        a.update(kw)
        if quantize:
            return lib.moe_quantize_int4(*[a[x] for x in ("x", "t", "r", "k", "g", "c", "s", "b", "st")], None)
        return lib.moe_dequant_int4(*[a[x] for x in ("c", "s", "b", "st", "r", "k", "g", "x", "t")], None)
    assert call(r=-1) == ARG and call(k=0) == ARG and call(t=F8) == ARG and call(st=F8) == ARG and call(t=-1) == ARG
    assert call(g=16) == UNSUP and call(g=0) == UNSUP and call(g=256) == UNSUP and call(k=192) == UNSUP
    assert call(r=2**41 // 256) == UNSUP and call(r=2**62, k=2**62) == UNSUP
    for p in ("x", "c", "s"):
        assert call(**{p: None}) == ARG, p
    assert call(x=_at(8)) == UNSUP and call(c=_at(2)) == UNSUP and call(s=_at(2)) == UNSUP and call(b=_at(2)) == UNSUP
    assert call(r=0, x=None, c=None, s=None) == 0


def test_int4_product_errors():
    def call(**kw):
        a = dict(x=FAKE, r=8, k=256, i=FAKE, e=4, w=FAKE, s=FAKE, b=None, u=None, us=None, ub=None, st=BF16, g=64,
                 n=64, y=FAKE, yt=BF16, wk=FAKE, wb=1 << 20)
        a.update(kw)
        return lib.moe_gather_gemm_int4(*[a[x] for x in ("x", "r", "k", "i", "e", "w", "s", "b", "u", "us", "ub", "st",
                                                         "g", "n", "y", "yt", "wk", "wb")], None)
    assert call(r=-1) == ARG and call(k=0) == ARG and call(n=0) == ARG and call(e=0) == ARG
    assert call(st=F8) == ARG and call(yt=F8) == ARG
    assert call(u=FAKE) == ARG and call(us=FAKE) == ARG and call(ub=FAKE) == ARG
    assert call(u=FAKE, us=FAKE, b=FAKE) == ARG and call(u=FAKE, us=FAKE, ub=FAKE) == ARG
    assert call(g=48) == UNSUP and call(g=256) == UNSUP and call(k=96) == UNSUP and call(e=1025) == UNSUP
    assert call(k=(1 << 22) + 64) == UNSUP and call(n=(1 << 22) + 1) == UNSUP and call(r=2**31) == UNSUP
    assert call(r=2**31 - 1, n=1 << 22) == UNSUP
    assert b"too many tiles" in lib.moe_last_error()
    for p in ("x", "i", "w", "s", "y"):
        assert call(**{p: None}) == ARG, p
    for p in ("x", "w", "y"):
        assert call(**{p: _at(8)}) == UNSUP, p
    assert call(u=_at(8), us=FAKE) == UNSUP and call(u=FAKE, us=_at(2)) == UNSUP
    assert call(s=_at(2)) == UNSUP and call(b=_at(2)) == UNSUP and call(i=_at(2)) == UNSUP
    need = lib.moe_gather_gemm_int4_workspace_bytes(8, 4)
    assert need > 0 and call(wb=need - 1) == WS and call(wk=None) == WS and call(wk=_at(64)) == WS
    assert call(r=0, x=None, i=None, w=None, s=None, y=None, wk=None, wb=0) == 0
    f = lib.moe_gather_gemm_int4_workspace_bytes
    assert f(-1, 8) == 0 and f(8, 0) == 0 and f(8, 1025) == 0 and f(2**31, 8) == 0


CALLS = [("moe_balance_loss", 2), ("moe_quantize_int4", 1), ("moe_dequant_int4", 2), ("moe_gather_gemm_int4", 4)]


@pytest.mark.parametrize("fn,n", CALLS)
@pytest.mark.parametrize("bad", [None, 3, [1, 2], np.zeros((4, 64), np.uint8)])
def test_no_tensor(fn, n, bad):
    with pytest.raises(TypeError, match="must be a tensor"):
        getattr(moe, fn)(*[bad] * n)


def test_no_device_tensor():
    t = torch.zeros((4, 64))
    for fn, n in CALLS:
        with pytest.raises(ValueError, match="device tensor"):
            getattr(moe, fn)(*[t] * n)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_balance_loss_backward(t, t, t, 2, t)
    with pytest.raises(TypeError, match="must be a tensor"):
        moe.moe_balance_loss_backward(None, None, None, 2, None)
