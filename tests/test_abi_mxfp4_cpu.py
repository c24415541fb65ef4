"""The MXFP4 entry points reject bad arguments before touching the GPU (no call
here reaches a launch)."""
import ctypes

import pytest

from combine_moe_route_topk_amd import _lib

lib = _lib.lib
ARG, UNSUP, WS = _lib.MOE_ERR_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
FAKE = ctypes.c_void_p(0x1000)      # never dereferenced


def _at(offset):
    return ctypes.c_void_p(0x1000 + offset)


def test_quantize_errors():
    def call(**kw):
        a = dict(x=FAKE, t=1, r=4, k=64, c=FAKE, s=FAKE)
        a.update(kw)
        return lib.moe_quantize_mxfp4(a["x"], a["t"], a["r"], a["k"], a["c"], a["s"], None)
    assert call(r=-1) == ARG and call(k=0) == ARG and call(t=2) == ARG and call(t=-1) == ARG
    assert call(k=48) == UNSUP and call(r=2**41 // 64) == UNSUP and call(r=2**62, k=2**62) == UNSUP
    assert call(x=None) == ARG and call(c=None) == ARG and call(s=None) == ARG
    assert call(x=_at(8)) == UNSUP and call(c=_at(2)) == UNSUP
    assert call(r=0, x=None, c=None, s=None) == 0


def test_dequant_errors():
    def call(**kw):
        a = dict(c=FAKE, s=FAKE, r=4, k=64, o=FAKE, t=1)
        a.update(kw)
        return lib.moe_dequant_mxfp4(a["c"], a["s"], a["r"], a["k"], a["o"], a["t"], None)
    assert call(r=-1) == ARG and call(k=0) == ARG and call(t=2) == ARG
    assert call(k=40) == UNSUP and call(r=2**41 // 64) == UNSUP
    assert call(c=None) == ARG and call(s=None) == ARG and call(o=None) == ARG
    assert call(o=_at(8)) == UNSUP and call(c=_at(1)) == UNSUP
    assert call(r=0, c=None, s=None, o=None) == 0


@pytest.mark.parametrize("gather", [False, True])
def test_product_errors(gather):
    def call(**kw):
        a = dict(x=FAKE, xs=FAKE, r=8, k=128, idx=FAKE, e=4, w=FAKE, ws=FAKE, u=None, us=None, n=64,
                 y=FAKE, wk=FAKE, wkb=1 << 20)
        a.update(kw)
        args = [a["x"], a["xs"], a["r"], a["k"], a["idx"], a["e"], a["w"], a["ws"], a["u"], a["us"],
                a["n"], a["y"]]
        if gather:
            return lib.moe_gather_gemm_mxfp4(*args, a["wk"], a["wkb"], None)
        return lib.moe_grouped_gemm_mxfp4(*args, None)
    assert call(r=-1) == ARG and call(k=0) == ARG and call(n=0) == ARG and call(e=0) == ARG
    assert call(u=FAKE) == ARG and call(us=FAKE) == ARG
    assert call(k=64) == UNSUP and call(k=192) == UNSUP and call(e=1025) == UNSUP
    assert call(k=(1 << 22) + 128) == UNSUP and call(n=(1 << 22) + 1) == UNSUP
    assert call(r=2**31) == UNSUP
    assert call(r=2**31 - 1, n=1 << 22) == UNSUP
    assert b"too many tiles" in lib.moe_last_error()
    for p in ("x", "xs", "idx", "w", "ws", "y"):
        assert call(**{p: None}) == ARG, p
    for p in ("x", "w", "y"):
        assert call(**{p: _at(8)}) == UNSUP, p
    assert call(u=_at(8), us=FAKE) == UNSUP and call(u=FAKE, us=_at(2)) == UNSUP
    for p in ("xs", "ws", "idx"):
        assert call(**{p: _at(2)}) == UNSUP, p
    assert call(r=0, x=None, xs=None, idx=None, w=None, ws=None, y=None, wk=None, wkb=0) == 0
    if gather:
        need = lib.moe_gather_gemm_mxfp4_workspace_bytes(8, 4)
        assert need > 0 and call(wkb=need - 1) == WS and call(wk=None) == WS and call(wk=_at(64)) == WS


def test_gather_workspace_sizes():
    f = lib.moe_gather_gemm_mxfp4_workspace_bytes
    assert f(0, 1) > 0 and f(1024, 256) >= 8 * 1024
    assert f(-1, 8) == 0 and f(8, 0) == 0 and f(8, 1025) == 0 and f(2**31, 8) == 0
