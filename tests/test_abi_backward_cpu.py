"""The gradient entry points reject bad arguments before touching the GPU (no
call here reaches a launch)."""
import ctypes

from combine_moe_route_topk_amd import _lib

lib = _lib.lib
ARG, UNSUP = _lib.MOE_ERR_ARG, _lib.MOE_ERR_UNSUPPORTED
FAKE = ctypes.c_void_p(0x1000)      # never dereferenced


def test_combine_backward_errors():
    def call(**kw):
        a = dict(g=FAKE, gt=1, y=FAKE, yt=1, n=4, d=64, k=2, pos=FAKE, w=FAKE, dy=FAKE, dw=FAKE)
        a.update(kw)
        return lib.moe_combine_backward(a["g"], a["gt"], a["y"], a["yt"], a["n"], a["d"], a["k"],
                                        a["pos"], a["w"], a["dy"], a["dw"], None)
    assert call(n=-1) == ARG and call(d=0) == ARG and call(k=0) == ARG
    assert call(gt=2) == ARG and call(yt=5) == ARG and call(yt=-1) == ARG
    assert call(k=65) == UNSUP
    assert call(n=2**30, k=2) == UNSUP and call(n=2**62, k=64) == UNSUP
    for p in ("g", "y", "pos", "w", "dy", "dw"):
        assert call(**{p: None}) == ARG, p
    assert call(y=ctypes.c_void_p(0x1001)) == ARG                    # bf16: 2 bytes
    assert call(y=ctypes.c_void_p(0x1002), yt=0) == ARG              # f32: 4 bytes
    assert call(dw=ctypes.c_void_p(0x1002)) == ARG
    assert b"aligned" in lib.moe_last_error()
    assert call(n=0, g=None, y=None, pos=None, w=None, dy=None, dw=None) == 0


def test_dispatch_backward_errors():
    def call(**kw):
        a = dict(r=FAKE, rt=1, n=4, d=64, k=2, pos=FAKE, dx=FAKE, xt=1)
        a.update(kw)
        return lib.moe_dispatch_backward(a["r"], a["rt"], a["n"], a["d"], a["k"], a["pos"], a["dx"],
                                         a["xt"], None)
    assert call(n=-1) == ARG and call(d=0) == ARG and call(k=0) == ARG
    assert call(rt=2) == ARG and call(xt=3) == ARG
    assert call(k=65) == UNSUP and call(n=2**31, k=1) == UNSUP
    for p in ("r", "pos", "dx"):
        assert call(**{p: None}) == ARG, p
    assert call(dx=ctypes.c_void_p(0x1002), xt=0) == ARG
    assert call(n=0, r=None, pos=None, dx=None) == 0


def test_route_topk_backward_errors():
    def call(**kw):
        a = dict(l=FAKE, idx=FAKE, w=FAKE, dw=FAKE, n=4, e=8, k=2, rn=0, dl=FAKE)
        a.update(kw)
        return lib.moe_route_topk_backward(a["l"], a["idx"], a["w"], a["dw"], a["n"], a["e"], a["k"],
                                           a["rn"], a["dl"], None)
    assert call(n=-1) == ARG and call(e=0) == ARG and call(k=0) == ARG and call(k=9) == ARG
    assert call(e=2048) == UNSUP and call(k=65, e=128) == UNSUP
    for p in ("l", "idx", "w", "dw", "dl"):
        assert call(**{p: None}) == ARG, p
    assert call(dl=ctypes.c_void_p(0x1002)) == ARG
    assert call(n=0, l=None, idx=None, w=None, dw=None, dl=None) == 0
