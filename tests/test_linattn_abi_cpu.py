"""Refusals of the linear-attention and layer-norm entry points, on the CPU:
every bad call returns its status before anything is enqueued."""

import ctypes
import os

import pytest
import torch

from log_linear_attention_chunkwise_gb300 import binding

P, ODD, NULL = ctypes.c_void_p(256), ctypes.c_void_p(256 + 8), None
BIG = 1 << 40
OK, ARG, SHAPE, WS = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from log_linear_attention_chunkwise_gb300 import build
        build.build()
    return binding.load()


def call_fwd(lib, q=P, k=P, v=P, ld=P, lens=NULL, si=NULL, out=P, so=NULL, B=1, H=1, T=64, dk=64, dv=64, dt=1, ws=P,
             wsb=BIG):
    return lib.lla_linattn_fwd(q, k, v, ld, lens, si, out, so, B, H, T, dk, dv, dt, 0, ws, wsb, NULL, NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(dk=48), SHAPE), (dict(dv=8), SHAPE), (dict(dk=256), SHAPE), (dict(T=(1 << 24) + 1), SHAPE),
    (dict(B=70000), SHAPE), (dict(B=-1), ARG), (dict(T=-1), ARG), (dict(H=-1), ARG), (dict(dt=2), ARG),
    (dict(q=NULL), ARG), (dict(k=NULL), ARG), (dict(v=NULL), ARG), (dict(out=NULL), ARG), (dict(ld=NULL), ARG),
    (dict(q=ODD), ARG), (dict(v=ODD), ARG), (dict(out=ODD), ARG), (dict(si=ODD), ARG), (dict(so=ODD), ARG),
    (dict(T=1 << 20, wsb=0), WS), (dict(T=1 << 20, ws=NULL), ARG), (dict(T=1 << 20, ws=ctypes.c_void_p(256 + 16)), ARG),
    (dict(B=0, q=NULL, ld=NULL), OK), (dict(H=0), OK), (dict(T=0, q=NULL, k=NULL, v=NULL, out=NULL), OK),
])
def test_fwd_refusals(lib, kw, code):
    assert call_fwd(lib, **kw) == code


def test_workspace_queries(lib):
    f, b = lib.lla_linattn_fwd_workspace_bytes, lib.lla_linattn_bwd_workspace_bytes
    assert f(1, 1, 1 << 20, 128, 128, 1) > 0 and f(1, 1, 1 << 20, 128, 128, 1) % 256 == 0
    # one tile, or heads that fill the SMs: nothing to split
    for dtype in (0, 1):
        assert f(1, 1, 64, 128, 128, dtype) == 0 and f(64, 16, 4096, 128, 128, dtype) == 0
    assert b(1, 1, 1 << 20, 128, 64, 1) > 0
    for bad in ((1, 1, 64, 48, 64, 1), (0, 1, 64, 64, 64, 1), (1, 1, 0, 64, 64, 1), (1, 1, 64, 64, 64, 5)):
        assert f(*bad) == 0 and b(*bad) == 0
    n = lib.lla_linattn_norm_bwd_workspace_bytes(2, 3, 100, 64, 32, 1)
    assert n >= 2 * 3 * 100 * 32 * 2 + lib.lla_layer_norm_bwd_workspace_bytes(2, 3, 100, 32, 1)


def test_long_walks_are_cut(lib):
    # a walk's accumulator takes 256 tiles at most, however many heads there are; fp32 sums need no such cut
    f, b = lib.lla_linattn_fwd_workspace_bytes, lib.lla_linattn_bwd_workspace_bytes
    for tiles in (512, 513, 131072):
        n = (tiles + 255) // 256
        assert f(4, 76, 128 * tiles, 128, 64, 1) >= 4 * 76 * n * 128 * 64 * 4
        assert b(4, 76, 128 * tiles, 128, 64, 1) >= 2 * 4 * 76 * n * 128 * 64 * 4
    assert f(4, 76, 65536, 128, 64, 0) == 0


def test_bwd_refusals(lib):
    def bwd(q=P, do=P, dq=P, dv=P, ld=P, si=NULL, dso=NULL, dsi=NULL, B=1, T=64, dk=64, dt=1, ws=P, wsb=BIG):
        return lib.lla_linattn_bwd(q, P, P, ld, NULL, si, do, dso, dq, P, dv, dsi, B, 1, T, dk, 64, dt, 0, ws, wsb,
                                   NULL, NULL)
    assert bwd(dk=48) == SHAPE
    assert bwd(dt=9) == ARG
    for kw in (dict(q=NULL), dict(do=NULL), dict(dq=NULL), dict(dv=NULL), dict(ld=NULL), dict(do=ODD), dict(dq=ODD),
               dict(si=ODD), dict(dso=ODD), dict(dsi=ODD)):
        assert bwd(**kw) == ARG, kw
    assert bwd(dso=P, dsi=P) == ARG                # dk reads dstate_out while dstate_in is written
    assert bwd(si=P, dsi=P) == ARG                 # and dq state_in
    assert bwd(T=1 << 20, wsb=0) == WS
    assert bwd(B=0, q=NULL) == OK
    assert bwd(T=0, q=NULL, do=NULL, dq=NULL, dv=NULL) == OK


def test_decode_refusals(lib):
    def dec(S=P, q=P, ld=P, slots=NULL, out=P, pool=4, B=2, H=1, dk=64, dv=64, dt=1):
        return lib.lla_linattn_decode_step(S, q, P, P, ld, slots, out, pool, B, H, dk, dv, dt, 0, NULL, NULL)
    assert dec(dk=48) == SHAPE and dec(dv=12) == SHAPE and dec(B=70000, pool=70000) == SHAPE
    assert dec(dt=7) == ARG and dec(B=-1) == ARG and dec(pool=-1) == ARG
    assert dec(pool=1) == ARG                      # without slots every sequence has its own state
    for kw in (dict(S=NULL), dict(S=ODD), dict(q=NULL), dict(out=NULL), dict(ld=NULL), dict(q=ODD)):
        assert dec(**kw) == ARG, kw
    assert dec(B=0, S=NULL) == OK


def test_norm_refusals(lib):
    def fwd(x=P, w=P, y=P, B=1, H=1, T=3, N=100, eps=1e-5, dt=0):
        return lib.lla_layer_norm_fwd(x, w, NULL, NULL, y, NULL, NULL, B, H, T, N, eps, dt, 0, NULL, NULL)

    def bwd(x=P, w=P, mean=P, dy=P, dx=P, dw=P, B=1, T=3, N=100, dt=0, ws=P, wsb=BIG):
        return lib.lla_layer_norm_bwd(x, w, mean, P, NULL, dy, dx, dw, NULL, B, 1, T, N, dt, 0, ws, wsb, NULL, NULL)
    for f in (fwd, bwd):
        assert f(N=0) == SHAPE and f(N=16385) == SHAPE and f(B=70000) == SHAPE
        assert f(B=-1) == ARG and f(T=-1) == ARG and f(dt=3) == ARG
        assert f(x=NULL) == ARG and f(x=ODD) == ARG and f(w=ODD) == ARG
    assert fwd(eps=-1.0) == ARG and fwd(eps=float("nan")) == ARG and fwd(eps=float("inf")) == ARG
    assert fwd(y=NULL) == ARG and fwd(T=0, x=NULL) == OK
    assert bwd(mean=NULL) == ARG and bwd(dy=NULL) == ARG and bwd(dx=ODD) == ARG
    assert bwd(wsb=0) == WS and bwd(ws=NULL) == ARG


def test_norm_pair_refusals(lib):
    def fwd(q=P, o=P, y=P, w=P, eps=1e-5, T=64, dk=64):
        return lib.lla_linattn_norm_fwd(q, P, P, P, NULL, NULL, w, NULL, eps, o, y, NULL, NULL, NULL, 1, 1, T, dk, 64, 1,
                                        0, P, BIG, NULL, NULL)
    for kw in (dict(q=NULL), dict(o=NULL), dict(y=NULL), dict(y=ODD), dict(w=ODD), dict(eps=-1.0)):
        assert fwd(**kw) == ARG, kw
    assert fwd(dk=40) == SHAPE

    def bwd(q=P, o=P, mean=P, dy=P, dso=NULL, dsi=NULL, ld=P, dt=1, ws=P, wsb=BIG):
        return lib.lla_linattn_norm_bwd(q, P, P, ld, NULL, NULL, o, P, mean, P, dy, dso, P, P, P, P, P, dsi, 1, 1, 64,
                                        64, 64, dt, 0, ws, wsb, NULL, NULL)
    for kw in (dict(q=NULL), dict(o=NULL), dict(mean=NULL), dict(dy=ODD), dict(ld=NULL), dict(dso=P, dsi=P), dict(dt=4),
               dict(ws=NULL)):
        assert bwd(**kw) == ARG, kw
    assert bwd(wsb=0) == WS


def test_zero_padding_refusals(lib):
    def call(n=1, p=256, rb=64, rows=1, lens=P, B=1, H=1, T=8):
        ptrs, i32 = (ctypes.c_void_p * max(n, 1))(*[p] * max(n, 1)), ctypes.c_int32 * max(n, 1)
        return lib.lla_zero_padding(ptrs, i32(*[rb] * max(n, 1)), i32(*[rows] * max(n, 1)), n, lens, B, H, T, NULL)
    assert call(n=-1) == ARG and call(B=-1) == ARG and call(T=-1) == ARG and call(rb=-1) == ARG
    assert call(p=0) == ARG and call(lens=NULL) == ARG
    assert call(n=9) == SHAPE and call(B=70000) == SHAPE
    assert call(n=0) == OK and call(B=0) == OK and call(T=0, p=0) == OK and call(rb=0, p=0) == OK


def host(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


CALLS = {
    "linattn_fwd": lambda: binding.linattn_fwd(host(1, 2, 8, 16), host(1, 2, 8, 16), host(1, 2, 8, 16), host(2)),
    "linattn_bwd": lambda: binding.linattn_bwd(host(1, 2, 8, 16), host(1, 2, 8, 16), host(1, 2, 8, 16), host(2),
                                               host(1, 2, 8, 16)),
    "linattn_decode_step": lambda: binding.linattn_decode_step(host(3, 2, 16, 16), host(1, 2, 16), host(1, 2, 16),
                                                               host(1, 2, 16), host(2)),
    "layer_norm_fwd": lambda: binding.layer_norm_fwd(host(1, 1, 4, 8)),
    "layer_norm_bwd": lambda: binding.layer_norm_bwd(host(1, 1, 4, 8), None, host(1, 1, 4), host(1, 1, 4),
                                                     host(1, 1, 4, 8)),
    "linattn_norm_fwd": lambda: binding.linattn_norm_fwd(host(1, 2, 8, 16), host(1, 2, 8, 16), host(1, 2, 8, 16),
                                                         host(2)),
    "linattn_norm_bwd": lambda: binding.linattn_norm_bwd(host(1, 2, 8, 16), host(1, 2, 8, 16), host(1, 2, 8, 16),
                                                         host(2), host(1, 2, 8, 16), None, host(1, 2, 8),
                                                         host(1, 2, 8), host(1, 2, 8, 16)),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_host_tensors_are_refused(name, lib):
    with pytest.raises(ValueError, match="CUDA tensor"):
        CALLS[name]()
