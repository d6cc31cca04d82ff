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


# ---- outputs that overlap what the call reads, or one another

def at(i, shift=0):
    return ctypes.c_void_p((i << 40) + shift)


N_ROWS, N_STATE = 2 * 3 * 100 * 64 * 2, 2 * 3 * 64 * 64 * 4  # bytes of [2,3,100,64] bf16, of the states


def spans(base, size):
    """The buffer itself, and overlaps by its last and by its first 16 bytes."""
    return [at(base), at(base, size - 16), at(base, 16 - size)]


def test_fwd_overlaps_are_refused(lib):
    def fwd(out=at(4), so=at(6), norm=False, y=at(7), mean=at(8), rstd=at(9)):
        a = (at(1), at(2), at(3), at(10), NULL, at(5))
        if norm:
            return lib.lla_linattn_norm_fwd(*a, at(11), at(12), 1e-5, out, y, mean, rstd, so, 2, 3, 100, 64, 64, 1, 0,
                                            at(13), BIG, NULL, NULL)
        return lib.lla_linattn_fwd(*a, out, so, 2, 3, 100, 64, 64, 1, 0, at(13), BIG, NULL, NULL)

    for norm in (False, True):
        for base, size in ((1, N_ROWS), (2, N_ROWS), (3, N_ROWS), (5, N_STATE)):
            for p in spans(base, min(size, N_ROWS)):
                assert fwd(out=p, norm=norm) == ARG, (norm, base)
        for base in (1, 2, 3, 4):
            for p in spans(base, N_ROWS):
                assert fwd(so=p, norm=norm) == ARG, (norm, base)
        for p in spans(5, N_STATE)[1:]:  # a part of state_in; the whole of it is allowed
            assert fwd(so=p, norm=norm) == ARG, norm
    for p in spans(4, N_ROWS)[1:]:       # a part of o; the whole of it is allowed
        assert fwd(y=p, norm=True) == ARG
    for kw in (dict(y=at(6)), dict(mean=at(4)), dict(rstd=at(8)), dict(mean=at(7)), dict(y=at(11)), dict(rstd=at(6))):
        assert fwd(norm=True, **kw) == ARG, kw


def test_bwd_overlaps_are_refused(lib):
    def bwd(norm=False, dw=at(14), db=at(15), **kw):
        o = {"dq": at(7), "dk": at(8), "dv": at(9), "ds": at(10), **kw}
        a, tail = (at(1), at(2), at(3), at(11), NULL, at(5)), (2, 3, 100, 64, 64, 1, 0, at(13), BIG, NULL, NULL)
        if norm:
            return lib.lla_linattn_norm_bwd(*a, at(16), at(17), at(18), at(19), at(4), at(6), o["dq"], o["dk"], o["dv"],
                                            dw, db, o["ds"], *tail)
        return lib.lla_linattn_bwd(*a, at(4), at(6), o["dq"], o["dk"], o["dv"], o["ds"], *tail)

    for norm in (False, True):
        for name in ("dq", "dk", "dv", "ds"):
            for base, size in ((1, N_ROWS), (2, N_ROWS), (3, N_ROWS), (5, N_STATE), (6, N_STATE)):
                for p in spans(base, min(size, N_ROWS)):
                    assert bwd(norm, **{name: p}) == ARG, (norm, name, base)
        for a, b in (("dq", 8), ("dk", 9), ("dv", 7), ("ds", 7), ("dq", 10)):
            assert bwd(norm, **{a: at(b, 32)}) == ARG, (norm, a, b)
    assert bwd(dq=at(4)) == ARG
    for kw in (dict(dw=at(15)), dict(dw=at(16)), dict(db=at(4)), dict(dw=at(17)), dict(db=at(1)), dict(dw=at(9))):
        assert bwd(True, **kw) == ARG, kw


def test_norm_overlaps_are_refused(lib):
    size = 3 * 50 * 100 * 4

    def fwd(y=at(4), mean=at(5), rstd=at(6)):
        return lib.lla_layer_norm_fwd(at(1), at(2), at(3), NULL, y, mean, rstd, 1, 3, 50, 100, 1e-5, 0, 0, NULL, NULL)

    def bwd(dx=at(6), dw=at(7), db=at(8)):
        return lib.lla_layer_norm_bwd(at(1), at(2), at(3), at(4), NULL, at(5), dx, dw, db, 1, 3, 50, 100, 0, 0, at(13),
                                      BIG, NULL, NULL)
    for p in spans(1, size)[1:]:
        assert fwd(y=p) == ARG and bwd(dx=p) == ARG
    for p in spans(5, size)[1:]:
        assert bwd(dx=p) == ARG
    for kw in (dict(y=at(2)), dict(y=at(3)), dict(y=at(5)), dict(mean=at(1)), dict(rstd=at(1, 64)), dict(mean=at(6)),
               dict(mean=at(2))):
        assert fwd(**kw) == ARG, kw
    for kw in (dict(dx=at(2)), dict(dx=at(3)), dict(dx=at(4)), dict(dx=at(7)), dict(dw=at(8)), dict(dw=at(1)),
               dict(db=at(5)), dict(dw=at(3)), dict(db=at(2))):
        assert bwd(**kw) == ARG, kw


def test_decode_overlaps_are_refused(lib):
    def dec(state=at(1), out=at(5), dt=0):
        return lib.lla_linattn_decode_step(state, at(2), at(3), at(4), at(6), NULL, out, 4, 2, 3, 64, 64, dt, 0, NULL, NULL)
    for base, size in ((1, 2 * 3 * 64 * 4), (2, 2 * 3 * 64 * 4), (3, 2 * 3 * 64 * 4), (4, 2 * 3 * 64 * 4)):
        for p in spans(base, size):
            assert dec(out=p) == ARG, base
    for base in (2, 3, 4):
        assert dec(state=at(base)) == ARG and dec(state=at(base, 256)) == ARG


def test_a_stream_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    stream = type("Stream", (), {"device": torch.device("cuda", 1), "cuda_stream": 16})()
    called = []
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        binding._launch(stream, called.append)
    assert not called
