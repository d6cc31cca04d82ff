"""GPU parity of layer norm and of the normalised linear-attention layer
against fp64.

Bounds.  A row sum of a thread's 16 values and the tree over the threads has
fewer than K = 64 roundings on the way of any term (16384 columns: 16 + 15),
products and powers among them, so with u = 2^-24 a centred value is off by at
most K u max|x| and y by K u (max|x| rstd + |h|) |w| besides its own rounding
(half a step, 2^-8 in bf16).  dx: every term carries at most K roundings.  dweight,
dbias: a term meets at most as many additions as there are rows."""

import numpy as np
import pytest
import torch

from linattn_reference import U16, U32, assert_close, f64, lin_inputs, linattn, linattn_grads, norm, norm_grads
from log_linear_attention_chunkwise_gb300 import binding

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
K = 64


def half(dtype):
    return U16 if dtype == BF16 else U32


def within(got, ref, bound, what):
    g = f64(got)
    assert np.isfinite(g).all(), what
    r = np.abs(g - ref) / (bound + 1e-37)
    assert (r <= 1).all(), (what, float(r.max()))


def inputs(B, H, T, N, dtype, seed, offset=1.0):
    gen = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    return ((randn(B, H, T, N) * 2 + offset).to(dtype), 1 + 0.3 * randn(H, N), 0.5 * randn(H, N),
            randn(B, H, T, N).to(dtype))


def y_bound(x, w, b, eps, dtype):
    y, mean, rstd = norm(x, w, b, eps)
    h = np.abs(f64(x) - mean[..., None]) * rstd[..., None]
    aw = 1.0 if w is None else np.abs(f64(w))[None, :, None]
    ab = 0.0 if b is None else np.abs(f64(b))[None, :, None]
    return y, mean, rstd, K * U32 * ((np.abs(f64(x)).max(-1) * rstd)[..., None] * (1 + h) + h) * aw + \
        2 * U32 * ab + half(dtype) * (np.abs(y) + 1e-5)


SIZES = [(1, 1, 1, 1), (1, 1, 3, 2), (1, 2, 5, 7), (2, 3, 9, 16), (1, 4, 33, 32), (2, 2, 70, 64), (3, 2, 129, 128),
         (1, 1, 6, 129), (1, 1, 5, 256), (1, 1, 9, 500), (1, 1, 4, 999), (1, 2, 3, 1024), (1, 1, 3, 2048), (1, 1, 5, 3001),
         (1, 1, 2, 4096), (1, 1, 2, 8191), (1, 1, 2, 8192), (1, 1, 2, 16384), (1, 1, 1, 16383), (1, 1, 5000, 24),
         (1, 1, 40, 6443), (2, 1, 5, 8191)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,H,T,N", SIZES)
def test_fwd_and_bwd(B, H, T, N, dtype, cuda_device):
    x, w, b, dy = inputs(B, H, T, N, dtype, seed=N + T)
    xd, wd, bd, dyd = (t.cuda() for t in (x, w, b, dy))
    y, mean, rstd = binding.layer_norm_fwd(xd, wd, bd, return_stats=True)
    ref, m, r, bound = y_bound(x, w, b, 1e-5, dtype)
    within(y, ref, bound, "y")
    big = np.abs(f64(x)).max(-1)
    within(mean, m, K * U32 * big, "mean")
    within(rstd, r, K * U32 * r * (1 + big * r), "rstd")
    dx, dw, db = binding.layer_norm_bwd(xd, wd, mean, rstd, dyd)
    # the given mean and rstd are inputs of the backward: compare at them
    gx, gw, gb = norm_grads(x, w, mean, rstd, dy)
    h = np.abs((f64(x) - f64(mean)[..., None]) * f64(rstd)[..., None])
    g = np.abs(f64(dy) * f64(w)[None, :, None])
    scale = f64(rstd)[..., None] * (g + g.mean(-1, keepdims=True) + h * (g * h).mean(-1, keepdims=True))
    within(dx, gx, K * U32 * scale + half(dtype) * (np.abs(gx) + K * U32 * scale), "dx")
    n = B * T + K
    within(dw, gw, n * U32 * (np.abs(f64(dy)) * h).sum((0, 2)), "dweight")
    within(db, gb, n * U32 * np.abs(f64(dy)).sum((0, 2)), "dbias")
    again = binding.layer_norm_bwd(xd, wd, mean, rstd, dyd)
    assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))


@pytest.mark.parametrize("B,H,T,N", [(1, 1, 8192, 2048), (2, 16, 4096, 128), (1, 3, 3000, 250), (1, 1, 500, 8192)])
def test_many_rows_many_times(B, H, T, N, cuda_device):
    """One call after the other without a wait, on two sets of inputs in turn: the same bits every time, the
    column sums those of fp64."""
    sets = []
    for seed in (1, 2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        sets.append((randn(B, H, T, N).to(BF16), 1 + 0.1 * randn(H, N), randn(H, N), randn(B, H, T, N).to(BF16)))

    def step(x, w, b, dy):
        y, mean, rstd = binding.layer_norm_fwd(x, w, b, return_stats=True)
        return (y, mean, rstd) + binding.layer_norm_bwd(x, w, mean, rstd, dy)

    first = [step(*s) for s in sets]
    torch.cuda.synchronize()
    for _ in range(10):
        again = [step(*s) for s in sets + sets]
        assert all(torch.equal(p, q) for r, f in zip(again, first + first) for p, q in zip(r, f))
    for (x, w, b, dy), (y, mean, rstd, dx, dw, db) in zip(sets, first):
        h = (x.double() - mean.double()[..., None]) * rstd.double()[..., None]
        for got, r, mag in ((dw, dy.double() * h, (dy.double() * h).abs()), (db, dy.double(), dy.double().abs())):
            assert bool(((got.double() - r.sum((0, 2))).abs() <= (B * T + K) * U32 * mag.sum((0, 2))).all())


def test_without_weight_and_bias(cuda_device):
    x, _, _, dy = inputs(2, 2, 10, 64, BF16, seed=1)
    y, mean, rstd = binding.layer_norm_fwd(x.cuda(), return_stats=True)
    ref, _, _, bound = y_bound(x, None, None, 1e-5, BF16)
    within(y, ref, bound, "y")
    dx, dw, db = binding.layer_norm_bwd(x.cuda(), None, mean, rstd, dy.cuda())
    one = binding.layer_norm_bwd(x.cuda(), torch.ones(2, 64, device="cuda"), mean, rstd, dy.cuda())
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), one))


@pytest.mark.parametrize("N,dtype", [(128, F32), (999, F32), (2048, F32)])
def test_a_large_mean_costs_no_digits_beyond_the_inputs(N, dtype, cuda_device):
    x, w, b, _ = inputs(1, 1, 6, N, dtype, seed=2, offset=1000.0)
    y = binding.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda())
    ref, _, _, bound = y_bound(x, w, b, 1e-5, dtype)
    within(y, ref, bound, "y")


def test_constant_rows(cuda_device):
    x = torch.full((1, 1, 3, 128), 2.5, dtype=BF16, device="cuda")
    y, mean, rstd = binding.layer_norm_fwd(x, bias=torch.full((1, 128), 0.5, device="cuda"), eps=1e-4, return_stats=True)
    assert bool((y == 0.5).all()) and bool((mean == 2.5).all())
    np.testing.assert_allclose(f64(rstd), 100.0, rtol=1e-6)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,H,T", [(1, 1, 38), (2, 3, 500)])
def test_rows_of_one_column(B, H, T, dtype, cuda_device):
    """Such a row is its own mean: y is the bias and x has no gradient, exactly, whatever g rounds to."""
    x, w, b, dy = (t.cuda() for t in inputs(B, H, T, 1, dtype, seed=4))
    y, mean, rstd = binding.layer_norm_fwd(x, w, b, return_stats=True)
    assert torch.equal(y, b.to(dtype)[None, :, None].expand_as(y)) and torch.equal(mean, x[..., 0].float())
    dx, dw, db = binding.layer_norm_bwd(x, w, mean, rstd, dy)
    assert bool((dx == 0).all()) and bool((dw == 0).all())
    n = B * T
    assert bool(((db.double()[:, 0] - dy.double().sum((0, 2, 3))).abs() <= n * U32 * dy.double().abs().sum((0, 2, 3))).all())


@pytest.mark.parametrize("N,dtype", [(64, BF16), (100, F32), (2048, BF16)])
def test_padded_batch(N, dtype, cuda_device):
    B, H, T = 4, 2, 37
    lens = [37, 0, 1, 20]
    x, w, b, dy = inputs(B, H, T, N, dtype, seed=3)
    xd, dyd = x.cuda(), dy.cuda()
    for i, n in enumerate(lens):
        xd[i, :, n:] = float("nan")
        dyd[i, :, n:] = float("inf")
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full((B, H, T, N), 7.0, dtype=dtype, device="cuda")
    y, mean, rstd = binding.layer_norm_fwd(xd, w.cuda(), b.cuda(), lens=ln, out=out, return_stats=True)
    ref, _, _, bound = y_bound(x, w, b, 1e-5, dtype)
    keep = np.arange(T)[None] < np.array(lens)[:, None]
    for i, n in enumerate(lens):
        assert bool((y[i, :, n:] == 7.0).all())
        within(y[i, :, :n], ref[i, :, :n], bound[i, :, :n], "y")
    dx, dw, db = binding.layer_norm_bwd(xd, w.cuda(), mean, rstd, dyd, lens=ln)
    gx, gw, gb = norm_grads(x, w, mean, rstd, dy, keep)
    np.testing.assert_allclose(f64(dw), gw, atol=1e-4, rtol=1e-5)
    np.testing.assert_allclose(f64(db), gb, atol=1e-4, rtol=1e-5)
    assert np.abs(f64(dx) - gx).max() <= 2 * U16 * np.abs(gx).max()
    for i, n in enumerate(lens):
        assert bool((dx[i, :, n:] == 0).all())
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ln[1] = T + 1
    binding.layer_norm_fwd(xd, lens=ln, device_error=err)
    assert binding.device_error_check(err) == 3


def test_in_place_and_empty(cuda_device):
    x, w, b, dy = (t.cuda() for t in inputs(2, 2, 50, 128, BF16, seed=4))
    want, mean, rstd = binding.layer_norm_fwd(x, w, b, return_stats=True)
    y = x.clone()
    assert binding.layer_norm_fwd(y, w, b, out=y) is y and torch.equal(y, want)
    e = x[:, :, :0].contiguous()
    assert binding.layer_norm_fwd(e, w, b).shape == (2, 2, 0, 128)
    dx, dw, db = binding.layer_norm_bwd(e, w, mean[:, :, :0].contiguous(), rstd[:, :, :0].contiguous(), e)
    assert dx.numel() == 0 and bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("B,H,T,d,dtype,lens", [(2, 3, 200, 128, BF16, None), (3, 2, 150, 64, F32, [150, 0, 70]),
                                                (1, 1, 1300, 128, BF16, None), (2, 2, 90, 32, BF16, [1, 90])])
def test_normalised_linear_attention(B, H, T, d, dtype, lens, cuda_device):
    """The two together, forward and backward, as a training step and a prompt call them."""
    x = lin_inputs(B, H, T, d, d, dtype, seed=T)
    h = {n: t.cuda() for n, t in x.items()}
    _, w, b, dy = inputs(B, H, T, d, dtype, seed=T + 1)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    names = ("q", "k", "v", "log_decay")
    args = [h[n] for n in names]
    y, o, mean, rstd, st = binding.linattn_norm_fwd(*args, w.cuda(), b.cuda(), lens=ln, state_in=h["state"], keep=True,
                                                    return_state=True)
    # the pair is its two parts, in place too
    o1, st1 = binding.linattn_fwd(*args, lens=ln, state_in=h["state"], return_state=True)
    y1, m1, r1 = binding.layer_norm_fwd(o1, w.cuda(), b.cuda(), lens=ln, return_stats=True)
    assert all(torch.equal(p, q) for p, q in zip((y, o, mean, rstd, st), (y1, o1, m1, r1, st1)))
    # in place, the state asked for as above (without it the last bits of o may differ)
    assert torch.equal(binding.linattn_norm_fwd(*args, w.cuda(), b.cuda(), lens=ln, state_in=h["state"],
                                                return_state=True)[0], y)
    got = binding.linattn_norm_bwd(*args, o, w.cuda(), mean, rstd, dy.cuda(), lens=ln, state_in=h["state"],
                                   dstate_out=h["dstate"], return_dstate=True)
    do, dw, db = binding.layer_norm_bwd(o, w.cuda(), mean, rstd, dy.cuda(), lens=ln)
    want = binding.linattn_bwd(*args, do, lens=ln, state_in=h["state"], dstate_out=h["dstate"], return_dstate=True)
    assert all(torch.equal(p, q) for p, q in zip(got, want[:3] + (dw, db) + want[3:]))
    # and against fp64 from the layer's own kept values
    keep = None if lens is None else np.arange(T)[None] < np.array(lens)[:, None]
    gd, gw, gb = norm_grads(o, w, mean, rstd, dy, keep)
    np.testing.assert_allclose(f64(dw), gw, atol=1e-3, rtol=1e-5)
    np.testing.assert_allclose(f64(db), gb, atol=1e-3, rtol=1e-5)
    ref = linattn_grads(x["q"], x["k"], x["v"], x["log_decay"], do, lens, x["state"], x["dstate"])
    wgt = linattn_grads(*(x[n].abs() for n in "qkv"), x["log_decay"], do.abs(), lens, x["state"].abs(), x["dstate"].abs())
    for name, g, r, a in zip(("dq", "dk", "dv", "dstate"), got[:3] + got[5:], ref, wgt):
        assert_close(g, r, a, F32 if name == "dstate" else dtype, d, d, T, name)


def test_refusals(cuda_device):
    x = torch.zeros(1, 2, 3, 64, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        binding.layer_norm_fwd(x, torch.ones(64, device="cuda"))
    with pytest.raises(TypeError):
        binding.layer_norm_fwd(x.half())
    with pytest.raises(binding.LLAError, match="INVALID_ARGUMENT"):
        binding.layer_norm_fwd(x, eps=-1.0)
    with pytest.raises(binding.LLAError, match="UNSUPPORTED_SHAPE"):
        binding.layer_norm_fwd(torch.zeros(1, 1, 1, 16385, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        binding.layer_norm_fwd(torch.zeros(1, 2, 64, 3, device="cuda").transpose(2, 3))


@pytest.mark.parametrize("B,H,T,N", [(1, 1, 20000, 132), (2, 3, 2100, 160), (1, 2, 9001, 252), (1, 1, 20000, 256), (3, 2, 17, 192)])
def test_fp32_rows_of_two_pieces_a_thread(B, H, T, N, cuda_device):
    """132 to 256 columns in single precision, many turns a CTA."""
    test_fwd_and_bwd(B, H, T, N, F32, cuda_device)


def raw_bwd(x, w, mean, rstd, dy, dx, dw, db, ws):
    """lla_layer_norm_bwd itself: outputs that may be absent or the same buffer as an input."""
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    B, H, T, N = x.shape
    return binding.load().lla_layer_norm_bwd(
        p(x), p(w), p(mean), p(rstd), None, p(dy), p(dx), p(dw), p(db), B, H, T, N, int(x.dtype == BF16), 0, p(ws),
        0 if ws is None else ws.numel(), None, torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("N,dtype", [(64, BF16), (256, F32), (999, BF16), (2048, F32)])
def test_gradients_that_are_not_asked_for_and_in_place(N, dtype, cuda_device):
    x, w, b, dy = (t.cuda() for t in inputs(2, 3, 40, N, dtype, seed=6))
    _, mean, rstd = binding.layer_norm_fwd(x, w, b, return_stats=True)
    dx, dw, db = binding.layer_norm_bwd(x, w, mean, rstd, dy)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    for names in ((), ("dw",), ("db",), ("dw", "db")):
        got = {n: torch.full_like(dw, 7.0) for n in names}
        for into in ("new", "dy", "x"):
            gx, gdy, gin = torch.full_like(x, 7.0), dy.clone(), x.clone()
            gx = {"new": gx, "dy": gdy, "x": gin}[into]
            assert raw_bwd(gin, w, mean, rstd, gdy, gx, got.get("dw"), got.get("db"), ws if names else None) == 0
            assert torch.equal(gx, dx)
            assert all(torch.equal(g, {"dw": dw, "db": db}[n]) for n, g in got.items())
