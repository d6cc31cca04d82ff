"""GPU parity of linear attention with per-head decays (forward, backward,
single tokens) against the fp64 recurrence.  Bounds: linattn_reference."""

import numpy as np
import pytest
import torch

from linattn_reference import U16, assert_close, f64, lin_inputs, linattn, linattn_grads
from log_linear_attention_chunkwise_gb300 import binding

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def dev(x):
    return {n: t.cuda() for n, t in x.items()}


def absolute(x):
    return {n: (t if n == "log_decay" else t.abs()) for n, t in x.items()}


def check_fwd(x, lens, state, got, T):
    dk, dv = x["q"].shape[-1], x["v"].shape[-1]
    ax = absolute(x)
    ref = linattn(x["q"], x["k"], x["v"], x["log_decay"], lens, x["state"] if state else None)
    wgt = linattn(ax["q"], ax["k"], ax["v"], x["log_decay"], lens, ax["state"] if state else None)
    assert_close(got[0], ref[0], wgt[0], x["q"].dtype, dk, dv, T, "out")
    if len(got) > 1:
        assert_close(got[1], ref[1], wgt[1], F32, dk, dv, T, "state")


SHAPES = [
    # B, H, T, dk, dv, dtype, state, lens
    (1, 1, 1, 128, 128, BF16, False, None), (2, 2, 1, 64, 64, BF16, True, None), (1, 2, 2, 16, 16, F32, True, None),
    (1, 2, 127, 128, 128, BF16, True, None), (1, 2, 128, 128, 128, BF16, False, None),
    (2, 1, 129, 128, 128, BF16, True, None), (1, 3, 255, 64, 64, BF16, True, None), (1, 2, 333, 64, 64, F32, True, None),
    (1, 2, 500, 128, 128, F32, True, None), (2, 2, 200, 128, 64, BF16, True, None), (1, 2, 200, 64, 128, BF16, True, None),
    (1, 2, 150, 16, 128, F32, False, None), (1, 1, 150, 128, 16, BF16, True, None), (1, 2, 97, 32, 32, BF16, True, None),
    # padded batches: empty, one-token and tile-edge sequences among full ones
    (5, 2, 300, 128, 128, BF16, True, [300, 0, 1, 129, 256]), (4, 2, 130, 64, 64, BF16, False, [0, 130, 64, 65]),
    (3, 2, 140, 32, 64, F32, True, [140, 0, 77]), (2, 1, 128, 128, 128, BF16, True, [0, 0]),
    # few heads, many tokens: cut into segments
    (1, 1, 2000, 128, 128, BF16, True, None), (1, 2, 1500, 64, 64, BF16, True, None), (1, 1, 1700, 32, 32, F32, True, None),
    (2, 1, 1900, 128, 128, BF16, True, [1900, 700]), (2, 1, 1400, 128, 128, F32, False, [0, 1291]),
]


@pytest.mark.parametrize("B,H,T,dk,dv,dtype,state,lens", SHAPES)
def test_fwd(B, H, T, dk, dv, dtype, state, lens, cuda_device):
    x = lin_inputs(B, H, T, dk, dv, dtype, seed=B * 1000 + T + dk)
    d = dev(x)
    if lens is not None:  # whatever stands behind a sequence's end is not read
        for b, n in enumerate(lens):
            for name in ("q", "k", "v"):
                d[name][b, :, n:] = float("nan") if b % 2 else float("inf")
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((B, H, T, dv), 7.0, dtype=dtype, device="cuda")
    got = binding.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], lens=ln, state_in=d["state"] if state else None,
                              return_state=True, out=out, device_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    o = f64(got[0])
    for b, n in enumerate(lens or []):
        assert (o[b, :, n:] == 7.0).all(), "rows behind the sequence changed"
        got[0][b, :, n:] = 0
    check_fwd(x, lens, state, got, T)
    again = binding.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], lens=ln, state_in=d["state"] if state else None,
                                return_state=True)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])  # the same bits every time


@pytest.mark.parametrize("B,H,T,dk,dv,dtype,state,lens", SHAPES)
def test_bwd(B, H, T, dk, dv, dtype, state, lens, cuda_device):
    x = lin_inputs(B, H, T, dk, dv, dtype, seed=B * 1000 + T + dk + 1)
    d, ax = dev(x), absolute(x)
    if lens is not None:
        for b, n in enumerate(lens):
            for name in ("q", "k", "v", "dout"):
                d[name][b, :, n:] = float("inf") if b % 2 else float("nan")
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    kw = dict(lens=ln, state_in=d["state"] if state else None, dstate_out=d["dstate"] if state else None)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = binding.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["dout"], return_dstate=True, device_error=err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    both = [linattn_grads(u["q"], u["k"], u["v"], x["log_decay"], u["dout"], lens, u["state"] if state else None,
                          u["dstate"] if state else None) for u in (x, ax)]
    for name, g, r, w in zip(("dq", "dk", "dv", "dstate"), got, *both):
        assert_close(g, r, w, F32 if name == "dstate" else dtype, dk, dv, T, name)
    again = binding.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["dout"], return_dstate=True, **kw)
    assert all(torch.equal(a, g) for a, g in zip(again, got))


@pytest.mark.parametrize("B,H,T,d,padded", [(8, 16, 1000, 128, False), (8, 16, 1000, 128, True), (1, 16, 2432, 128, False),
                                            (12, 16, 700, 64, True), (2, 16, 2500, 64, False), (40, 8, 300, 128, True)])
def test_many_tiles_many_times(B, H, T, d, padded, cuda_device):
    """Walks of many tiles on every SM, one after the other without a wait: every call gives the same bits, and
    the right ones (against fp64 products on the GPU, block by block of the definition)."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    q, v, do = ((randn(B, H, T, d) / n).to(BF16) for n in (d ** 0.5, 1.0, 1.0))
    k = randn(B, H, T, d)
    k = (k / k.norm(dim=-1, keepdim=True)).to(BF16)
    ld = -torch.exp2(-8.0 + 4.0 * torch.rand(H, generator=gen, device="cuda"))
    S0, dS = randn(B, H, d, d), randn(B, H, d, d)
    lens = torch.randint(0, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32) if padded else None
    kw = dict(lens=lens, state_in=S0)

    def step():
        return binding.linattn_fwd(q, k, v, ld, return_state=True, **kw) + (binding.linattn_fwd(q, k, v, ld, **kw),) + \
            binding.linattn_bwd(q, k, v, ld, do, dstate_out=dS, return_dstate=True, **kw)

    first = step()
    for _ in range(6):
        again = [step() for _ in range(3)]
        assert all(torch.equal(a, b) for r in again for a, b in zip(r, first))
    n = torch.full((B,), T, device="cuda") if lens is None else lens.long()
    t = torch.arange(T, device="cuda")
    on = t < n[:, None]
    names = ("out", "state", "out without state", "dq", "dk", "dv", "dstate")
    worst = dict.fromkeys(names, (0.0, 0.0))
    for h in range(H):
        a = ld[h].double()
        w = torch.where(t[:, None] >= t, torch.exp(a * (t[:, None] - t).clamp_min(0)), 0.0)
        to_end = torch.where(on, torch.exp(a * (n[:, None] - 1 - t).clamp_min(0)), 0.0)[..., None]
        after, an = torch.exp(a * (t + 1))[:, None], torch.exp(a * n)[:, None, None]
        x, y, z, g = (torch.where(on[..., None], u[:, h].double(), 0.0) for u in (q, k, v, do))
        P, R = x @ y.mT * w, g @ z.mT * w
        S, D = S0[:, h].double(), dS[:, h].double()
        out = P @ z + after * (x @ S)
        ref = (out, y.mT @ (to_end * z) + an * S, out, R @ y + after * (g @ S.mT), R.mT @ x + to_end * (z @ D.mT),
               P.mT @ g + to_end * (y @ D), x.mT @ (after * g) + an * D)
        for name, r, f in zip(names, ref, first):
            r = r if r.shape[1] != T or "state" == name or name == "dstate" else torch.where(on[..., None], r, 0.0)
            e, s = worst[name]
            worst[name] = (e + float((f[:, h].double() - r).square().sum()), s + float(r.square().sum()))
    for name, (e, s) in worst.items():
        assert (e / s) ** 0.5 <= (1e-5 if name in ("state", "dstate") else U16), (name, (e / s) ** 0.5)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 32)])
def test_decay_extremes(dtype, d, cuda_device):
    """a = 1 (plain sums), a = 0 from -inf and from a huge rate (each token sees itself), and fast decays
    whose powers underflow inside a tile."""
    x = lin_inputs(1, 5, 300, d, d, dtype, seed=5)
    x["log_decay"] = torch.tensor([0.0, float("-inf"), -1e30, -5.0, -40.0])
    h = dev(x)
    got = binding.linattn_fwd(h["q"], h["k"], h["v"], h["log_decay"], state_in=h["state"], return_state=True)
    check_fwd(x, None, True, got, 300)
    g = binding.linattn_bwd(h["q"], h["k"], h["v"], h["log_decay"], h["dout"], state_in=h["state"],
                            dstate_out=h["dstate"], return_dstate=True)
    ax = absolute(x)
    both = [linattn_grads(u["q"], u["k"], u["v"], x["log_decay"], u["dout"], None, u["state"], u["dstate"])
            for u in (x, ax)]
    for name, a, r, w in zip(("dq", "dk", "dv", "dstate"), g, *both):
        assert_close(a, r, w, F32 if name == "dstate" else dtype, d, d, 300, name)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 64)])
def test_prompt_in_pieces_then_single_tokens(dtype, d, cuda_device):
    """A prompt taken in two pieces in place, then decoded token by token, is one long sequence."""
    B, H, T = 3, 2, 310
    x = lin_inputs(B, H, T, d, d, dtype, seed=9)
    h = dev(x)
    cut, end = 190, 300
    part = lambda n, a, b: h[n][:, :, a:b].contiguous()  # noqa: E731
    pool = torch.zeros(B + 2, H, d, d, device="cuda")
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    state = h["state"].clone()
    outs = []
    for a, b in ((0, cut), (cut, end)):
        o, s = binding.linattn_fwd(part("q", a, b), part("k", a, b), part("v", a, b), h["log_decay"], state_in=state,
                                   state_out=state)
        assert s is state
        outs.append(o)
    pool[slots.long()] = state
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    steps = []
    for t in range(end, T):
        steps.append(binding.linattn_decode_step(pool, *(h[n][:, :, t].contiguous() for n in "qkv"), h["log_decay"],
                                                 slots=slots, device_error=err))
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    ax = absolute(x)
    ref = linattn(x["q"], x["k"], x["v"], x["log_decay"], None, x["state"])
    wgt = linattn(ax["q"], ax["k"], ax["v"], x["log_decay"], None, ax["state"])
    assert_close(torch.cat(outs, 2), ref[0][:, :, :end], wgt[0][:, :, :end], dtype, d, d, T, "prompt")
    # the fp32 read-out of an fp32 state: fp32 bounds for bf16 inputs too
    assert_close(torch.stack(steps, 2), ref[0][:, :, end:], wgt[0][:, :, end:], F32, d, d, T, "tokens")
    assert_close(pool[slots.long()], ref[1], wgt[1], F32, d, d, T, "states")
    assert bool((pool[[1, 3]] == 0).all())


@pytest.mark.parametrize("dk,dv,dtype", [(128, 128, BF16), (16, 16, F32), (32, 128, BF16), (128, 16, F32), (64, 32, BF16)])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 5)])
def test_decode(B, H, dk, dv, dtype, cuda_device):
    x = lin_inputs(B, H, 1, dk, dv, dtype, seed=dk + dv)
    h, ax = dev(x), absolute(x)
    state = h["state"].clone()
    q, k, v = (h[n][:, :, 0].contiguous() for n in "qkv")
    o = binding.linattn_decode_step(state, q, k, v, h["log_decay"])
    ref = linattn(x["q"], x["k"], x["v"], x["log_decay"], None, x["state"])
    wgt = linattn(ax["q"], ax["k"], ax["v"], x["log_decay"], None, ax["state"])
    assert_close(o, ref[0][:, :, 0], wgt[0][:, :, 0], F32, dk, dv, 1, "out")
    assert_close(state, ref[1], wgt[1], F32, dk, dv, 1, "state")


def test_decode_slots_that_are_padding_out_of_range_or_named_twice(cuda_device):
    B, H, d, pool = 6, 2, 64, 5
    x = dev(lin_inputs(B, H, 1, d, d, BF16, seed=3))
    q, k, v = (x[n][:, :, 0].contiguous() for n in "qkv")
    base = torch.randn(pool, H, d, d, device="cuda")
    clean = base[:B - 1].clone()

    def step(slots):
        state, out = base.clone(), torch.full((B, H, d), 3.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        binding.linattn_decode_step(state, q, k, v, x["log_decay"], out=out, device_error=err,
                                    slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
        return state, out, int(err.item())

    state, out, err = step([2, -1, 0, 4, -1, 1])
    assert err == 0 and bool((out[[1, 4]] == 3.0).all()) and torch.equal(state[3], clean[3])
    assert bool((out[[0, 2, 3, 5]] != 3.0).any(-1).all())
    state, out, err = step([2, 5, 0, 4, 1, 3])       # 5 is outside the pool
    assert err == 2 and bool((out[1] == 3.0).all())
    state, out, err = step([2, -1, 0, 2, 1, 3])      # 0 and 3 name the same state
    assert err in (1, 4) and bool((out[[0, 3]] == 3.0).all()) and torch.equal(state[2], clean[2])
    assert not torch.equal(state[0], clean[0])
    # rows of an out made here are 0 where no state was read, on memory that held other values
    torch.full((B, H, d), 3.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = binding.linattn_decode_step(base.clone(), q, k, v, x["log_decay"], device_error=err,
                                      slots=torch.tensor([2, -1, 0, 2, 1, 9], dtype=torch.int32, device="cuda"))
    assert bool((out[[0, 1, 3, 5]] == 0).all()) and bool((out[[2, 4]] != 0).any(-1).all()) and int(err.item()) in (1, 4, 6)


@pytest.mark.parametrize("T,H", [(300, 2), (1700, 1)])
def test_bad_length_is_reported_and_its_sequence_left_alone(T, H, cuda_device):
    x = lin_inputs(3, H, T, 128, 128, BF16, seed=2)
    h = dev(x)
    for bad in (-1, T + 1):
        lens = torch.tensor([T, bad, 5], dtype=torch.int32, device="cuda")
        out, st = torch.full_like(h["v"], 7.0), torch.full((3, H, 128, 128), 7.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        binding.linattn_fwd(h["q"], h["k"], h["v"], h["log_decay"], lens=lens, out=out, state_out=st, device_error=err)
        assert binding.device_error_check(err) == 3
        assert bool((out[1] == 7.0).all()) and bool((st[1] == 7.0).all())
        ref, _ = linattn(x["q"][[0, 2]], x["k"][[0, 2]], x["v"][[0, 2]], x["log_decay"], [T, 5])
        np.testing.assert_allclose(f64(out[[0, 2]])[1, :, :5], ref[1, :, :5], atol=2e-2)
        err.zero_()
        g = binding.linattn_bwd(h["q"], h["k"], h["v"], h["log_decay"], h["dout"], lens=lens, device_error=err)
        assert binding.device_error_check(err) == 3 and all(bool((t[1] == 0).all()) for t in g)


def test_no_tokens(cuda_device):
    x = dev(lin_inputs(2, 3, 0, 32, 16, F32, seed=4))
    o, s = binding.linattn_fwd(x["q"], x["k"], x["v"], x["log_decay"], state_in=x["state"], return_state=True)
    assert o.shape == (2, 3, 0, 16) and torch.equal(s, x["state"])
    _, s = binding.linattn_fwd(x["q"], x["k"], x["v"], x["log_decay"], return_state=True)
    assert bool((s == 0).all())
    g = binding.linattn_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["dout"], dstate_out=x["dstate"], return_dstate=True)
    assert torch.equal(g[3], x["dstate"]) and g[0].shape == (2, 3, 0, 32)


@pytest.mark.parametrize("T,d,dtype", [(400, 128, BF16), (1500, 128, BF16), (300, 32, F32)])
def test_graph_and_streams(T, d, dtype, cuda_device):
    """Captured and replayed on new inputs, and run on a stream of its own."""
    xs = [dev(lin_inputs(1, 2, T, d, d, dtype, seed=s)) for s in (1, 2)]
    buf = {n: t.clone() for n, t in xs[0].items()}
    names = ("q", "k", "v", "log_decay")

    def step(x):
        o, s = binding.linattn_fwd(*(x[n] for n in names), state_in=x["state"], return_state=True)
        return (o, s) + binding.linattn_bwd(*(x[n] for n in names), x["dout"], state_in=x["state"],
                                            dstate_out=x["dstate"], return_dstate=True)

    want = [[t.clone() for t in step(x)] for x in xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(buf)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step(buf)
    for x, w in ((xs[1], want[1]), (xs[0], want[0])):
        for n in buf:
            buf[n].copy_(x[n])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, w))
    # the same call, the state asked for as above: without it the last bits of out may differ
    o, _ = binding.linattn_fwd(*(xs[1][n] for n in names), state_in=xs[1]["state"], return_state=True, stream=side)
    side.synchronize()
    assert torch.equal(o, want[1][0])


@pytest.mark.parametrize("T,H,d,padded", [(1500, 2, 128, False), (700, 24, 64, True), (260, 40, 128, True)])
def test_two_streams_at_once(T, H, d, padded, cuda_device):
    """Calls that share the GPU (split, whole, with the state's pass behind them) give what they give alone."""
    xs = [dev(lin_inputs(2, H, T, d, d, BF16, seed=s)) for s in (3, 4)]
    lens = torch.tensor([T, T // 3], dtype=torch.int32, device="cuda") if padded else None

    def step(x):
        a = tuple(x[n] for n in ("q", "k", "v", "log_decay"))
        y = binding.linattn_norm_fwd(*a, lens=lens, state_in=x["state"], keep=True, return_state=True)
        return y + binding.linattn_norm_bwd(*a, y[1], None, y[2], y[3], x["dout"], lens=lens, state_in=x["state"],
                                            dstate_out=x["dstate"], return_dstate=True)

    want = [[t.clone() for t in step(x)] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(step(xs[i]))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for call in g:
            assert all(torch.equal(t, u) for t, u in zip(call, w))


def test_offsets_past_32_bits(cuda_device):
    """Tensors of more than 2^31 values: the last head's rows are what that head gives alone (to the roundings of
    another cut into segments), the last rows of a norm the same bits, and a state far into a pool is the one used."""
    H, T, d = 130, 131072, 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((1, H, T, d), generator=gen, device="cuda", dtype=BF16) / d ** 0.5
    ld = torch.full((H,), -0.01, device="cuda")
    last = x[:, H - 1:].contiguous()

    def close(a, b):
        a, b = a.double(), b.double()
        assert bool(((a - b).norm() <= 2 * U16 * b.norm()))

    lens = torch.tensor([T - 5], dtype=torch.int32, device="cuda")
    out, state = binding.linattn_fwd(x, x, x, ld, lens=lens, return_state=True)
    alone = binding.linattn_fwd(last, last, last, ld[:1], lens=lens, return_state=True)
    close(out[:, H - 1:], alone[0])
    assert bool((out[0, H - 1, T - 5:] == 0).all())
    np.testing.assert_allclose(f64(state[:, H - 1:]), f64(alone[1]), rtol=0, atol=1e-5 * float(alone[1].abs().max()))
    del out
    grads = binding.linattn_bwd(x, x, x, ld, x, lens=lens)
    for g, r in zip(grads, binding.linattn_bwd(last, last, last, ld[:1], last, lens=lens)):
        close(g[:, H - 1:], r)
    del grads
    rows, N = x.view(1, 1, -1, 8192), 8192
    end = rows[:, :, -40:].contiguous()
    y, mean, rstd = binding.layer_norm_fwd(rows, return_stats=True)
    y2, mean2, rstd2 = binding.layer_norm_fwd(end, return_stats=True)
    assert torch.equal(y[:, :, -40:], y2) and torch.equal(mean[:, :, -40:], mean2)
    del y
    dx = binding.layer_norm_bwd(rows, None, mean, rstd, rows)[0]
    assert torch.equal(dx[:, :, -40:], binding.layer_norm_bwd(end, None, mean2, rstd2, end)[0])
    del dx, rows, x
    pool, slots = torch.zeros((135000, 1, d, d), device="cuda"), [134999, 3]
    few = torch.randn((2, 1, d, d), generator=gen, device="cuda")
    pool[slots] = few
    q = last[0, 0, :2, None].contiguous()
    o = binding.linattn_decode_step(pool, q, q, q, ld[:1], slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    assert torch.equal(o, binding.linattn_decode_step(few, q, q, q, ld[:1])) and torch.equal(pool[slots], few)
    del pool
    torch.cuda.empty_cache()


@pytest.mark.parametrize("shape,dtype", [((3, 2, 37, 128), BF16), ((3, 2, 37, 5), BF16), ((3, 1, 2000, 64), F32), ((3, 2, 9), F32)])
def test_zero_padding(shape, dtype, cuda_device):
    T = shape[2]
    lens = torch.tensor([T, 0, T // 2], dtype=torch.int32, device="cuda")
    x, y = (torch.full(shape, 5.0, dtype=dtype, device="cuda") for _ in range(2))
    around = torch.full((y.numel() + 8,), 5.0, dtype=dtype, device="cuda")
    z = around[4:-4].view(shape)  # a base that is not 16-byte aligned, with neighbours to keep
    binding.zero_padding([x, y, z], lens)
    for t in (x, y, z):
        for b, n in enumerate(lens.tolist()):
            assert bool((t[b, :, :n] == 5.0).all()) and bool((t[b, :, n:] == 0).all())
    assert bool((around[:4] == 5.0).all()) and bool((around[-4:] == 5.0).all())
    lens[0] = T + 1  # a length that makes no sense leaves no row of the sequence
    binding.zero_padding([x], lens)
    assert bool((x[0] == 0).all())
    with pytest.raises(ValueError):
        binding.zero_padding([x, x[:, :1].contiguous()] if shape[1] > 1 else [x, x[:2].contiguous()], lens)


def test_refusals(cuda_device):
    x = dev(lin_inputs(1, 2, 20, 64, 64, BF16, seed=1))
    f = lambda **kw: binding.linattn_fwd(**{**{n: x[n] for n in ("q", "k", "v", "log_decay")}, **kw})  # noqa: E731
    with pytest.raises(ValueError, match="contiguous"):
        f(q=x["q"].transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(TypeError):
        f(k=x["k"].float())
    with pytest.raises(TypeError):
        f(**{n: x[n].half() for n in "qkv"})
    with pytest.raises(ValueError, match="shape"):
        f(log_decay=x["log_decay"][:1].contiguous())
    with pytest.raises(ValueError, match="shape"):
        f(lens=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        f(lens=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(binding.LLAError, match="UNSUPPORTED_SHAPE"):
        f(q=x["q"][..., :48].contiguous(), k=x["k"][..., :48].contiguous())
    odd = torch.empty(1 * 2 * 20 * 64 + 1, dtype=BF16, device="cuda")[1:].view(1, 2, 20, 64)
    with pytest.raises(binding.LLAError, match="INVALID_ARGUMENT"):
        f(q=odd)
    with pytest.raises(binding.LLAError, match="INVALID_ARGUMENT"):
        binding.linattn_decode_step(torch.zeros(1, 2, 64, 64, device="cuda"), *(torch.zeros(2, 2, 64, device="cuda"),) * 3,
                                    x["log_decay"])


@pytest.mark.parametrize("T,d", [(524288, 16), (262144, 128)])
def test_long_sums_without_decay(T, d, cuda_device):
    """a = 1 over 4096 and 2048 tiles, a head on every SM: a walk's own state, which is not rounded to nearest, must not
    drift with T.  The last 32768 tokens (for the gradients of k and v the first) are compared with a call on those
    alone from the state of the others, which is handed out in fp32 accuracy.  The share by which the outputs fall
    short is their projection on those; what roundings to nearest leave of it is random: 2^-8 / sqrt(3) of an operand,
    shared by the d d elements of a head's state, of which at least d count (q = k, a growing diagonal): four
    deviations over 152 d of them are less than 2^-12."""
    H, part = 152, 32768
    x = torch.empty((1, H, T, d), device="cuda", dtype=BF16)
    gen = torch.Generator(device="cuda").manual_seed(6)
    for h in range(H):
        x[0, h] = torch.randn((T, d), generator=gen, device="cuda") / d ** 0.5
    ld = torch.zeros(H, device="cuda")

    def check(got, ref, name):
        a = r = 0.0
        for h in range(H):
            g, f = got[0, h].double(), ref[0, h].double()
            a, r = a + float((g * f).sum()), r + float(f.square().sum())
        assert abs(a / r - 1.0) <= 2.0 ** -12, (name, a / r - 1.0)

    first, last = x[:, :, :part].contiguous(), x[:, :, -part:].contiguous()
    rest = x[:, :, :-part].contiguous()
    state = binding.linattn_fwd(rest, rest, rest, ld, return_state=True)[1]
    for h in range(0, H, 19):  # the state handed out, against fp64
        S = sum(c.double().T @ c.double() for c in rest[0, h].split(65536))
        assert float((state[0, h].double() - S).norm()) <= 1e-5 * float(S.norm())
    rest = x[:, :, part:].contiguous()
    dstate = binding.linattn_bwd(rest, rest, rest, ld, rest, return_dstate=True)[3]
    del rest
    out = binding.linattn_fwd(x, x, x, ld)[:, :, -part:]
    check(out, binding.linattn_fwd(last, last, last, ld, state_in=state), "out")
    del out
    dq, dk, dv = binding.linattn_bwd(x, x, x, ld, x)
    del x
    check(dq[:, :, -part:], binding.linattn_bwd(last, last, last, ld, last, state_in=state)[0], "dq")
    _, k1, v1 = binding.linattn_bwd(first, first, first, ld, first, dstate_out=dstate)
    check(dk[:, :, :part], k1, "dk")
    check(dv[:, :, :part], v1, "dv")
    del dq, dk, dv, k1, v1, first, last
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,d,dtype", [(300, 128, BF16), (300, 64, BF16), (2000, 128, BF16), (300, 32, F32), (1700, 64, F32)])
def test_a_decay_that_is_nan_shows(T, d, dtype, cuda_device):
    """Every output of such a head is NaN (a sequence without tokens hands its state through), no other head's changes."""
    x = dev(lin_inputs(2, 3, T, d, d, dtype, seed=8))
    nan = x["log_decay"].clone()
    nan[1] = float("nan")
    lens = torch.tensor([T - 7, 0], dtype=torch.int32, device="cuda")
    token = [x[n][:, :, 0].contiguous() for n in "qkv"]

    def step(ld):
        pool = x["state"].clone()
        fwd = binding.linattn_fwd(x["q"], x["k"], x["v"], ld, lens=lens, state_in=x["state"], return_state=True)
        bwd = binding.linattn_bwd(x["q"], x["k"], x["v"], ld, x["dout"], lens=lens, state_in=x["state"],
                                  dstate_out=x["dstate"], return_dstate=True)
        return dict(zip(("out", "state", "dq", "dk", "dv", "dstate"), fwd + bwd)), (
            binding.linattn_decode_step(pool, *token, ld), pool)

    (rows, tok), (want, want_tok) = step(nan), step(x["log_decay"])
    for name, g in rows.items():
        at = g[0, 1] if "state" in name else g[0, 1, :T - 7]
        assert bool(at.isnan().all()), name
        assert torch.equal(g[:, [0, 2]], want[name][:, [0, 2]]) and torch.equal(g[1], want[name][1]), name
    assert torch.equal(rows["state"][1], x["state"][1]) and torch.equal(rows["dstate"][1], x["dstate"][1])
    for g, w in zip(tok, want_tok):
        assert bool(g[:, 1].isnan().all()) and torch.equal(g[:, [0, 2]], w[:, [0, 2]])


def test_decode_on_an_empty_pool(cuda_device):
    """pool = 0: padding only, and any other slot is out of range."""
    x = dev(lin_inputs(3, 2, 1, 64, 64, BF16, seed=3))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(slots):
        return binding.linattn_decode_step(torch.empty((0, 2, 64, 64), device="cuda"), *(x[n][:, :, 0].contiguous() for n in "qkv"),
                                           x["log_decay"], device_error=err,
                                           slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))

    assert bool((step([-1, -1, -1]) == 0).all()) and int(err.item()) == 0
    assert bool((step([-1, 0, -1]) == 0).all()) and int(err.item()) == 2
    with pytest.raises(binding.LLAError, match="INVALID_ARGUMENT"):  # without slots every sequence needs a state
        binding.linattn_decode_step(torch.empty((0, 2, 64, 64), device="cuda"), *(x[n][:, :, 0].contiguous() for n in "qkv"),
                                    x["log_decay"])


@pytest.mark.parametrize("dk,dv,dtype", [(16, 16, F32), (64, 32, BF16)])
def test_decode_of_thousands_with_slots_named_twice(dk, dv, dtype, cuda_device):
    B, H, pool = 5000, 2, 6000
    x = lin_inputs(B, H, 1, dk, dv, dtype, seed=12)
    gen = torch.Generator().manual_seed(13)
    base = torch.randn((pool, H, dk, dv), generator=gen)
    slots = torch.randperm(pool, generator=gen)[:B]
    slots[[0, 4999]] = int(slots[2500])                    # one slot three times
    slots[4097] = int(slots[129])                          # another one twice, far apart
    slots[[7, 3333]] = -1
    slots[[1000]] = pool
    skip = torch.zeros(B, dtype=torch.bool)
    skip[[0, 4999, 2500, 4097, 129, 7, 3333, 1000]] = True
    state, err = base.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = binding.linattn_decode_step(state, *(x[n][:, :, 0].contiguous().cuda() for n in "qkv"), x["log_decay"].cuda(),
                                      slots=slots.to(torch.int32).cuda(), device_error=err)
    torch.cuda.synchronize()
    assert int(err.item()) - 1 in (0, 4999, 2500, 4097, 129, 1000)
    on = slots[~skip]
    keep = {n: x[n][~skip] for n in "qkv"}
    ax = absolute(keep)
    ref = linattn(*(keep[n] for n in "qkv"), x["log_decay"], None, base[on])
    wgt = linattn(*(ax[n] for n in "qkv"), x["log_decay"], None, base[on].abs())
    assert_close(out[~skip.cuda()], ref[0][:, :, 0], wgt[0][:, :, 0], F32, dk, dv, 1, "out")
    assert_close(state[on.cuda()], ref[1], wgt[1], F32, dk, dv, 1, "state")
    rest = torch.ones(pool, dtype=torch.bool)
    rest[on] = False
    assert bool((out[skip.cuda()] == 0).all()) and torch.equal(state[rest.cuda()].cpu(), base[rest])


@pytest.mark.parametrize("T,H,dtype", [(300, 2, BF16), (1700, 1, BF16), (1700, 1, F32)])
@pytest.mark.parametrize("bad", [-1, None])
def test_sequences_beside_a_bad_length_are_right(T, H, dtype, bad, cuda_device):
    """All rows and states of the other sequences, forward and backward, at the bounds of every other test."""
    d = 64
    x = lin_inputs(3, H, T, d, d, dtype, seed=14)
    h, ax = dev(x), absolute(x)
    bad = T + 1 if bad is None else bad
    lens = torch.tensor([T, bad, T // 2], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = [h[n] for n in ("q", "k", "v", "log_decay")]
    got = binding.linattn_fwd(*args, lens=lens, state_in=h["state"], return_state=True, device_error=err) + \
        binding.linattn_bwd(*args, h["dout"], lens=lens, state_in=h["state"], dstate_out=h["dstate"], return_dstate=True,
                            device_error=err)
    assert binding.device_error_check(err) == 3
    good = [T, 0, T // 2]
    both = [linattn(u["q"], u["k"], u["v"], x["log_decay"], good, u["state"]) +
            linattn_grads(u["q"], u["k"], u["v"], x["log_decay"], u["dout"], good, u["state"], u["dstate"]) for u in (x, ax)]
    for name, g, r, w in zip(("out", "state", "dq", "dk", "dv", "dstate"), got, *both):
        assert bool((g[1] == 0).all()), name  # the skipped one, in outputs made by the call
        assert_close(g[[0, 2]], r[[0, 2]], w[[0, 2]], F32 if "state" in name else dtype, d, d, T, name)
