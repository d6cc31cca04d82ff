"""Device-detected failures reach the caller.

The tensor-core kernels bound every wait on a shared-memory barrier; a wait
that runs out records an lla_device_error code in the caller's device_error
word and the kernel runs to its end.  The library's test hook withholds the
first product of each tile (nothing is issued for it, so no copy or product
is left in flight) and bounds the waits at a few thousand polls, so the
waits on that product run out on purpose, in a small case, without any
fault.  The word must then read LLA_DEVERR_SYNC_TIMEOUT through
lla_device_error_check (status LLA_ERR_DEVICE_REPORTED), the GPU must stay
usable, and a normal call afterwards must leave the word at zero and match
the oracle.
"""

import ctypes

import pytest
import torch

import oracle
from log_linear_attention_chunkwise_gb300 import binding
from log_linear_attention_chunkwise_gb300 import workloads as W
from parity import assert_parity

pytestmark = pytest.mark.gpu

LLA_DEVERR_COPY_TIMEOUT = 1
LLA_DEVERR_SYNC_TIMEOUT = 2


def _inputs(T=384, H=2):
    cfg = W.small_fwd_config(1, H, T, 128, 128, 64, torch.bfloat16, seed=77)
    x = W.make_fwd_inputs(cfg)
    return x, {n: t.cuda() for n, t in x.items()}


def test_clean_call_leaves_the_word_at_zero():
    x, xd = _inputs()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = binding.fwd(xd["q"], xd["k"], xd["v"], xd["g"], xd["lam"], chunk=64, device_error=err)
    assert binding.device_error_check(err) == 0
    assert_parity(out, oracle.naive(x["q"], x["k"], x["v"], x["g"], x["lam"]), torch.bfloat16, "clean")


def test_withheld_product_is_reported_and_the_gpu_recovers():
    x, xd = _inputs()
    lib = binding.load()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.debug_withhold_first_product(True)
    try:
        binding.fwd(xd["q"], xd["k"], xd["v"], xd["g"], xd["lam"], chunk=64, device_error=err)
        code = ctypes.c_int32(0)
        stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        rc = lib.lla_device_error_check(ctypes.c_void_p(err.data_ptr()), ctypes.byref(code), stream)
    finally:
        binding.debug_withhold_first_product(False)
    assert rc == 5, binding.STATUS.get(rc, rc)          # LLA_ERR_DEVICE_REPORTED
    assert code.value == LLA_DEVERR_SYNC_TIMEOUT
    # the context is intact: a normal call on the same inputs is correct and clean
    err.zero_()
    out = binding.fwd(xd["q"], xd["k"], xd["v"], xd["g"], xd["lam"], chunk=64, device_error=err)
    assert binding.device_error_check(err) == 0
    assert_parity(out, oracle.naive(x["q"], x["k"], x["v"], x["g"], x["lam"]), torch.bfloat16,
                  "after the withheld call")


def test_host_and_noalloc_entry_points_report_too():
    x, xd = _inputs(T=256, H=1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    hx = {n: t.pin_memory() for n, t in x.items()}
    binding.debug_withhold_first_product(True)
    try:
        binding.fwd_host(hx["q"], hx["k"], hx["v"], hx["g"], hx["lam"], chunk=64, device_error=err)
        host_code = binding.device_error_check(err)
        err.zero_()
        lib = binding.load()
        out = torch.empty((1, 1, 256, 128), device="cuda")
        p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
        stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        rc = lib.lla_fwd_noalloc(p(xd["q"]), p(xd["k"]), p(xd["v"]), p(xd["g"]), p(xd["lam"]), p(out),
                                 1, 1, 256, 128, 128, 64, 1, 0, p(err), stream)
        assert rc == 0
        noalloc_code = binding.device_error_check(err)
    finally:
        binding.debug_withhold_first_product(False)
    assert host_code == LLA_DEVERR_SYNC_TIMEOUT
    assert noalloc_code == LLA_DEVERR_SYNC_TIMEOUT


@pytest.mark.parametrize("T,H,d", [(300, 2, 128), (300, 2, 64), (2000, 1, 128)])
def test_withheld_products_of_linear_attention_are_reported(T, H, d):
    """Whole walks with a state's pass behind them, and segments with the pass before them: both kinds of waits run
    out, the call ends and reports, without a word too, and the calls after it are right."""
    gen = torch.Generator().manual_seed(5)
    q, k, v, do = (torch.randn((1, H, T, d), generator=gen).to(torch.bfloat16).cuda() / d ** 0.5 for _ in range(4))
    ld = torch.full((H,), -0.02, device="cuda")
    lens = torch.tensor([T - 3], dtype=torch.int32, device="cuda")

    def calls(**kw):
        return (binding.linattn_fwd(q, k, v, ld, lens=lens, return_state=True, **kw),
                binding.linattn_bwd(q, k, v, ld, do, lens=lens, return_dstate=True, **kw))

    want = calls()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.debug_withhold_first_product(True)
    try:
        codes = []
        for one in (binding.linattn_fwd, lambda *a, **kw: binding.linattn_bwd(*a, do, **kw)):
            err.zero_()
            one(q, k, v, ld, lens=lens, device_error=err)
            codes.append(binding.device_error_check(err))
        calls()
        torch.cuda.synchronize()
    finally:
        binding.debug_withhold_first_product(False)
    assert codes == [LLA_DEVERR_SYNC_TIMEOUT] * 2
    err.zero_()
    got = calls(device_error=err)
    assert binding.device_error_check(err) == 0
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))


@pytest.mark.parametrize("N,dtype", [(128, torch.bfloat16), (2048, torch.bfloat16), (128, torch.float32)])
def test_withheld_copies_of_layer_norm_are_reported(N, dtype):
    """A CTA of many turns (of widths that come in by bulk copies) whose first copy never comes: the call ends in a few
    limits, not one a turn."""
    gen = torch.Generator().manual_seed(5)
    x, dy = (torch.randn((1, 1, 200000 if N < 2048 else 30000, N), generator=gen).to(dtype).cuda() for _ in range(2))
    want, mean, rstd = binding.layer_norm_fwd(x, return_stats=True)
    grads = binding.layer_norm_bwd(x, None, mean, rstd, dy)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.debug_withhold_first_product(True)
    try:
        codes = []
        for call in (lambda: binding.layer_norm_fwd(x, device_error=err),
                     lambda: binding.layer_norm_bwd(x, None, mean, rstd, dy, device_error=err)):
            err.zero_()
            start = torch.cuda.Event(enable_timing=True)
            end = torch.cuda.Event(enable_timing=True)
            start.record()
            call()
            end.record()
            codes.append(binding.device_error_check(err))
            assert start.elapsed_time(end) < 20e3
    finally:
        binding.debug_withhold_first_product(False)
    assert codes == [LLA_DEVERR_COPY_TIMEOUT] * 2
    err.zero_()
    assert torch.equal(binding.layer_norm_fwd(x, device_error=err), want)
    got = binding.layer_norm_bwd(x, None, mean, rstd, dy, device_error=err)
    assert binding.device_error_check(err) == 0 and all(torch.equal(a, b) for a, b in zip(got, grads))
