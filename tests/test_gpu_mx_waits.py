"""Bounded waits of the MX operators: what their limit counts, and what it reports."""
import numpy as np
import pytest
import torch

import fsa_inputs
import mx_ref as ref
from gpu_util import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fsa():
    import __graft_entry__
    __graft_entry__.build()
    import matrix_core_softmax_gb300 as m
    return m


def _bf16(shape, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    return to_dev(fsa_inputs.to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32)))


def _zeros(fsa, rows, cols, fmt):
    op = fsa.mx_new_operand(rows, cols, fmt)
    op.codes.zero_(), op.scales.fill_(127)
    return op


@pytest.mark.parametrize("T,N", [(300, 2048), (700, 1500), (2600, 2000), (1, 600), (300, 600)])
def test_time_of_the_kernel_before_does_not_count(fsa, T, N):
    """A short product right behind one that takes longer than the short one's limit and
    leaves SMs free, on which the short one's first tiles begin early and wait."""
    K, limit = 512, 1
    far = _zeros(fsa, 2048, 1 << 20, "mxfp8"), _zeros(fsa, 1280, 1 << 20, "mxfp8")
    x, w = fsa.mx_pack(_bf16((T, K), 1), "mxfp8"), fsa.mx_pack(_bf16((N, K), 2, K ** -0.5), "mxfp4")
    y0 = torch.empty(2048, 1280, dtype=torch.bfloat16, device="cuda")
    want, out = fsa.mx_linear(x, w), torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    fsa.mx_linear(*far, out=y0)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    fsa.mx_linear(*far, out=y0)
    b.record()
    torch.cuda.synchronize()
    assert a.elapsed_time(b) > 1.2 * limit
    assert fsa.get_device_error() == 0
    for _ in range(3):
        out.fill_(7.0)
        fsa.mx_linear(*far, out=y0)
        fsa.mx_linear(x, w, out=out, wait_timeout_ms=limit)
        assert fsa.get_device_error() == 0
        assert torch.equal(out, want) and (y0 == 0).all()


# rows enough for the blocks to stay: one warp a row, eight, sixteen
RINGS = [(20000, 1024), (3000, 8192), (700, 16384)]


@pytest.mark.parametrize("flags", ["SKIP_KV_ARRIVE", "LOSE_ONE_WAIT"])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("R,K", RINGS)
def test_a_norm_that_gives_up_says_so(fsa, R, K, residual, flags):
    """A place of the ring that never arrives, and a wait that runs out in one lane while
    the lane that fetches goes on."""
    x, g = _bf16((R, K), 3), _bf16((K,), 4)
    kw = dict(residual=x if residual else None)
    good = fsa.rms_norm_mx(x, g, **kw)
    assert fsa.get_device_error() == 0
    fsa.rms_norm_mx(x, g, wait_timeout_ms=5, debug_flags=getattr(fsa, "DEBUG_" + flags), **kw)
    assert fsa.get_device_error() == 5 and fsa.get_device_error() == 0
    again = fsa.rms_norm_mx(x, g, wait_timeout_ms=500, **kw)
    assert fsa.get_device_error() == 0
    if residual:
        assert torch.equal(again[1], good[1])
        good, again = good[0], again[0]
    assert torch.equal(again.codes, good.codes)
    assert torch.equal(fsa.mx_unpack(again), fsa.mx_unpack(good))


def test_few_rows_wait_for_nothing(fsa):
    x, g = _bf16((5, 512), 5), _bf16((512,), 6)
    good = fsa.rms_norm_mx(x, g)
    got = fsa.rms_norm_mx(x, g, wait_timeout_ms=1, debug_flags=fsa.DEBUG_SKIP_KV_ARRIVE | fsa.DEBUG_LOSE_ONE_WAIT)
    assert fsa.get_device_error() == 0 and torch.equal(got.codes, good.codes)


MODES = [("mxfp4", "mxfp4"), ("mxfp8", "mxfp4"), ("mxfp8", "mxfp8")]
# pairs of CTAs on tiles of 256, 192 and 128 outputs, rows and outputs that end inside one
PAIRS = [(1024, 8192, 1024), (2500, 2500, 1100), (300, 5000, 2500), (300, 2048, 600)]


@pytest.mark.parametrize("fx,fw", MODES)
@pytest.mark.parametrize("T,N,K", PAIRS)
def test_pairs_that_give_up_leave_nothing_behind(fsa, T, N, K, fx, fw):
    """The second stage never counts as arrived while both CTAs' copies are on their way;
    what runs next on the same SMs is not disturbed by them."""
    x, w = fsa.mx_pack(_bf16((T, K), 7), fx), fsa.mx_pack(_bf16((N, K), 8, K ** -0.5), fw)
    good = fsa.mx_linear(x, w)
    ref.check_product(good, ref.values(x), ref.values(w))
    for _ in range(3):
        fsa.mx_linear(x, w, wait_timeout_ms=3, debug_flags=fsa.DEBUG_SKIP_KV_ARRIVE)
        y = fsa.mx_linear(x, w)
        assert fsa.get_device_error() == 5 and fsa.get_device_error() == 0
        assert torch.equal(y, good)


@pytest.mark.parametrize("fx,fw", MODES)
def test_pairs_repeat_beside_one_another(fsa, fx, fw):
    """Products of every tile width on streams of their own: each stage's copies of both
    CTAs are there when its products run, however late they land."""
    ops = [(fsa.mx_pack(_bf16((T, K), 9 + i), fx), fsa.mx_pack(_bf16((N, K), 19 + i, K ** -0.5), fw))
           for i, (T, N, K) in enumerate(PAIRS)]
    want = [fsa.mx_linear(x, w) for x, w in ops]
    streams = [torch.cuda.Stream() for _ in ops]
    torch.cuda.synchronize()
    for _ in range(25):
        got = []
        for (x, w), st in zip(ops, streams):
            with torch.cuda.stream(st):
                got.append(fsa.mx_linear(x, w))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert fsa.get_device_error() == 0
