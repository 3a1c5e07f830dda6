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
