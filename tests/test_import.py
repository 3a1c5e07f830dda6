"""The package imports, and its entry points allocate, without torch's private allocation."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_without_the_private_function():
    code = ("import torch\n"
            "if hasattr(torch._C._dynamo.guards, '_empty_strided_cuda'): del torch._C._dynamo.guards._empty_strided_cuda\n"
            "import matrix_core_softmax_gb300 as fsa\n"
            "assert fsa._empty_cuda is fsa._empty_dispatched\n"
            "op = fsa.mx_new_operand(3, 200, 'mxfp8', device='cpu')\n"
            "assert op.codes.shape == (3, 256)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


@pytest.mark.gpu
def test_the_same_outputs_from_either_allocation(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import matrix_core_softmax_gb300 as fsa

    x = torch.linspace(-3, 3, 5 * 200, device="cuda").view(5, 200).bfloat16()

    def outputs():
        op, h = fsa.rms_norm_mx(x, x[0].clone(), residual=x)
        y = fsa.mx_linear(op, fsa.mx_pack(x))
        return op.codes, h, y, fsa.mx_unpack(op)

    want = outputs()
    monkeypatch.setattr(fsa, "_empty_cuda", fsa._empty_dispatched)
    for a, b in zip(outputs(), want):
        assert torch.equal(a, b) and a.device == b.device and a.stride() == b.stride()
