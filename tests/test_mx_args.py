"""Host checks of the MX operands' entry points: wrong arguments are refused before
anything touches a device."""
import ctypes

import pytest
import torch

import matrix_core_softmax_gb300 as fsa
from matrix_core_softmax_gb300 import build as fsa_build

P = ctypes.c_void_p
INVALID, UNSUPPORTED = 1, 2
E4M3, E2M3, E2M1 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    fsa_build.build()
    return fsa.load()


def _pack(lib, x=256, xs=100, rows=3, cols=100, elem=E2M1, codes=256, scales=256):
    return lib.fsa_mx_pack(P(x), xs, rows, cols, elem, P(codes), P(scales), None)


def _unpack(lib, x=256, xs=100, rows=3, cols=100, elem=E2M1, codes=256, scales=256):
    return lib.fsa_mx_unpack(P(codes), P(scales), rows, cols, elem, P(x), xs, None)


@pytest.mark.parametrize("call", [_pack, _unpack])
def test_operand_refused(lib, call):
    for bad in [dict(x=0), dict(x=255), dict(codes=0), dict(scales=0), dict(codes=272), dict(scales=264), dict(xs=-1),
                dict(xs=1 << 36), dict(rows=-1), dict(rows=(1 << 30) + 1), dict(cols=0), dict(cols=(1 << 20) + 1),
                dict(elem=3), dict(elem=-1)]:
        assert call(lib, **bad) == INVALID, bad
    assert call(lib, elem=E2M3) == UNSUPPORTED
    assert call(lib, rows=0, x=0, codes=0, scales=0) == 0       # nothing to do: no device needed


def test_unpack_refuses_overlapping_rows(lib):
    assert _unpack(lib, xs=99) == INVALID


def _norm(lib, x=256, xs=64, r=256, rs=64, g=256, eps=1e-6, rows=3, cols=64, elem=E4M3, s=256, ss=64, codes=256, scales=256):
    return lib.fsa_rms_norm_mx(P(x), xs, P(r), rs, P(g), eps, rows, cols, elem, P(s), ss, P(codes), P(scales), None)


def test_norm_refused(lib):
    nan, inf = float("nan"), float("inf")
    for bad in [dict(x=0), dict(x=1), dict(g=0), dict(g=3), dict(s=0), dict(s=5), dict(r=7), dict(ss=63), dict(ss=0), dict(xs=-1),
                dict(rs=-8), dict(eps=0.0), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(cols=32769, ss=40000),
                dict(cols=0), dict(rows=-1), dict(codes=8), dict(scales=8), dict(elem=4)]:
        assert _norm(lib, **bad) == INVALID, bad
    assert _norm(lib, elem=E2M3) == UNSUPPORTED
    assert _norm(lib, rows=0, x=0, r=0, s=0, codes=0, scales=0) == 0


def _linear(lib, xc=256, xs=256, ex=E4M3, wc=256, ws=256, ew=E2M1, T=4, N=128, K=64, y=256, st=128, opt=None):
    return lib.fsa_mx_linear(P(xc), P(xs), ex, P(wc), P(ws), ew, T, N, K, P(y), st, opt, None)


def test_linear_refused(lib):
    for bad in [dict(xc=0), dict(xs=0), dict(wc=0), dict(ws=0), dict(y=0), dict(xc=16), dict(wc=16), dict(xs=8), dict(ws=8),
                dict(y=1), dict(st=127), dict(st=-128), dict(T=-1), dict(N=-1), dict(K=0), dict(K=(1 << 20) + 1),
                dict(T=(1 << 30) + 1), dict(N=(1 << 30) + 1, st=1 << 31), dict(T=1 << 30, N=1 << 12, st=1 << 12), dict(ex=5),
                dict(ew=7), dict(opt=ctypes.byref(fsa.Options()), y=0)]:
        assert _linear(lib, **bad) == INVALID, bad
    assert _linear(lib, ex=E2M1, ew=E4M3) == UNSUPPORTED
    assert _linear(lib, ex=E2M3) == UNSUPPORTED and _linear(lib, ew=E2M3) == UNSUPPORTED
    assert _linear(lib, T=0, xc=0, xs=0, y=0) == 0 and _linear(lib, N=0, wc=0, ws=0, y=0) == 0


def test_binding_refuses_host_and_mismatched_tensors():
    x, g = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    op = fsa.mx_new_operand(4, 64, "mxfp4", device="cpu")
    assert op.codes.shape == (4, 64) and op.scales.shape == (1, 1, 512)
    assert fsa.mx_new_operand(129, 200, "mxfp8", device="cpu").codes.shape == (129, 256)
    for call in (lambda: fsa.mx_pack(x), lambda: fsa.mx_unpack(op), lambda: fsa.rms_norm_mx(x, g), lambda: fsa.mx_linear(op, op),
                 lambda: fsa.mx_new_operand(4, 0, "mxfp4", device="cpu"), lambda: fsa.mx_new_operand(-1, 8, "mxfp4", device="cpu"),
                 lambda: fsa.mx_new_operand(4, 64, "mxfp6", device="cpu")):
        with pytest.raises(ValueError):
            call()


def test_operand_of_given_tensors():
    codes, scales = torch.zeros(130, 128, dtype=torch.uint8), torch.zeros(2, 2, 512, dtype=torch.uint8)
    op = fsa.MxOperand(codes, scales, 200, "mxfp4")
    assert op.codes is codes and op.scales is scales and (op.rows, op.cols, op.fmt) == (130, 200, "mxfp4")
    for bad in ((codes, scales, 128, "mxfp4"), (codes, scales, 300, "mxfp4"), (codes, scales, 200, "mxfp8"),
                (codes, scales, 200, "mxfp6"), (codes, scales[:1], 200, "mxfp4"), (codes[:, :64], scales, 200, "mxfp4"),
                (codes.int(), scales, 200, "mxfp4"), (codes, scales.float(), 200, "mxfp4"), (codes.T, scales, 200, "mxfp4"),
                (torch.zeros(130, 256, dtype=torch.uint8)[:, ::2], scales, 200, "mxfp4"), (codes[0], scales, 200, "mxfp4"),
                (codes, scales, 0, "mxfp4")):
        with pytest.raises(ValueError):
            fsa.MxOperand(*bad)


@pytest.mark.parametrize("rows,cols,fmt", [(0, 5, "mxfp4"), (1, 1, "mxfp8"), (200, 300, "mxfp4"), (128, 128, "mxfp8")])
def test_new_operand_holds_both_parts(rows, cols, fmt):
    op = fsa.mx_new_operand(rows, cols, fmt, device="cpu")
    atoms, groups = -(-cols // 128), -(-rows // 128)
    assert op.codes.shape == (rows, atoms * (64 if fmt == "mxfp4" else 128)) and op.scales.shape == (groups, atoms, 512)
    assert op.codes is op.codes and op.codes.is_contiguous() and op.scales.is_contiguous()
    op.codes.fill_(1), op.scales.fill_(2)
    assert (op.codes == 1).all() and (op.scales == 2).all()
    if rows:
        assert op._pointers() == (op.codes.data_ptr(), op.scales.data_ptr())


def test_operands_are_copied_and_stored(tmp_path):
    import copy
    op = fsa.mx_new_operand(5, 200, "mxfp8", device="cpu")
    op.codes.copy_(torch.arange(5 * 256).view(5, 256) % 251), op.scales.fill_(120)
    torch.save(op, tmp_path / "op")
    for other in (copy.deepcopy(op), torch.load(tmp_path / "op", weights_only=False)):
        assert (other.rows, other.cols, other.fmt, other.elem) == (op.rows, op.cols, op.fmt, op.elem)
        assert torch.equal(other.codes, op.codes) and torch.equal(other.scales, op.scales)
        assert other._pointers() == (other.codes.data_ptr(), other.scales.data_ptr())
        assert other.codes.data_ptr() != op.codes.data_ptr() and repr(other) == repr(op)
