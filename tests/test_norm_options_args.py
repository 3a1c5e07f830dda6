"""Host checks of the norm's entry point with options."""
import ctypes

import pytest

import matrix_core_softmax_gb300 as fsa
from matrix_core_softmax_gb300 import build as fsa_build

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    fsa_build.build()
    return fsa.load()


@pytest.mark.parametrize("options", [None, dict(wait_timeout_ms=5), dict(wait_timeout_ms=-1, debug_flags=3)])
def test_refuses_what_the_short_form_refuses(lib, options):
    opt = None if options is None else ctypes.byref(fsa.Options(**options))

    def call(x=256, xs=64, r=256, rs=64, g=256, eps=1e-6, rows=3, cols=64, elem=fsa.ELEM_E4M3, s=256, ss=64, codes=256, scales=256):
        args = [P(x), xs, P(r), rs, P(g), eps, rows, cols, elem, P(s), ss, P(codes), P(scales)]
        st = lib.fsa_rms_norm_mx_ex(*args, opt, None)
        assert st == lib.fsa_rms_norm_mx(*args, None)
        return st

    for bad in [dict(x=0), dict(g=0), dict(s=0), dict(ss=63), dict(xs=-1), dict(eps=0.0), dict(eps=float("nan")),
                dict(cols=32769, ss=40000), dict(cols=0), dict(rows=-1), dict(codes=8), dict(scales=8), dict(elem=4)]:
        assert call(**bad) == 1, bad
    assert call(elem=fsa.ELEM_E2M3) == 2
    assert call(rows=0, x=0, r=0, s=0, codes=0, scales=0) == 0
