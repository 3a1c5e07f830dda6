"""Host checks of the serving entry points that take fsa_options."""
import ctypes

import pytest

import matrix_core_softmax_gb300 as fsa
from matrix_core_softmax_gb300 import build as fsa_build

P = ctypes.c_void_p
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    fsa_build.build()
    return fsa.load()


def _opt(**kw):
    return ctypes.byref(fsa.Options(**kw))


def _attend(lib, opt, D=64, max_pages=5, q=256):
    return lib.fsa_kv4_attention_fwd_ex(P(q), 1024, P(256), P(256), P(256), P(256), None, 1, 1, 8, 1, D, 3, 64, max_pages, opt,
                                        None)


def test_cache_attention_options(lib):
    assert _attend(lib, _opt(sm_scale=float("nan"))) == INVALID
    assert _attend(lib, None, q=8) == INVALID and _attend(lib, None, D=96) == UNSUPPORTED
    need = lib.fsa_kv4_attention_workspace_size(1, 1, 8, 1, 128, 64, 2048)
    assert need > 0
    for kw in (None, dict(workspace=256, workspace_bytes=need - 1), dict(workspace=264, workspace_bytes=need),
               dict(workspace=0, workspace_bytes=need)):
        assert _attend(lib, kw if kw is None else _opt(**kw), D=128, max_pages=2048) == INVALID, kw


def test_packed_attention_options(lib):
    def call(opt, D=64, k=256):
        return lib.fsa_varlen_attention_fwd_ex(P(256), P(k), P(256), 256, 128, 128, P(256), P(256), P(256), None, 1, 8, 8, 4, 2,
                                               D, 1, opt, None)
    assert call(_opt(sm_scale=float("inf"))) == INVALID
    assert call(None, k=8) == INVALID and call(None, D=96) == UNSUPPORTED
