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


@pytest.mark.parametrize("page", [32, 64, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_workspace_on_both_sides_of_the_split(lib, page, D):
    # up to 1024 keys a block takes a segment, up to 2048 from 64 segments on; longer
    # tables are split and joined through the workspace
    def size(B, Sq, Hq, Hkv, keys):
        return lib.fsa_kv4_attention_workspace_size(B, Sq, Hq, Hkv, D, page, keys // page)
    for B, Hkv in ((1, 1), (7, 9), (63, 1)):
        assert size(B, 1, 4 * Hkv, Hkv, 1024) == 0
        assert size(B, 1, 4 * Hkv, Hkv, 1024 + 256) > 0
    for B, Hkv in ((8, 8), (64, 1)):
        assert size(B, 1, 4 * Hkv, Hkv, 2048) == 0
        assert size(B, 1, 4 * Hkv, Hkv, 2048 + 256) > 0
    # pieces of at most two segments of 8 or 16 rows a team, in FP32 with their log-sum-exp
    assert size(1, 1, 8, 1, 131072) == 304 * 2 * 8 * (D + 1) * 4
    assert size(1, 5, 8, 1, 131072) == 152 * 2 * 16 * (D + 1) * 4
