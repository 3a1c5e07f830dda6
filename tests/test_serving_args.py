"""Host checks of the four-bit cache and packed-attention entry points: wrong
arguments are refused before anything touches a device."""
import ctypes

import pytest
import torch

import matrix_core_softmax_gb300 as fsa
from matrix_core_softmax_gb300 import build as fsa_build

P = ctypes.c_void_p
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    fsa_build.build()
    return fsa.load()


def test_page_bytes(lib):
    assert lib.fsa_kv4_page_bytes(1, 32, 64) == 34 * 64
    assert lib.fsa_kv4_page_bytes(8, 64, 128) == 8 * 2 * 34 * 128
    for H, page, D in [(0, 32, 64), (1, 0, 64), (1, 16, 64), (1, 48, 64), (1, 32, 96), (65536, 32, 64), (1, 65568, 64),
                       (-1, 32, 64), (1, -32, 64)]:
        assert lib.fsa_kv4_page_bytes(H, page, D) == 0


def _append(lib, k=256, v=256, ks=128, vs=128, slots=256, T=4, H=2, D=64, cache=256, pages=3, page=32):
    return lib.fsa_kv4_append(P(k), P(v), ks, vs, P(slots), T, H, D, P(cache), pages, page, None)


def _read(lib, k=256, v=256, ks=128, vs=128, slots=256, T=4, H=2, D=64, cache=256, pages=3, page=32):
    return lib.fsa_kv4_read(P(cache), pages, page, P(slots), T, H, D, P(k), P(v), ks, vs, None)


@pytest.mark.parametrize("call", [_append, _read])
def test_rows_refused(lib, call):
    for bad in [dict(k=0), dict(v=0), dict(slots=0), dict(cache=0), dict(k=8), dict(v=24), dict(cache=8), dict(slots=260),
                dict(ks=100), dict(vs=-128), dict(T=-1), dict(T=1 << 31), dict(H=0), dict(pages=0), dict(pages=1 << 31),
                dict(page=48), dict(page=0), dict(ks=1 << 36),
                dict(pages=(1 << 31) - 1, page=128), dict(T=(1 << 31) - 1, H=65, ks=65 * 64, vs=65 * 64)]:
        assert call(lib, **bad) == INVALID, bad
    assert call(lib, D=96) == UNSUPPORTED
    assert call(lib, T=0, k=0, v=0, slots=0) == 0        # nothing to do: no device needed


def test_read_refuses_overlapping_rows(lib):
    assert _read(lib, ks=64) == INVALID                  # two heads of 64 need 128


def _attend(lib, q=256, qs=256, cache=256, table=256, lens=256, o=256, lse=0, B=2, Sq=1, Hq=4, Hkv=2, D=64, pages=3, page=32,
            max_pages=5, sm=0.0, ws=0, wsb=0):
    return lib.fsa_kv4_attention_fwd(P(q), qs, P(cache), P(table), P(lens), P(o), P(lse), B, Sq, Hq, Hkv, D, pages, page,
                                     max_pages, sm, P(ws), wsb, None)


def test_cache_attention_refused(lib):
    for bad in [dict(q=0), dict(cache=0), dict(table=0), dict(lens=0), dict(o=0), dict(q=8), dict(o=8), dict(cache=4),
                dict(table=258), dict(lens=258), dict(lse=258), dict(qs=4), dict(qs=-8), dict(B=0), dict(B=65536), dict(Sq=0),
                dict(Hq=5), dict(Hkv=0), dict(Hq=0), dict(pages=0), dict(page=40), dict(max_pages=0),
                dict(max_pages=1 << 26), dict(Sq=40000), dict(B=65535, Hkv=65535, Hq=65535),
                dict(B=65535, Hkv=8, Hq=8, max_pages=1 << 25),
                dict(pages=1 << 30, page=64), dict(sm=float("nan")), dict(sm=float("inf"))]:
        assert _attend(lib, **bad) == INVALID, bad
    assert _attend(lib, D=80) == UNSUPPORTED


def test_cache_attention_workspace(lib):
    assert lib.fsa_kv4_attention_workspace_size(0, 1, 4, 2, 64, 32, 5) == 0
    assert lib.fsa_kv4_attention_workspace_size(1, 1, 5, 2, 64, 32, 5) == 0
    # one sequence over a long context is split and joined through the workspace
    need = lib.fsa_kv4_attention_workspace_size(1, 1, 8, 1, 128, 64, 2048)
    if need:
        kw = dict(B=1, Hq=8, Hkv=1, D=128, page=64, max_pages=2048, qs=1024)
        assert _attend(lib, **kw) == INVALID
        assert _attend(lib, ws=256, wsb=need - 1, **kw) == INVALID
        assert _attend(lib, ws=264, wsb=need, **kw) == INVALID


def _varlen(lib, q=256, k=256, v=256, qs=256, ks=128, vs=128, cq=256, ck=256, o=256, lse=0, B=1, Tq=8, Tk=8, Hq=4, Hkv=2, D=64,
            causal=1, sm=0.0):
    return lib.fsa_varlen_attention_fwd(P(q), P(k), P(v), qs, ks, vs, P(cq), P(ck), P(o), P(lse), B, Tq, Tk, Hq, Hkv, D, causal,
                                        sm, None)


def test_varlen_refused(lib):
    for bad in [dict(q=0), dict(k=0), dict(v=0), dict(o=0), dict(cq=0), dict(ck=0), dict(q=8), dict(k=8), dict(v=8), dict(o=8),
                dict(cq=258), dict(ck=2), dict(lse=2), dict(qs=248), dict(ks=64), dict(vs=132), dict(B=0), dict(Tq=-1),
                dict(Tk=-1), dict(Tq=(1 << 26) + 1), dict(Tk=(1 << 26) + 1), dict(B=1 << 30), dict(Hq=5), dict(Hkv=0), dict(Hq=258, Hkv=2, qs=258 * 64), dict(causal=2),
                dict(sm=float("inf"))]:
        assert _varlen(lib, **bad) == INVALID, bad
    assert _varlen(lib, D=96) == UNSUPPORTED
    assert _varlen(lib, Tq=0, q=0, o=0) == 0


def test_binding_refuses_host_and_mismatched_tensors(lib):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        fsa.varlen_attention_fwd(x, x, x, cu)
    with pytest.raises(ValueError):
        fsa.kv4_append(torch.zeros(1, 2, 1, 34 * 64, dtype=torch.uint8), x, x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        fsa.kv4_read(torch.zeros(1, 2, 1, 100, dtype=torch.uint8), torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        fsa.kv4_new_cache(1, 16, 2, 64)
    with pytest.raises(ValueError):
        fsa.kv4_new_cache(0, 32, 2, 64)
    with pytest.raises(ValueError):
        fsa.kv4_new_cache(1, 32, 2, 80)
