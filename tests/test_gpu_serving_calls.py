"""Calls of the serving operators as a serving loop makes them."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fsa():
    import __graft_entry__
    __graft_entry__.build()
    import matrix_core_softmax_gb300 as m
    return m


def test_an_empty_batch(fsa):
    # as append, read-back and packed attention, which take no tokens
    cache = fsa.kv4_new_cache(2, 32, 2, 64)
    q = torch.empty(0, 1, 8, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    lens = torch.empty(0, dtype=torch.int32, device="cuda")
    o, lse = fsa.kv4_attention_fwd(q, cache, table, lens, return_lse=True)
    assert o.shape == q.shape and lse.shape == (0, 1, 8)
    out = torch.empty_like(q)
    assert fsa.kv4_attention_fwd(q, cache, table, lens, out=out) is out
    with pytest.raises(ValueError):
        fsa.kv4_attention_fwd(q, cache, table, lens[:0].long())
    with pytest.raises(ValueError):
        fsa.kv4_attention_fwd(q[:, :0], cache, table, lens)
    assert fsa.get_device_error() == 0
