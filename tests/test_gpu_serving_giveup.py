"""The attention kernels of the serving operators when a wait runs out: every
role leaves, the call reports it, and the next call on the context works."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fsa():
    import __graft_entry__
    __graft_entry__.build()
    import matrix_core_softmax_gb300 as m
    return m


# (64-token pages) one block a segment of eight and of four warps, the split form
# of one and of two teams a block, 16 rows to a key head; two groups or more to a
# warp in all of them
@pytest.mark.parametrize("lens,width,Sq,Hq,Hkv,D", [([700, 40], 16, 1, 8, 2, 128), ([2000] * 64, 32, 1, 8, 8, 64),
                                                    ([20000, 60, 60000], 960, 1, 8, 2, 128),
                                                    ([40000, 40, 30000], 4096, 1, 15, 3, 128),
                                                    ([30000, 700], 480, 3, 8, 1, 64)])
def test_cache_attention_whose_copies_never_arrive(fsa, lens, width, Sq, Hq, Hkv, D):
    B, page = len(lens), 64
    need = [-(-n // page) for n in lens]
    cache = fsa.kv4_new_cache(sum(need), page, Hkv, D)
    slots = torch.arange(sum(need) * page, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(len(slots), Hkv, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    fsa.kv4_append(cache, k, v, slots)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(sum(need[:b]), sum(need[:b + 1]), device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn(B, Sq, Hq, D, generator=gen, device="cuda").bfloat16()
    want = fsa.kv4_attention_fwd(q, cache, table, n)
    assert fsa.get_device_error() == 0
    fsa.kv4_attention_fwd(q, cache, table, n, wait_timeout_ms=200, debug_flags=fsa.DEBUG_SKIP_KV_ARRIVE)
    assert fsa.get_device_error() == 5 and fsa.get_device_error() == 0
    # a limit that does not run out changes nothing
    assert torch.equal(fsa.kv4_attention_fwd(q, cache, table, n, wait_timeout_ms=500), want)
    assert torch.equal(fsa.kv4_attention_fwd(q, cache, table, n), want)
    assert fsa.get_device_error() == 0


# one item; some of several items; more items than SMs, whose numbers CTAs take over
@pytest.mark.parametrize("lens,Hq,Hkv,D", [([300], 1, 1, 64), ([100, 700, 1, 400], 8, 2, 128), ([600] * 40, 10, 2, 128),
                                           ([128] * 10 + [600] * 60, 16, 4, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_packed_attention_whose_key_tile_never_arrives(fsa, lens, Hq, Hkv, D, causal):
    T = sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn(T, h, D, generator=gen, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
    want = fsa.varlen_attention_fwd(q, k, v, cu, causal=causal)
    assert fsa.get_device_error() == 0
    fsa.varlen_attention_fwd(q, k, v, cu, causal=causal, wait_timeout_ms=200, debug_flags=fsa.DEBUG_SKIP_KV_ARRIVE)
    assert fsa.get_device_error() == 5 and fsa.get_device_error() == 0
    assert torch.equal(fsa.varlen_attention_fwd(q, k, v, cu, causal=causal, wait_timeout_ms=500), want)
    assert torch.equal(fsa.varlen_attention_fwd(q, k, v, cu, causal=causal), want)
    assert fsa.get_device_error() == 0
