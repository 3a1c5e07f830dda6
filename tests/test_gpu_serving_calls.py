"""Calls of the serving operators as a serving loop makes them."""
import numpy as np
import pytest
import torch

import fsa_inputs
import serving_ref as ref
from gpu_util import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fsa():
    import __graft_entry__
    __graft_entry__.build()
    import matrix_core_softmax_gb300 as m
    return m


def _rows(shape, seed):
    rng = np.random.default_rng(seed)
    return fsa_inputs.to_bf16_bits(rng.standard_normal(shape).astype(np.float32))


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


@pytest.mark.parametrize("D,G,Hkv", [(128, 4, 2), (64, 5, 3)])
def test_a_captured_step_follows_tokens_slots_lengths_and_pages(fsa, D, G, Hkv):
    """Append, attend and read-back captured once, replayed for step after step:
    new rows, slots, lengths and page tables, a place that falls empty and one
    that another sequence takes over."""
    page, B, width = 32, 3, 40
    Hq = G * Hkv
    cache = fsa.kv4_new_cache(B * width, page, Hkv, D)
    order = torch.randperm(B * width, generator=torch.Generator().manual_seed(3)).int().view(B, width)
    held = [[np.zeros((0, Hkv, D)), np.zeros((0, Hkv, D))] for _ in range(B)]
    for b, n in enumerate((1100, 30, 63)):  # (1100 of 1280 keys: the split form)
        k, v = _rows((n, Hkv, D), 10 + b), _rows((n, Hkv, D), 20 + b)
        j = torch.arange(n)
        fsa.kv4_append(cache, to_dev(k), to_dev(v), (order[b, j // page].long() * page + j % page).cuda())
        held[b] = [ref.held_rows(k), ref.held_rows(v)]
    q = torch.zeros(B, 1, Hq, D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros(B, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.full((B,), -1, dtype=torch.int64, device="cuda")
    table, lens = order.cuda(), torch.zeros(B, dtype=torch.int32, device="cuda")
    back = torch.zeros(5, dtype=torch.int64, device="cuda")

    def step():
        fsa.kv4_append(cache, k, v, slots)
        return (*fsa.kv4_attention_fwd(q, cache, table, lens, return_lse=True), *fsa.kv4_read(cache, back))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse, bk, bv = step()
    for i in range(6):
        if i == 3:   # sequence 1 has ended
            held[1] = [x[:0] for x in held[1]]
        if i == 4:   # another one takes its place, its pages in another order
            order[1] = order[1].flip(0)
        live = [b for b in range(B) if not (b == 1 and i == 3)]
        kb, vb, qb = _rows((B, Hkv, D), 100 + i), _rows((B, Hkv, D), 200 + i), _rows((B, 1, Hq, D), 300 + i)
        new = torch.full((B,), -1, dtype=torch.int64)
        for b in live:
            n = len(held[b][0])
            new[b] = int(order[b, n // page]) * page + n % page
            held[b] = [np.concatenate([x, ref.held_rows(y[b:b + 1])]) for x, y in zip(held[b], (kb, vb))]
        k.copy_(to_dev(kb)), v.copy_(to_dev(vb)), q.copy_(to_dev(qb))
        slots.copy_(new), table.copy_(order)
        lens.copy_(torch.tensor([len(h[0]) for h in held], dtype=torch.int32))
        back.copy_(torch.cat([new, new[:1], torch.tensor([-1])]))
        g.replay()
        torch.cuda.synchronize()
        for b in range(B):
            n = len(held[b][0])
            r = ref.attend(q[b].double().cpu(), torch.from_numpy(held[b][0]), torch.from_numpy(held[b][1]),
                           torch.tensor([n - 1]), ref.default_scale(D))
            ref.check(o[b].cpu(), lse[b].cpu(), r, ref.F16)
        # the rows just written, by the call and by the cache's own bytes
        want = ref.cache_rows(cache, back.tolist())
        assert np.array_equal(bk.double().cpu().numpy(), want[0]) and np.array_equal(bv.double().cpu().numpy(), want[1])
        for b in live:
            assert np.array_equal(want[0][b], held[b][0][-1]) and np.array_equal(want[1][b], held[b][1][-1])
    assert fsa.get_device_error() == 0
