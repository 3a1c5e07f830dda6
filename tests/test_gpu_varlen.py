"""Attention over packed sequences on the GPU against 64 bits."""
import numpy as np
import pytest
import torch

import fsa_inputs
import serving_ref as ref
from gpu_util import to_dev

pytestmark = pytest.mark.gpu
BF16 = ref.BF16


@pytest.fixture(scope="module")
def fsa():
    import __graft_entry__
    __graft_entry__.build()
    import matrix_core_softmax_gb300 as m
    return m


def _bf16(shape, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    return to_dev(fsa_inputs.to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32)))


def _cu(lens, first=0):
    return torch.tensor(np.cumsum([first] + list(lens)), dtype=torch.int32, device="cuda")


def _check(o, lse, q, k, v, cq, ck, causal, sm):
    for b in range(len(cq) - 1):
        a, c = slice(int(cq[b]), int(cq[b + 1])), slice(int(ck[b]), int(ck[b + 1]))
        nq, nk = a.stop - a.start, c.stop - c.start
        last = (nk - nq if causal else nk) + torch.arange(nq, device=q.device)
        r = ref.attend(q[a].double(), k[c].double(), v[c].double(), last, sm)
        ref.check(o[a], lse[a], r, BF16)


CASES = [
    # query lengths, key lengths (None: the same), Hq, Hkv, D
    ([1], None, 1, 1, 64),
    ([1, 2, 127, 128, 129, 0, 300], None, 8, 2, 128),
    ([64, 65, 63], None, 2, 2, 64),
    ([5, 1, 40, 16], [200, 1, 40, 513], 5, 1, 128),          # pieces that continue a context
    ([33, 50, 7, 20], [10, 0, 7, 256], 6, 3, 64),             # more queries than keys: rows that see nothing
    ([257, 511], [1000, 511], 21, 3, 128),                    # seven heads to a key head
    ([100, 37], None, 24, 2, 64),                             # twelve
    ([40], None, 128, 1, 64),                                 # one hundred and twenty-eight
    ([9, 3], None, 100, 1, 128),
    ([1500], None, 4, 4, 128),
    ([2100, 900], [2100, 4000], 16, 2, 128),
    ([1] * 300, None, 2, 1, 64),                              # many tiny sequences
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[2]}-{c[3]}-{c[4]}")
def test_matches_64_bits(fsa, case, causal):
    nq, nk, Hq, Hkv, D = case
    nk = nk or nq
    q, k, v = _bf16((sum(nq), Hq, D), 1, 2.0), _bf16((sum(nk), Hkv, D), 2), _bf16((sum(nk), Hkv, D), 3)
    cq, ck = _cu(nq), _cu(nk)
    o, lse = fsa.varlen_attention_fwd(q, k, v, cq, ck, causal=causal, return_lse=True)
    assert fsa.get_device_error() == 0
    _check(o, lse, q, k, v, cq, ck, causal, ref.default_scale(D))
    assert torch.equal(o, fsa.varlen_attention_fwd(q, k, v, cq, ck, causal=causal))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 128), (8, 1, 64), (1, 1, 128)])
def test_ends_of_key_halves(fsa, Hq, Hkv, D, causal):
    # keys that end at, before and behind each 64th, under one and many query tokens
    nk = [n + d for n in (64, 128, 192, 256, 320) for d in (-1, 0, 1)] + [32, 33, 96, 97, 160]
    nq = [(1, 64, 5, n)[i % 4] if n >= 64 else n for i, n in enumerate(nk)]
    q, k, v = _bf16((sum(nq), Hq, D), 21, 2.0), _bf16((sum(nk), Hkv, D), 22), _bf16((sum(nk), Hkv, D), 23)
    cq, ck = _cu(nq), _cu(nk)
    o, lse = fsa.varlen_attention_fwd(q, k, v, cq, ck, causal=causal, return_lse=True)
    assert fsa.get_device_error() == 0
    _check(o, lse, q, k, v, cq, ck, causal, ref.default_scale(D))


@pytest.mark.parametrize("seed", range(8))
def test_random_shapes(fsa, seed):
    rng = np.random.default_rng(2000 + seed)
    D, causal = int(rng.choice([64, 128])), bool(rng.random() < 0.7)
    Hkv, G, B = (int(rng.integers(1, m)) for m in (5, 18, 40))
    nq = [int(x) for x in (rng.random(B) ** 2 * rng.choice([20, 300, 1200])).astype(int)]
    nk = [max(0, n + int(rng.integers(-20, 500) if rng.random() < 0.6 else 0)) for n in nq]
    q, k, v = _bf16((sum(nq), G * Hkv, D), seed, 2.0), _bf16((sum(nk), Hkv, D), seed + 50), _bf16((sum(nk), Hkv, D), seed + 90)
    cq, ck = _cu(nq), _cu(nk)
    o, lse = fsa.varlen_attention_fwd(q, k, v, cq, ck, causal=causal, return_lse=True)
    assert fsa.get_device_error() == 0
    _check(o, lse, q, k, v, cq, ck, causal, ref.default_scale(D))


@pytest.mark.parametrize("kind", ["growing", "huge", "zero", "sink"])
def test_score_ranges(fsa, kind):
    n, Hq, Hkv, D = 700, 4, 2, 64
    q, k, v = _bf16((n, Hq, D), 4), _bf16((n, Hkv, D), 5), _bf16((n, Hkv, D), 6)
    if kind == "growing":        # the running maximum grows in every tile
        k = (k.float() * torch.linspace(0.1, 12, n, device="cuda")[:, None, None]).bfloat16()
        q = q.abs()
        k = k.abs()
    elif kind == "huge":
        q, k = (q.float() * 30).bfloat16(), (k.float() * 30).bfloat16()
    elif kind == "zero":
        q, k = q * 0, k * 0
    elif kind == "sink":
        k = k.clone()
        k[0] = (q.float().mean(0)[:Hkv] * 300).bfloat16()
    cu = _cu([n])
    o, lse = fsa.varlen_attention_fwd(q, k, v, cu, return_lse=True)
    _check(o, lse, q, k, v, cu, cu, True, ref.default_scale(D))


@pytest.mark.parametrize("D", [64, 128])
def test_strides_rows_outside_and_neighbours(fsa, D):
    """Views of one projection; rows before the first and behind the last sequence
    hold NaN and are left alone; a sequence of NaN does not reach its neighbours."""
    Hq, Hkv, lens = 4, 2, [130, 57, 200]
    T = 20 + sum(lens) + 40
    proj = _bf16((T, Hq + 2 * Hkv, D), 7)
    proj[:20] = float("nan")
    proj[20 + sum(lens):] = float("inf")
    proj[20 + 130:20 + 187] = float("nan")
    q, k, v = proj[:, :Hq], proj[:, Hq:Hq + Hkv], proj[:, Hq + Hkv:]
    cu = _cu(lens, 20)
    out = torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 5.0, device="cuda")
    o, l = fsa.varlen_attention_fwd(q, k, v, cu, out=out, lse=lse, return_lse=True)
    assert o is out and l is lse and fsa.get_device_error() == 0
    end = 20 + sum(lens)
    assert (o[:20] == 3).all() and (o[end:] == 3).all() and (l[:20] == 5).all() and (l[end:] == 5).all()
    for b in (0, 2):
        s = slice(int(cu[b]), int(cu[b + 1]))
        r = ref.attend(q[s].double(), k[s].double(), v[s].double(), torch.arange(lens[b], device="cuda"), ref.default_scale(D))
        ref.check(o[s], l[s], r, BF16)


def test_no_tokens(fsa):
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    ek = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert fsa.varlen_attention_fwd(e, ek, ek, _cu([0, 0])).shape == (0, 4, 64)
    # queries without any keys
    q = _bf16((10, 4, 64), 8)
    o, lse = fsa.varlen_attention_fwd(q, ek, ek, _cu([10]), _cu([0]), return_lse=True)
    assert (o == 0).all() and torch.isinf(lse).all() and fsa.get_device_error() == 0


def test_bad_bounds_are_reported(fsa):
    Hq, Hkv, D = 4, 2, 64
    q, k, v = _bf16((60, Hq, D), 9), _bf16((60, Hkv, D), 10), _bf16((60, Hkv, D), 11)
    good = fsa.varlen_attention_fwd(q, k, v, _cu([20, 20, 20]))
    for bounds in ([0, 20, 10, 60], [0, 20, 40, 61], [-3, 20, 40, 60], [0, 20, 40, 0x7FFFFFFF], [0, 20, -5, 60]):
        out = torch.full((60, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
        cu = torch.tensor(bounds, dtype=torch.int32, device="cuda")
        fsa.varlen_attention_fwd(q, k, v, cu, _cu([20, 20, 20]), out=out)
        assert fsa.get_device_error() == 1 and fsa.get_device_error() == 0
        if bounds[:2] == [0, 20]:
            assert torch.equal(out[:20], good[:20])
        out = torch.full((60, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
        fsa.varlen_attention_fwd(q, k, v, _cu([20, 20, 20]), cu, out=out)
        assert fsa.get_device_error() == 1
        if bounds[:2] == [0, 20]:
            assert torch.equal(out[:20], good[:20])


def test_a_bad_bound_behind_long_sequences(fsa):
    # more pairs of query tiles than SMs: the sequences before the wrong bound are
    # whole, the others left alone
    Hq = Hkv = 16
    lens = [2000, 1500, 300, 700]
    q, k, v = (_bf16((sum(lens), Hq, 64), 40 + i) for i in range(3))
    good = fsa.varlen_attention_fwd(q, k, v, _cu(lens))
    bad = _cu(lens)
    bad[3] = 3000
    out = torch.full_like(q, 3.0)
    fsa.varlen_attention_fwd(q, k, v, bad, _cu(lens), out=out)
    assert fsa.get_device_error() == 1 and fsa.get_device_error() == 0
    assert torch.equal(out[:3500], good[:3500]) and (out[3500:] == 3).all()


def test_streams_and_graphs(fsa):
    Hq, Hkv, D = 8, 2, 128
    runs = []
    for s in range(2):
        lens = [300 + s, 17, 129]
        T = sum(lens)
        a = _bf16((T, Hq, D), 12 + s), _bf16((T, Hkv, D), 14 + s), _bf16((T, Hkv, D), 16 + s), _cu(lens)
        runs.append((a, fsa.varlen_attention_fwd(*a)))
    graphs, outs = [], []
    for a, _ in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fsa.varlen_attention_fwd(*a))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, (_, want) in zip(outs, runs):
        assert torch.equal(o, want)
    # the captured call follows new lengths
    a, _ = runs[0]
    a[3].copy_(_cu([100, 217, 129]))
    want = fsa.varlen_attention_fwd(*a)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want)
    assert fsa.get_device_error() == 0


def test_equals_the_dense_kernel_within_rounding(fsa):
    # one sequence, every key seen: the dense BF16 kernel's case
    H, S, D = 3, 260, 128
    q, k, v = (_bf16((S, H, D), 20 + i) for i in range(3))
    o, lse = fsa.varlen_attention_fwd(q, k, v, _cu([S]), causal=False, return_lse=True)
    dense = fsa.bf16_attention_fwd(*(x.transpose(0, 1).contiguous()[None] for x in (q, k, v)))[0].transpose(0, 1)
    r = ref.attend(q.double(), k.double(), v.double(), torch.full((S,), S, device="cuda"), ref.default_scale(D))
    ref.check(o, lse, r, BF16)
    ref.check(dense, lse, r, BF16)


def test_many_sequences_of_one_token(fsa):
    # more than 65535 (tile, head) pairs
    n, Hq = 70000, 2
    q, k, v = (_bf16((n, Hq, 64), 30 + i) for i in range(3))
    cu = _cu([1] * n)
    o = fsa.varlen_attention_fwd(q, k, v, cu)
    assert torch.equal(o, v) and fsa.get_device_error() == 0
