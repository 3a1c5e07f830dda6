"""The serving operators on finite inputs of extreme range, against 64 bits."""
import math

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


def _bits(x):
    return fsa_inputs.to_bf16_bits(np.asarray(x, np.float32))


def _cached(fsa, k, v, page=64):
    """One sequence's rows [n, Hkv, D] (float64) in a cache, pages in reverse order:
    cache, page table, length and the held rows."""
    n, H, D = k.shape
    pages = -(-n // page)
    cache = fsa.kv4_new_cache(pages, page, H, D)
    table = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    j = torch.arange(n, device="cuda")
    kb, vb = _bits(k), _bits(v)
    fsa.kv4_append(cache, to_dev(kb), to_dev(vb), table[0, j // page].long() * page + j % page)
    held = tuple(torch.from_numpy(ref.held_rows(x)) for x in (kb, vb))
    return cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), held


# A key without a value whose score leads by `lead` (log2), then values 2^growth
# larger.  1024 keys: a block takes the segment, four groups a warp; 160000: two
# groups a warp of the split form.
@pytest.mark.parametrize("n", [1024, 160000])
@pytest.mark.parametrize("lead,growth", [(64, 70), (100, 40), (90, 36), (100, 10), (40, 100), (87, 42), (110, 96)])
def test_a_leading_key_without_value_before_larger_values(fsa, n, lead, growth):
    D, page, G = 64, 64, 4
    rng = np.random.default_rng(n + lead)
    u = rng.choice([-1.0, 1.0], D)
    k = np.zeros((n, 1, D))
    v = np.rint(rng.uniform(1, 7, (n, 1, D))) / 4
    group = np.arange(n) // 32
    leaders = (np.arange(n) % 32 == 7) & (group % 2 == 0)
    k[leaders, 0] = 1.5 * u
    v[leaders] = 0
    v[group % 2 == 1] *= 2.0 ** growth
    cache, table, lens, (hk, hv) = _cached(fsa, k, v, page)
    q = np.array([1.0, 0.75, 0.5, -1.0])[None, None, :, None] * u
    sm = float(np.float32(lead * math.log(2) / (1.5 * D)))
    qb = to_dev(_bits(q))
    o, lse = fsa.kv4_attention_fwd(qb, cache, table, lens, sm_scale=sm, return_lse=True)
    assert fsa.get_device_error() == 0
    r = ref.attend(qb[0].double().cpu(), hk, hv, torch.tensor([n - 1]), sm)
    ref.check(o[0].cpu(), lse[0].cpu(), r, ref.F16)


# One channel carries the scores, so that they are exact: of all keys one wins.
# What a row then gets is that key's value, whatever the scores' size.
@pytest.mark.parametrize("size", [2.0 ** 40, 2.0 ** 64, 2.0 ** 115], ids=["2^40", "2^64", "2^115"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("n", [1, 300, 5000])
def test_cache_scores_far_from_zero(fsa, n, sign, size):
    D, G = 128, 4
    rng = np.random.default_rng(n)
    k, q = np.zeros((n, 1, D)), np.zeros((1, 1, G, D))
    k[:, 0, 5] = np.where(sign > 0, 1.0, 4.0) * math.sqrt(size)
    win = n // 3
    k[win, 0, 5] = np.where(sign > 0, 4.0, 1.0) * math.sqrt(size)
    q[..., 5] = sign * math.sqrt(size)
    v = np.rint(rng.uniform(-4, 4, (n, 1, D)))
    cache, table, lens, (hk, hv) = _cached(fsa, k, v)
    o, lse = fsa.kv4_attention_fwd(to_dev(_bits(q)), cache, table, lens, sm_scale=0.5, return_lse=True)
    assert fsa.get_device_error() == 0
    want = hv[win, 0]
    assert torch.equal(o.double().cpu()[0, 0], want.expand(G, D))
    s = 0.5 * float(hk[win, 0, 5]) * sign * float(torch.tensor(math.sqrt(size)).bfloat16())
    assert (lse.double().cpu() - s).abs().max() <= 2.0 ** -21 * abs(s)


@pytest.mark.parametrize("size", [2.0 ** 24, 2.0 ** 40, 2.0 ** 64, 2.0 ** 116], ids=["2^24", "2^40", "2^64", "2^116"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("n,causal", [(1, True), (300, True), (300, False), (1500, True)])
def test_packed_scores_far_from_zero(fsa, n, causal, sign, size):
    D, Hq, Hkv = 64, 6, 2
    g = torch.Generator().manual_seed(n)
    k, q = torch.zeros(n, Hkv, D), torch.zeros(n, Hq, D)
    root = math.sqrt(size)
    # scores in steps (the sizes are even powers, so k = root * step / 128 is a bf16 value
    # and equal scores are those of equal steps): the largest is another from row to row
    step = torch.randperm(n, generator=g) % 120 + 128
    k[:, :, 9] = root * step[:, None] / 128
    q[:, :, 9] = sign * root * 1.25
    v = torch.randn(n, Hkv, D, generator=g)
    q, k, v = (x.bfloat16().cuda() for x in (q, k, v))
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    o, lse = fsa.varlen_attention_fwd(q, k, v, cu, causal=causal, sm_scale=0.35, return_lse=True)
    assert fsa.get_device_error() == 0
    # the keys of the largest score share the weight; the others' lies below 2^-1000
    # of it or so at these sizes (2^24: steps of 2^17 * 1.25 * 0.35)
    s = sign * step.double()
    seen = torch.ones(n, n).tril() if causal else torch.ones(n, n)
    s = torch.where(seen > 0, s, -math.inf)
    w = (s == s.max(1, keepdim=True).values).double()
    w /= w.sum(1, keepdim=True)
    vv = v.double().cpu()
    want = torch.stack([w @ vv[:, h // (Hq // Hkv)] for h in range(Hq)], 1)
    big = torch.stack([w @ vv[:, h // (Hq // Hkv)].abs() for h in range(Hq)], 1)
    # equal weights, one rounding of them to bf16 and one of the result
    assert ((o.double().cpu() - want).abs() <= 2.0 ** -7 * big).all()
    top = s.max(1).values / 128 * float(torch.tensor(root).bfloat16()) * float(q[0, 0, 9].abs()) * 0.35
    assert torch.isfinite(lse).all()
    err = (lse.double().cpu() - top[:, None]).abs()
    assert (err <= 2.0 ** -21 * top.abs()[:, None] + math.log(n) + 2.0 ** -10).all()


# Keys and queries at opposite ends of bf16's exponents, scores of normal size
@pytest.mark.parametrize("e", [126, 118, 100, -100, -119, -124, -127, -130])
@pytest.mark.parametrize("n,D", [(200, 64), (3000, 128)])
def test_cache_keys_at_the_ends_of_the_exponents(fsa, n, D, e):
    rng = np.random.default_rng(n)
    k = np.clip(rng.standard_normal((n, 2, D)), -1.9, 1.9) * 2.0 ** e
    v = rng.standard_normal((n, 2, D))
    q = np.clip(rng.standard_normal((1, 1, 10, D)), -1.9, 1.9) * 2.0 ** min(-e, 126)
    cache, table, lens, (hk, hv) = _cached(fsa, k, v)
    qb = to_dev(_bits(q))
    sm = 0.3 * 2.0 ** (-e - min(-e, 126))
    o, lse = fsa.kv4_attention_fwd(qb, cache, table, lens, sm_scale=sm, return_lse=True)
    assert fsa.get_device_error() == 0
    r = ref.attend(qb[0].double().cpu(), hk, hv, torch.tensor([n - 1]), float(np.float32(sm)))
    ref.check(o[0].cpu(), lse[0].cpu(), r, ref.F16)


@pytest.mark.parametrize("e", [125, -110, -126, -130])
def test_cache_values_at_the_ends_of_the_exponents(fsa, e):
    n, D = 700, 128
    rng = np.random.default_rng(5)
    k, v = rng.standard_normal((n, 2, D)), np.clip(rng.standard_normal((n, 2, D)), -1.9, 1.9) * 2.0 ** e
    cache, table, lens, (hk, hv) = _cached(fsa, k, v)
    qb = to_dev(_bits(rng.standard_normal((1, 1, 6, D))))
    o, lse = fsa.kv4_attention_fwd(qb, cache, table, lens, return_lse=True)
    assert fsa.get_device_error() == 0
    r = ref.attend(qb[0].double().cpu(), hk, hv, torch.tensor([n - 1]), ref.default_scale(D))
    ref.check(o[0].cpu(), lse[0].cpu(), r, ref.F16)


# The layout is public: a cache that its owner filled, with the scale bytes that
# fsa_kv4_append never writes (2^127)
@pytest.mark.parametrize("n,D", [(200, 64), (3000, 128)])
def test_a_cache_with_the_largest_scales(fsa, n, D):
    page, H = 64, 2
    pages = -(-n // page)
    rng = np.random.default_rng(n)
    c = np.zeros((pages, H, page // 32, 34 * D), np.uint8)
    nibbles = np.array([0, 1, 2, 8, 9, 10], np.uint8)  # 0, 0.5, 1 and their negatives
    c[..., :32 * D] = rng.choice(nibbles, c[..., :32 * D].shape) | (rng.choice(nibbles, c[..., :32 * D].shape) << 4)
    c[..., 32 * D:33 * D] = rng.choice(np.array([0, 1, 126, 253, 254], np.uint8), c[..., 32 * D:33 * D].shape)
    c[..., 33 * D:] = rng.integers(120, 135, c[..., 33 * D:].shape)
    cache = torch.from_numpy(c).cuda()
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    hk, hv = (torch.from_numpy(x) for x in ref.cache_rows(cache, list(range(n))))
    q = to_dev(_bits(np.clip(rng.standard_normal((1, 1, 8, D)), -1.9, 1.9) * 2.0 ** -126))
    o, lse = fsa.kv4_attention_fwd(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), sm_scale=0.25,
                                   return_lse=True)
    assert fsa.get_device_error() == 0
    r = ref.attend(q[0].double().cpu(), hk, hv, torch.tensor([n - 1]), 0.25)
    ref.check(o[0].cpu(), lse[0].cpu(), r, ref.F16)
