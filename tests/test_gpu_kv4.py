"""The four-bit key/value cache on the GPU: writing, reading back, attention
over it, and a short generation through all of the serving operators."""
import numpy as np
import pytest
import torch

import fsa_inputs
import serving_ref as ref
from gpu_util import to_dev

pytestmark = pytest.mark.gpu
F16 = ref.F16


@pytest.fixture(scope="module")
def fsa():
    import __graft_entry__
    __graft_entry__.build()
    import matrix_core_softmax_gb300 as m
    return m


def _bits(shape, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    return fsa_inputs.to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32))


def _values(bits):
    return fsa_inputs.bf16_bits_to_f32(bits).astype(np.float64)


# ---------------------------------------------------------- write and read --

@pytest.mark.parametrize("T,H,D,page", [(1, 1, 64, 32), (7, 3, 128, 32), (100, 2, 64, 96), (65, 8, 128, 64),
                                        (33, 5, 128, 256)])
def test_append_bytes_and_read_back(fsa, T, H, D, page):
    pages = -(-T // page) + 2
    rng = np.random.default_rng(T + H)
    slots = rng.permutation(pages * page)[:T]
    k, v = _bits((T, H, D), 1), _bits((T, H, D), 2, 50.0)
    cache = torch.full_like(fsa.kv4_new_cache(pages, page, H, D), 0xA5)
    fsa.kv4_append(cache, to_dev(k), to_dev(v), torch.from_numpy(slots).cuda())
    got = cache.cpu().numpy()
    want = np.full_like(got, 0xA5)              # bytes of other slots stay as they were
    for bits, order, at, sat in ((k, ref.key_order(D), 0, 32 * D), (v, ref.value_order(D), 16 * D, 33 * D)):
        codes, scales = ref.pack_rows(bits.reshape(T * H, D), order)
        codes, scales = codes.reshape(T, H, -1), scales.reshape(T, H, -1)
        for i, s in enumerate(slots):
            r = s % 32
            want[s // page, :, s % page // 32, at + r * D // 2: at + (r + 1) * D // 2] = codes[i]
            want[s // page, :, s % page // 32, sat + r * D // 32: sat + (r + 1) * D // 32] = scales[i]
    assert np.array_equal(got, want)
    rk, rv = fsa.kv4_read(cache, torch.from_numpy(slots).cuda())
    assert fsa.get_device_error() == 0
    assert np.array_equal(rk.double().cpu().numpy(), ref.held_rows(k))
    assert np.array_equal(rv.double().cpu().numpy(), ref.held_rows(v))


@pytest.mark.parametrize("D", [64, 128])
def test_special_blocks(fsa, D):
    rows = np.stack([np.zeros(D, np.uint16), np.full(D, 0x8000, np.uint16), np.full(D, 0x0001, np.uint16),
                     np.full(D, 0x807F, np.uint16), np.full(D, 0x0080, np.uint16),
                     fsa_inputs.to_bf16_bits(np.tile(np.array([6, 5, 2.5, 0.25, -0.75, 1.25, -1.75, 3.5], np.float32), D // 8)),
                     fsa_inputs.to_bf16_bits(np.tile(np.array([6.03125, -1e-30], np.float32), D // 2)),
                     fsa_inputs.to_bf16_bits(np.full(D, 2.0 ** 126, np.float32))])[:, None]
    T = len(rows)
    cache = fsa.kv4_new_cache(1, 32, 1, D)
    slots = torch.arange(T, device="cuda")
    fsa.kv4_append(cache, to_dev(rows), to_dev(rows), slots)
    k, v = fsa.kv4_read(cache, slots)
    want = ref.held_rows(rows)
    assert np.array_equal(k.double().cpu().numpy(), want) and np.array_equal(v.double().cpu().numpy(), want)


def test_strided_rows_padding_and_bad_slots(fsa):
    T, H, D, page = 40, 2, 128, 32
    proj = to_dev(_bits((T, 7, D), 3))                       # 3 query heads, 2 key heads, 2 value heads
    k, v = proj[:, 3:5], proj[:, 5:7]
    slots = torch.randperm(64, device="cuda")[:T].clone()
    slots[5], slots[17] = -1, -(1 << 40)
    cache, plain = fsa.kv4_new_cache(2, page, H, D), fsa.kv4_new_cache(2, page, H, D)
    fsa.kv4_append(cache, k, v, slots)
    keep = slots >= 0
    fsa.kv4_append(plain, k[keep].contiguous(), v[keep].contiguous(), slots[keep])
    assert torch.equal(cache, plain) and fsa.get_device_error() == 0
    both = torch.full((T, 2, H + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    rk, rv = fsa.kv4_read(cache, slots, out_k=both[:, 0, :H], out_v=both[:, 1, :H])
    assert (rk[~keep] == 0).all() and (both[:, :, H] == 7.0).all()
    ck, cv = fsa.kv4_read(cache, slots)
    assert torch.equal(rk, ck) and torch.equal(rv, cv)
    # a slot behind the cache: skipped, reported, nothing else touched
    before = cache.clone()
    bad = torch.tensor([64, 1 << 50], device="cuda")
    fsa.kv4_append(cache, k[:2], v[:2], bad)
    assert fsa.get_device_error() == 1 and fsa.get_device_error() == 0
    assert torch.equal(cache, before)
    rk, rv = fsa.kv4_read(cache, bad)
    assert fsa.get_device_error() == 1
    assert (rk == 0).all() and (rv == 0).all()
    # no tokens: nothing happens
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    fsa.kv4_append(cache, k[:0], v[:0], none)
    assert fsa.kv4_read(cache, none)[0].shape == (0, H, D)


# --------------------------------------------------------------- attention --

def _sequences(fsa, lens, Hkv, D, page, seed, kscale=1.0, vscale=1.0, edit=None):
    """A cache of sequences on scattered pages, the unused slots and pages full of
    garbage.  Returns cache, page table, lengths and the held rows (float64)."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    cache = torch.from_numpy(rng.integers(0, 256, (pages, Hkv, page // 32, 34 * D), dtype=np.uint8)).cuda()
    perm = rng.permutation(pages)
    table = np.full((len(lens), max(max(need), 1) + 1), 0x7FFFFFFF, np.int32)
    k = [_bits((n, Hkv, D), seed + 10 * b, kscale) for b, n in enumerate(lens)]
    v = [_bits((n, Hkv, D), seed + 10 * b + 1, vscale) for b, n in enumerate(lens)]
    if edit:
        edit(k, v)
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        if n:
            j = np.arange(n)
            slots = table[b, j // page].astype(np.int64) * page + j % page
            fsa.kv4_append(cache, to_dev(k[b]), to_dev(v[b]), torch.from_numpy(slots).cuda())
    held = [(torch.from_numpy(ref.held_rows(a)), torch.from_numpy(ref.held_rows(c))) for a, c in zip(k, v)]
    return cache, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), held


def _check_sequences(fsa, o, lse, q, held, sm):
    Sq = q.shape[1]
    for b, (k, v) in enumerate(held):
        n = k.shape[0]
        r = ref.attend(q[b].double().cpu(), k, v, n - Sq + torch.arange(Sq), sm)
        ref.check(o[b].cpu(), lse[b].cpu(), r, F16)


CASES = [
    # lens, Sq, Hq, Hkv, D, page
    ([1], 1, 1, 1, 64, 32),
    ([0, 1, 31, 32, 33, 64, 65, 300], 1, 8, 2, 128, 32),
    ([0, 1, 2, 3, 40, 129], 4, 6, 2, 64, 64),         # rows that see nothing
    ([500, 97], 1, 5, 1, 128, 96),
    ([257, 256, 255], 3, 21, 3, 128, 256),            # 7 heads to a key head, 21 rows
    ([1000, 1], 2, 32, 2, 64, 128),                   # 32 rows to a key head
    ([5000, 20000], 1, 16, 4, 128, 64),
    ([4097], 1, 40, 8, 128, 64),
    ([3000], 9, 12, 1, 64, 32),                       # 108 rows
    ([70] * 40, 1, 3, 3, 128, 32),
    ([0, 700, 0, 0, 33, 1, 2500, 64, 0], 1, 6, 3, 128, 64),    # empty sequences inside and at the end
    ([17 * i % 400 for i in range(64)], 1, 8, 8, 64, 32),       # more whole segments than fit at once
    ([13 * i % 300 for i in range(64)], 3, 32, 8, 128, 64),     # the same with 12 rows
    ([311 * i % 3000 for i in range(50)], 1, 4, 2, 64, 128),    # segments that end inside every warp's part
    ([0] * 7, 2, 4, 2, 64, 32),
    ([3, 0, 5] * 700, 1, 2, 1, 64, 32),                         # more sequences than a block has threads
    ([40000, 5], 1, 3, 1, 64, 256),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[1]}-{c[2]}-{c[3]}-{c[4]}-{c[5]}")
def test_attention_matches_the_held_values(fsa, case):
    lens, Sq, Hq, Hkv, D, page = case
    cache, table, n, held = _sequences(fsa, lens, Hkv, D, page, seed=sum(lens) + Hq)
    q = to_dev(_bits((len(lens), Sq, Hq, D), 5, 2.0))
    o, lse = fsa.kv4_attention_fwd(q, cache, table, n, return_lse=True)
    assert fsa.get_device_error() == 0
    _check_sequences(fsa, o, lse, q, held, ref.default_scale(D))
    again = fsa.kv4_attention_fwd(q, cache, table, n)
    assert torch.equal(o, again)


@pytest.mark.parametrize("kind", ["sink", "value_outlier", "block_outlier", "tiny_values", "huge_keys", "zero_keys",
                                  "growing", "one_hot", "late_outlier", "outliers_growing", "zero_then_large"])
def test_attention_over_uneven_rows(fsa, kind):
    """Rows of very different sizes: weights that span the range of f16, value
    scales that differ between tokens and between the blocks of a token."""
    lens, Hq, Hkv, D, page = [700, 96], 8, 2, 128, 64
    queries = _values(_bits((2, 1, Hq, D), 6)).reshape(2, Hkv, Hq // Hkv, D)

    def edit(k, v):
        for b, (a, c) in enumerate(zip(k, v)):
            ka, va = _values(a), _values(c)
            away = -queries[b].sum(1) * np.sqrt(D) / D     # a key that every head scores about -1
            if kind == "sink":
                ka[0] *= 12
                va[0] *= 2.0 ** -10
            elif kind == "value_outlier":
                va[50] *= 2.0 ** 15
            elif kind == "block_outlier":
                va[40, :, :32] *= 2.0 ** 12
                va[41, :, 32:64] *= 2.0 ** -12
            elif kind == "tiny_values":
                va *= 2.0 ** -100
            elif kind == "huge_keys":
                ka *= 30
            elif kind == "zero_keys":
                ka[:] = 0
                va[:32] = 0
            elif kind == "growing":
                ka *= np.linspace(0.1, 8, len(ka))[:, None, None]
                va *= np.exp2(np.linspace(-12, 12, len(va)))[:, None, None]
            elif kind == "one_hot":
                ka[len(ka) // 2] *= 100
            elif kind == "late_outlier":      # weight 2^-20 or so, value 2^20: counts as much as the others
                ka[-40] = 14 * away
                va[-40] *= 2.0 ** 20
            elif kind == "outliers_growing":  # the same again and again, each larger and further off
                for i in range(1, 9):
                    ka[i * len(ka) // 9] = 8 * i * away
                    va[i * len(ka) // 9] *= 2.0 ** (11 * i)
            elif kind == "zero_then_large":   # no values at all at first
                va[:len(va) // 2] = 0
                va[len(va) // 2:] *= 2.0 ** 100
            a[:] = fsa_inputs.to_bf16_bits(ka.astype(np.float32))
            c[:] = fsa_inputs.to_bf16_bits(va.astype(np.float32))
    cache, table, n, held = _sequences(fsa, lens, Hkv, D, page, seed=3, edit=edit)
    q = to_dev(_bits((2, 1, Hq, D), 6))
    o, lse = fsa.kv4_attention_fwd(q, cache, table, n, return_lse=True)
    assert fsa.get_device_error() == 0
    _check_sequences(fsa, o, lse, q, held, ref.default_scale(D))


@pytest.mark.parametrize("amp", [0.0, 2.0 ** -120, 2.0 ** 60])
def test_attention_query_sizes(fsa, amp):
    # scores from nothing to a single survivor
    lens, Hq, Hkv, D, page = [130], 4, 1, 64, 32
    cache, table, n, held = _sequences(fsa, lens, Hkv, D, page, seed=8)
    qf = (np.random.default_rng(9).standard_normal((1, 1, Hq, D)) * amp).astype(np.float32)
    qf[..., 3] *= 2.0 ** -12
    q = to_dev(fsa_inputs.to_bf16_bits(qf))
    sm = 0.125 if amp < 2 else 2.0 ** -58
    o, lse = fsa.kv4_attention_fwd(q, cache, table, n, sm_scale=sm, return_lse=True)
    _check_sequences(fsa, o, lse, q, held, sm)


@pytest.mark.parametrize("Hkv,D,Sq", [(8, 128, 1), (2, 64, 3)])
def test_attention_with_a_wide_page_table(fsa, Hkv, D, Sq):
    """Room for far longer sequences than there are: the work is cut for the long
    ones (half shares), most blocks have none."""
    lens, page, B = [60, 0, 900, 3] * 16, 64, 64
    cache, table, n, held = _sequences(fsa, lens, Hkv, D, page, seed=10)
    wide = torch.full((B, 40960 // page), -7, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = to_dev(_bits((B, Sq, 4 * Hkv, D), 11, 2.0))
    o, lse = fsa.kv4_attention_fwd(q, cache, wide, n, return_lse=True)
    assert fsa.get_device_error() == 0
    _check_sequences(fsa, o, lse, q, held, ref.default_scale(D))


@pytest.mark.parametrize("Hkv,D,G", [(3, 128, 5), (3, 64, 8), (3, 128, 1)])
def test_attention_over_long_parts(fsa, Hkv, D, G):
    # two teams of warps a block: long sequences, short ones between them
    lens, page = [9000, 40, 0, 7000, 1, 700, 12000], 128
    cache, table, n, held = _sequences(fsa, lens, Hkv, D, page, seed=14)
    wide = torch.full((len(lens), 163840 // page), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = to_dev(_bits((len(lens), 1, G * Hkv, D), 15, 2.0))
    o, lse = fsa.kv4_attention_fwd(q, cache, wide, n, return_lse=True)
    assert fsa.get_device_error() == 0
    _check_sequences(fsa, o, lse, q, held, ref.default_scale(D))


@pytest.mark.parametrize("seed", range(8))
def test_attention_of_random_shapes(fsa, seed):
    rng = np.random.default_rng(1000 + seed)
    D, page = int(rng.choice([64, 128])), 32 * int(rng.integers(1, 9))
    Hkv, G, Sq, B = (int(rng.integers(1, m)) for m in (5, 18, 6, 12))
    lens = [int(x) for x in (rng.random(B) ** 2 * rng.choice([40, 700, 6000])).astype(int)]
    cache, table, n, held = _sequences(fsa, lens, Hkv, D, page, seed=seed, kscale=float(rng.choice([0.3, 1, 3])))
    q = to_dev(_bits((B, Sq, G * Hkv, D), seed, 1.5))
    o, lse = fsa.kv4_attention_fwd(q, cache, table, n, return_lse=True)
    assert fsa.get_device_error() == 0
    _check_sequences(fsa, o, lse, q, held, ref.default_scale(D))


def test_attention_strides_outputs_and_workspace(fsa):
    lens, Sq, Hq, Hkv, D, page = [300, 41, 2000], 2, 8, 2, 128, 64
    cache, table, n, held = _sequences(fsa, lens, Hkv, D, page, seed=12)
    proj = to_dev(_bits((3 * Sq, Hq + 2 * Hkv, D), 13))
    q = proj[:, :Hq].unflatten(0, (3, Sq))
    o, lse = fsa.kv4_attention_fwd(q, cache, table, n, return_lse=True)
    _check_sequences(fsa, o, lse, q, held, ref.default_scale(D))
    need = fsa.kv4_attention_workspace_size(3, Sq, Hq, Hkv, D, page, table.shape[1])
    ws = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    out, out_lse = torch.empty_like(o), torch.empty_like(lse)
    got = fsa.kv4_attention_fwd(q.contiguous(), cache, table, n, out=out, lse=out_lse, return_lse=True,
                                workspace=ws[:need + 256])
    assert got[0] is out and got[1] is out_lse
    assert torch.equal(out, o) and torch.equal(out_lse, lse)
    assert (ws[need + 256:] == 0xFF).all()


def test_sequences_that_share_pages(fsa):
    # two continuations of one prefix, and a page that a sequence holds twice
    Hq, Hkv, D, page = 8, 2, 128, 32
    cache, table, _, held = _sequences(fsa, [300], Hkv, D, page, seed=17)
    k, v = held[0]
    t = table[0, :10].repeat(3, 1)
    t[1, 9] = t[0, 2]                      # 9 common pages, another last one
    t[2, 1:4] = t[2, 0]
    n = torch.tensor([300, 310, 128], dtype=torch.int32, device="cuda")
    q = to_dev(_bits((3, 1, Hq, D), 18))
    o, lse = fsa.kv4_attention_fwd(q, cache, t, n, return_lse=True)
    assert fsa.get_device_error() == 0
    rows = [(k, v), *((torch.cat([x[:288], x[64:86]]) for x in (k, v)),), *((torch.cat([x[:32]] * 4) for x in (k, v)),)]
    _check_sequences(fsa, o, lse, q, [tuple(r) for r in rows], ref.default_scale(D))


def test_bad_pages_and_lengths_are_reported(fsa):
    lens, Hq, Hkv, D, page = [100, 100, 64], 4, 1, 128, 32
    cache, table, n, held = _sequences(fsa, lens, Hkv, D, page, seed=15)
    q = to_dev(_bits((3, 1, Hq, D), 16))
    good = fsa.kv4_attention_fwd(q, cache, table, n)
    assert fsa.get_device_error() == 0
    for bad in (-1, cache.shape[0], 0x7FFFFFFF):
        t = table.clone()
        t[1, 1] = bad
        o, lse = fsa.kv4_attention_fwd(q, cache, t, n, return_lse=True)
        assert fsa.get_device_error() == 1 and fsa.get_device_error() == 0
        assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])
        # the page's keys are left out
        k, v = (torch.cat([x[:32], x[64:]]) for x in held[1])
        ref.check(o[1].cpu(), lse[1].cpu(), ref.attend(q[1].double().cpu(), k, v, torch.tensor([67]), ref.default_scale(D)), F16)
    # lengths outside the table are clamped and reported
    wide = table[:, :2].contiguous()
    o, lse = fsa.kv4_attention_fwd(q, cache, wide, torch.tensor([64, -5, 1 << 30], dtype=torch.int32, device="cuda"),
                                   return_lse=True)
    assert fsa.get_device_error() == 1
    assert (o[1] == 0).all() and torch.isinf(lse[1]).all()
    assert torch.equal(o[2], good[2])


def test_cache_beyond_32_bit_offsets(fsa):
    # 4.9 GB of pages, the sequence in the last ones
    Hkv, D, page = 8, 128, 64
    pages = (5 << 30) // (Hkv * 2 * 34 * D)
    cache = torch.empty((pages, Hkv, page // 32, 34 * D), dtype=torch.uint8, device="cuda")
    assert cache.numel() > 1 << 32
    n = 150
    k, v = _bits((n, Hkv, D), 20), _bits((n, Hkv, D), 21)
    ids = np.array([pages - 1, 1, pages - 2], np.int32)
    j = np.arange(n)
    slots = torch.from_numpy(ids[j // page].astype(np.int64) * page + j % page).cuda()
    fsa.kv4_append(cache, to_dev(k), to_dev(v), slots)
    rk, _ = fsa.kv4_read(cache, slots)
    assert np.array_equal(rk.double().cpu().numpy(), ref.held_rows(k))
    q = to_dev(_bits((1, 1, 16, D), 22))
    o, lse = fsa.kv4_attention_fwd(q, cache, torch.from_numpy(ids)[None].cuda(),
                                   torch.tensor([n], dtype=torch.int32, device="cuda"), return_lse=True)
    assert fsa.get_device_error() == 0
    _check_sequences(fsa, o, lse, q, [(torch.from_numpy(ref.held_rows(k)), torch.from_numpy(ref.held_rows(v)))],
                     ref.default_scale(D))


def test_streams_and_graphs(fsa):
    """A step (append, attend) captured once and replayed with new tokens, lengths
    and pages; two captured steps with memory of their own replayed at once."""
    B, Hq, Hkv, D, page = 2, 8, 2, 64, 32
    steps = []
    for s in range(2):
        lens = [90 + s, 2100]
        cache, table, n, held = _sequences(fsa, lens, Hkv, D, page, seed=30 + s)
        q = to_dev(_bits((B, 1, Hq, D), 33 + s))
        want = fsa.kv4_attention_fwd(q, cache, table, n)
        steps.append((cache, table, n, q, want))
    graphs, outs = [], []
    for cache, table, n, q, _ in steps:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            fsa.kv4_attention_fwd(q, cache, table, n)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fsa.kv4_attention_fwd(q, cache, table, n))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, step in zip(outs, steps):
        assert torch.equal(o, step[4])
    # the same graph after its sequence shrank
    cache, table, n, q, _ = steps[0]
    n[1] = 64
    want = fsa.kv4_attention_fwd(q, cache, table, n)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want)
    # a given stream: outputs belong to it
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o = fsa.kv4_attention_fwd(q, cache, table, n, stream=st)
    st.synchronize()
    assert torch.equal(o, want)
    assert fsa.get_device_error() == 0


# --------------------------------------------- all of them, as they are used --

@pytest.mark.parametrize("D,G", [(128, 4), (64, 3)])
def test_prompt_then_tokens(fsa, D, G):
    """Prompts of different lengths attended as one pack and written to the cache;
    one of them continued by a second piece that reads its prefix back; then
    tokens one at a time: each result against 64 bits on the values it saw."""
    Hkv, page = 2, 32
    Hq = G * Hkv
    lens, sm = [70, 1, 131], ref.default_scale(D)
    T = sum(lens)
    proj = to_dev(_bits((T, Hq + 2 * Hkv, D), 40))
    q, k, v = proj[:, :Hq], proj[:, Hq:Hq + Hkv], proj[:, Hq + Hkv:]
    cu = torch.tensor([0, 70, 71, 202], dtype=torch.int32, device="cuda")
    o, lse = fsa.varlen_attention_fwd(q, k, v, cu, return_lse=True)
    host = [x.double().cpu() for x in (q, k, v)]
    for b, n in enumerate(lens):
        s = slice(int(cu[b]), int(cu[b + 1]))
        r = ref.attend(host[0][s], host[1][s], host[2][s], torch.arange(n), sm)
        ref.check(o[s].cpu(), lse[s].cpu(), r, ref.BF16)
    # into the cache: eight pages a sequence
    cache = fsa.kv4_new_cache(24, page, Hkv, D)
    table = torch.randperm(24, device="cuda").int().view(3, 8)
    pos = torch.cat([torch.arange(n) for n in lens]).cuda()
    seq = torch.repeat_interleave(torch.arange(3), torch.tensor(lens)).cuda()

    def slots_of(seq, pos):
        return table[seq, pos // page].long() * page + pos % page
    fsa.kv4_append(cache, k, v, slots_of(seq, pos))
    held = [[torch.from_numpy(ref.held_rows(x[int(cu[b]):int(cu[b + 1])].contiguous().view(torch.int16).cpu().numpy()
                                            .view(np.uint16))) for x in (k, v)] for b in range(3)]
    # a second piece of prompt for sequence 2: its prefix comes back from the cache
    m = 45
    more = to_dev(_bits((m, Hq + 2 * Hkv, D), 41))
    mq, mk, mv = more[:, :Hq], more[:, Hq:Hq + Hkv], more[:, Hq + Hkv:]
    pk, pv = fsa.kv4_read(cache, slots_of(torch.full((131,), 2, device="cuda"), torch.arange(131, device="cuda")))
    ak, av = torch.cat([pk, mk]), torch.cat([pv, mv])
    o, lse = fsa.varlen_attention_fwd(mq, ak, av, torch.tensor([0, m], dtype=torch.int32, device="cuda"),
                                      torch.tensor([0, 131 + m], dtype=torch.int32, device="cuda"), return_lse=True)
    r = ref.attend(mq.double().cpu(), torch.cat([held[2][0], mk.double().cpu()]), torch.cat([held[2][1], mv.double().cpu()]),
                   131 + torch.arange(m), sm)
    ref.check(o.cpu(), lse.cpu(), r, ref.BF16)
    fsa.kv4_append(cache, mk, mv, slots_of(torch.full((m,), 2, device="cuda"), 131 + torch.arange(m, device="cuda")))
    held[2] = [torch.cat([a, torch.from_numpy(ref.held_rows(x.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)))])
               for a, x in zip(held[2], (mk, mv))]
    n = torch.tensor([70, 1, 131 + m], device="cuda")
    for step in range(4):
        tok = to_dev(_bits((3, Hq + 2 * Hkv, D), 50 + step))
        q, k, v = tok[:, :Hq], tok[:, Hq:Hq + Hkv], tok[:, Hq + Hkv:]
        fsa.kv4_append(cache, k, v, slots_of(torch.arange(3, device="cuda"), n))
        n = n + 1
        o, lse = fsa.kv4_attention_fwd(q[:, None], cache, table, n.int(), return_lse=True)
        for b in range(3):
            held[b] = [torch.cat([a, torch.from_numpy(ref.held_rows(x[b:b + 1].contiguous().view(torch.int16).cpu().numpy()
                                                                    .view(np.uint16)))]) for a, x in zip(held[b], (k, v))]
        _check_sequences(fsa, o, lse, q[:, None], held, sm)
    assert fsa.get_device_error() == 0
