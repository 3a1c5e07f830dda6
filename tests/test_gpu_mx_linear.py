"""The product of two MX operands on the GPU against 64 bits."""
import numpy as np
import pytest
import torch

import fsa_inputs
import mx_ref as ref
import serving_ref
from gpu_util import to_dev

pytestmark = pytest.mark.gpu

MODES = [("mxfp4", "mxfp4"), ("mxfp8", "mxfp4"), ("mxfp8", "mxfp8")]


@pytest.fixture(scope="module")
def fsa():
    import __graft_entry__
    __graft_entry__.build()
    import matrix_core_softmax_gb300 as m
    return m


def _bf16(shape, seed, scale=1.0, wide=0.0):
    """N(0, scale^2) rows; wide: rows and columns of different size, e^(wide N(0, 1)) each."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape) * scale
    x *= np.exp(wide * rng.standard_normal((1, shape[1]))) * np.exp(wide * rng.standard_normal((shape[0], 1)))
    return to_dev(fsa_inputs.to_bf16_bits(x.astype(np.float32)))


def _operands(fsa, T, N, K, fx, fw, seed=0, wide=0.8):
    return (fsa.mx_pack(_bf16((T, K), seed, 1.0, wide), fx), fsa.mx_pack(_bf16((N, K), seed + 1, K ** -0.5, wide / 2), fw))


SHAPES = [
    # T, N, K
    (1, 1, 1), (1, 16, 32), (2, 5, 33), (1, 128, 128), (3, 129, 127), (16, 256, 256), (17, 130, 129), (31, 100, 300),
    (1, 6144, 4096), (5, 1000, 5120), (64, 512, 1024), (65, 384, 640), (127, 200, 257), (128, 128, 128), (129, 128, 4128),
    (200, 777, 96), (300, 264, 8192), (513, 1111, 500), (1024, 1280, 256),
    # many tiles of many tokens
    (1300, 4000, 300), (2305, 2100, 257), (20000, 200, 128), (300, 10000, 640), (129, 20000, 96), (2048, 2560, 1024),
    (5000, 1300, 33), (512, 4096, 500), (1440, 2000, 1100), (400, 5000, 900), (2050, 5120, 640),
    # one and two CTAs an SM, rings of all depths, tiles of more than 128 tokens in parts
    (16, 20480, 1000), (128, 20000, 700), (100, 10000, 2100), (40, 4000, 6000), (256, 4096, 1100), (1000, 1000, 2900),
    # long rows
    (2, 130, 100000), (300, 200, 40001),
]


@pytest.mark.parametrize("fx,fw", MODES)
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_matches_64_bits(fsa, T, N, K, fx, fw):
    x, w = _operands(fsa, T, N, K, fx, fw, T + N + K)
    y = fsa.mx_linear(x, w)
    assert fsa.get_device_error() == 0
    ref.check_product(y, ref.values(x), ref.values(w))
    assert torch.equal(y, fsa.mx_linear(x, w))


@pytest.mark.parametrize("fx,fw", MODES)
@pytest.mark.parametrize("T,N,K", [(1, 256, 512), (9, 200, 384), (130, 300, 640), (19500, 200, 384)])
def test_whole_numbers_are_exact(fsa, T, N, K, fx, fw):
    """Elements 0 .. 6 of either sign under scales of 1 and 2: every sum is a whole
    number below 2^24, so y is its rounding to bf16 and nothing else."""
    rng = np.random.default_rng(T)
    big = np.array([0, 1, 2, 3, 4, 6], np.float32)

    def rows(n):
        v = big[rng.integers(0, 6, (n, K))] * rng.choice([-1, 1], (n, K))
        v[:, ::32] = 6.0                      # every block has the largest element
        two = rng.integers(0, 2, (n, K // 32)).repeat(32, 1)
        return v * (1 + two)

    a, b = (torch.from_numpy(rows(n).astype(np.float32)).cuda() for n in (T, N))
    x, w = fsa.mx_pack(a.bfloat16(), fx), fsa.mx_pack(b.bfloat16(), fw)
    assert torch.equal(fsa.mx_unpack(x).float(), a) and torch.equal(fsa.mx_unpack(w).float(), b)
    want = (a.double() @ b.double().T).float().bfloat16()
    assert torch.equal(fsa.mx_linear(x, w), want)


@pytest.mark.parametrize("fx,fw", MODES)
@pytest.mark.parametrize("times,N", [(1, 200), (70, 200), (5, 2000), (16, 2000)])
def test_one_element_at_a_time(fsa, fx, fw, times, N):
    """x holds one element 1 in each row, at every column in turn: y's rows are w's
    columns, so a wrong place of a code or a scale shows."""
    K = 288
    w = fsa.mx_pack(_bf16((N, K), 3, 1.0, 1.0), fw)
    x = torch.zeros(K, K, dtype=torch.bfloat16, device="cuda")
    x.fill_diagonal_(1.0)
    y = fsa.mx_linear(fsa.mx_pack(x.repeat(times, 1), fx), w)
    assert torch.equal(y, fsa.mx_unpack(w).T.repeat(times, 1))


@pytest.mark.parametrize("seed", range(10))
def test_random_shapes(fsa, seed):
    rng = np.random.default_rng(300 + seed)
    fx, fw = MODES[int(rng.integers(3))]
    T, N, K = (int(np.exp(rng.uniform(0, np.log(m)))) for m in (1500, 3000, 6000))
    x, w = _operands(fsa, T, N, K, fx, fw, seed)
    y = fsa.mx_linear(x, w)
    assert fsa.get_device_error() == 0
    ref.check_product(y, ref.values(x), ref.values(w))


@pytest.mark.parametrize("fx,fw", MODES)
@pytest.mark.parametrize("pad,first", [(8, 0), (4, 4), (1, 0), (3, 1)])
@pytest.mark.parametrize("T", [3, 140, 19800])
def test_output_rows_at_a_distance(fsa, fx, fw, pad, first, T):
    N, K = 200, 160
    x, w = _operands(fsa, T, N, K, fx, fw)
    want = fsa.mx_linear(x, w)
    out = torch.full((T, first + N + pad), 5.0, dtype=torch.bfloat16, device="cuda")
    view = out[:, first:first + N]
    assert fsa.mx_linear(x, w, out=view) is view
    assert torch.equal(view, want) and (out[:, :first] == 5).all() and (out[:, first + N:] == 5).all()


@pytest.mark.parametrize("fx,fw", MODES)
@pytest.mark.parametrize("T", [70, 10070])
def test_scales_behind_the_last_row_and_neighbours(fsa, fx, fw, T):
    # NaN scales in rows behind the last one, and in a row of x and of w, stay there
    N, K = 300, 400
    x, w = _operands(fsa, T, N, K, fx, fw)
    good = fsa.mx_linear(x, w)
    for op, rows in ((x, T), (w, N)):
        s = op.scales.view(op.scales.shape[0], op.scales.shape[1], 32, 4, 4)
        r = torch.arange(op.scales.shape[0] * 128, device="cuda")
        r = r[r >= rows]
        s[r // 128, :, r % 32, r % 128 // 32] = 255
        s[0, 1, 7, 1] = 255        # row 39
    y = fsa.mx_linear(x, w)
    keep_t, keep_n = [t for t in range(T) if t != 39], [n for n in range(N) if n != 39]
    assert torch.equal(y[keep_t][:, keep_n], good[keep_t][:, keep_n])
    assert torch.isnan(y[39]).all() and torch.isnan(y[:, 39]).all()


def test_parts_of_a_weight(fsa):
    x, w = _operands(fsa, 20, 640, 512, "mxfp8", "mxfp4")
    y = fsa.mx_linear(x, w)
    for a, b in ((0, 128), (128, 512), (512, 640)):
        part = fsa.MxOperand(w.codes[a:b], w.scales[a // 128:b // 128], 512, "mxfp4")
        ref.check_product(fsa.mx_linear(x, part), ref.values(x), ref.values(part))
        assert (fsa.mx_linear(x, part).float() - y[:, a:b].float()).abs().max() < 0.1


@pytest.mark.parametrize("fx,fw", MODES)
def test_extreme_scales(fsa, fx, fw):
    # blocks at both ends of the exponent range, whose products are of normal size
    T, N, K = 20, 140, 320
    x, w = _bf16((T, K), 1).float(), _bf16((N, K), 2).float()
    for b, e in enumerate((100, -100, 60, -60, 118, -118, 0, 30, -30, 5)):
        x[:, 32 * b:32 * b + 32] *= 2.0 ** e
        w[:, 32 * b:32 * b + 32] *= 2.0 ** -e
    x, w = fsa.mx_pack(x.bfloat16(), fx), fsa.mx_pack(w.bfloat16(), fw)
    ref.check_product(fsa.mx_linear(x, w), ref.values(x), ref.values(w))


def test_outputs_beyond_32_bits(fsa):
    # 2.6e9 outputs; a few rows and columns from everywhere, the last ones among them
    T, N, K = 65700, 40000, 64
    x, w = _operands(fsa, T, N, K, "mxfp8", "mxfp4")
    y = fsa.mx_linear(x, w)
    assert fsa.get_device_error() == 0
    t = torch.tensor([0, 1, 33000, 53687, 53688, 65535, T - 1], device="cuda")
    n = torch.tensor([0, 127, 128, 20001, N - 1], device="cuda")
    ref.check_product(y[t], ref.values(x)[t.cpu()], ref.values(w))
    ref.check_product(y[:, n].contiguous(), ref.values(x), ref.values(w)[n.cpu()])


def test_nothing_to_do(fsa):
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    x, w = _operands(fsa, 4, 128, 256, "mxfp4", "mxfp4")
    assert fsa.mx_linear(fsa.mx_pack(e), w).shape == (0, 128)
    assert fsa.mx_linear(x, fsa.mx_pack(e)).shape == (4, 0)


@pytest.mark.parametrize("T,N", [(2, 512), (300, 600), (2600, 2000)])
def test_streams_and_graphs(fsa, T, N):
    K = 1024
    g = to_dev(fsa_inputs.to_bf16_bits(np.ones(K, np.float32)))
    w = [fsa.mx_pack(_bf16((N, K), 50 + i, K ** -0.5), "mxfp4") for i in range(2)]
    x = [_bf16((T, K), 60 + i) for i in range(2)]

    def step(i):
        return fsa.mx_linear(fsa.rms_norm_mx(x[i], g), w[i])

    want = [step(i) for i in range(2)]
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(i))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    x[0].copy_(x[1])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], fsa.mx_linear(fsa.rms_norm_mx(x[1], g), w[0]))
    assert fsa.get_device_error() == 0


@pytest.mark.parametrize("T", [1, 300, 10000])
def test_giving_up(fsa, T):
    # the second stage of every tile's ring never counts as arrived
    x, w = _operands(fsa, T, 600, 2048, "mxfp8", "mxfp4")
    good = fsa.mx_linear(x, w)
    fsa.mx_linear(x, w, wait_timeout_ms=5, debug_flags=fsa.DEBUG_SKIP_KV_ARRIVE)
    assert fsa.get_device_error() == 5 and fsa.get_device_error() == 0
    assert torch.equal(fsa.mx_linear(x, w), good) and fsa.get_device_error() == 0


@pytest.mark.parametrize("T,fmt", [(1, "mxfp8"), (1, "mxfp4"), (150, "mxfp8")])
def test_a_layer_as_it_is_served(fsa, T, fmt):
    """Norm, the query, key and value projections as one product, append, attention over
    the cache, output projection, and the next norm: each against 64 bits on what the
    step before it gave."""
    Hq, Hkv, D, page = 8, 2, 64, 32
    width = Hq * D
    g = _bf16((1, width), 70, 0.2).view(-1) + 1
    h, d = _bf16((T, width), 71, 1.0, 0.5), _bf16((T, width), 72)
    wqkv = fsa.mx_pack(_bf16(((Hq + 2 * Hkv) * D, width), 73, width ** -0.5), "mxfp4")
    wo = fsa.mx_pack(_bf16((width, width), 74, width ** -0.5), "mxfp4")
    before = 40  # tokens already in the cache
    cache = fsa.kv4_new_cache(8, page, Hkv, D)
    kv = _bf16((before, 2 * Hkv * D), 75).view(before, 2 * Hkv, D)
    slots = torch.arange(before + T, device="cuda")
    fsa.kv4_append(cache, kv[:, :Hkv], kv[:, Hkv:], slots[:before])

    x, h1 = fsa.rms_norm_mx(d, g, residual=h, fmt=fmt)
    assert torch.equal(h1, (h.float() + d.float()).bfloat16())
    ref.check_norm_operand(x, ref.norm(h1.double(), g.double(), 1e-6))
    qkv = fsa.mx_linear(x, wqkv)
    ref.check_product(qkv, ref.values(x), ref.values(wqkv))
    heads = qkv.view(T, Hq + 2 * Hkv, D)
    q, k, v = heads[:, :Hq], heads[:, Hq:Hq + Hkv], heads[:, Hq + Hkv:]
    fsa.kv4_append(cache, k, v, slots[before:])
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    o, lse = fsa.kv4_attention_fwd(q[None], cache, table, torch.tensor([before + T], dtype=torch.int32, device="cuda"),
                                   return_lse=True)
    hk, hv = fsa.kv4_read(cache, slots)
    r = serving_ref.attend(q.double(), hk.double(), hv.double(), before + torch.arange(T, device="cuda"),
                           serving_ref.default_scale(D))
    serving_ref.check(o[0], lse[0], r, serving_ref.F16)
    a = fsa.mx_pack(o.view(T, width), fmt)
    y = fsa.mx_linear(a, wo)
    ref.check_product(y, ref.values(a), ref.values(wo))
    nxt, h2 = fsa.rms_norm_mx(y, g, residual=h1, fmt=fmt, out_sum=h1)
    ref.check_norm_operand(nxt, ref.norm(h2.double(), g.double(), 1e-6))
    assert fsa.get_device_error() == 0


@pytest.mark.parametrize("T", [1, 40, 300, 2600])
def test_buffers_that_every_call_reuses(fsa, T):
    """Product, packing and norm in turn over the same buffers: what one call reads the
    next but one writes, called one after another and replayed."""
    n = 512
    w = [fsa.mx_pack(_bf16((n, n), 80 + i, n ** -0.5), f) for i, f in enumerate(("mxfp4", "mxfp8", "mxfp4"))]
    g = to_dev(fsa_inputs.to_bf16_bits(np.ones(n, np.float32)))
    x0 = _bf16((T, n), 90)

    def chain(keep):
        h, op = x0.clone(), None
        y = torch.empty_like(x0) if keep else None
        op8, op4 = (fsa.mx_new_operand(T, n, f) if keep else None for f in ("mxfp8", "mxfp4"))
        for i in range(12):
            kw = dict(out=op8, out_sum=h) if keep else {}
            op, h = fsa.rms_norm_mx(h if i == 0 else y, g, residual=h, **kw)
            y = fsa.mx_linear(op, w[i % 3], out=y if keep else None)
            op = fsa.mx_pack(y, "mxfp4", out=op4)
            y = fsa.mx_linear(op, w[0], out=y if keep else None)
        return h, y

    want = chain(False)
    for _ in range(5):
        got = chain(True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(True)
    for _ in range(10):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and fsa.get_device_error() == 0


@pytest.mark.parametrize("fx,fw", MODES)
@pytest.mark.parametrize("T,N,K", [(1, 1920, 4200), (3, 2048, 4096), (20, 4600, 4100), (7, 4736, 4096), (50, 9500, 3000), (12, 9600, 4096),
                                   (100, 19456, 1300), (200, 1024, 5120), (256, 2300, 2500), (257, 1500, 2500), (140, 4700, 1100)])
def test_as_many_clusters_as_run_at_once(fsa, T, N, K, fx, fw):
    """Tiles around the numbers that parts of K in two, four and eight leave at work."""
    x, w = _operands(fsa, T, N, K, fx, fw, T + N + K)
    y = fsa.mx_linear(x, w)
    assert fsa.get_device_error() == 0
    ref.check_product(y, ref.values(x), ref.values(w))


def test_all_kinds_at_once(fsa):
    """Products in tiles of every kind, norms and the packed attention, each on a stream of
    its own, give what they give alone."""
    shapes = [(1, 2048, 2048), (30, 9000, 1024), (100, 20000, 512), (200, 1500, 2048), (512, 4096, 1024), (3000, 3000, 512)]
    ops = [_operands(fsa, T, N, K, *MODES[i % 3], seed=i) for i, (T, N, K) in enumerate(shapes)]
    jobs = [lambda x=x, w=w: fsa.mx_linear(x, w) for x, w in ops]
    h, g = _bf16((6000, 1024), 40), _bf16((1, 1024), 41).view(-1)
    jobs.append(lambda: fsa.mx_unpack(fsa.rms_norm_mx(h, g)))
    q, kv = _bf16((2000, 8 * 64), 42).view(2000, 8, 64), _bf16((2000, 4 * 64), 43).view(2000, 4, 64)
    ends = torch.tensor([0, 700, 2000], dtype=torch.int32, device="cuda")
    jobs.append(lambda: fsa.varlen_attention_fwd(q, kv[:, :2], kv[:, 2:], ends))
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(15):
        got = []
        for job, st in zip(jobs, streams):
            with torch.cuda.stream(st):
                got.append(job())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert fsa.get_device_error() == 0


@pytest.mark.parametrize("T", [1, 400])
def test_captured_beside_copies_and_forks(fsa, T):
    """Calls captured right behind a fill, a copy, and a join with another stream."""
    K, N = 1024, 768
    w = fsa.mx_pack(_bf16((N, K), 1, K ** -0.5), "mxfp4")
    src = [_bf16((T, K), 2 + i) for i in range(2)]
    x, z, op = torch.empty_like(src[0]), torch.empty(T, N, dtype=torch.bfloat16, device="cuda"), fsa.mx_new_operand(T, K, "mxfp8")
    side = torch.cuda.Stream()

    def step():
        z.zero_()
        x.copy_(src[0])
        fsa.mx_pack(x, "mxfp8", out=op)
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            a = fsa.mx_linear(op, w)
        fsa.mx_linear(op, w, out=z)
        here.wait_stream(side)
        back = fsa.mx_unpack(op)
        op2 = fsa.mx_pack(back, "mxfp4")
        x.fill_(0)
        return fsa.mx_linear(op2, w), a, z

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for s in (src[1], src[0]):
        src[0].copy_(s.clone())
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        first = fsa.mx_pack(src[0], "mxfp8")
        want = fsa.mx_linear(first, w)
        assert torch.equal(got[1], want) and torch.equal(got[2], want)
        assert torch.equal(got[0], fsa.mx_linear(fsa.mx_pack(fsa.mx_unpack(first), "mxfp4"), w))
    assert fsa.get_device_error() == 0
