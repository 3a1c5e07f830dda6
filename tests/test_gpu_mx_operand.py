"""MX operands on the GPU: packed, read back, and written by the norm."""
import numpy as np
import pytest
import torch

import fsa_inputs
import mx_ref as ref
from gpu_util import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fsa():
    import __graft_entry__
    __graft_entry__.build()
    import matrix_core_softmax_gb300 as m
    return m


def _bits(shape, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    return fsa_inputs.to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32))


def _check_pack(op, bits):
    codes, scales = ref.quantized(bits, op.fmt)
    c, s = ref.plain_codes(op)
    R, K = bits.shape
    assert np.array_equal(c[:, :K], codes) and (c[:, K:] == 0).all()
    assert np.array_equal(s[:R, :scales.shape[1]], scales) and (s[:R, scales.shape[1]:] == 127).all()


SHAPES = [(1, 1), (1, 32), (3, 31), (2, 33), (5, 127), (130, 128), (7, 129), (257, 96), (4, 4100), (1, 8192), (33, 640),
          (1000, 300), (5000, 64), (5001, 100), (4870, 128), (100, 2100)]


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("R,K", SHAPES)
def test_pack_and_back(fsa, R, K, fmt):
    bits = _bits((R, K), R + K, 3.0)
    x = to_dev(bits)
    op = fsa.mx_pack(x, fmt)
    assert fsa.get_device_error() == 0
    _check_pack(op, bits)
    assert torch.equal(fsa.mx_unpack(op).double().cpu(), ref.values(op))


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("pad,first", [(8, 0), (24, 8), (1, 0), (2, 1), (33, 3)])
def test_strides(fsa, fmt, pad, first):
    R, K = 37, 200
    wide = _bits((R, K + pad + first), 5)
    x = to_dev(wide)[:, first:first + K]
    op = fsa.mx_pack(x, fmt)
    _check_pack(op, wide[:, first:first + K])
    out = torch.full((R, K + pad + first), 7.0, dtype=torch.bfloat16, device="cuda")
    fsa.mx_unpack(op, out=out[:, first:first + K])
    assert torch.equal(out[:, first:first + K].double().cpu(), ref.values(op))
    assert (out[:, :first] == 7).all() and (out[:, first + K:] == 7).all()
    # a row that is repeated
    op = fsa.mx_pack(x[3:4].expand(R, K), fmt)
    _check_pack(op, np.repeat(wide[3:4, first:first + K], R, 0))


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_every_magnitude(fsa, fmt):
    # every finite bf16, in blocks of neighbours and in blocks of all sizes; zeros
    bits = np.arange(0x7F80, dtype=np.uint16)
    near = np.concatenate([bits, bits | 0x8000]).reshape(-1, 32 * 17)
    rng = np.random.default_rng(1)
    mixed = rng.permutation(near.reshape(-1)).reshape(near.shape)
    small = rng.integers(0, 0x0100, (20, 96)).astype(np.uint16)
    for b in (near, mixed, small, np.zeros((3, 64), np.uint16), np.full((2, 40), 0x8000, np.uint16)):
        op = fsa.mx_pack(to_dev(b), fmt)
        _check_pack(op, b)
        want = ref.values(op)
        got = fsa.mx_unpack(op).double().cpu()
        want = torch.where(want.abs() >= 2.0 ** 128, torch.copysign(torch.full_like(want, float("inf")), want),
                           want.float().bfloat16().double())
        assert torch.equal(got, want)


def test_rows_behind_and_given_operands(fsa):
    for fmt in ("mxfp4", "mxfp8"):
        bits = _bits((130, 200), 8)
        op = fsa.mx_new_operand(130, 200, fmt)
        op.codes.fill_(0xAB), op.scales.fill_(0xCD)
        assert fsa.mx_pack(to_dev(bits), fmt, out=op) is op
        _check_pack(op, bits)
        assert (ref.plain_codes(op)[1][130:] == 0xCD).all()
        # whole groups of rows are an operand
        part = fsa.MxOperand(op.codes[128:], op.scales[1:], 200, fmt)
        assert torch.equal(fsa.mx_unpack(part), fsa.mx_unpack(op)[128:])
    empty = fsa.mx_pack(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert empty.codes.shape == (0, 64) and fsa.mx_unpack(empty).shape == (0, 64)


NORMS = [(1, 1), (1, 32), (2, 33), (5, 128), (9, 200), (300, 64), (130, 1024), (3, 4100), (1, 5120), (700, 5120), (2, 20480),
         (3, 20500), (1, 32768), (40, 8192),
         # rows enough for the blocks to stay (on 16 bytes and off them)
         (2001, 5120), (3000, 1001), (20005, 64), (700, 16384), (9000, 200)]


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("R,K", NORMS)
def test_norm(fsa, R, K, residual, fmt):
    x, r, g = to_dev(_bits((R, K), 1)), to_dev(_bits((R, K), 2, 3.0)), to_dev(_bits((K,), 3))
    got = fsa.rms_norm_mx(x, g, residual=r if residual else None, eps=1e-5, fmt=fmt)
    h = x
    if residual:
        got, total = got
        h = (x.float() + r.float()).bfloat16()
        assert torch.equal(total, h)
    assert fsa.get_device_error() == 0
    ref.check_norm_operand(got, ref.norm(h.double(), g.double(), 1e-5))


@pytest.mark.parametrize("R,K", [(6, 96), (5, 4096), (300, 5000), (2500, 2048)])
@pytest.mark.parametrize("pad,off", [(7, 3), (16, 8)])
def test_norm_strides_and_sums_in_place(fsa, R, K, pad, off):
    g = to_dev(_bits((K + 1,), 3))[1:] if K % 8 == 0 else to_dev(_bits((K,), 3))   # (gain off 16 bytes)
    xw, rw = to_dev(_bits((R, K + 24), 4)), to_dev(_bits((R, K + pad), 5))
    x, r = xw[:, 8:8 + K], rw[:, off:off + K]
    h = (x.float() + r.float()).bfloat16()
    y = ref.norm(h.double(), g.double(), 1e-6)
    left = rw[:, :off].clone(), rw[:, off + K:].clone()
    op, total = fsa.rms_norm_mx(x, g, residual=r, out_sum=r)
    assert total is r and torch.equal(r, h) and torch.equal(rw[:, :off], left[0]) and torch.equal(rw[:, off + K:], left[1])
    ref.check_norm_operand(op, y)
    # the same with the sum in x's place, and one residual row for all
    one = to_dev(_bits((1, K), 6))
    h = (x.float() + one.float()).bfloat16()
    op, total = fsa.rms_norm_mx(x, g, residual=one.expand(R, K), out_sum=x)
    assert total is x and torch.equal(x, h)
    ref.check_norm_operand(op, ref.norm(h.double(), g.double(), 1e-6))


@pytest.mark.parametrize("K", [32, 1000, 8192])
@pytest.mark.parametrize("size,eps", [(2.0 ** 100, 1e-6), (2.0 ** 62, 1e-6), (2.0 ** -70, 1e-6), (2.0 ** -70, 1e-38),
                                      (2.0 ** -120, 1e-44), (2.0 ** -40, 1e-12), (0.0, 1e-6), (0.0, 1e-44)])
def test_norm_ranges(fsa, K, size, eps):
    # squares beyond FP32 at either end; a row of ordinary size beside them
    x = to_dev(_bits((5, K), 9)).float()
    x[1::2] *= size
    x = x.bfloat16()
    g = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    op = fsa.rms_norm_mx(x, g, eps=eps)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    y = ref.norm(x.double(), g.double(), eps)
    ref.check_norm_operand(op, y)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_offsets_beyond_32_bits(fsa, fmt):
    # 2.3e9 elements; the rows around 2^31 elements and 2^32 bytes and the last ones
    R, K = 70000, 32768
    at = [0, 1, 32767, 32768, 65535, 65536, 65537, R - 1]
    bits, gain = _bits((len(at), K), 1), _bits((K,), 2)
    x = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    x[at] = to_dev(bits)
    op = fsa.mx_pack(x, fmt)
    back = fsa.mx_unpack(op)
    small = fsa.mx_pack(to_dev(bits), fmt)
    assert torch.equal(back[at], fsa.mx_unpack(small)) and torch.equal(op.codes[at], small.codes)
    assert (back[2:30000] == 0).all() and (back[40000:60000] == 0).all()
    del back
    g = to_dev(gain)
    want, total = fsa.rms_norm_mx(to_dev(bits), g, residual=to_dev(bits), fmt=fmt)
    got, h = fsa.rms_norm_mx(x, g, residual=x, fmt=fmt, out=op)
    assert got is op and torch.equal(got.codes[at], want.codes) and torch.equal(h[at], total)
    assert fsa.get_device_error() == 0


def test_norm_rows_stand_alone(fsa):
    # a row of NaN or infinity does not reach its neighbours
    for R, K in ((9, 64), (5, 5120)):
        x, g = to_dev(_bits((R, K), 1)), to_dev(_bits((K,), 3))
        good = fsa.mx_unpack(fsa.rms_norm_mx(x, g))
        x[1] = float("nan")
        x[3, 5] = float("inf")
        got = fsa.mx_unpack(fsa.rms_norm_mx(x, g))
        keep = [r for r in range(R) if r not in (1, 3)]
        assert torch.equal(got[keep], good[keep])
    assert fsa.get_device_error() == 0


def test_operands_on_other_streams(fsa):
    x, g = to_dev(_bits((64, 512), 1)), to_dev(_bits((512,), 2))
    want = fsa.mx_unpack(fsa.mx_pack(x, "mxfp8")), fsa.mx_unpack(fsa.rms_norm_mx(x, g))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (fsa.mx_unpack(fsa.mx_pack(x, "mxfp8", stream=side), stream=side),
           fsa.mx_unpack(fsa.rms_norm_mx(x, g, stream=side), stream=side))
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_operands_live_as_long_as_their_tensors(fsa):
    x = to_dev(_bits((1000, 512), 1))
    op = fsa.mx_pack(x, "mxfp8")
    codes, scales = op.codes, op.scales
    want = codes.clone(), scales.clone()
    assert op.codes is codes and op.device == x.device
    del op
    others = [fsa.mx_pack(torch.zeros_like(x), "mxfp8") for _ in range(8)]
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    again = fsa.MxOperand(codes, scales, 512, "mxfp8")
    assert torch.equal(fsa.mx_unpack(again), fsa.mx_unpack(fsa.mx_pack(x, "mxfp8")))
    del others
    before = torch.cuda.memory_allocated()
    for _ in range(50):
        fsa.mx_pack(x, "mxfp8")
    assert torch.cuda.memory_allocated() == before
