"""The norm's root is a rounded one: values next to a border between two codes."""
import numpy as np
import pytest
import torch

import fsa_inputs
import mx_ref as ref
from gpu_util import to_dev


@pytest.fixture(scope="module")
def fsa():
    import __graft_entry__
    __graft_entry__.build()
    import matrix_core_softmax_gb300 as m
    return m


def whole_row(h, S, K):
    """K whole numbers of 0 .. 255, the first of them h, whose squares add up to S (or None)."""
    rest = S - h * h
    a = int(np.sqrt(rest / (K - 5)))
    left = rest - (K - 5) * a * a
    more, left = left // (2 * a + 1), left % (2 * a + 1)
    if a < 1 or a > 254 or more > K - 5:
        return None
    row = [h] + [a + 1] * more + [a] * (K - 5 - more)
    for p in range(int(np.sqrt(left)), -1, -1):     # four squares
        for q in range(int(np.sqrt(left - p * p)), -1, -1):
            for r in range(int(np.sqrt(left - p * p - q * q)), -1, -1):
                s = int(np.sqrt(left - p * p - q * q - r * r) + 0.5)
                if p * p + q * q + r * r + s * s == left:
                    return row + [p, q, r, s]
    return None


def near_borders(K, most):
    """(rows [R, K], sides [R]): the first value of a row, h / sqrt(S / K), lies above (+1)
    or below (-1) a border between two E4M3 elements, close to it but farther than the
    roundings of the root (2^-24 relative) and, unless h is a power of two, of the product
    with it (2^-24).  Squares' sums S are whole numbers below 2^24 and K a power of two, so
    mean and sum are exact in any order."""
    rows, sides = [], []
    for h in range(1, 256):
        error = 2.0 ** -24 if h & (h - 1) == 0 else 2.0 ** -23
        for j in range(8):
            border = 1 + (2 * j + 1) / 16
            for e in range(-8, 9):
                at = K * h * h / (border * 2.0 ** e) ** 2
                if not 2 ** 21 <= at < 2 ** 24 - 64:
                    continue
                for S in range(int(at) - 6, int(at) + 8):
                    # y / border - 1, the difference of S and `at` being exact enough
                    off = np.sqrt(at / S) - 1
                    if not error * (1 + 2.0 ** -10) < abs(off) < most * error:
                        continue
                    row = whole_row(h, S, K)
                    if row:
                        rows.append(row)
                        sides.append(1 if off > 0 else -1)
    return np.array(rows, np.float32), np.array(sides)


def test_rows_are_what_they_say():
    rows, _ = near_borders(512, 1.5)
    assert len(rows) > 2000 and rows.max() <= 255 and rows.min() >= 0
    assert (rows.astype(np.int64) ** 2).sum(1).max() < 2 ** 24


@pytest.mark.gpu
@pytest.mark.parametrize("K", [512, 1024])
def test_values_next_to_borders(fsa, K):
    """y = h / sqrt(S / K) with a rounding of the root's inverse and one of the product, gain
    1 and an eps that S / K does not see: the code is that of the side on which the exact
    value lies.  A root with an error of a unit in the last place (2^-23) puts some 300
    values in 10000 on the other side."""
    rows, sides = near_borders(K, 2.0)
    x = to_dev(fsa_inputs.to_bf16_bits(rows))
    assert torch.equal(x.float().cpu(), torch.from_numpy(rows))
    op = fsa.rms_norm_mx(x, torch.ones(K, dtype=torch.bfloat16, device="cuda"), eps=1e-30, fmt="mxfp8")
    assert fsa.get_device_error() == 0
    got = ref.values(op)[:, 0].numpy()
    y = rows[:, 0] / np.sqrt((rows.astype(np.float64) ** 2).sum(1) / K)
    step = 2.0 ** (np.floor(np.log2(y)) - 3)
    down = np.floor(y / step) * step               # the element below
    want = np.where(sides > 0, down + step, down)
    wrong = got != want
    assert not wrong.any(), f"{wrong.sum()} of {len(rows)} values on the wrong side of their border"
