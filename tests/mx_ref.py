"""Plain 64-bit forms of the MX operands, the norm that writes one and their product,
and the bounds the GPU's outputs are held to."""
import numpy as np
import torch

import oracle

ELEM = {"mxfp8": 0, "mxfp4": 2}     # oracle.mx_quantize's element numbers
MOST = {"mxfp8": 448.0, "mxfp4": 6.0}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
E2M1 = np.concatenate([E2M1, -E2M1])
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)])
E4M3[127] = np.nan
E4M3 = np.concatenate([E4M3, -E4M3])


def quantized(bits, fmt):
    """bf16 patterns [R, K] -> (codes [R, K], scale bytes [R, ceil(K / 32)]) of the oracle."""
    codes, scales = oracle.mx_quantize(np.ascontiguousarray(bits)[None], 1, ELEM[fmt])
    return codes[0], scales[0]


def plain_codes(op):
    """(codes [R, 128 A], scale bytes [128 ceil(R / 128), 4 A]) of an operand, one to a byte."""
    c, s = op.codes.cpu().numpy(), op.scales.cpu().numpy()
    if op.fmt == "mxfp4":
        c = np.stack([c & 15, c >> 4], -1).reshape(c.shape[0], -1)
    G, A, _ = s.shape
    r, b = np.arange(128 * G)[:, None], np.arange(4 * A)[None]
    return c, s[r // 128, b // 4, r % 32 * 16 + r % 128 // 32 * 4 + b % 4]


def values(op):
    """The values that an operand holds, float64 torch [R, cols] on the CPU."""
    c, s = plain_codes(op)
    v = (E2M1 if op.fmt == "mxfp4" else E4M3)[c] * np.exp2(np.repeat(s[:c.shape[0]].astype(np.float64) - 127, 32, axis=1))
    return torch.from_numpy(v[:, :op.cols])


def check_product(y, x, w):
    """y bf16 [T, N] against x [T, K] and w [N, K] in float64.

    Products of the elements are exact.  An instruction adds 64 of them at most (32 in
    eight bits) and the sum so far, each kept in 22 bits at least of the largest:
    2^-22 (64 max |p| + |sum|), which over the row's n instructions comes to at most
    (64 + n) 2^-22 S with S = sum |x w|; the FP32 additions of up to eight parts of K
    are inside of it (8 2^-24 S).  The output is rounded to bf16 (2^-8)."""
    x, w = x.to(y.device), w.to(y.device)
    ref, S = x @ w.T, x.abs() @ w.abs().T
    n = -(-x.shape[1] // 32)
    tol = (64 + n + 2) * 2.0 ** -22 * S
    tol = tol + 2.0 ** -8 * (ref.abs() + tol) + 2.0 ** -133
    bad = (y.double() - ref).abs() > tol
    assert torch.isfinite(y).all(), "output not finite"
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outputs beyond their bound, worst "
                           f"{((y.double() - ref).abs() / tol).max():.3g} x, first at {bad.nonzero()[0].tolist()}")


def norm(x, gain, eps):
    """y in float64 of rows x (float64)."""
    return x / torch.sqrt(x.square().mean(1, keepdim=True) + eps) * gain


def check_norm_operand(op, y):
    """An operand against the rows y (float64) that it quantizes.

    The GPU's y is FP32: squares and their sum in FP32 (each lane adds at most 40, then
    5 + 5 levels: 50 roundings, halved by the root), division, root and two products:
    2^-24 (25 + 4) < 2^-19 relative.  So a block's scale is the least one that holds y's
    largest magnitude, within 2^-19 of it, and a value the nearest element to y, within
    2^-19 |y| of half a step."""
    c, s = plain_codes(op)
    R, K = y.shape
    A = -(-K // 128)
    y = torch.nn.functional.pad(y.cpu(), (0, 128 * A - K)).numpy().reshape(R, 4 * A, 32)
    v = (E2M1 if op.fmt == "mxfp4" else E4M3)[c].reshape(R, 4 * A, 32)
    X = s[:R].astype(np.float64) - 127
    most, top, slack = MOST[op.fmt], np.abs(y).max(2), 2.0 ** -19
    blocks = -(-K // 32)
    assert (s[:R, blocks:] == 127).all() and (v[:, blocks:] == 0).all()
    X, top, y, v = X[:, :blocks], top[:, :blocks], y[:, :blocks], v[:, :blocks]
    assert (top <= most * np.exp2(X) * (1 + slack)).all(), "a scale too small"
    low = X > -127
    assert (top[low] > most * np.exp2(X[low] - 1) * (1 - slack)).all(), "a scale too large"
    z = np.abs(y) / np.exp2(X)[..., None]
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.maximum(z, 1e-300)))
    step = np.exp2(np.maximum(e, 0) - 1) if op.fmt == "mxfp4" else np.exp2(np.maximum(e, -6) - 3)
    off = np.abs(v * np.sign(np.where(y == 0, 1, y)) - z)
    # (at the lower end of a binade the step below is half: within the slack either fits;
    # above the largest element only the slack is left)
    tol = step / 2 * (1 + 2.0 ** -18) + slack * z + 2.0 ** -40
    bad = off > tol
    assert not bad.any(), f"{bad.sum()} values, worst {np.max(off / tol):.3g} x"
