"""Plain 64-bit forms of the serving operators (four-bit cache, packed
attention) for their tests, and the bounds their outputs are held to."""
import math

import numpy as np
import torch

import oracle

INF = float("inf")


def key_order(D):
    """d of every nibble of a key row of the cache, low nibble first."""
    return np.array([32 * b + 8 * t + i for t in range(4) for b in range(D // 32) for i in range(8)])


def value_order(D):
    return np.array([32 * b + 4 * g + i for g in range(8) for b in range(D // 32) for i in range(4)])


def pack_rows(bits, order):
    """bf16 patterns [N, D] -> (code bytes [N, D/2], scale bytes [N, D/32]) of the cache."""
    codes, scales = oracle.mx_quantize(np.ascontiguousarray(bits)[None], 1, 2)
    c = codes[0][:, order]
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8), scales[0]


E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
E2M1 = np.concatenate([E2M1, -E2M1])


def held_rows(bits):
    """The values that bf16 rows [..., D] have once held in the cache, float64."""
    flat = np.ascontiguousarray(bits).reshape(1, -1, bits.shape[-1])
    codes, scales = oracle.mx_quantize(flat, 1, 2)
    v = E2M1[codes] * np.exp2(np.repeat(scales.astype(np.float64) - 127, 32, axis=-1))
    return v.reshape(bits.shape)


def cache_rows(cache, slots):
    """(k, v) float64 [T, H, D] that a cache tensor holds at the slots, from its bytes."""
    c = cache.cpu().numpy()
    pages, H, groups, last = c.shape
    D, P = last // 34, 32 * groups
    out = []
    for order, at, sat in ((key_order(D), 0, 32 * D), (value_order(D), 16 * D, 32 * D + D)):
        rows = np.zeros((len(slots), H, D))
        for i, s in enumerate(slots):
            if s < 0:
                continue
            g = c[s // P, :, s % P // 32]
            r = s % 32
            code = g[:, at + r * D // 2: at + (r + 1) * D // 2]
            nib = np.stack([code & 15, code >> 4], -1).reshape(H, D)
            sc = g[:, sat + r * D // 32: sat + (r + 1) * D // 32].astype(np.float64) - 127
            rows[i][:, order] = E2M1[nib]
            rows[i] *= np.exp2(np.repeat(sc, 32, axis=-1))
        out.append(rows)
    return out


def attend(q, k, v, last, sm):
    """One sequence in float64: q [nq, Hq, D], k and v [nk, Hkv, D] torch; query
    i sees keys j <= last[i].  Returns o, lse, and for the bounds A = sum of
    weight * |v|, the largest sm * sum |q k| of each row, and N (see check)."""
    nq, Hq, D = q.shape
    nk, Hkv = k.shape[0], k.shape[1]
    G = Hq // Hkv
    o = torch.zeros(nq, Hq, D, dtype=torch.float64, device=q.device)
    A, N = torch.zeros_like(o), torch.zeros_like(o)
    lse = torch.full((nq, Hq), -INF, dtype=torch.float64, device=q.device)
    S = torch.zeros_like(lse)
    if nk == 0 or nq == 0:
        return o, lse, A, S, N
    hidden = torch.arange(nk, device=q.device)[None] > last[:, None]
    some = ~hidden.all(1)
    for h in range(Hq):
        kk, vv = k[:, h // G], v[:, h // G]
        s = (q[:, h] @ kk.T) * sm
        sabs = (q[:, h].abs() @ kk.abs().T) * sm
        s = s.masked_fill(hidden, -INF)
        sabs = sabs.masked_fill(hidden, 0.0)
        r = torch.logsumexp(s, 1)
        w = torch.exp(s - torch.where(some, r, torch.zeros_like(r))[:, None])
        w = torch.where(some[:, None], w, torch.zeros_like(w))
        o[:, h], A[:, h], lse[:, h], S[:, h] = w @ vv, w @ vv.abs(), r, sabs.max(1).values
        size = vv.abs().unflatten(1, (-1, 32)).amax(2)                     # of a key's blocks
        top = size.amax(0)
        rho = (size / top.clamp(min=1e-300)).amax(1)                       # of a key among the keys
        N[:, h] = nk * ((w * rho).amax(1, keepdim=True) * top).repeat_interleave(32, 1)
    return o, lse, A, S, N


# Bounds.  s carries FP32 sums of at most 128 exact products, kept in at least
# 22 bits by the tensor core: 2^-20 of sum |q k|, in the weight and in the
# normaliser.  The exponential's argument (|x| < 128 in units of log 2 where
# the weight matters) is rounded to 24 bits: 2^-17 twice; the hardware
# exponential is good to 2^-22.  Together under 2^-15 + 2^-19 S of A.  A weight
# is then rounded to f16 (2^-11) or bf16 (2^-8), and the output to bf16 (2^-8).
# Small weights have an absolute error instead.  In FP32 and bf16 a weight
# below 2^-126 of the row's largest is lost: 2^-126 N.  In f16 (weights
# p 2^(X - R), X the scale of the key's block, R the largest one, normalised by
# the largest p 2^(X - R) over keys and blocks) the error is 2^-25 of that
# normaliser a key, times 2^R and a code of at most 6.  The largest value of a
# block lies in (3, 6] 2^X, so max p 2^(X - R) <= 2 max (w rho) and 6 * 2^R <=
# 2 top: 4 * 2^-25 N, with N = keys * max (w rho) * top.

F16, BF16 = (2.0 ** -11, 2.0 ** -23), (2.0 ** -8, 2.0 ** -126)


def check(o, lse, ref, weights):
    ro, rl, A, S, N = ref
    eps, small = weights
    o, lse = o.double(), lse.double()
    rel = eps + 2.0 ** -15 + 2.0 ** -19 * S[..., None]
    tol = rel * A + small * N
    tol = tol + 2.0 ** -8 * (ro.abs() + tol) + 2.0 ** -133
    bad = (o - ro).abs() > tol
    assert torch.isfinite(o).all(), "output not finite"
    assert not bad.any(), f"{int(bad.sum())} outputs beyond their bound, worst {((o - ro).abs() / tol).max():.3g} x"
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    d = (lse - rl)[~empty].abs()
    ltol = (2.0 ** -15 + 2.0 ** -20 * S + 2.0 ** -22 * rl.abs())[~empty]
    assert (d <= ltol).all(), f"log-sum-exp off by {(d / ltol).max():.3g} x its bound"


def default_scale(D):
    return 1.0 / math.sqrt(D)
