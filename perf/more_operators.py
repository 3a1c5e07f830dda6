"""Speed cases of the operators around the attention of a served language model:
matrices in microscaled formats (packed and read back), the root-mean-square norm
with the residual's addition whose output is such a matrix, and the product of two.

`run` makes one pass on what `prepare` made.  With `own` false it computes the
operator's plain form from elementary torch operations in 32 bits; with `own` true
it calls the library.

A matrix [rows, cols] in "mxfp4" (E2M1) or "mxfp8" (E4M3) has one E8M0 scale for 32
elements of a row.  codes: bytes [rows, pitch], pitch = 64 (mxfp4: two codes a byte,
low nibble first) or 128 (mxfp8) times ceil(cols / 128); codes behind cols are zero.
scales: bytes [ceil(rows / 128), ceil(cols / 128), 512]; the scale of row r and
block b (32 elements) is byte (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4 of
[r // 128, b // 4]; those of blocks behind cols are 127.
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token's activations, packed for a product: launch latency
        dict(name="pack-token-1x4096", op="pack", T=1, K=4096, fmt="mxfp4", pad=0),
        # activations of a ragged batch, every other column block of a wider tensor, 8 bits
        dict(name="pack-batch-1111x5100", op="pack", T=1111, K=5100, fmt="mxfp8", pad=20),
        # a weight matrix laid out when a model is loaded
        dict(name="pack-weight-20480x8192", op="pack", T=20480, K=8192, fmt="mxfp4", pad=0),
        # a decoding step's norm, one token: launch latency
        dict(name="norm-token-1x5120", op="norm", T=1, K=5120, fmt="mxfp8", residual=True),
        # a prompt's first norm (nothing to add yet), an odd number of tokens
        dict(name="norm-first-777x4096", op="norm", T=777, K=4096, fmt="mxfp8", residual=False),
        # the norms of long prompts: memory bound
        dict(name="norm-prompt-16384x8192", op="norm", T=16384, K=8192, fmt="mxfp8", residual=True),
        # one decoded token through the query, key and value projections of 32 / 8 heads of 128
        dict(name="linear-token-1x4096x6144", op="linear", T=1, K=4096, N=6144, fx="mxfp4", fw="mxfp4"),
        # a decoding batch through a norm and the first product of a feed-forward layer, 8-bit activations
        dict(name="norm-linear-batch-24x5120x20480", op="normlinear", T=24, K=5120, N=20480, fx="mxfp8", fw="mxfp4", residual=True),
        # a short ragged piece of a prompt, sizes that end inside tiles
        dict(name="linear-piece-333x4128x5000", op="linear", T=333, K=4128, N=5000, fx="mxfp8", fw="mxfp4"),
        # a prompt in 8 bits on both sides, 40 heads of 128
        dict(name="linear-prompt-4096x5120x5120", op="linear", T=4096, K=5120, N=5120, fx="mxfp8", fw="mxfp8"),
        # a large prompt with 8-bit activations and 4-bit weights
        dict(name="linear-prompt-8192x4096x16384", op="linear", T=8192, K=4096, N=16384, fx="mxfp8", fw="mxfp4"),
        # the largest prompt, four bits on both sides: tensor bound
        dict(name="linear-prompt-8192x8192x16384", op="linear", T=8192, K=8192, N=16384, fx="mxfp4", fw="mxfp4"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _width(rng, lo, hi):
    """A number of columns or outputs: mostly whole blocks, now and then any number."""
    n = _log(rng, lo, hi)
    step = rng.choice([128, 64, 32, 32, 8, 1])
    return max(1, n // step * step)


def draw(rng):
    op = rng.choice(["pack", "norm", "normlinear", "linear", "linear", "linear"])
    if op == "pack":
        T, K = _log(rng, 1, 20480), _width(rng, 32, 8192)
        return dict(op=op, T=T, K=K, fmt=rng.choice(["mxfp4", "mxfp8"]), pad=rng.choice([0, 0, 8, 33]))
    if op == "norm":
        return dict(op=op, T=_log(rng, 1, 16384), K=_width(rng, 32, 8192), fmt="mxfp8", residual=rng.random() < 0.7)
    fx, fw = rng.choice([("mxfp4", "mxfp4"), ("mxfp8", "mxfp4"), ("mxfp8", "mxfp4"), ("mxfp8", "mxfp8")])
    T = _log(rng, 1, rng.choice([8, 128, 8192, 8192]))
    case = dict(op=op, T=T, K=_width(rng, 32, 8192), N=_width(rng, 16, 20480), fx=fx, fw=fw)
    while case["T"] * case["K"] * case["N"] > 8192 * 8192 * 16384:
        case["T"] //= 2
    if op == "normlinear":
        case["residual"] = rng.random() < 0.7
    return case


# ------------------------------------------------------------------- data --

def _rand(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda")


def _activations(T, K, gen, pad=0):
    """Activations of normal size with some channels larger than others, bf16 [T, K]:
    a view of a tensor with `pad` more columns."""
    x = _rand((T, K + pad), gen) * torch.exp(0.6 * _rand((K + pad,), gen))
    return x.bfloat16()[:, :K]


def _pow2(n):
    """2^n in 32 bits for integers n from -126 to 127, exactly (0 for -127)."""
    return ((n.int() + 127) << 23).view(torch.float32)


def _scaled(x, fmt):
    """(values on the format's grid, exponents X) of blocks x [..., 32] in 32 bits."""
    amax = x.abs().amax(-1, keepdim=True)
    f, e = torch.frexp(amax)  # amax = f 2^e, f in [0.5, 1)
    if fmt == "mxfp4":
        X = e - 3 + (f > 0.75).to(e.dtype)
    else:
        X = e - 9 + (f > 0.875).to(e.dtype)
    X = torch.where(amax > 0, X, torch.full_like(e, -127)).clamp(-127, 127)
    y = x * _pow2(-X)
    a = y.abs()
    if fmt == "mxfp4":
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    else:
        step = _pow2((torch.frexp(a)[1] - 4).clamp(min=-9))
    return torch.round(y / step) * step, X


def _held(x, fmt):
    """The values that rows x [T, K] in 32 bits have once held in the format."""
    T, K = x.shape
    blocks = torch.nn.functional.pad(x, (0, -K % 32)).view(T, -1, 32)
    y, X = _scaled(blocks, fmt)
    return (y * _pow2(X)).flatten(1)[:, :K]


def _lay_out(x, fmt):
    """Rows x [R, K] in 32 bits -> (codes, scales) as described above."""
    R, K = x.shape
    A = -(-K // 128)
    y, X = _scaled(torch.nn.functional.pad(x, (0, 128 * A - K)).view(R, 4 * A, 32), fmt)
    if fmt == "mxfp4":
        a = y.abs()
        code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
        code = (code + 8 * torch.signbit(y).to(torch.uint8)).view(R, 128 * A)
        codes = code[:, 0::2] + 16 * code[:, 1::2]
    else:
        codes = y.to(torch.float8_e4m3fn).view(torch.uint8).view(R, 128 * A)
    byte = (X.view(R, 4 * A) + 127).to(torch.uint8)
    byte[:, -(-K // 32):] = 127
    full = torch.full((-(-R // 128) * 128, 4 * A), 127, dtype=torch.uint8, device=x.device)
    full[:R] = byte
    scales = full.view(-1, 4, 32, A, 4).permute(0, 3, 2, 1, 4).reshape(-1, A, 512)
    return codes.contiguous(), scales.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, T, K = case["op"], case["T"], case["K"]
    st = dict(case=case, x=_activations(T, K, gen, case.get("pad", 0)))
    if op in ("norm", "normlinear"):
        st["gain"] = (1 + 0.2 * _rand((K,), gen)).bfloat16()
        st["residual"] = (3 * _activations(T, K, gen).float()).bfloat16() if case["residual"] else None
    if op in ("linear", "normlinear"):
        N = case["N"]
        codes, scales = [], []
        for r in range(0, N, 4096):  # whole 128-row groups at a time
            c, s = _lay_out((_rand((min(4096, N - r), K), gen) * K ** -0.5).bfloat16().float(), case["fw"])
            codes.append(c)
            scales.append(s)
        st["wc"], st["ws"] = torch.cat(codes), torch.cat(scales)
    return st


# ------------------------------------------------------------- plain forms --

def _plain_weight(st):
    """The weights [N, K] in 32 bits."""
    c, K, N = st["wc"], st["case"]["K"], st["case"]["N"]
    if st["case"]["fw"] == "mxfp4":
        grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=c.device)
        v = torch.cat([grid, -grid])[torch.stack([c & 15, c >> 4], -1).flatten(1).int()]
    else:
        v = c.view(torch.float8_e4m3fn).float()
    A = st["ws"].shape[1]
    X = st["ws"].view(-1, A, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, 4 * A)[:N].int() - 127
    return (v.view(N, 4 * A, 32) * _pow2(X)[..., None]).flatten(1)[:, :K]


def _plain_norm(st):
    """(normed rows in 32 bits, the sum in bf16 or None)"""
    h, total = st["x"].float(), None
    if st["residual"] is not None:
        total = (h + st["residual"].float()).bfloat16()
        h = total.float()
    inv = 1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
    return h * inv * st["gain"].float(), total


def _plain(st):
    c = st["case"]
    if c["op"] == "pack":
        return _held(st["x"].float(), c["fmt"]).bfloat16()
    if c["op"] == "linear":
        return (_held(st["x"].float(), c["fx"]) @ _plain_weight(st).T).bfloat16()
    y, total = _plain_norm(st)
    if c["op"] == "norm":
        return _held(y, c["fmt"]).bfloat16(), total
    return (_held(y, c["fx"]) @ _plain_weight(st).T).bfloat16(), total


def run(state):
    if not own:
        return _plain(state)
    import matrix_core_softmax_gb300 as fsa
    c = state["case"]
    if c["op"] == "pack":
        return fsa.mx_unpack(fsa.mx_pack(state["x"], c["fmt"]))
    total = None
    if c["op"] == "linear":
        x = fsa.mx_pack(state["x"], c["fx"])
    else:
        x = fsa.rms_norm_mx(state["x"], state["gain"], residual=state["residual"], eps=EPS, fmt=c.get("fmt") or c["fx"])
        if state["residual"] is not None:
            x, total = x
        if c["op"] == "norm":
            return fsa.mx_unpack(x), total
    y = fsa.mx_linear(x, fsa.MxOperand(state["wc"], state["ws"], c["K"], c["fw"]))
    return y if c["op"] == "linear" else (y, total)


# -------------------------------------------------------------------- work --

def work(case):
    T, K = case["T"], case["K"]
    held = {"mxfp4": 0.5 + 1 / 32, "mxfp8": 1 + 1 / 32}
    bytes_ = 2 * T * K  # the bf16 rows
    if case["op"] in ("norm", "normlinear"):
        bytes_ += 2 * K + (4 * T * K if case["residual"] else 0)
    if case["op"] in ("pack", "norm"):  # the operand out and in again, its values out
        return {"bytes": bytes_ + 2 * held[case["fmt"]] * T * K + 2 * T * K, "flops": 0}
    N = case["N"]
    return {"bytes": bytes_ + held[case["fw"]] * N * K + 2 * T * N, "flops": 2 * T * N * K}


# ------------------------------------------------------------------- exact --

def _exact_pow2(n):
    """2^n in 64 bits for integral n, exactly (a device's pow is not)."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_held(x, fmt):
    """Held values of rows x in 64 bits: the least scale 2^X under which the largest
    magnitude of a block does not pass the largest element, the nearest element, and of
    two equally near ones the even code."""
    if fmt == "mxfp4":
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    else:
        low = [i * 2.0 ** -9 for i in range(8)]
        grid = low + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
        grid = torch.tensor(grid[:127], dtype=torch.float64, device=x.device)  # up to 448
    most = grid[-1]
    T, K = x.shape
    out = torch.empty_like(x)
    for b in range(0, K, 32):
        v = x[:, b:b + 32]
        top = v.abs().amax(1, keepdim=True)
        X = torch.ceil(torch.log2(torch.where(top > 0, top, 2.0 ** -140) / most))
        X = torch.where(most * _exact_pow2(X - 1) >= top, X - 1, X)
        X = torch.where(most * _exact_pow2(X) < top, X + 1, X)
        X = X.clamp(-127, 127)
        z = v.abs() / _exact_pow2(X)
        up = torch.bucketize(z, grid).clamp(1, len(grid) - 1)
        lo, hi = grid[up - 1], grid[up]
        code = torch.where((z - lo < hi - z) | ((z - lo == hi - z) & (up % 2 == 1)), up - 1, up)
        out[:, b:b + 32] = torch.sign(v) * grid[code] * _exact_pow2(X)
    return out


def _exact_weight(st):
    N, K, four = st["case"]["N"], st["case"]["K"], st["case"]["fw"] == "mxfp4"
    w = torch.empty((N, K), dtype=torch.float64, device=st["wc"].device)
    size = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0) if four else tuple(
        m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8))
    table = torch.tensor(size + tuple(-s for s in size), dtype=torch.float64, device=w.device)
    r = torch.arange(N, device=w.device)
    at = r % 32 * 16 + r % 128 // 32 * 4
    for b in range(-(-K // 32)):
        k = torch.arange(32 * b, min(K, 32 * b + 32), device=w.device)
        if four:
            code = (st["wc"][:, k // 2] >> (4 * (k % 2)).to(torch.uint8)) & 15
        else:
            code = st["wc"][:, k]
        scale = st["ws"][r // 128, b // 4, at + b % 4].long() - 127
        w[:, k] = table[code.long()] * _exact_pow2(scale)[:, None]
    return w


def exact(case, seed):
    st = prepare(case, seed)
    x, total = st["x"].double(), None
    if case["op"] == "pack":
        return _exact_held(x, case["fmt"])
    if case["op"] != "linear":
        if st["residual"] is not None:
            total = x + st["residual"].double()
            x = total.bfloat16().double()  # the norm is that of the sum as it is stored
        x = x / torch.sqrt(x.square().mean(1, keepdim=True) + EPS) * st["gain"].double()
        if case["op"] == "norm":
            return _exact_held(x, case["fmt"]), total
    y = _exact_held(x, case["fx"]) @ _exact_weight(st).T
    return y if case["op"] == "linear" else (y, total)
