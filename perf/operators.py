"""Speed cases of the serving operators: the four-bit key/value cache (written,
read back, attended) and causal attention over packed prompts.

`run` makes one call of an operator on what `prepare` made.  With `own` false
it computes the operator's plain form from elementary torch operations in 32
bits; with `own` true it calls the library.

The cache is a byte tensor [pages][kv heads][page_size / 32][34 D].  The last
axis is one 32-key group of one head: the key codes (32 rows of D / 2 bytes),
the value codes (the same), the key scales (32 rows of D / 32 bytes) and the
value scales.  Codes are E2M1, two to a byte (low nibble first), scales E8M0
bytes of the 32-element blocks along D.  Inside a row the bytes are ordered for
a tensor-core fragment: byte t (D / 8) + 4 b + j of a key row holds d = 32 b +
8 t + 2 j and the next one, byte g (D / 16) + 2 b + j of a value row holds
d = 32 b + 4 g + 2 j and the next one.
"""
import math
import random

import torch

own = False

GROUP = 32  # keys of a cache group


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decoding step of a few small sequences: launch latency
        dict(name="append-step-4", op="append", T=4, pad=0, Hkv=2, D=64, page=32),
        # one decoding step of a full batch, some of its places empty
        dict(name="append-step-128", op="append", T=128, pad=5, Hkv=8, D=128, page=64),
        # a long prompt's keys and values into the cache
        dict(name="append-prompt-65537", op="append", T=65537, pad=0, Hkv=8, D=128, page=64),
        # a short cached prefix back as bf16, for attention over a prompt that continues it
        dict(name="read-prefix-777", op="read", T=777, pad=9, Hkv=4, D=128, page=32),
        # a long cached context back as bf16
        dict(name="read-context-131072", op="read", T=131072, pad=0, Hkv=8, D=128, page=128),
        # one user, a short conversation, one token: launch latency
        dict(name="decode-1x300", op="decode", B=1, Sq=1, Hq=32, Hkv=8, D=128, page=64, longest=300, mix=0),
        # checking four drafted tokens a sequence, ragged lengths, some shorter than the draft
        dict(name="decode-draft-16x5000", op="decode", B=16, Sq=4, Hq=16, Hkv=2, D=64, page=32, longest=5000, mix=3),
        # one user, a context of 128 Ki tokens: the keys split over the GPU and joined
        dict(name="decode-1x131072", op="decode", B=1, Sq=1, Hq=40, Hkv=8, D=128, page=128, longest=131072, mix=0),
        # a full serving batch of ragged long contexts: memory bound
        dict(name="decode-64x32768", op="decode", B=64, Sq=1, Hq=32, Hkv=8, D=128, page=64, longest=32768, mix=7),
        # three short prompts in one pack, one of them a single token
        dict(name="prompt-3x130", op="prompt", B=3, Hq=8, Hkv=2, D=64, longest=130, more=0, mix=5, causal=True),
        # pieces of prompts that continue cached prefixes, ragged, five query heads to a key head
        dict(name="prompt-8x2500-chunk", op="prompt", B=8, Hq=40, Hkv=8, D=128, longest=2500, more=1500, mix=11, causal=True),
        # one whole prompt of 16 Ki tokens
        dict(name="prompt-1x16384", op="prompt", B=1, Hq=32, Hkv=8, D=128, longest=16384, more=0, mix=0, causal=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "decode", "prompt", "prompt"])
    D = rng.choice([64, 128, 128])
    page = rng.choice([32, 64, 96, 128, 256])
    if op in ("append", "read"):
        T = _log(rng, 1, 65537 if op == "append" else 131072)
        return dict(op=op, T=T, pad=min(T - 1, rng.choice([0, 0, 1, 7])), Hkv=rng.choice([1, 2, 3, 5, 8]), D=D, page=page)
    Hkv = rng.choice([1, 2, 3, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    if op == "decode":
        Sq = rng.choice([1, 1, 1, 2, 3, 5])
        B = _log(rng, 1, 64)
        longest = _log(rng, 1, 131072)
        while B * longest * Hkv > 64 * 32768 * 4:
            longest = max(1, longest // 2)
        return dict(op=op, B=B, Sq=Sq, Hq=G * Hkv, Hkv=Hkv, D=D, page=page, longest=longest, mix=rng.randrange(1 << 20))
    B = _log(rng, 1, 24)
    longest = _log(rng, 1, 8192)
    more = rng.choice([0, 0, _log(rng, 1, 4096)])
    while B * G * Hkv * longest * (longest + more) > 16 * 16384 * 16384 or B * longest > 65536:
        longest = max(1, longest // 2)
        more //= 2
    return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, D=D, longest=longest, more=more, mix=rng.randrange(1 << 20),
                causal=rng.random() < 0.85)


def _lengths(case):
    """Lengths of the case's sequences (decode: keys; prompt: queries and keys): the
    longest one first, the others spread below it, now and then an empty one."""
    r = random.Random(1000003 * case["mix"] + 7 * case["B"] + case["longest"])
    n = [case["longest"]]
    for i in range(1, case["B"]):
        n.append(0 if case["B"] > 6 and i == 5 else 1 + int(case["longest"] * r.random() ** 0.7 * 0.999))
    if case["op"] == "decode":
        return n, n
    return n, [x + (r.randrange(case["more"] + 1) if case["more"] else 0) for x in n]


# ------------------------------------------------------------------- data --

def _e2m1(x):
    """(values on the E2M1 grid, exponent X) of 32-element blocks x [..., 32] in 32 bits."""
    amax = x.abs().amax(-1, keepdim=True)
    f, e = torch.frexp(amax)
    X = torch.where(amax > 0, e - 3 + (f > 0.75).to(e.dtype), torch.full_like(e, -127)).clamp(-127, 127)
    y = torch.ldexp(x, -X)
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.round(y / step) * step, X


def _key_order(D, device):
    """d of every nibble of a key row, in the order of the row's bytes, low nibble first."""
    t, b, j, h = torch.meshgrid(*(torch.arange(n, device=device) for n in (4, D // 32, 4, 2)), indexing="ij")
    return (32 * b + 8 * t + 2 * j + h).reshape(-1)


def _value_order(D, device):
    g, b, j, h = torch.meshgrid(*(torch.arange(n, device=device) for n in (8, D // 32, 2, 2)), indexing="ij")
    return (32 * b + 4 * g + 2 * j + h).reshape(-1)


def _pack(x, order):
    """Rows x [N, D] in 32 bits -> (code bytes [N, D / 2], scale bytes [N, D / 32])."""
    N, D = x.shape
    y, X = _e2m1(x.view(N, D // 32, 32))
    a = y.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code + 8 * torch.signbit(y).to(torch.uint8)).view(N, D)[:, order]
    return code[:, 0::2] + 16 * code[:, 1::2], (X.view(N, D // 32) + 127).to(torch.uint8)


def _unpack(codes, scales, order):
    """(code bytes [..., D / 2], scale bytes [..., D / 32]) -> values [..., D] in 32 bits."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    grid = torch.cat([grid, -grid])
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    c = c[..., torch.argsort(order)]
    v = grid[c.int()]
    return torch.ldexp(v.unflatten(-1, (-1, 32)), scales.int().unsqueeze(-1) - 127).flatten(-2)


def _rand(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda")


def _new_cache(pages, Hkv, page, D):
    return torch.zeros((pages, Hkv, page // GROUP, 34 * D), dtype=torch.uint8, device="cuda")


def _parts(cache):
    """Views of a cache: key codes, value codes, key scales, value scales, each
    [pages, heads, groups, 32, bytes of a row]."""
    D = cache.shape[-1] // 34
    sizes = [GROUP * D // 2, GROUP * D // 2, GROUP * D // 32, GROUP * D // 32]
    return [p.unflatten(-1, (GROUP, -1)) for p in cache.split(sizes, -1)]


def _fill(cache, gen):
    """Keys (some channels larger than others) and values of normal size in every slot."""
    pages, H, groups, last = cache.shape
    D = last // 34
    kc, vc, ks, vs = _parts(cache)
    amp = torch.exp(0.5 * _rand((H, 1, 1, D), gen))
    piece = max(1, (1 << 25) // (H * groups * GROUP * D))
    for p in range(0, pages, piece):
        n = min(piece, pages - p)
        for codes, scales, order, a in ((kc, ks, _key_order(D, "cuda"), amp), (vc, vs, _value_order(D, "cuda"), 1.0)):
            x = (_rand((n, H, groups, GROUP, D), gen) * a).bfloat16().float()
            c, s = _pack(x.view(-1, D), order)
            codes[p:p + n] = c.view(n, H, groups, GROUP, D // 2)
            scales[p:p + n] = s.view(n, H, groups, GROUP, D // 32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, D, Hkv = case["op"], case["D"], case["Hkv"]
    st = dict(case=case)
    if op in ("append", "read"):
        T, page = case["T"], case["page"]
        pages = -(-T // page) + 3
        slots = torch.randperm(pages, generator=gen, device="cuda").repeat_interleave(page) * page
        slots = (slots + torch.arange(page, device="cuda").repeat(pages))[3:T + 3].clone()
        if case["pad"]:
            slots[T - case["pad"]:] = -1
        st.update(slots=slots, cache=_new_cache(pages, Hkv, page, D))
        if op == "append":
            # keys and values as one projection gives them: views of one tensor
            kv = _rand((T, 2, Hkv, D), gen)
            kv[:, 0] *= torch.exp(0.5 * _rand((Hkv, D), gen))
            kv = kv.bfloat16()
            st.update(k=kv[:, 0], v=kv[:, 1])
        else:
            _fill(st["cache"], gen)
    elif op == "decode":
        _, lens = _lengths(case)
        page = case["page"]
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 1
        perm = torch.randperm(pages, generator=gen, device="cuda").int()
        table = torch.full((case["B"], max(1, max(need))), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        st.update(cache=_new_cache(pages, Hkv, page, D), table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                  q=_rand((case["B"], case["Sq"], case["Hq"], D), gen).bfloat16())
        _fill(st["cache"], gen)
    else:
        nq, nk = _lengths(case)
        cq = torch.tensor([sum(nq[:i]) for i in range(len(nq) + 1)], dtype=torch.int32)
        ck = torch.tensor([sum(nk[:i]) for i in range(len(nk) + 1)], dtype=torch.int32)
        st.update(cu_q=cq.cuda(), cu_k=ck.cuda(), longest_q=max(nq), longest_k=max(nk),
                  q=_rand((sum(nq), case["Hq"], D), gen).bfloat16(),
                  k=(_rand((sum(nk), Hkv, D), gen) * torch.exp(0.5 * _rand((Hkv, D), gen))).bfloat16(),
                  v=_rand((sum(nk), Hkv, D), gen).bfloat16())
    return st


# ------------------------------------------------------------- plain forms --

def _rows_of(x, slots, page):
    """Rows of a cache part [pages, H, groups, 32, n] at the slots: [T, H, n]."""
    s = slots.clamp(min=0)
    return x[s // page, :, s % page // GROUP, s % GROUP]


def _plain_append(st):
    def held(x):
        y, X = _e2m1(x.float().unflatten(-1, (-1, 32)))
        y = torch.ldexp(y, X).flatten(-2)
        return torch.where((st["slots"] >= 0)[:, None, None], y, 0.0).bfloat16()
    return held(st["k"]), held(st["v"])


def _plain_read(st):
    page, D = st["case"]["page"], st["case"]["D"]
    kc, vc, ks, vs = _parts(st["cache"])
    there = (st["slots"] >= 0)[:, None, None]
    k = _unpack(_rows_of(kc, st["slots"], page), _rows_of(ks, st["slots"], page), _key_order(D, "cuda"))
    v = _unpack(_rows_of(vc, st["slots"], page), _rows_of(vs, st["slots"], page), _value_order(D, "cuda"))
    return torch.where(there, k, 0.0).bfloat16(), torch.where(there, v, 0.0).bfloat16()


def _attend(q, k, v, seen):
    """Softmax attention in 32 bits: q [B, H, G, Sq, D], k and v [B, H, Sk, D], seen
    [B, Sq, Sk]: outputs (zero where a row sees nothing) and log-sum-exps."""
    B, H, G, Sq, D = q.shape
    s = (q.reshape(B, H, G * Sq, D) / math.sqrt(D)) @ k.transpose(-1, -2)
    s = s.view(B, H, G, Sq, -1).masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, H, G * Sq, -1) @ v).view(B, H, G, Sq, D) / total.clamp(min=1e-30)
    return o, (m + torch.log(total)).squeeze(-1)


def _plain_decode(st):
    c = st["case"]
    B, Sq, Hq, Hkv, D = c["B"], c["Sq"], c["Hq"], c["Hkv"], c["D"]
    kc, vc, ks, vs = (p[st["table"].long().clamp(min=0)].transpose(1, 2).flatten(2, 4) for p in _parts(st["cache"]))
    k = _unpack(kc, ks, _key_order(D, "cuda"))
    v = _unpack(vc, vs, _value_order(D, "cuda"))
    key = torch.arange(k.shape[2], device="cuda")
    last = st["lens"][:, None] - Sq + torch.arange(Sq, device="cuda")  # the last key that query i sees
    seen = key <= last[:, :, None]
    q = st["q"].float().view(B, Sq, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    o, lse = _attend(q, k, v, seen)
    return o.permute(0, 3, 1, 2, 4).reshape(B, Sq, Hq, D).bfloat16(), lse.permute(0, 3, 1, 2).reshape(B, Sq, Hq)


def _plain_prompt(st):
    c = st["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    nq, nk = st["cu_q"].diff(), st["cu_k"].diff()
    iq, ik = torch.arange(st["longest_q"], device="cuda"), torch.arange(st["longest_k"], device="cuda")
    at_q = (st["cu_q"][:-1, None] + iq).clamp(max=st["q"].shape[0] - 1)
    at_k = (st["cu_k"][:-1, None] + ik).clamp(max=st["k"].shape[0] - 1)
    seen = (ik < nk[:, None])[:, None, :].expand(-1, len(iq), -1)
    if c["causal"]:
        seen = seen & (ik <= (nk - nq)[:, None, None] + iq[None, :, None])
    q = st["q"].float()[at_q].unflatten(2, (Hkv, Hq // Hkv)).permute(0, 2, 3, 1, 4)
    k, v = (st[n].float()[at_k].transpose(1, 2) for n in ("k", "v"))
    o, lse = _attend(q, k, v, seen)
    valid = iq < nq[:, None]
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3)[valid].bfloat16(), lse.permute(0, 3, 1, 2).flatten(2, 3)[valid]


def run(state):
    op = state["case"]["op"]
    if own:
        import matrix_core_softmax_gb300 as fsa
        if op == "append":
            fsa.kv4_append(state["cache"], state["k"], state["v"], state["slots"])
            return fsa.kv4_read(state["cache"], state["slots"])
        if op == "read":
            return fsa.kv4_read(state["cache"], state["slots"])
        if op == "decode":
            return fsa.kv4_attention_fwd(state["q"], state["cache"], state["table"], state["lens"], return_lse=True)
        return fsa.varlen_attention_fwd(state["q"], state["k"], state["v"], state["cu_q"], state["cu_k"],
                                        causal=state["case"]["causal"], return_lse=True)
    return {"append": _plain_append, "read": _plain_read, "decode": _plain_decode, "prompt": _plain_prompt}[op](state)


# -------------------------------------------------------------------- work --

def work(case):
    op, D, Hkv = case["op"], case["D"], case["Hkv"]
    row = Hkv * D * 2              # a token's keys, or values, in bf16
    held = 2 * Hkv * (D // 2 + D // 32)  # a token's keys and values in the cache
    if op in ("append", "read"):
        n = case["T"] - case["pad"]
        if op == "append":  # the bf16 rows in, the cache out and in again, the values out
            return {"bytes": 2 * row * n + 2 * held * n + 2 * row * case["T"] + 8 * case["T"], "flops": 0}
        return {"bytes": held * n + 2 * row * case["T"] + 8 * case["T"], "flops": 0}
    nq, nk = _lengths(case)
    if op == "decode":
        Sq, Hq = case["Sq"], case["Hq"]
        rows = case["B"] * Sq * Hq
        pages = sum(-(-n // case["page"]) for n in nk)
        pairs = sum(max(0, n - Sq + 1 + i) for n in nk for i in range(Sq))
        return {"bytes": held * sum(nk) + rows * (4 * D + 4) + 4 * pages + 4 * case["B"], "flops": 4 * D * Hq * pairs}
    pairs = 0
    for a, b in zip(nq, nk):
        pairs += a * b - (a * (a - 1) // 2 if case["causal"] else 0)
    return {"bytes": sum(nq) * case["Hq"] * (4 * D + 4) + 2 * row * sum(nk), "flops": 4 * D * case["Hq"] * pairs}


# ------------------------------------------------------------------- exact --

def _exact_rows(q, k, v, first):
    """One sequence and one key head in 64 bits: q [G, Sq, D], k and v [Sk, D];
    query i sees the keys up to and including first + i."""
    G, Sq, D = q.shape
    o = torch.zeros((G, Sq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((G, Sq), -math.inf, dtype=torch.float64, device=q.device)
    for i0 in range(0, Sq, 2048):
        i1 = min(Sq, i0 + 2048)
        n = min(k.shape[0], first + i1)
        if n <= 0:
            continue
        s = torch.einsum("gid,jd->gij", q[:, i0:i1], k[:n]) * D ** -0.5
        hidden = torch.arange(n, device=q.device)[None] > first + torch.arange(i0, i1, device=q.device)[:, None]
        s[:, hidden] = -math.inf
        lse[:, i0:i1] = torch.logsumexp(s, -1)
        some = torch.isfinite(lse[:, i0:i1, None])
        w = torch.where(some, torch.exp(s - torch.where(some, lse[:, i0:i1, None], 0.0)), 0.0)
        o[:, i0:i1] = torch.einsum("gij,jd->gid", w, v[:n])
    return o, lse


def _exact_cache_values(cache, which):
    """All values of a cache as held, in 64 bits: [pages, H, page, D], byte by byte
    from the layout's definition."""
    pages, H, groups, last = cache.shape
    D = last // 34
    size = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
    table = torch.tensor(size, dtype=torch.float64, device=cache.device)
    out = torch.empty((pages, H, groups, GROUP, D), dtype=torch.float64, device=cache.device)
    at = which * GROUP * D // 2
    code = cache[..., at:at + GROUP * D // 2].reshape(pages, H, groups, GROUP, D // 2)
    at = GROUP * D + which * GROUP * D // 32
    scale = cache[..., at:at + GROUP * D // 32].reshape(pages, H, groups, GROUP, D // 32)
    for d in range(D):
        b, r = divmod(d, 32)
        if which == 0:
            byte = (r // 8) * (D // 8) + 4 * b + (r % 8) // 2
        else:
            byte = (r // 4) * (D // 16) + 2 * b + (r % 4) // 2
        nibble = (code[..., byte] >> (4 * (d % 2))) & 15
        out[..., d] = table[nibble.long()] * torch.pow(2.0, scale[..., b].double() - 127)
    return out.view(pages, H, groups * GROUP, D)


def exact(case, seed):
    op, D, Hkv = case["op"], case["D"], case["Hkv"]
    if op != "append" and work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    if op == "append":
        def held(x):
            x = x.double().unflatten(-1, (-1, 32))
            top = x.abs().amax(-1, keepdim=True)
            X = torch.ceil(torch.log2(torch.where(top > 0, top, 2.0 ** -125) / 6))
            X = torch.where(6 * torch.pow(2.0, X - 1) >= top, X - 1, X)
            X = torch.where(6 * torch.pow(2.0, X) < top, X + 1, X)
            grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
            y = x.abs() / torch.pow(2.0, X)
            # nearest grid value; of two equally near ones that of the even code
            up = torch.bucketize(y, grid).clamp(1, 7)
            lo, hi = grid[up - 1], grid[up]
            code = torch.where((y - lo < hi - y) | ((y - lo == hi - y) & (up % 2 == 1)), up - 1, up)
            val = torch.sign(x) * grid[code] * torch.pow(2.0, X)
            val = val.flatten(-2)
            val[st["slots"] < 0] = 0
            return val
        return held(st["k"]), held(st["v"])
    if op == "read":
        page, res = case["page"], []
        for which in (0, 1):
            x = _exact_cache_values(st["cache"], which)
            s = st["slots"].clamp(min=0)
            x = x[s // page, :, s % page]
            x[st["slots"] < 0] = 0
            res.append(x)
        return tuple(res)
    Hq, G = case["Hq"], case["Hq"] // Hkv
    if op == "decode":
        B, Sq = case["B"], case["Sq"]
        o = torch.zeros((B, Sq, Hq, D), dtype=torch.float64, device="cuda")
        lse = torch.zeros((B, Sq, Hq), dtype=torch.float64, device="cuda")
        lens = st["lens"].tolist()
        for h in range(Hkv):
            kx, vx = (_exact_cache_values(st["cache"][:, h:h + 1], which) for which in (0, 1))
            for b in range(B):
                n = lens[b]
                pages = st["table"][b, :-(-n // case["page"])].long()
                k, v = kx[pages, 0].reshape(-1, D)[:n], vx[pages, 0].reshape(-1, D)[:n]
                r = _exact_rows(st["q"][b, :, h * G:(h + 1) * G].double().transpose(0, 1), k, v, n - Sq)
                o[b, :, h * G:(h + 1) * G], lse[b, :, h * G:(h + 1) * G] = r[0].transpose(0, 1), r[1].transpose(0, 1)
        return o, lse
    o = torch.zeros((st["q"].shape[0], Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((st["q"].shape[0], Hq), dtype=torch.float64, device="cuda")
    cq, ck = st["cu_q"].tolist(), st["cu_k"].tolist()
    for b in range(case["B"]):
        nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        for h in range(Hkv):
            k, v = (st[n][ck[b]:ck[b + 1], h].double() for n in ("k", "v"))
            q = st["q"][cq[b]:cq[b + 1], h * G:(h + 1) * G].double().transpose(0, 1)
            r = _exact_rows(q, k, v, nk - nq if case["causal"] else nk)
            o[cq[b]:cq[b + 1], h * G:(h + 1) * G], lse[cq[b]:cq[b + 1], h * G:(h + 1) * G] = r[0].transpose(0, 1), r[1].transpose(0, 1)
    return o, lse
