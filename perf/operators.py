"""Workloads of the attention operators: position rotation, appending to the paged 8-bit key/value
cache, single-token attention over that cache, and causal attention over packed prompts.

Each case is a dict of plain values.  `own = False` computes the operators in plain torch operations
(32-bit arithmetic, 64-bit angles); `own = True` calls the framework.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
# Smallest and largest exponent of a block's power-of-two scale.
EXP_LO, EXP_HI = -100, 100


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # One decode step's queries of a small batch, rotated on their own: the latency of a small call.
        dict(name="rotary decode 8x32x128", op="rotary", T=8, H=32, D=128, R=128, layout="half", dtype="bf16",
             scaling="none", factor=1.0, inverse=False, far=1000),
        # The queries of an 8192-token prompt over 96 heads, positions scaled for a long context.
        dict(name="rotary prompt 8192x96x128", op="rotary", T=8192, H=96, D=128, R=128, layout="half", dtype="bf16",
             scaling="yarn", factor=8.0, inverse=False, far=60000),
        # Half of each head rotated in interleaved pairs, fp32, an odd token count at far positions (a
        # million-token context served in pieces), undoing the rotation.
        dict(name="rotary partial 4099x12x64", op="rotary", T=4099, H=12, D=64, R=32, layout="interleaved",
             dtype="f32", scaling="linear", factor=4.0, inverse=True, far=1048575),
        # A decode step of 256 sequences around position 1000: one new token each, its queries rotated too.
        dict(name="append decode 256", op="append", B=256, Hq=64, Hk=8, D=128, R=128, P=64, layout="half",
             scaling="none", factor=1.0, new_lo=1, new_hi=1, ctx_lo=900, ctx_hi=1100, return_k=False, lens_seed=1),
        # Eight whole prompts packed (512 to 16384 tokens), whose rotated keys and queries feed the prompt attention.
        dict(name="append prompts 8x[512,16384]", op="append", B=8, Hq=32, Hk=8, D=128, R=128, P=64, layout="half",
             scaling="yarn", factor=4.0, new_lo=512, new_hi=16384, ctx_lo=0, ctx_hi=0, return_k=True, lens_seed=2),
        # Pieces of 37 prompts continuing part-filled pages: small heads, small pages, part of the head rotated.
        dict(name="append pieces 37x[1,100]", op="append", B=37, Hq=10, Hk=2, D=64, R=32, P=16, layout="interleaved",
             scaling="none", factor=1.0, new_lo=1, new_hi=100, ctx_lo=1, ctx_hi=5000, return_k=True, lens_seed=3),
        # One user's decode step at position 1000: the latency of a small call.
        dict(name="decode 1x1000", op="decode", B=1, Hq=32, Hk=8, D=128, P=64, len_lo=1000, len_hi=1000, lens_seed=4),
        # A decode batch of 256 sequences around position 1000.
        dict(name="decode 256x[900,1100]", op="decode", B=256, Hq=64, Hk=8, D=128, P=64, len_lo=900, len_hi=1100,
             lens_seed=5),
        # A few long documents of very different lengths, small pages.
        dict(name="decode 8x[8192,131072]", op="decode", B=8, Hq=40, Hk=8, D=128, P=16, len_lo=8192, len_hi=131072,
             lens_seed=6),
        # A short prompt with small heads: the latency of a small call.
        dict(name="prompt 1x100 d64", op="prompt", B=1, Hq=8, Hk=2, D=64, Dv=64, len_lo=100, len_hi=100, prefix=0,
             lens_seed=7),
        # One 8192-token prompt, four query heads to each key/value head.
        dict(name="prompt 1x8192 d128", op="prompt", B=1, Hq=32, Hk=8, D=128, Dv=128, len_lo=8192, len_hi=8192,
             prefix=0, lens_seed=8),
        # Packed prompts of different lengths with 32 heads of 192 (keys) and 128 (values), the widths of the
        # stack's full-attention layers.
        dict(name="prompt 8x[100,4096] d192", op="prompt", B=8, Hq=32, Hk=32, D=192, Dv=128, len_lo=100, len_hi=4096,
             prefix=0, lens_seed=9),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rotary", "append", "decode", "prompt"])
    seed = rng.randrange(1 << 20)
    while True:
        if op == "rotary":
            D = rng.choice([64, 128, 192, 256])
            c = dict(op=op, T=_log(rng, 1, 32768), H=rng.choice([1, 2, 5, 8, 12, 32, 64, 96]), D=D,
                     R=rng.choice([D, D, D // 2, 32]), layout=rng.choice(["half", "interleaved"]),
                     dtype=rng.choice(["bf16", "bf16", "f32"]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                     factor=float(rng.choice([1, 2, 8, 32])), inverse=rng.random() < 0.25,
                     far=_log(rng, 1000, 1048575))
            cost, most = c["T"] * c["H"] * D * (2 if c["dtype"] == "bf16" else 4), 8192 * 96 * 128 * 2
        elif op == "append":
            D = rng.choice([64, 128])
            Hk = rng.choice([1, 2, 4, 8, 16])
            one = rng.random() < 0.4
            lo = 1 if one else _log(rng, 1, 2000)
            hi = 1 if one else _log(rng, lo, 16384)
            ctx = _log(rng, 1, 20000)
            c = dict(op=op, B=_log(rng, 1, 512 if one else 64), Hq=Hk * rng.choice([1, 3, 4, 5, 8, 16]), Hk=Hk, D=D,
                     R=rng.choice([D, D, D // 2]), P=rng.choice([16, 32, 64, 128]),
                     layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                     factor=float(rng.choice([1, 4, 16])), new_lo=lo, new_hi=hi, ctx_lo=rng.choice([0, ctx // 2]),
                     ctx_hi=ctx, return_k=rng.random() < 0.5, lens_seed=seed)
            new, ctxs = _lens(c, "new"), _lens(c, "ctx")
            slots = sum(-(-(n + x) // c["P"]) * c["P"] for n, x in zip(new, ctxs))
            cost = sum(new) * (c["Hq"] + 2 * Hk) * D + slots * Hk * D // 8
            most = 41000 * 48 * 128
        elif op == "decode":
            Hk = rng.choice([1, 2, 4, 8, 16])
            lo = _log(rng, 1, 32768)
            c = dict(op=op, B=_log(rng, 1, 512), Hq=Hk * rng.choice([1, 2, 4, 5, 7, 8, 12, 16, 24]), Hk=Hk,
                     D=rng.choice([64, 128]), P=rng.choice([16, 32, 64, 128]), len_lo=lo,
                     len_hi=_log(rng, lo, 131072), lens_seed=seed)
            lens = _lens(c, "len")
            cost, most = len(lens) * max(lens) * Hk * c["D"], 8 * 131072 * 8 * 128 // 2
        else:
            Hk = rng.choice([1, 2, 4, 8, 32])
            D, Dv = rng.choice([(64, 64), (128, 128), (192, 128)])
            lo = _log(rng, 1, 4096)
            c = dict(op=op, B=_log(rng, 1, 24), Hq=Hk * rng.choice([1, 2, 3, 4, 8]), Hk=Hk, D=D, Dv=Dv, len_lo=lo,
                     len_hi=_log(rng, lo, 8192), prefix=rng.choice([0, 0, _log(rng, 1, 2000)]), lens_seed=seed)
            q, kv = _lens(c, "q"), _lens(c, "kv")
            cost, most = len(q) * c["Hq"] * max(q) * max(kv) * (D + Dv), 32 * 8192 * 8192 * 256
            if c["Hq"] > 64:
                continue
        if cost <= most:
            return c


def _spread(rng, lo, hi, n):
    if lo <= 0:
        return [rng.randint(lo, hi) for _ in range(n)]
    return [_log(rng, lo, hi) for _ in range(n)]


def _lens(c, what):
    """The case's sequence lengths: fixed by the case, so that the work is."""
    rng = random.Random("%s-%d" % ("len" if what in ("q", "kv") else what, c["lens_seed"]))
    if what == "new":
        return _spread(rng, c["new_lo"], c["new_hi"], c["B"])
    if what == "ctx":
        return _spread(rng, c["ctx_lo"], c["ctx_hi"], c["B"])
    lens = _spread(rng, c["len_lo"], c["len_hi"], c["B"])
    if what == "kv" and c["prefix"]:  # earlier tokens of each sequence, whose keys and values are there already
        return [n + rng.randint(0, c["prefix"]) for n in lens]
    return lens


def _inv_freq(c):
    """(angle per position of each pair, factor on the rotated part), in 64 bits on the host.

    linear: positions divided by the factor; ntk: the base raised so that the slowest pair turns `factor`
    times slower; yarn: pairs that turn at least 32 times within the original 4096 positions are kept, those
    that turn at most once are divided by the factor, the others in between, magnitude 0.1 ln(factor) + 1.
    """
    R, base, s = c["R"], 10000.0, c["factor"]
    e = torch.arange(0, R, 2, dtype=torch.float64) / R
    if c["scaling"] == "ntk" and R > 2:
        base = base * s ** (R / (R - 2))
    f = base ** -e
    if c["scaling"] == "linear":
        f = f / s
    if c["scaling"] == "yarn":
        keep = ((4096 * f / (2 * math.pi) - 1) / (32 - 1)).clamp(0, 1)
        return f * keep + f / s * (1 - keep), 0.1 * math.log(s) + 1.0
    return f, 1.0


# ---------------------------------------------------------------------------
# inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cum(v):
    out = [0]
    for n in v:
        out.append(out[-1] + n)
    return out


def _heads(g, T, H, D, spread=0.5):
    """bf16 activations: unit normal, with channels of different size, as keys and queries have."""
    ch = torch.exp(spread * torch.randn((H, D), generator=g, device=DEV))
    return (torch.randn((T, H, D), generator=g, device=DEV) * (ch / ch.square().mean(-1, keepdim=True).sqrt())).bfloat16()


def _pages(g, n, Hk, P, D):
    """A filled part of the cache: e4m3 codes and a power-of-two scale for each page and head."""
    codes = (torch.randn((n, Hk, P, D), generator=g, device=DEV, dtype=torch.bfloat16) * 64).to(torch.float8_e4m3fn)
    return codes, torch.exp2(torch.randint(-7, -4, (n, Hk), generator=g, device=DEV).float())


def _block_table(g, slots, P):
    """[B, widest] page numbers, every page once, in random order; the places behind a sequence's last page hold 0."""
    need = [-(-n // P) for n in slots]
    total = max(1, sum(need))
    order = torch.randperm(total, generator=g, device=DEV).int()
    w = max(1, max(need))
    n = _ints(need).long()
    first = torch.cumsum(n, 0) - n
    j = torch.arange(w, device=DEV)
    at = first[:, None] + j[None, :]
    return torch.where(j[None, :] < n[:, None], order[at.clamp(max=total - 1)], 0).int().contiguous(), total


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "rotary":
        f, s["magnitude"] = _inv_freq(c)
        s["inv_freq"] = f.to(DEV)
        start = torch.randint(0, max(1, c["far"] - c["T"] + 1), (1,), generator=g, device=DEV)
        s["positions"] = ((start + torch.arange(c["T"], device=DEV)) % (c["far"] + 1)).int()
        s["x"] = torch.randn((c["T"], c["H"], c["D"]), generator=g, device=DEV).to(
            torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
    elif c["op"] == "append":
        f, s["magnitude"] = _inv_freq(c)
        s["inv_freq"] = f.to(DEV)
        new, ctx = _lens(c, "new"), _lens(c, "ctx")
        s["block_table"], pages = _block_table(g, [a + b for a, b in zip(new, ctx)], c["P"])
        s["context_lens"] = _ints(ctx)
        s["cu_seqlens"] = _ints(_cum(new)) if c["new_hi"] > 1 else None
        T = sum(new)
        s["q"], s["k"] = _heads(g, T, c["Hq"], c["D"]), _heads(g, T, c["Hk"], c["D"])
        s["v"] = _heads(g, T, c["Hk"], c["D"], 0.1)
        kc, ks = _pages(g, pages, c["Hk"], c["P"], c["D"])
        vc, vs = _pages(g, pages, c["Hk"], c["P"], c["D"])
        s["cache"] = (kc, vc, ks, vs)
    elif c["op"] == "decode":
        lens = _lens(c, "len")
        s["block_table"], pages = _block_table(g, lens, c["P"])
        s["seq_lens"] = _ints(lens)
        s["q"] = _heads(g, c["B"], c["Hq"], c["D"])
        kc, ks = _pages(g, pages, c["Hk"], c["P"], c["D"])
        vc, vs = _pages(g, pages, c["Hk"], c["P"], c["D"])
        s["cache"] = (kc, vc, ks, vs)
    else:
        q, kv = _lens(c, "q"), _lens(c, "kv")
        s["cu_seqlens"] = _ints(_cum(q))
        s["cu_seqlens_k"] = _ints(_cum(kv)) if c["prefix"] else None
        # what the plain form pads to; the framework's call has no need of it
        s["widest"] = (max(q), max(kv))
        s["q"], s["k"] = _heads(g, sum(q), c["Hq"], c["D"]), _heads(g, sum(kv), c["Hk"], c["D"])
        s["v"] = _heads(g, sum(kv), c["Hk"], c["Dv"], 0.1)
    return s


# ---------------------------------------------------------------------------
# plain forms

def _rotate(x, positions, inv_freq, magnitude, R, layout, sign=1.0):
    """x [T, H, D] in 32 bits, its first R channels rotated; angles in 64 bits."""
    angle = positions.double()[:, None] * inv_freq[None, :]
    cos = (torch.cos(angle) * magnitude).float()[:, None, :]
    sin = (torch.sin(angle) * (magnitude * sign)).float()[:, None, :]
    x = x.float()
    if layout == "half":
        a, b = x[..., : R // 2], x[..., R // 2 : R]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_rotary(s):
    c = s["case"]
    y = _rotate(s["x"], s["positions"], s["inv_freq"], s["magnitude"], c["R"], c["layout"], -1.0 if c["inverse"] else 1.0)
    return y.to(s["x"].dtype)


def _need(amax):
    """The smallest exponent e with amax <= 448 * 2^e, within the limits."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    return torch.where(amax > 0, (e - 9 + (m > 0.875).int()).clamp(EXP_LO, EXP_HI), EXP_LO)


def _write_blocks(x, codes, scale, tok_page, tok_off, slot, pages, first_off):
    """Quantises x [T, H, D] into its pages.  slot: each token's place among `pages`, the pages written;
    first_off: where each page's new tokens begin (what lies before is kept)."""
    amax = torch.zeros((pages.numel(), x.shape[1]), device=x.device)
    amax = amax.index_reduce_(0, slot, x.abs().amax(-1), "amax")
    need = _need(amax)
    old = torch.frexp(scale[pages])[1] - 1
    e = torch.where(first_off[:, None] > 0, torch.maximum(old, need), need)
    # earlier tokens of the page, moved to the new scale where it grew
    kept = codes[pages].float() * torch.exp2((old - e).float())[:, :, None, None]
    keep = torch.arange(codes.shape[2], device=x.device)[None, :] < first_off[:, None]
    moved = torch.where(keep[:, None, :, None], kept.to(torch.float8_e4m3fn).view(torch.uint8), codes[pages].view(torch.uint8))
    codes.view(torch.uint8)[pages] = moved
    scale[pages] = torch.exp2(e.float())
    q = (x * torch.exp2(-e.float())[slot][..., None]).to(torch.float8_e4m3fn)
    codes.view(torch.uint8)[tok_page, :, tok_off] = q.view(torch.uint8)


def _plain_append(s):
    c = s["case"]
    kc, vc, ks, vs = s["cache"]
    T, P = s["k"].shape[0], c["P"]
    t = torch.arange(T, device=DEV)
    b = t if s["cu_seqlens"] is None else torch.searchsorted(s["cu_seqlens"][1:].contiguous(), t.int(), right=True)
    i = t - (t if s["cu_seqlens"] is None else s["cu_seqlens"].long()[b])
    pos = s["context_lens"].long()[b] + i
    page, off = s["block_table"].long()[b, pos // P], pos % P
    first = torch.full((kc.shape[0],), P, dtype=torch.long, device=DEV).index_reduce_(0, page, off, "amin")
    pages = torch.nonzero(first < P).flatten()
    slot = torch.searchsorted(pages, page)
    q = _rotate(s["q"], pos, s["inv_freq"], s["magnitude"], c["R"], c["layout"]).bfloat16()
    k = _rotate(s["k"], pos, s["inv_freq"], s["magnitude"], c["R"], c["layout"])
    _write_blocks(k, kc, ks, page, off, slot, pages, first[pages])
    _write_blocks(s["v"].float(), vc, vs, page, off, slot, pages, first[pages])
    return [q, k.bfloat16() if c["return_k"] else None, kc, vc, ks, vs]


def _softmax_sum(scores, mask, v):
    """(sum of softmax(scores) v, log of the sum of exponentials) over the last axis; rows without a key give 0 and -inf."""
    scores = scores.masked_fill(~mask, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, 1.0)
    return o, (torch.log(total) + top).squeeze(-1)


def _plain_decode(s):
    c = s["case"]
    kc, vc, ks, vs = s["cache"]
    G, P, D = c["Hq"] // c["Hk"], c["P"], c["D"]
    bt = s["block_table"].long()
    B, w = bt.shape

    def gather(codes, scale):  # [B, Hk, w * P, D]
        x = codes.view(torch.uint8)[bt].view(torch.float8_e4m3fn).float() * scale[bt][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, c["Hk"], w * P, D)

    q = s["q"].float().view(B, c["Hk"], G, D)
    scores = q @ gather(kc, ks).transpose(-1, -2) * D ** -0.5
    mask = torch.arange(w * P, device=DEV)[None, :] < s["seq_lens"][:, None]
    o, lse = _softmax_sum(scores, mask[:, None, None, :], gather(vc, vs))
    return [o.reshape(B, c["Hq"], D).bfloat16(), lse.reshape(B, c["Hq"])]


def _plain_prompt(s):
    c = s["case"]
    G = c["Hq"] // c["Hk"]
    Lq, Lk = s["widest"]
    cq = s["cu_seqlens"].long()
    ck = cq if s["cu_seqlens_k"] is None else s["cu_seqlens_k"].long()
    nq, nk = cq[1:] - cq[:-1], ck[1:] - ck[:-1]
    iq, ik = torch.arange(Lq, device=DEV), torch.arange(Lk, device=DEV)
    at_q = (cq[:-1, None] + iq).clamp(max=s["q"].shape[0] - 1)
    at_k = (ck[:-1, None] + ik).clamp(max=s["k"].shape[0] - 1)
    B = at_q.shape[0]
    q = s["q"].float()[at_q].view(B, Lq, c["Hk"], G, c["D"]).permute(0, 2, 3, 1, 4)
    k = s["k"].float()[at_k].permute(0, 2, 3, 1)[:, :, None]
    v = s["v"].float()[at_k].permute(0, 2, 1, 3)[:, :, None]
    # query i of a sequence sees its keys up to i + (keys - queries)
    mask = (ik[None, None, :] <= iq[None, :, None] + (nk - nq)[:, None, None]) & (ik[None, None, :] < nk[:, None, None])
    o, lse = _softmax_sum(q @ k * c["D"] ** -0.5, mask[:, None, None], v)
    live = (iq[None, :] < nq[:, None]).flatten()
    o = o.permute(0, 3, 1, 2, 4).reshape(B * Lq, c["Hq"], c["Dv"])[live]
    lse = lse.permute(0, 3, 1, 2).reshape(B * Lq, c["Hq"])[live]
    return [o.bfloat16(), lse]


def run(state):
    s, c = state, state["case"]
    if own:
        import kimi_delta_attention_gated_gb300 as kda

        if c["op"] == "rotary":
            return kda.rotary(s["x"], s["positions"], s["inv_freq"], magnitude=s["magnitude"], layout=c["layout"],
                              inverse=c["inverse"])
        if c["op"] == "append":
            q, k = kda.kv_append(s["k"], s["v"], s["cache"], s["block_table"], s["context_lens"],
                                 cu_seqlens=s["cu_seqlens"], inv_freq=s["inv_freq"], magnitude=s["magnitude"],
                                 layout=c["layout"], q=s["q"], return_k=c["return_k"])
            return [q, k, *s["cache"]]
        if c["op"] == "decode":
            return list(kda.attn_decode(s["q"], s["cache"], s["block_table"], s["seq_lens"], return_lse=True))
        return list(kda.attn_prompt(s["q"], s["k"], s["v"], cu_seqlens=s["cu_seqlens"],
                                    cu_seqlens_k=s["cu_seqlens_k"], return_lse=True))
    return {"rotary": _plain_rotary, "append": _plain_append, "decode": _plain_decode, "prompt": _plain_prompt}[c["op"]](s)


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "rotary":
        n = c["T"] * c["H"] * c["D"]
        return {"bytes": 2 * n * (2 if c["dtype"] == "bf16" else 4) + 4 * c["T"], "flops": 3 * n}
    if c["op"] == "append":
        T = sum(_lens(c, "new"))
        k = T * c["Hk"] * c["D"]
        q = T * c["Hq"] * c["D"]
        # k and v in 16 bits in, 8 bits out; q (and k, where it is wanted) in and out in 16 bits
        return {"bytes": 2 * 3 * k + 4 * q + (2 * k if c["return_k"] else 0), "flops": 3 * (q + k) + 4 * k}
    if c["op"] == "decode":
        n = sum(_lens(c, "len"))
        pages = sum(-(-x // c["P"]) for x in _lens(c, "len"))
        q = c["B"] * c["Hq"]
        return {"bytes": 2 * n * c["Hk"] * c["D"] + 8 * pages * c["Hk"] + 4 * pages + 4 * q * c["D"] + 4 * q,
                "flops": 4 * n * c["Hq"] * c["D"]}
    q, kv = _lens(c, "q"), _lens(c, "kv")
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(q, kv))
    return {"bytes": 2 * (sum(q) * c["Hq"] + sum(kv) * c["Hk"]) * (c["D"] + c["Dv"]) + 4 * sum(q) * c["Hq"],
            "flops": 2 * pairs * c["Hq"] * (c["D"] + c["Dv"])}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits: complex rotation, token by token pages, one sequence and head group at a time

def _turn64(x, positions, f, magnitude, layout, sign=1):
    x = x.double()
    R = 2 * f.numel()
    pairs = x[..., :R].unflatten(-1, (2, -1)).transpose(-1, -2) if layout == "half" else x[..., :R].unflatten(-1, (-1, 2))
    turn = torch.polar(torch.full((positions.numel(), f.numel()), float(magnitude), dtype=torch.float64, device=x.device),
                       sign * torch.outer(positions.double(), f))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
    out = x.clone()
    out[..., :R] = (z.transpose(-1, -2) if layout == "half" else z).flatten(-2)
    return out


def _to_e4m3_64(x):
    """x (64 bits, at most 448 in size) rounded to the nearest e4m3 value, ties to even."""
    step = torch.exp2((torch.frexp(x)[1] - 4).clamp(min=-9).double())
    return torch.round(x / step) * step


def _exact_append(c, s):
    kc, vc, ks, vs = s["cache"]
    new, ctx, P = _lens(c, "new"), _lens(c, "ctx"), c["P"]
    pos = torch.cat([torch.arange(x, x + n) for n, x in zip(new, ctx)]).to(DEV)
    q = _turn64(s["q"], pos, s["inv_freq"], s["magnitude"], c["layout"])
    k = _turn64(s["k"], pos, s["inv_freq"], s["magnitude"], c["layout"])
    bt = s["block_table"].cpu()
    codes, scales = [], []
    for x, cd, sc in ((k, kc, ks), (s["v"].double(), vc, vs)):
        cd, sc = cd.float(), sc.double().cpu().clone()
        amax = x.abs().amax(-1).cpu()
        t0 = 0
        for b in range(c["B"]):
            for j in range(ctx[b] // P, (ctx[b] + new[b] - 1) // P + 1):
                lo, hi = max(ctx[b], j * P), min(ctx[b] + new[b], (j + 1) * P)
                a, z = t0 + lo - ctx[b], t0 + hi - ctx[b]
                page, most = int(bt[b, j]), amax[a:z].amax(0)
                e = torch.ceil(torch.log2(most / E4M3_MAX)).clamp(EXP_LO, EXP_HI)
                old = torch.log2(sc[page])
                if lo > j * P:
                    e = torch.maximum(e, old)
                    shrink = torch.exp2(old - e).to(DEV)[:, None, None]
                    cd[page, :, : lo - j * P] = _to_e4m3_64(cd[page, :, : lo - j * P].double() * shrink).float()
                sc[page] = torch.exp2(e)
                y = x[a:z] * torch.exp2(-e).to(DEV)[None, :, None]
                cd[page, :, lo - j * P : hi - j * P] = _to_e4m3_64(y).float().transpose(0, 1)
            t0 += new[b]
        codes.append(cd)
        scales.append(sc.to(DEV))
    return [q, k if c["return_k"] else None, codes[0], codes[1], scales[0], scales[1]]


def _attend64(q, k, v, seen):
    """q [G, n, D], k [L, D], v [L, Dv]; row i of each head sees the first seen[i] keys."""
    s = q @ k.T * q.shape[-1] ** -0.5
    s = s.masked_fill(torch.arange(k.shape[0], device=DEV)[None, :] >= seen[:, None], -math.inf)
    lse = torch.logsumexp(s, -1)
    return torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None]) @ v, lse


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rotary":
        return _turn64(s["x"], s["positions"], s["inv_freq"], s["magnitude"], c["layout"], -1 if c["inverse"] else 1)
    if c["op"] == "append":
        return _exact_append(c, s)
    G = c["Hq"] // c["Hk"]
    if c["op"] == "decode":
        kc, vc, ks, vs = s["cache"]
        o = torch.zeros((c["B"], c["Hq"], c["D"]), dtype=torch.float64, device=DEV)
        lse = torch.full((c["B"], c["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
        for b, n in enumerate(_lens(c, "len")):
            at = s["block_table"][b, : -(-n // c["P"])].long()
            kb, vb = kc.view(torch.uint8)[at].view(kc.dtype).double(), vc.view(torch.uint8)[at].view(vc.dtype).double()
            for h in range(c["Hk"]):
                k = (kb[:, h] * ks[at, h].double()[:, None, None]).flatten(0, 1)[:n]
                v = (vb[:, h] * vs[at, h].double()[:, None, None]).flatten(0, 1)[:n]
                hs = slice(h * G, (h + 1) * G)
                r, l = _attend64(s["q"][b, hs].double()[:, None], k, v, torch.tensor([n], device=DEV))
                o[b, hs], lse[b, hs] = r[:, 0], l[:, 0]
        return [o, lse]
    cq, ck = _cum(_lens(c, "q")), _cum(_lens(c, "kv"))
    o = torch.zeros((cq[-1], c["Hq"], c["Dv"]), dtype=torch.float64, device=DEV)
    lse = torch.full((cq[-1], c["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        n, m = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        seen = torch.arange(n, device=DEV) + 1 + m - n
        for h in range(c["Hk"]):
            hs = slice(h * G, (h + 1) * G)
            q = s["q"][cq[b] : cq[b + 1], hs].double().transpose(0, 1)
            r, l = _attend64(q, s["k"][ck[b] : ck[b + 1], h].double(), s["v"][ck[b] : ck[b + 1], h].double(), seen)
            o[cq[b] : cq[b + 1], hs], lse[cq[b] : cq[b + 1], hs] = r.transpose(0, 1), l.transpose(0, 1)
    return [o, lse]
