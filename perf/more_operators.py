"""Workloads of the latent-attention operators: one vector of 512 + 64 channels a token stands for the keys
and values of all heads.  Appending it to its paged cache (normalised, its 64 position channels turned),
taking queries into its space, attention over the cache there, bringing the result back to each head's
values, and expanding packed latents to whole keys and values for a prompt.

Each case is a dict of plain values.  `own = False` computes the operators in plain torch operations
(32-bit arithmetic, 64-bit angles); `own = True` calls the framework.
"""
import math
import random

import torch

own = False

DEV = "cuda"
# Channels: the shared latent, the shared position part of a key, a head's own key and value.
C, R, DK, DV = 512, 64, 128, 128
EPS = 1e-5


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # A decode step of 256 sequences around position 1000: one new token's latent each, without positions.
        dict(name="append decode 256", op="append", B=256, P=64, turned=0, layout="half", scaling="none", factor=1.0,
             new_lo=1, new_hi=1, ctx_lo=900, ctx_hi=1100, norm=True, rows=False, beside=0, lens_seed=1),
        # Eight new prompts, the latents a part of a wider projection's rows, kept in a row too for the expanded form.
        dict(name="append prompts 8x[512,16384]", op="append", B=8, P=64, turned=64, layout="interleaved",
             scaling="yarn", factor=8.0, new_lo=512, new_hi=16384, ctx_lo=0, ctx_hi=0, norm=True, rows=True,
             beside=1536, lens_seed=2),
        # The queries of a small decode step: the latency of a small call.
        dict(name="queries 8x32", op="queries", T=8, H=32, turned=0, layout="half", scaling="none", factor=1.0, far=2000),
        # The queries of a decode step of 256 sequences with 128 heads, with positions.
        dict(name="queries 256x128", op="queries", T=256, H=128, turned=64, layout="interleaved", scaling="yarn",
             factor=8.0, far=60000),
        # One user's decode step at 1000 tokens: latency.
        dict(name="attn 1x1000 h32", op="attn", B=1, H=32, P=64, n_lo=1, n_hi=1, ctx_lo=999, ctx_hi=999, lens_seed=3),
        # The ordinary decode step of a batch.
        dict(name="attn 128x[900,1100] h32", op="attn", B=128, H=32, P=64, n_lo=1, n_hi=1, ctx_lo=900, ctx_hi=1100,
             lens_seed=4),
        # Long contexts of very different lengths, many heads.
        dict(name="attn 8x[8192,131072] h96", op="attn", B=8, H=96, P=128, n_lo=1, n_hi=1, ctx_lo=8192, ctx_hi=131072,
             lens_seed=5),
        # Drafted tokens being verified: one to six a sequence, causal among themselves, small pages.
        dict(name="attn drafts 37x[1,6] h16", op="attn", B=37, H=16, P=16, n_lo=1, n_hi=6, ctx_lo=1, ctx_hi=5000,
             lens_seed=6),
        # The way back for a small decode step, and for 256 sequences with 128 heads.
        dict(name="values 8x32", op="values", T=8, H=32),
        dict(name="values 256x128", op="values", T=256, H=128),
        # Keys and values of a short prompt, and of an 8192-token one.
        dict(name="expand 100x16", op="expand", T=100, H=16),
        dict(name="expand 8192x32", op="expand", T=8192, H=32),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


_HEADS = [1, 2, 5, 8, 12, 16, 20, 32, 48, 64, 96, 128]


def draw(rng):
    op = rng.choice(["append", "queries", "attn", "attn", "values", "expand"])
    seed = rng.randrange(1 << 20)
    pos = dict(turned=rng.choice([0, 64, 64, 32]), layout=rng.choice(["half", "interleaved"]),
               scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=float(rng.choice([1, 4, 16])))
    while True:
        if op == "append":
            one = rng.random() < 0.4
            lo = 1 if one else _log(rng, 1, 2000)
            hi = 1 if one else _log(rng, lo, 16384)
            ctx = _log(rng, 1, 20000)
            c = dict(op=op, B=_log(rng, 1, 512 if one else 64), P=rng.choice([16, 32, 64, 128]), new_lo=lo, new_hi=hi,
                     ctx_lo=rng.choice([0, ctx // 2]), ctx_hi=ctx, norm=rng.random() < 0.8, rows=rng.random() < 0.5,
                     beside=rng.choice([0, 0, 64, 1536]), lens_seed=seed, **pos)
            slots = sum(-(-(n + x) // c["P"]) * c["P"] for n, x in zip(_lens(c, "new"), _lens(c, "ctx")))
            cost, most = sum(_lens(c, "new")) + slots // 8, 41000
        elif op == "attn":
            lo = _log(rng, 1, 32768)
            n = rng.choice([1, 1, 1, 4, 8, _log(rng, 1, 300)])
            c = dict(op=op, B=_log(rng, 1, 512), H=rng.choice(_HEADS), P=rng.choice([16, 32, 64, 128]),
                     n_lo=rng.choice([1, n]), n_hi=n, ctx_lo=rng.choice([0, lo]), ctx_hi=_log(rng, lo, 131072),
                     lens_seed=seed)
            most_n, most_len = max(_lens(c, "n")), max(a + b for a, b in zip(_lens(c, "n"), _lens(c, "ctx")))
            cost, most = c["B"] * most_len * max(most_n * c["H"], 48), 8 * 131072 * 96
        else:
            c = dict(op=op, T=_log(rng, 1, 16384), H=rng.choice(_HEADS))
            if op == "queries":
                c.update(far=_log(rng, 1000, 1048575), **pos)
            cost, most = c["T"] * c["H"], 8192 * 32
        if cost <= most:
            return c


def _spread(rng, lo, hi, n):
    if lo <= 0:
        return [rng.randint(lo, hi) for _ in range(n)]
    return [_log(rng, lo, hi) for _ in range(n)]


def _lens(c, what):
    """The case's lengths ("new" or "n": tokens of the call, "ctx": those before): fixed by the case, so that
    the work is."""
    return _spread(random.Random("%s-%d" % (what, c["lens_seed"])), c[what + "_lo"], c[what + "_hi"], c["B"])


def _inv_freq(c):
    """(angle per position of each pair, factor on the turned part), in 64 bits on the host.

    linear: positions divided by the factor; ntk: the base raised so that the slowest pair turns `factor`
    times slower; yarn: pairs that turn at least 32 times within the original 4096 positions are kept, those
    that turn at most once are divided by the factor, the others in between, magnitude 0.1 ln(factor) + 1.
    """
    n, base, s = c["turned"], 10000.0, c["factor"]
    e = torch.arange(0, n, 2, dtype=torch.float64) / n
    if c["scaling"] == "ntk":
        base = base * s ** (n / (n - 2))
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


def _rows(g, *shape, spread=0.5):
    """bf16 activations: unit normal, with channels of different size."""
    ch = torch.exp(spread * torch.randn(shape[-1], generator=g, device=DEV))
    return (torch.randn(shape, generator=g, device=DEV) * (ch / ch.square().mean().sqrt())).bfloat16()


def _weights(g, H):
    """The projection from the latent to every head's keys and values, as trained: [H, keys then values, latent]."""
    return (torch.randn((H, DK + DV, C), generator=g, device=DEV) * C ** -0.5).bfloat16()


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
    s = {"case": c, "inv_freq": None, "magnitude": 1.0}
    if c.get("turned"):
        f, s["magnitude"] = _inv_freq(c)
        s["inv_freq"] = f.to(DEV)
    if c["op"] == "append":
        new, ctx = _lens(c, "new"), _lens(c, "ctx")
        s["block_table"], pages = _block_table(g, [a + b for a, b in zip(new, ctx)], c["P"])
        s["context_lens"] = _ints(ctx)
        s["cu_seqlens"] = _ints(_cum(new)) if c["new_hi"] > 1 else None
        s["x"] = _rows(g, sum(new), c["beside"] + C + R)[:, c["beside"]:]
        s["norm_w"] = 1 + 0.1 * torch.randn(C, generator=g, device=DEV) if c["norm"] else None
        s["cache"] = _rows(g, pages, c["P"], C + R)
    elif c["op"] == "queries":
        start = torch.randint(0, c["far"] + 1, (c["T"],), generator=g, device=DEV)
        s["positions"] = start.int() if c["turned"] else None
        s["q"], s["w"] = _rows(g, c["T"], c["H"], DK + R), _weights(g, c["H"])
    elif c["op"] == "attn":
        n, ctx = _lens(c, "n"), _lens(c, "ctx")
        lens = [a + b for a, b in zip(n, ctx)]
        s["block_table"], pages = _block_table(g, lens, c["P"])
        s["seq_lens"] = _ints(lens)
        s["cu_seqlens"] = _ints(_cum(n)) if c["n_hi"] > 1 else None
        s["most"] = max(n)  # what the plain form pads to; the framework's call has no need of it
        s["q"], s["cache"] = _rows(g, sum(n), c["H"], C + R), _rows(g, pages, c["P"], C + R)
    elif c["op"] == "values":
        s["o"], s["w"] = _rows(g, c["T"], c["H"], C), _weights(g, c["H"])
    else:
        s["rows"], s["w"] = _rows(g, c["T"], C + R), _weights(g, c["H"])
    return s


# ---------------------------------------------------------------------------
# plain forms

def _turn(x, positions, s):
    """x [T, .., R] in 32 bits, its first channels turned in pairs; angles in 64 bits."""
    if s["inv_freq"] is None:
        return x
    n = s["case"]["turned"]
    angle = positions.double()[:, None] * s["inv_freq"][None, :]
    angle = angle.view(angle.shape[0], *([1] * (x.dim() - 2)), angle.shape[1])
    cos, sin = (torch.cos(angle) * s["magnitude"]).float(), (torch.sin(angle) * s["magnitude"]).float()
    if s["case"]["layout"] == "half":
        a, b = x[..., : n // 2], x[..., n // 2 : n]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:n:2], x[..., 1:n:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, x[..., n:]], -1)


def _plain_append(s):
    P = s["case"]["P"]
    t = torch.arange(s["x"].shape[0], device=DEV)
    b = t if s["cu_seqlens"] is None else torch.searchsorted(s["cu_seqlens"][1:].contiguous(), t.int(), right=True)
    i = t - (t if s["cu_seqlens"] is None else s["cu_seqlens"].long()[b])
    pos = s["context_lens"].long()[b] + i
    x = s["x"].float()
    lat = x[:, :C]
    if s["norm_w"] is not None:
        lat = lat * torch.rsqrt(lat.square().mean(-1, keepdim=True) + EPS) * s["norm_w"]
    rows = torch.cat([lat, _turn(x[:, C:], pos, s)], -1).bfloat16()
    s["cache"][s["block_table"].long()[b, pos // P], pos % P] = rows
    return [s["cache"], rows if s["case"]["rows"] else None]


def _plain_queries(s):
    q = s["q"].float()
    lat = torch.einsum("thd,hdc->thc", q[..., :DK], s["w"][:, :DK].float())
    return torch.cat([lat, _turn(q[..., DK:], s["positions"], s)], -1).bfloat16()


def _plain_attn(s):
    c, m = s["case"], s["most"]
    B, H = c["B"], c["H"]
    kv = s["cache"][s["block_table"].long()].flatten(1, 2).float()  # [B, places, C + R]
    cu = torch.arange(B + 1, device=DEV) if s["cu_seqlens"] is None else s["cu_seqlens"].long()
    n, i = cu[1:] - cu[:-1], torch.arange(m, device=DEV)
    q = s["q"].float()[(cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)]  # [B, m, H, C + R]
    seen = s["seq_lens"][:, None] - n[:, None] + i + 1
    scores = (q.flatten(1, 2) @ kv.transpose(1, 2) * (DK + R) ** -0.5).view(B, m, H, -1)
    scores.masked_fill_((torch.arange(kv.shape[1], device=DEV) >= seen[..., None])[:, :, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores.sub_(torch.where(top == -math.inf, 0.0, top)))
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(1, 2) @ kv[..., :C]).view(B, m, H, C) / torch.where(total > 0, total, 1.0)
    live = i < n[:, None]
    return [o[live].bfloat16(), (torch.log(total) + top)[..., 0][live]]


def _plain_values(s):
    return torch.einsum("thc,hdc->thd", s["o"].float(), s["w"][:, DK:].float()).bfloat16()


def _plain_expand(s):
    x, H = s["rows"].float(), s["case"]["H"]
    kv = (x[:, :C] @ s["w"].float().flatten(0, 1).T).view(-1, H, DK + DV)
    k = torch.cat([kv[..., :DK], x[:, None, C:].expand(-1, H, -1)], -1)
    return [k.bfloat16(), kv[..., DK:].bfloat16()]


def run(state):
    s, c = state, state["case"]
    if own:
        import kimi_delta_attention_gated_gb300 as kda

        if c["op"] == "append":
            rows = kda.latent_append(s["x"], s["cache"], s["block_table"], s["context_lens"], cu_seqlens=s["cu_seqlens"],
                                     norm_w=s["norm_w"], eps=EPS, inv_freq=s["inv_freq"], magnitude=s["magnitude"],
                                     layout=c["layout"], return_rows=c["rows"])
            return [s["cache"], rows]
        if c["op"] == "queries":
            return kda.latent_queries(s["q"], s["w"], positions=s["positions"], inv_freq=s["inv_freq"],
                                      magnitude=s["magnitude"], layout=c["layout"])
        if c["op"] == "attn":
            return list(kda.attn_latent(s["q"], s["cache"], s["block_table"], s["seq_lens"], cu_seqlens=s["cu_seqlens"],
                                        return_lse=True))
        if c["op"] == "values":
            return kda.latent_values(s["o"], s["w"])
        return list(kda.latent_expand(s["rows"], s["w"]))
    return {"append": _plain_append, "queries": _plain_queries, "attn": _plain_attn, "values": _plain_values,
            "expand": _plain_expand}[c["op"]](s)


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "append":
        T = sum(_lens(c, "new"))
        return {"bytes": 2 * (C + R) * T * (3 if c["rows"] else 2), "flops": 4 * T * C + 3 * T * c["turned"]}
    if c["op"] == "attn":
        n, ctx = _lens(c, "n"), _lens(c, "ctx")
        kept, rows = sum(a + b for a, b in zip(n, ctx)), sum(n) * c["H"]
        pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(n, ctx))
        return {"bytes": 2 * (C + R) * kept + 2 * rows * (C + R + C) + 4 * rows,
                "flops": 2 * pairs * c["H"] * (C + R + C)}
    T, H = c["T"], c["H"]
    if c["op"] == "queries":
        return {"bytes": 2 * T * H * (DK + R + C + R) + 2 * H * DK * C, "flops": 2 * T * H * DK * C}
    if c["op"] == "values":
        return {"bytes": 2 * T * H * (C + DV) + 2 * H * DV * C, "flops": 2 * T * H * DV * C}
    return {"bytes": 2 * T * (C + R) + 2 * T * H * (DK + R + DV) + 2 * H * (DK + DV) * C,
            "flops": 2 * T * H * (DK + DV) * C}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits: complex rotation, one sequence or head at a time, keys and values of each
# head where the plain form works on the latent

def _turn64(x, positions, s):
    x = x.double()
    f = s["inv_freq"]
    if f is None:
        return x
    n = 2 * f.numel()
    half = s["case"]["layout"] == "half"
    pairs = x[..., :n].unflatten(-1, (2, -1)).transpose(-1, -2) if half else x[..., :n].unflatten(-1, (-1, 2))
    turn = torch.polar(torch.full((positions.numel(), f.numel()), float(s["magnitude"]), dtype=torch.float64, device=DEV),
                       torch.outer(positions.double(), f))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
    out = x.clone()
    out[..., :n] = (z.transpose(-1, -2) if half else z).flatten(-2)
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "append":
        new, ctx, P = _lens(c, "new"), _lens(c, "ctx"), c["P"]
        cache, bt, t0, kept = s["cache"].double(), s["block_table"].long(), 0, []
        for b in range(c["B"]):
            x = s["x"][t0 : t0 + new[b]].double()
            t0 += new[b]
            place = torch.arange(ctx[b], ctx[b] + new[b], device=DEV)
            lat = x[:, :C]
            if s["norm_w"] is not None:
                lat = s["norm_w"].double() * lat / torch.sqrt((lat * lat).sum(1) / C + EPS)[:, None]
            row = torch.cat([lat, _turn64(x[:, None, C:], place, s)[:, 0]], 1)
            cache.view(-1, C + R)[bt[b, place // P] * P + place % P] = row
            kept.append(row)
        return [cache, torch.cat(kept) if c["rows"] else None]
    if c["op"] == "queries":
        out = torch.empty((c["T"], c["H"], C + R), dtype=torch.float64, device=DEV)
        for h in range(c["H"]):
            out[:, h, :C] = s["q"][:, h, :DK].double() @ s["w"][h, :DK].double()
        out[..., C:] = _turn64(s["q"][..., DK:], s["positions"], s)
        return out
    if c["op"] == "attn":
        n, ctx, t0 = _lens(c, "n"), _lens(c, "ctx"), 0
        if sum(a * (a + b) for a, b in zip(n, ctx)) * c["H"] > 8 * 131072 * 96:
            return None
        o = torch.zeros((sum(n), c["H"], C), dtype=torch.float64, device=DEV)
        lse = torch.full((sum(n), c["H"]), -math.inf, dtype=torch.float64, device=DEV)
        for b in range(c["B"]):
            L = n[b] + ctx[b]
            kv = s["cache"][s["block_table"][b, : -(-L // c["P"])].long()].flatten(0, 1)[:L].double()
            for i in range(n[b]):
                k = kv[: ctx[b] + i + 1]
                z = s["q"][t0 + i].double() @ k.T / math.sqrt(DK + R)
                lse[t0 + i] = torch.logsumexp(z, -1)
                o[t0 + i] = torch.softmax(z, -1) @ k[:, :C]
            t0 += n[b]
        return [o, lse]
    if c["op"] == "values":
        out = torch.empty((c["T"], c["H"], DV), dtype=torch.float64, device=DEV)
        for h in range(c["H"]):
            out[:, h] = s["o"][:, h].double() @ s["w"][h, DK:].double().T
        return out
    x = s["rows"].double()
    k = torch.empty((c["T"], c["H"], DK + R), dtype=torch.float64, device=DEV)
    v = torch.empty((c["T"], c["H"], DV), dtype=torch.float64, device=DEV)
    for h in range(c["H"]):
        k[:, h, :DK], v[:, h] = x[:, :C] @ s["w"][h, :DK].double().T, x[:, :C] @ s["w"][h, DK:].double().T
        k[:, h, DK:] = x[:, C:]
    return [k, v]
