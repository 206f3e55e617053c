"""GPU tests of the paged cache's append (kda_kv_append).  New codes are held to half an e4m3 step
of the 64-bit rotated value (plus the rotation's fp32 roundings), scales to the smallest power of
two that fits, earlier codes of a page to their exact shift, everything else to its old bits."""
import math

import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def filled_cache(pages, Hk, P, D, seed, exp=(-8, -3)):
    g = gen(seed)
    codes = lambda: (torch.randn((pages, Hk, P, D), generator=g, device="cuda") * 60).clamp(-448, 448).to(
        torch.float8_e4m3fn)
    scale = lambda: torch.exp2(torch.randint(*exp, (pages, Hk), generator=g, device="cuda").float())
    return kda.KVCache(codes(), codes(), scale(), scale())


def table_for(slots, P, seed, spare=2):
    need = [-(-s // P) for s in slots]
    order = torch.randperm(sum(need) + spare, generator=torch.Generator().manual_seed(seed)).int()
    t = torch.full((len(slots), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = order[at:at + n]
        at += n
    return t, sum(need) + spare


def bits(t):
    return t.view(torch.uint8).cpu()


def copy_of(cache):
    return kda.KVCache(*(t.view(torch.uint8).clone().view(t.dtype) if t.dtype == torch.float8_e4m3fn else t.clone()
                         for t in cache))


def verify_cache(old, new, table, ctx, lens, k64, v64, R, mag, layout):
    """Every page and head of `new` against `old` and the new tokens' 64-bit rows."""
    P, D = old.k.shape[2], old.k.shape[3]
    for which, rows in (("k", k64), ("v", v64)):
        oc, nc = bits(getattr(old, which)), bits(getattr(new, which))
        ov, nv = ref.f64(getattr(old, which)), ref.f64(getattr(new, which))
        os_, ns = ref.f64(getattr(old, which + "_scale")), ref.f64(getattr(new, which + "_scale"))
        slack = ref.ROTARY_ROUNDINGS * ref.HALF_F32 * ref.rotary_size(rows, R, mag, layout) if which == "k" and R else 0 * rows
        seen = torch.zeros(oc.shape[0], dtype=torch.bool)
        t0 = 0
        for n, (c, m) in enumerate(zip(ctx, lens)):
            for j in range(c // P, (c + m - 1) // P + 1) if m else ():
                lo, hi = max(c, j * P), min(c + m, (j + 1) * P)
                page = int(table[n, j]) if j < table.shape[1] else -1
                if page < 0 or page >= oc.shape[0]:
                    continue
                seen[page] = True
                x, sl = rows[t0 + lo - c:t0 + hi - c], slack[t0 + lo - c:t0 + hi - c]
                off, end = lo - j * P, hi - j * P
                for h in range(oc.shape[1]):
                    s = ns[page, h].item()
                    assert math.frexp(s)[0] == 0.5, "scales are powers of two"
                    amax = x[:, h].abs().max().item()
                    assert amax <= 448 * s * (1 + 1e-6)
                    tight = amax > 224 * s * (1 - 1e-6) or s == 2.0 ** -100
                    assert tight or (off > 0 and s == os_[page, h]), (which, page, h)
                    if off > 0:
                        assert s >= os_[page, h]
                        moved = torch.from_numpy(ref.to_e4m3(ov[page, h, :off] * (os_[page, h] / s)))
                        assert torch.equal(nv[page, h, :off], moved), "earlier codes move exactly"
                    ref.check(f"{which} codes", nv[page, h, off:end] * s, x[:, h],
                              (x[:, h].abs() * ref.HALF_E4M3).clamp(min=s * 2.0 ** -10) + 2 * sl[:, h])
                    assert torch.equal(nc[page, h, end:], oc[page, h, end:]), "places behind the last token stay"
            t0 += m
        assert torch.equal(nc[~seen], oc[~seen]) and torch.equal(ns[~seen], os_[~seen]), "other pages stay"


def run_case(ctx, lens, Hk, Hq, D, P, R, layout="half", seed=0, step=False, spread=0.0, return_k=True, mag=1.0):
    table, pages = table_for([c + m for c, m in zip(ctx, lens)], P, seed)
    T = sum(lens)
    g = gen(seed + 1)
    grow = torch.exp2(spread * torch.randn((T, Hk, 1), generator=g, device="cuda"))
    k = (torch.randn((T, Hk, D), generator=g, device="cuda") * grow).bfloat16()
    v = (torch.randn((T, Hk, D), generator=g, device="cuda") * grow).bfloat16()
    q = torch.randn((T, Hq, D), generator=g, device="cuda").bfloat16() if Hq else None
    cache = filled_cache(pages, Hk, P, D, seed + 2)
    old = copy_of(cache)
    f = kda.rotary_inv_freq(R)[0] if R else None
    cu = None if step else torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")
    qr, kr = kda.kv_append(k, v, cache, table.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"), cu_seqlens=cu,
                           inv_freq=f, magnitude=mag, layout=layout, q=q, return_k=return_k)
    torch.cuda.synchronize()
    pos = torch.cat([torch.arange(c, c + m) for c, m in zip(ctx, lens)])
    turn = lambda t: ref.rotary(ref.f64(t), pos, f.cpu(), mag, layout) if R else ref.f64(t)
    for got, x in ((qr, q), (kr, k)):
        if got is None:
            continue
        want = turn(x)
        tol = ref.HALF_BF16 * want.abs()
        if R:
            tol = tol + ref.ROTARY_ROUNDINGS * ref.HALF_F32 * ref.rotary_size(ref.f64(x), R, mag, layout)
        ref.check("rotated", got, want, tol)
    verify_cache(old, cache, table, ctx, lens, turn(k), ref.f64(v), R, mag, layout)
    return cache


@pytest.mark.parametrize("ctx,lens", [
    ([0], [1]), ([0], [64]), ([0], [129]), ([5], [1]), ([63], [2]), ([64], [64]), ([100, 0, 17], [30, 0, 1]),
    ([0, 0, 0], [0, 0, 3]), ([15, 16, 31, 1000], [1, 17, 33, 200]), ([3], [300])])
@pytest.mark.parametrize("P,D,layout", [(16, 64, "interleaved"), (64, 128, "half"), (128, 128, "interleaved"),
                                        (32, 64, "half")])
def test_runs(ctx, lens, P, D, layout):
    run_case(ctx, lens, Hk=2, Hq=6, D=D, P=P, R=D, layout=layout, seed=len(lens) + P)


@pytest.mark.parametrize("N,Hk,Hq", [(1, 1, 0), (1, 8, 64), (5, 3, 3), (37, 2, 10), (300, 1, 4)])
@pytest.mark.parametrize("P,D,R,layout", [(64, 128, 128, "half"), (16, 64, 32, "interleaved"), (128, 128, 64, "half"),
                                          (32, 64, 0, "half"), (16, 128, 16, "interleaved")])
def test_single_tokens(N, Hk, Hq, P, D, R, layout):
    ctx = [(i * 97) % 400 for i in range(N)]
    run_case(ctx, [1] * N, Hk, Hq, D, P, R, layout, seed=N, step=True, spread=3.0)


@pytest.mark.parametrize("R", [0, 32, 64])
def test_many_sequences_partial_rotation(R):
    """More sequences than threads of a CTA, so that the search for a run takes several passes."""
    lens = [(i * 7) % 5 for i in range(600)]
    ctx = [(i * 31) % 90 for i in range(600)]
    run_case(ctx, lens, Hk=1, Hq=2, D=64, P=16, R=R, seed=9, spread=2.0)


def test_growing_page_equals_its_steps():
    """A page filled token by token, each larger than the last: the codes of every step are the exact
    shift of the step before, and a later whole-page write takes a fresh scale."""
    P, D, Hk = 16, 64, 2
    cache = kda.kv_cache(3, Hk, D, P)
    table = torch.tensor([[2]], dtype=torch.int32, device="cuda")
    for i in range(P):
        x = (torch.randn((1, Hk, D), generator=gen(i), device="cuda") * 2.0 ** (i - 8)).bfloat16()
        old = copy_of(cache)
        kda.kv_append(x, x, cache, table, torch.tensor([i], dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        verify_cache(old, cache, table.cpu(), [i], [1], ref.f64(x), ref.f64(x), 0, 1.0, "half")
    small = torch.full((1, Hk, D), 2.0 ** -20, device="cuda").bfloat16()
    kda.kv_append(small, small, cache, table, torch.tensor([0], dtype=torch.int32, device="cuda"))
    assert (cache.k_scale[2] < 2.0 ** -27).all(), "place 0 opens the page anew"


def test_zero_infinite_and_nan_values():
    """A block of zeros takes the smallest scale; infinities and NaN are stored as NaN and leave the
    scale to the finite values."""
    P, D = 16, 64
    cache = kda.kv_cache(1, 1, D, P)
    k = torch.zeros((4, 1, D), device="cuda").bfloat16()
    v = torch.ones((4, 1, D), device="cuda").bfloat16()
    v[1, 0, 5], v[2, 0, 6], v[3, 0, 7] = float("inf"), float("-inf"), float("nan")
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda.kv_append(k, v, cache, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), zero, cu_seqlens=cu)
    assert cache.k_scale.item() == 2.0 ** -100 and (bits(cache.k)[0, 0, :4] == 0).all()
    assert cache.v_scale.item() == 2.0 ** -8
    got = cache.v.float()[0, 0, :4].cpu() * cache.v_scale.item()
    nan = got.isnan()
    assert nan[1, 5] and nan[2, 6] and nan[3, 7] and nan.sum() == 3 and (got[~nan] == 1.0).all()


@pytest.mark.parametrize("amax", [448.0, 450.0, 1.75, 1.7578125, 224.0])
def test_scale_at_its_border(amax):
    """448 * 2^e itself fits 2^e; the next bf16 value above takes 2^(e + 1)."""
    x = torch.zeros((1, 1, 64), device="cuda").bfloat16()
    x[0, 0, 9] = -amax
    cache = kda.kv_cache(1, 1, 64, 16)
    z = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    kda.kv_append(x, x, cache, z, z[0])
    assert cache.k_scale.item() == 2.0 ** math.ceil(math.log2(amax / 448))


@pytest.mark.parametrize("step", [False, True])
def test_padding_is_dropped(step):
    """Negative pages, pages out of range and tokens behind the block table store nothing; their
    rotated copies are still returned."""
    P, D, Hk = 16, 64, 2
    cache = filled_cache(4, Hk, P, D, 3)
    old = copy_of(cache)
    ctx = [0, 5, 16, 40]
    lens = [1] * 4 if step else [3, 2, 20, 1]
    table = torch.tensor([[-1], [7], [1], [2]], dtype=torch.int32)  # 16 and 40 lie behind a table of one page
    x = torch.randn((sum(lens), Hk, D), generator=gen(4), device="cuda").bfloat16()
    cu = None if step else torch.tensor([0, 3, 5, 25, 26], dtype=torch.int32, device="cuda")
    f, _ = kda.rotary_inv_freq(D)
    q, k = kda.kv_append(x, x, cache, table.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"), cu_seqlens=cu,
                         inv_freq=f, q=x, return_k=True)
    torch.cuda.synchronize()
    for a, b in zip(cache, old):
        assert torch.equal(bits(a), bits(b))
    assert torch.equal(q, k) and q.isfinite().all()


def test_strided_rows_and_bad_bounds():
    """k, v and q as slices of one projection; cu_seqlens that leaves the tensors is clamped."""
    T, Hk, Hq, D, P = 21, 2, 4, 64, 16
    fused = torch.randn((T, (Hq + 2 * Hk) * D), generator=gen(5), device="cuda").bfloat16()
    q, k, v = (t.unflatten(1, (-1, D)) for t in fused.split([Hq * D, Hk * D, Hk * D], 1))
    f, _ = kda.rotary_inv_freq(D)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = []
    for a, b, c, cu in ((q, k, v, [0, T]), (q.contiguous(), k.contiguous(), v.contiguous(), [-5, T + 100])):
        cache = kda.kv_cache(2, Hk, D, P)
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        r = kda.kv_append(b, c, cache, table, zero, cu_seqlens=cu, inv_freq=f, q=a, return_k=True)
        outs.append((*r, *cache))
    for i, (a, b) in enumerate(zip(*outs)):
        if i:  # a negative cu_seqlens[0] shifts the queries' positions, nothing else
            assert torch.equal(bits(a), bits(b)), i


@pytest.mark.parametrize("T", [40, 9000])
def test_rows_of_no_sequence_are_left_alone(T):
    """cu_seqlens that begins behind row 0 and ends before the last row; 9000 rows of 64 heads take the
    form with a launch of its own for the queries."""
    Hk, Hq, D, P = 1, 64, 64, 16
    g = gen(6)
    k = torch.randn((T, Hk, D), generator=g, device="cuda").bfloat16()
    q = torch.randn((T, Hq, D), generator=g, device="cuda").bfloat16()
    lo, hi = 5, T - 7
    pages = -(-(hi - lo) // P)
    cache = kda.kv_cache(pages, Hk, D, P)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    f, _ = kda.rotary_inv_freq(D)
    qo, ko = torch.full_like(q, 9.0), torch.full_like(k, 9.0)
    kda.kv_append(k, k, cache, table, zero, cu_seqlens=torch.tensor([lo, hi], dtype=torch.int32, device="cuda"),
                  inv_freq=f, q=q, q_out=qo, k_out=ko)
    for out, x in ((qo, q), (ko, k)):
        assert (out[:lo] == 9).all() and (out[hi:] == 9).all()
        want = kda.rotary(x[lo:hi], torch.arange(hi - lo, dtype=torch.int32, device="cuda"), f)
        assert torch.equal(out[lo:hi], want)


def test_graph_replays_append_where_the_lengths_say():
    """A captured step: each replay appends one token further on, as the lengths are counted up."""
    N, Hk, D, P = 3, 2, 64, 16
    table, pages = table_for([40] * N, P, 7)
    f, _ = kda.rotary_inv_freq(D)
    caches = [kda.kv_cache(pages, Hk, D, P) for _ in range(2)]
    ctx = torch.tensor([0, 15, 20], dtype=torch.int32, device="cuda")
    x = torch.randn((N, Hk, D), generator=gen(8), device="cuda").bfloat16()
    dt = table.cuda()
    kda.kv_append(x, x, kda.kv_cache(pages, Hk, D, P), dt, ctx, inv_freq=f)  # loaded before the capture
    torch.cuda.synchronize()
    graph, c = torch.cuda.CUDAGraph(), ctx.clone()
    with torch.cuda.graph(graph):
        kda.kv_append(x, x, caches[0], dt, c, inv_freq=f)
    for _ in range(5):
        graph.replay()
        kda.kv_append(x, x, caches[1], dt, ctx, inv_freq=f)
        c += 1
        ctx += 1
    torch.cuda.synchronize()
    for a, b in zip(*caches):
        assert torch.equal(bits(a), bits(b))


def test_refusals():
    cache = kda.kv_cache(2, 2, 64, 16)
    x = torch.zeros((3, 2, 64), device="cuda").bfloat16()
    table = torch.zeros((3, 1), dtype=torch.int32, device="cuda")
    ctx = torch.zeros(3, dtype=torch.int32, device="cuda")
    bad = [(dict(k=x[:, :1]), ValueError), (dict(k=x.float()), TypeError), (dict(context_lens=ctx[:2]), ValueError),
           (dict(block_table=table.long()), TypeError), (dict(context_lens=ctx.cpu()), ValueError),
           (dict(cu_seqlens=ctx), ValueError), (dict(q_out=x), ValueError), (dict(layout="x"), ValueError)]
    for over, err in bad:
        a = dict(k=x, v=x, cache=cache, block_table=table, context_lens=ctx)
        a.update(over)
        with pytest.raises(err):
            kda.kv_append(a.pop("k"), a.pop("v"), a.pop("cache"), a.pop("block_table"), a.pop("context_lens"), **a)
    with pytest.raises(kda.KDAError):  # one token per sequence without cu_seqlens
        kda.kv_append(x[:2], x[:2], cache, table, ctx)
    odd = kda.kv_cache(2, 2, 64, 24)
    with pytest.raises(kda.KDAError):
        kda.kv_append(x, x, odd, table, ctx)
