"""GPU tests of single-token attention over the paged 8-bit cache (kda_attn_decode) against 64-bit
attention over the same codes and scales.  Tolerance per output: one rounding to the output's
type; the weights' rounding to f16 (half a step, relative to sum p |v|); the scores' fp32
accumulation, whose error moves every weight: at most 2^-20 of the largest sum |q||k| * scale
(128 products, each accumulation step losing at most two units of 2^-24 of the running size)."""
import math

import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda
from tests import attn_reference as ref
from tests.test_kv_append_gpu import filled_cache, gen, table_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


def rows_of(cache, table, n, length, h):
    P = cache.k.shape[2]
    pages = table[n, : -(-length // P)].long()
    pick = lambda c, s: (ref.f64(c[pages.cuda(), h].float()) * ref.f64(s[pages.cuda(), h])[:, None, None]).flatten(0, 1)[:length]
    return pick(cache.k.float(), cache.k_scale), pick(cache.v.float(), cache.v_scale)


def verify(o, lse, q, cache, table, lens, scale=None):
    N, Hq, D = q.shape
    Hk = cache.k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    G = Hq // Hk
    for n in range(N):
        for h in range(Hk):
            hs = slice(h * G, (h + 1) * G)
            if lens[n] <= 0:
                assert (o[n, hs] == 0).all() and (lse[n, hs] == -math.inf).all()
                continue
            k, v = rows_of(cache, table, n, lens[n], h)
            want, wl, av, size = ref.attend(ref.f64(q[n, hs]), k, v, scale, [lens[n]] * G)
            moved = 2.0 ** -20 * size + 2.0 ** -20
            tol = (ref.HALF_F16 + 2 * moved)[:, None] * av + (ref.HALF_BF16 if o.dtype == torch.bfloat16 else 2.0 ** -20) * want.abs()
            ref.check(f"o[{n}, {h}]", o[n, hs], want, tol)
            ref.check(f"lse[{n}, {h}]", lse[n, hs], wl, moved + 2.0 ** -22 * wl.abs())


def case(lens, Hk, G, D, P, seed=0, exp=(-8, -5), out=torch.bfloat16, scale=None, sharp=1.0):
    table, pages = table_for([max(x, 1) for x in lens], P, seed)
    cache = filled_cache(pages, Hk, P, D, seed, exp)
    q = (sharp * torch.randn((len(lens), Hk * G, D), generator=gen(seed + 1), device="cuda")).bfloat16()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = kda.attn_decode(q, cache, table.cuda(), sl, return_lse=True, out_dtype=out, scale=scale)
    torch.cuda.synchronize()
    verify(o, lse, q, cache, table, lens, scale)
    return o, lse, q, cache, table, sl


@pytest.mark.parametrize("lens", [[1], [2, 0, 15], [16, 17, 31, 33], [64, 63, 65], [1000], [0, 0, 7], [300, 1, 4097]])
@pytest.mark.parametrize("Hk,G,D,P", [(1, 1, 128, 64), (2, 4, 64, 16), (2, 8, 128, 16), (1, 5, 64, 128),
                                      (3, 16, 128, 32), (1, 24, 128, 64), (2, 12, 64, 32), (1, 40, 64, 16)])
def test_lengths_and_groups(lens, Hk, G, D, P):
    case(lens, Hk, G, D, P, seed=len(lens) + G)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_long_and_ragged(out):
    """Pieces that span many sequences, and sequences that span many pieces."""
    case([20001, 5, 0, 3000, 129, 1, 0, 700] + [40] * 50, 2, 4, 128, 16, seed=3, out=out)


@pytest.mark.parametrize("N", [1, 130, 700])
def test_many_short_sequences(N):
    """More sequences than threads of a CTA; every CTA covers many heads."""
    case([(i * 13) % 50 for i in range(N)], 2, 2, 64, 16, seed=N)


def test_scales_far_apart():
    """Page scales from 2^-40 to 2^20, for keys with a small softmax scale: one accumulator holds
    values of very different pages."""
    case([500, 77], 2, 4, 128, 16, seed=5, exp=(-40, -4), out=torch.float32)
    case([500, 77], 2, 4, 128, 16, seed=6, exp=(-20, 20), out=torch.float32, scale=1e-9)


def test_sharp_and_large_scores():
    """Scores of several hundred, one token taking all the weight, and queries near bf16's extremes."""
    case([257], 1, 8, 128, 64, seed=7, sharp=30.0)
    case([257], 1, 8, 128, 64, seed=8, sharp=1e30, scale=1e-31)
    case([257], 1, 8, 64, 64, seed=9, sharp=1e-30, scale=1e29)


@pytest.mark.parametrize("D", [64, 128])
def test_what_lies_behind_a_sequence_does_not_count(D):
    """NaN codes behind each last token, NaN scales of pages nobody uses, garbage in the table."""
    lens = [5, 16, 33, 0, 100]
    o, lse, q, cache, table, sl = case(lens, 2, 4, D, 16, seed=11)
    P = 16
    for n, m in enumerate(lens):
        for j in range(table.shape[1]):
            if j * P >= m:
                table[n, j] = [-7, 10 ** 6][j & 1]
            elif m % P and j == m // P:
                cache.k.view(torch.uint8)[int(table[n, j]), :, m % P:] = 0x7F
                cache.v.view(torch.uint8)[int(table[n, j]), :, m % P:] = 0xFF
    o2, lse2 = kda.attn_decode(q, cache, table.cuda(), sl, return_lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_nan_stays_with_its_sequence_and_head():
    lens = [40, 40]
    o, lse, q, cache, table, sl = case(lens, 2, 2, 64, 16, seed=12)
    cache.v.view(torch.uint8)[int(table[1, 1]), 1, 3, 10] = 0x7F  # token 19 of sequence 1, head 1, channel 10
    o2 = kda.attn_decode(q, cache, table.cuda(), sl)
    bad = o2.isnan()
    assert bad[1, 2:, 10].all() and bad.sum() == 2
    q[0, 1, 5] = float("nan")
    o3 = kda.attn_decode(q, cache, table.cuda(), sl)
    assert o3[0, 1].isnan().all() and not o3[0, [0, 2, 3]].isnan().any()


@pytest.mark.parametrize("page", [-1, 1000])
def test_missing_page_gives_nan(page):
    """A page number out of range among a sequence's own pages: its rows are NaN, the others stand."""
    o, lse, q, cache, table, sl = case([40, 40, 7], 2, 2, 128, 16, seed=13)
    table[1, 2] = page
    o2 = kda.attn_decode(q, cache, table.cuda(), sl)
    assert o2[1].isnan().all() and torch.equal(o2[[0, 2]], o[[0, 2]])


def test_lengths_are_clamped():
    o, lse, q, cache, table, sl = case([48, 0], 1, 2, 64, 16, seed=14)
    sl2 = torch.tensor([10 ** 9, -5], dtype=torch.int32, device="cuda")
    o2 = kda.attn_decode(q, cache, table.cuda(), sl2)
    assert torch.equal(o2, o)


def test_same_bits_again_and_on_another_stream():
    args = case([5000, 3, 900], 2, 4, 128, 64, seed=15)
    o, lse, q, cache, table, sl = args
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        outs = [kda.attn_decode(q, cache, table.cuda(), sl) for _ in range(5)]
    st.synchronize()
    assert all(torch.equal(x, o) for x in outs)


def test_strided_queries():
    o, lse, q, cache, table, sl = case([33, 70], 2, 4, 128, 16, seed=16)
    fused = torch.zeros((2, 12, 128), device="cuda").bfloat16()
    fused[:, 2:10] = q
    assert torch.equal(kda.attn_decode(fused[:, 2:10], cache, table.cuda(), sl), o)


def test_graph_replays_with_grown_lengths():
    """A captured step replayed after the cache has grown: lengths, table and queries are read anew."""
    o, lse, q, cache, table, sl = case([700, 20], 2, 4, 64, 16, seed=17)
    dt = table.cuda()
    out = torch.empty_like(o)
    ws = torch.empty(kda.attn_decode_workspace_size(2, 8, 2, 64, dt.shape[1] * 16), dtype=torch.uint8, device="cuda")
    short = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    kda.attn_decode(q, cache, dt, short, o=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.attn_decode(q, cache, dt, short, o=out, workspace=ws)
    short.copy_(sl)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o)


def test_append_then_attend():
    """A decode run as it is used: prompt appended, then steps of append and attention, against exact
    attention over the rotated rows; what remains is the codes' rounding (half an e4m3 step of
    every key and value)."""
    N, Hk, G, D, P = 3, 2, 4, 128, 16
    Hq = Hk * G
    lens = [37, 1, 64]
    steps = 20
    table, pages = table_for([m + steps for m in lens], P, 21)
    table = table.cuda()
    cache = kda.kv_cache(pages, Hk, D, P)
    f, mag = kda.rotary_inv_freq(D, scaling="yarn", factor=4.0)
    g = gen(22)
    new = lambda t, h: torch.randn((t, h, D), generator=g, device="cuda").bfloat16()
    k0, v0 = new(sum(lens), Hk), new(sum(lens), Hk)
    cu = torch.tensor([0, 37, 38, 102], dtype=torch.int32, device="cuda")
    ctx = torch.zeros(N, dtype=torch.int32, device="cuda")
    kda.kv_append(k0, v0, cache, table, ctx, cu_seqlens=cu, inv_freq=f, magnitude=mag)
    ks = [list(x) for x in k0.split(lens)]
    vs = [list(x) for x in v0.split(lens)]
    ctx += torch.tensor(lens, dtype=torch.int32, device="cuda")
    for _ in range(steps):
        q, k, v = new(N, Hq), new(N, Hk), new(N, Hk)
        qr, _ = kda.kv_append(k, v, cache, table, ctx, inv_freq=f, magnitude=mag, q=q)
        ctx += 1
        o = kda.attn_decode(qr, cache, table, ctx)
        for n in range(N):
            ks[n].append(k[n])
            vs[n].append(v[n])
    for n in range(N):
        m = len(ks[n])
        kk = ref.rotary(ref.f64(torch.stack(ks[n])), torch.arange(m), f.cpu(), mag)
        vv = ref.f64(torch.stack(vs[n]))
        qq = ref.rotary(ref.f64(q[n][None]), torch.tensor([m - 1]), f.cpu(), mag)[0]
        for h in range(Hk):
            hs = slice(h * G, (h + 1) * G)
            want, _, av, size = ref.attend(qq[hs], kk[:, h], vv[:, h], D ** -0.5, [m] * G)
            # a key's code is off by half a step of each channel, so a score by at most that share of
            # sum |q||k| (and a bf16 rounding of q); a weight by e^(2 of that) - 1; a value by half a step
            off = (ref.HALF_E4M3 + ref.HALF_BF16) * size
            tol = ((torch.exp(2 * off) - 1)[:, None] + ref.HALF_E4M3 + 2.0 ** -8) * av + ref.HALF_BF16 * want.abs()
            ref.check(f"o[{n}, {h}]", o[n, hs], want, tol)


@pytest.mark.parametrize("D,P,Hq,Hk", [(64, 16, 2, 1), (128, 64, 24, 2), (128, 128, 3, 3)])
def test_short_tables_need_no_workspace(D, P, Hq, Hk):
    """A table that holds few tokens: a CTA for each head, nothing to join; empty sequences among them."""
    lens = [0, 1, 31, 33, 256, 0, 200]
    o, lse, q, cache, table, sl = case(lens, Hk, Hq // Hk, D, P, seed=23)
    assert kda.attn_decode_workspace_size(len(lens), Hq, Hk, D, table.shape[1] * P) == 0
    wide = torch.full((len(lens), 40 * 128 // P), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    assert kda.attn_decode_workspace_size(len(lens), Hq, Hk, D, wide.shape[1] * P) > 0
    o2, l2 = kda.attn_decode(q, cache, wide.cuda(), sl, return_lse=True)
    verify(o2, l2, q, cache, wide, lens)
    assert (o[0] == 0).all() and (lse[5] == float("-inf")).all()


def test_many_short_tables():
    """More heads than the GPU holds CTAs, whole; the lengths clamped to a table of 1024 tokens."""
    lens = [(37 * n) % 300 for n in range(130)] + [1000]
    o, lse, q, cache, table, sl = case(lens, 8, 1, 64, 64, seed=24)
    assert kda.attn_decode_workspace_size(len(lens), 8, 8, 64, table.shape[1] * 64) == 0
    o2 = kda.attn_decode(q, cache, table.cuda(), (sl + 100000) * (sl > 900) + sl * (sl <= 900))
    assert torch.equal(o2[:-1], o[:-1])  # the last one attends to the whole table now


def test_sequences_that_share_pages():
    """Two sequences with the same beginning: the pages stand in both rows of the table."""
    o, lse, q, cache, table, sl = case([100, 70], 2, 4, 64, 16, seed=18)
    table[1, :4] = table[0, :4]
    o2, l2 = kda.attn_decode(q, cache, table.cuda(), sl, return_lse=True)
    verify(o2, l2, q, cache, table, [100, 70])


def test_two_calls_at_once():
    """Two streams at the same time, each with a workspace from torch's allocator."""
    a, b = case([3000, 17], 2, 4, 128, 16, seed=19), case([900, 900, 5], 2, 4, 128, 16, seed=20)
    tables = [x[4].cuda() for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, (x, st) in enumerate(zip((a, b), streams)):
            with torch.cuda.stream(st):
                outs[i].append(kda.attn_decode(x[2], x[3], tables[i], x[5]))
    torch.cuda.synchronize()
    for x, got in zip((a, b), outs):
        assert all(torch.equal(y, x[0]) for y in got)


@pytest.mark.parametrize("Hk,G", [(1, 1), (1, 12), (4, 4)])
def test_one_long_sequence(Hk, G):
    """One sequence cut into as many pieces as the GPU takes; sampled against 64 bits."""
    case([30000], Hk, G, 128, 128, seed=21)
    case([30000], Hk, G, 64, 16, seed=22)


def test_refusals():
    cache = kda.kv_cache(4, 2, 64, 16)
    q = torch.zeros((2, 4, 64), device="cuda").bfloat16()
    table = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    sl = torch.ones(2, dtype=torch.int32, device="cuda")
    bad = [(dict(q=q.float()), TypeError), (dict(q=q[:1]), ValueError), (dict(seq_lens=sl.long()), TypeError),
           (dict(seq_lens=sl.cpu()), ValueError), (dict(q=torch.zeros((2, 4, 128), device="cuda").bfloat16()), ValueError),
           (dict(q=torch.zeros((2, 3, 64), device="cuda").bfloat16()), kda.KDAError),
           (dict(block_table=torch.zeros((2, 300), dtype=torch.int32, device="cuda"),
                 workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")), kda.KDAError),
           (dict(scale=float("nan")), kda.KDAError), (dict(out_dtype=torch.float16), TypeError)]
    for over, err in bad:
        a = dict(q=q, cache=cache, block_table=table, seq_lens=sl)
        a.update(over)
        with pytest.raises(err):
            kda.attn_decode(a.pop("q"), a.pop("cache"), a.pop("block_table"), a.pop("seq_lens"), **a)
