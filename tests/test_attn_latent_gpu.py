"""GPU tests of attention over the paged latent cache (kda_attn_latent) against 64-bit attention over the
same rows.  Tolerance per output: one rounding to the output's type; the weights' rounding to bf16 (half
a step, relative to sum p |v|); the scores' fp32 accumulation, whose error moves every weight: 576
products in 36 steps of 16, each losing at most two units of 2^-24 of the running size, below 2^-17 of
the largest sum |q||k| * scale; the products with the weights, a step for every 16 tokens that loses two
units; the sums of weights, 32 + tokens / 64 roundings; 2^-19 for references, factors and joining."""
import math

import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda
from tests import attn_reference as ref
from tests.test_kv_append_gpu import gen, table_for

pytestmark = pytest.mark.gpu
C, ROW = 512, 576


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


def cum(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def rows_of(cache, table, n, length):
    P = cache.shape[1]
    return ref.f64(cache[table[n, : -(-length // P)].long().cuda()]).flatten(0, 1)[:length]


def verify(o, lse, q, cache, table, lens, new=None, scale=None, heads=None, tokens=None):
    """tokens: which of each sequence's tokens are looked at (default all)."""
    H = q.shape[1]
    scale = 192 ** -0.5 if scale is None else scale
    hs = list(range(H)) if heads is None else heads
    t0 = 0
    for n, L in enumerate(lens):
        m = 1 if new is None else new[n]
        rows = rows_of(cache, table, n, max(L, 0))
        for i in range(m) if tokens is None else [t for t in tokens if t < m]:
            seen = L - m + i + 1
            at = t0 + i
            if seen <= 0:
                assert (o[at] == 0).all() and (lse[at] == -math.inf).all()
                continue
            k, qs = rows[:seen], ref.f64(q[at, hs])
            z = qs @ k.T * scale
            wl = torch.logsumexp(z, 1)
            p = torch.exp(z - wl[:, None])
            want, av = p @ k[:, :C], p @ k[:, :C].abs()
            size = (qs.abs() @ k.abs().T).amax(1) * abs(scale)
            moved = 2.0 ** -17 * size + 2.0 ** -19 + (32 + seen / 64) * 2.0 ** -24
            tol = (ref.HALF_BF16 + 2 * moved + (seen / 16 + 1) * 2.0 ** -23)[:, None] * av
            tol = tol + (ref.HALF_BF16 if o.dtype == torch.bfloat16 else 2.0 ** -20) * want.abs()
            ref.check(f"o[{n}, token {i}]", o[at, hs], want, tol)
            ref.check(f"lse[{n}, token {i}]", lse[at, hs], wl, moved + 2.0 ** -22 * wl.abs())
        t0 += m


def make(lens, H, P, seed, T, sharp=1.0):
    table, pages = table_for([max(x, 1) for x in lens], P, seed)
    g = gen(seed)
    cache = torch.randn((pages, P, ROW), generator=g, device="cuda").bfloat16()
    q = (sharp * torch.randn((T, H, ROW), generator=g, device="cuda")).bfloat16()
    return q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def case(lens, H, P, new=None, seed=0, out=torch.bfloat16, scale=None, sharp=1.0, **look):
    q, cache, table, sl = make(lens, H, P, seed, len(lens) if new is None else sum(new), sharp)
    cu = None if new is None else cum(new)
    o, lse = kda.attn_latent(q, cache, table.cuda(), sl, cu_seqlens=cu, return_lse=True, out_dtype=out, scale=scale)
    kda.device_status()
    verify(o, lse, q, cache, table, lens, new, scale, **look)
    return o, lse, q, cache, table, sl


@pytest.mark.parametrize("lens", [[1], [2, 0, 15], [63, 64, 65], [127, 129, 16], [1000], [0, 0, 7], [300, 1, 2049]])
@pytest.mark.parametrize("H,P", [(1, 64), (5, 16), (8, 128), (16, 32), (32, 64), (40, 16), (64, 64), (96, 128), (128, 16),
                                 (200, 64)])
def test_lengths_and_heads(lens, H, P):
    case(lens, H, P, seed=len(lens) + H)


@pytest.mark.parametrize("lens,new", [([5], [5]), ([70, 3, 200], [4, 3, 1]), ([64, 65, 1000], [2, 7, 0]), ([130, 9, 40], [1, 6, 17]),
                                      ([400], [100]), ([3, 0, 64], [5, 2, 66])])
@pytest.mark.parametrize("H,P", [(1, 64), (6, 16), (16, 32), (32, 128), (72, 64), (128, 64)])
def test_several_tokens(lens, new, H, P):
    """Drafted tokens and pieces, causal among themselves; more tokens than rows (leading ones see nothing)."""
    case(lens, H, P, new, seed=sum(lens) + H)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_long_and_ragged(out):
    """Pieces that span many sequences, and sequences that span many pieces."""
    case([20001, 5, 0, 3000, 129, 1, 0, 700] + [40] * 50, 16, 16, seed=3, out=out, heads=[0, 7, 15])


@pytest.mark.parametrize("H", [16, 128])
def test_one_long_sequence(H):
    case([30000], H, 128, seed=4, heads=[0, H // 2 + 1, H - 1])
    case([9000], H, 16, [5], seed=5, heads=[0, H - 1])


@pytest.mark.parametrize("N", [1, 130, 700])
def test_many_short_sequences(N):
    """More sequences than threads of a CTA; every CTA covers many units."""
    case([(i * 13) % 50 for i in range(N)], 4, 16, seed=N)


def test_rising_and_sharp_scores():
    """Scores of several hundred; rows that grow along the sequence, so that the reference is set anew in
    step after step; negative and tiny scales."""
    case([257], 16, 64, seed=7, sharp=30.0)
    case([257], 16, 64, seed=8, sharp=1e30, scale=1e-31)
    q, cache, table, sl = make([900], 24, 64, 9, 3)
    q = q.abs()
    P = 64
    grow = torch.linspace(0.1, 6, 960, device="cuda").view(-1, P, 1)
    cache[table[0].long().cuda()] = (cache[table[0].long().cuda()].abs().float() * grow).bfloat16()
    for scale in (None, -0.2, 1e-12):
        o, lse = kda.attn_latent(q, cache, table.cuda(), sl, cu_seqlens=cum([3]), return_lse=True, scale=scale)
        verify(o, lse, q, cache, table, [900], [3], scale)


@pytest.mark.parametrize("H", [16, 64])
def test_what_lies_behind_a_sequence_does_not_count(H):
    """NaN behind each last token, garbage in the table behind the pages in use."""
    lens = [5, 16, 33, 0, 100, 64]
    o, lse, q, cache, table, sl = case(lens, H, 16, seed=11)
    for n, m in enumerate(lens):
        for j in range(table.shape[1]):
            if j * 16 >= m:
                table[n, j] = [-7, 10 ** 6][j & 1]
            elif m % 16 and j == m // 16:
                cache[int(table[n, j]), m % 16:] = float("nan")
    o2, lse2 = kda.attn_latent(q, cache, table.cuda(), sl, return_lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("channel", [3, 300, 570])
def test_nothing_masked_enters(bad, channel):
    """A drafted token's row is not finite: tokens before it keep their values to the bit."""
    lens, new = [70, 200, 66], [4, 6, 5]
    o, lse, q, cache, table, sl = case(lens, 16, 32, new, seed=12)
    place = lens[1] - 3  # seen by the last three of the six
    cache[int(table[1, place // 32]), place % 32, channel] = bad
    o2, lse2 = kda.attn_latent(q, cache, table.cuda(), sl, cu_seqlens=cum(new), return_lse=True)
    blind = torch.ones(15, dtype=torch.bool, device="cuda")
    blind[4 + 3:4 + 6] = False
    assert torch.equal(o2[blind], o[blind]) and torch.equal(lse2[blind], lse[blind])
    if bad != bad:
        assert o2[~blind].isnan().all() and lse2[~blind].isnan().all()


def test_nan_stays_with_its_sequence_and_row():
    o, lse, q, cache, table, sl = case([40, 40], 8, 16, seed=13)
    cache[int(table[1, 1]), 3, 10] = float("nan")
    q[0, 1, 5] = float("nan")
    o2 = kda.attn_latent(q, cache, table.cuda(), sl)
    assert o2[1].isnan().all() and o2[0, 1].isnan().all()
    keep = [0, 2, 3, 4, 5, 6, 7]
    assert torch.equal(o2[0, keep], o[0, keep])


@pytest.mark.parametrize("page", [-1, 1000])
@pytest.mark.parametrize("P", [16, 128])
def test_missing_page_gives_nan(page, P):
    o, lse, q, cache, table, sl = case([300, 300, 7], 32, P, seed=14)
    table[1, 1] = page
    o2, l2 = kda.attn_latent(q, cache, table.cuda(), sl, return_lse=True)
    assert o2[1].isnan().all() and l2[1].isnan().all() and torch.equal(o2[[0, 2]], o[[0, 2]])


def test_lengths_are_clamped():
    o, lse, q, cache, table, sl = case([48, 0], 8, 16, seed=15)
    o2 = kda.attn_latent(q, cache, table.cuda(), torch.tensor([10 ** 9, -5], dtype=torch.int32, device="cuda"))
    assert torch.equal(o2, o)


def test_rows_of_no_sequence_stay():
    q, cache, table, sl = make([50, 60], 8, 16, 16, 12)
    cu = torch.tensor([2, 5, 9], dtype=torch.int32, device="cuda")
    o = torch.full((12, 8, C), 7.0, device="cuda").bfloat16()
    kda.attn_latent(q, cache, table.cuda(), sl, cu_seqlens=cu, o=o)
    assert (o[:2] == 7).all() and (o[9:] == 7).all()
    o2, lse = kda.attn_latent(q[2:9], cache, table.cuda(), sl, cu_seqlens=cu - 2, return_lse=True)
    verify(o2, lse, q[2:9], cache, table, [50, 60], [3, 4])
    wide = torch.tensor([-3, 5, 100], dtype=torch.int32, device="cuda")  # clamped to the rows
    a = kda.attn_latent(q, cache, table.cuda(), sl, cu_seqlens=wide)
    b = kda.attn_latent(q, cache, table.cuda(), sl, cu_seqlens=torch.tensor([0, 5, 12], dtype=torch.int32, device="cuda"))
    assert torch.equal(a, b)


def test_strided_queries():
    o, lse, q, cache, table, sl = case([33, 70], 8, 16, seed=17)
    fused = torch.zeros((2, 12, ROW), device="cuda").bfloat16()
    fused[:, 2:10] = q
    assert torch.equal(kda.attn_latent(fused[:, 2:10], cache, table.cuda(), sl), o)


def test_same_bits_again_and_on_another_stream():
    o, lse, q, cache, table, sl = case([5000, 3, 900], 32, 64, seed=18, heads=[0, 31])
    st = torch.cuda.Stream()
    dt = table.cuda()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        outs = [kda.attn_latent(q, cache, dt, sl) for _ in range(5)]
    st.synchronize()
    assert all(torch.equal(x, o) for x in outs)


def test_two_calls_at_once():
    a, b = case([3000, 17], 16, 64, seed=19, heads=[3]), case([900, 900, 5], 48, 16, seed=20, heads=[3])
    tables = [x[4].cuda() for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, (x, st) in enumerate(zip((a, b), streams)):
            with torch.cuda.stream(st):
                outs[i].append(kda.attn_latent(x[2], x[3], tables[i], x[5]))
    torch.cuda.synchronize()
    for x, got in zip((a, b), outs):
        assert all(torch.equal(y, x[0]) for y in got)


def test_graph_replays_with_grown_lengths():
    """A captured step replayed after the cache has grown: lengths, table and queries are read anew."""
    o, lse, q, cache, table, sl = case([700, 20], 16, 16, seed=21)
    dt, out = table.cuda(), torch.empty_like(o)
    ws = torch.empty(kda.attn_latent_workspace_size(2, 2, 16, dt.shape[1] * 16), dtype=torch.uint8, device="cuda")
    short = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    kda.attn_latent(q, cache, dt, short, o=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.attn_latent(q, cache, dt, short, o=out, workspace=ws)
    short.copy_(sl)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o)


def test_sequences_that_share_pages():
    o, lse, q, cache, table, sl = case([100, 70], 16, 16, seed=22)
    table[1, :4] = table[0, :4]
    o2, l2 = kda.attn_latent(q, cache, table.cuda(), sl, return_lse=True)
    verify(o2, l2, q, cache, table, [100, 70])


def test_no_tokens():
    q, cache, table, sl = make([5], 4, 16, 23, 1)
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert kda.attn_latent(q[:0], cache, table.cuda(), sl, cu_seqlens=cu).shape == (0, 4, C)


def test_refusals():
    cache = kda.latent_cache(4, 16)
    q = torch.zeros((2, 4, ROW), device="cuda").bfloat16()
    table = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    sl = torch.ones(2, dtype=torch.int32, device="cuda")
    bad = [(dict(q=q.float()), TypeError), (dict(q=q[:1]), ValueError), (dict(seq_lens=sl.long()), TypeError),
           (dict(seq_lens=sl.cpu()), ValueError), (dict(q=q[..., :512]), ValueError), (dict(cache=cache[:, :, :512]), ValueError),
           (dict(cache=cache.float()), TypeError), (dict(cu_seqlens=sl), ValueError), (dict(seq_lens=sl[:1]), ValueError),
           (dict(block_table=torch.zeros((2, 300), dtype=torch.int32, device="cuda"),
                 workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")), kda.KDAError),
           (dict(scale=float("nan")), kda.KDAError), (dict(scale=0.0), kda.KDAError), (dict(out_dtype=torch.float16), TypeError),
           (dict(o=torch.zeros((2, 4, ROW), device="cuda").bfloat16()), ValueError),
           (dict(cache=kda.latent_cache(4, 8)), kda.KDAError)]
    for over, err in bad:
        a = dict(q=q, cache=cache, block_table=table, seq_lens=sl)
        a.update(over)
        with pytest.raises(err):
            kda.attn_latent(a.pop("q"), a.pop("cache"), a.pop("block_table"), a.pop("seq_lens"), **a)
