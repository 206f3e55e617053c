"""GPU tests of single-token attention in the form that cuts the sequences' steps into pieces and
joins them (kda_attn_decode with a block table that holds many tokens), which needs a workspace.
Tolerances as in test_attn_decode_gpu.py."""
import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda
from tests.test_attn_decode_gpu import gen, verify
from tests.test_kv_append_gpu import filled_cache, table_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


@pytest.mark.parametrize("P", [16, 32, 128])
@pytest.mark.parametrize("D,Hk,G", [(128, 2, 4), (64, 1, 16)])
def test_each_step_takes_its_own_pages_scales(D, Hk, G, P):
    """Pages' scales are powers of two apart, so a step that read another step's scales would be off
    by far more than a rounding.  The same bits every time."""
    lens = [1000, 33, 16 * 37 + 1]
    table, pages = table_for(lens, P, 31)
    cache = filled_cache(pages, Hk, P, D, 31, (-12, -4))
    q = torch.randn((len(lens), Hk * G, D), generator=gen(32), device="cuda").bfloat16()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    dt = table.cuda()
    assert kda.attn_decode_workspace_size(len(lens), Hk * G, Hk, D, dt.shape[1] * P) > 0
    o, lse = kda.attn_decode(q, cache, dt, sl, return_lse=True)
    verify(o, lse, q, cache, table, lens)
    for _ in range(20):
        again = kda.attn_decode(q, cache, dt, sl, return_lse=True)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)


def wide_case(lens, Hk, G, D, P, seed=0, exp=(-8, -5), out=torch.bfloat16, scale=None):
    """The case with a table of just its pages and with one as wide as a server's (2048 tokens and more,
    -1 where there is no page), which is always cut; both against 64 bits."""
    table, pages = table_for([max(x, 1) for x in lens], P, seed)
    cache = filled_cache(pages, Hk, P, D, seed, exp)
    q = torch.randn((len(lens), Hk * G, D), generator=gen(seed + 1), device="cuda").bfloat16()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    wide = torch.full((len(lens), table.shape[1] + 2048 // P), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    assert kda.attn_decode_workspace_size(len(lens), Hk * G, Hk, D, wide.shape[1] * P) > 0
    for t in (table, wide):
        o, lse = kda.attn_decode(q, cache, t.cuda(), sl, return_lse=True, out_dtype=out, scale=scale)
        verify(o, lse, q, cache, t, lens, scale)
    return o, lse, q, cache, wide, sl


@pytest.mark.parametrize("Hk,G,D,P", [(2, 2, 64, 16), (1, 16, 128, 64), (4, 1, 128, 32)])
@pytest.mark.parametrize("N", [130, 300, 700])
def test_many_sequences(N, Hk, G, D, P):
    """More sequences than threads of a CTA, so that each measures several; pieces over many heads; heads
    that begin in one piece and end in the next; empty sequences in between."""
    wide_case([(i * 13) % 50 for i in range(N)], Hk, G, D, P, seed=N)


@pytest.mark.parametrize("lens", [[1], [2, 0, 15], [64, 63, 65], [300, 1, 900], [0, 0, 0], [0] * 40 + [5] + [0] * 200])
@pytest.mark.parametrize("Hk,G,D,P", [(1, 1, 128, 64), (2, 4, 64, 16), (3, 16, 128, 32), (1, 40, 64, 16)])
def test_lengths(lens, Hk, G, D, P):
    wide_case(lens, Hk, G, D, P, seed=len(lens) + G)


def test_scales_far_apart():
    wide_case([500, 77], 2, 4, 128, 16, seed=5, exp=(-40, -4), out=torch.float32)
    wide_case([500, 77], 2, 4, 128, 16, seed=6, exp=(-20, 20), out=torch.float32, scale=1e-9)


@pytest.mark.parametrize("D", [64, 128])
def test_what_lies_behind_a_sequence_does_not_count(D):
    lens, P = [5, 16, 33, 0, 100], 16
    o, lse, q, cache, table, sl = wide_case(lens, 2, 4, D, P, seed=11)
    for n, m in enumerate(lens):
        for j in range(table.shape[1]):
            if j * P >= m:
                table[n, j] = [-7, 10 ** 6][j & 1]
            elif m % P and j == m // P:
                cache.k.view(torch.uint8)[int(table[n, j]), :, m % P:] = 0x7F
                cache.v.view(torch.uint8)[int(table[n, j]), :, m % P:] = 0xFF
    o2, lse2 = kda.attn_decode(q, cache, table.cuda(), sl, return_lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("page", [-1, 10 ** 6])
@pytest.mark.parametrize("P", [16, 64])
def test_missing_page_and_nan_stay_with_their_sequence(page, P):
    lens = [70, 140] * 80
    o, lse, q, cache, table, sl = wide_case(lens, 2, 2, 128, P, seed=13)
    bad = table.clone()
    bad[101, 1] = page
    o2 = kda.attn_decode(q, cache, bad.cuda(), sl)
    rest = torch.arange(len(lens)) != 101
    assert o2[101].isnan().all() and torch.equal(o2[rest], o[rest])
    cache.v.view(torch.uint8)[int(table[100, 0]), 1, 3, 10] = 0x7F
    o3 = kda.attn_decode(q, cache, table.cuda(), sl)
    assert o3[100, 2:, 10].isnan().all() and o3.isnan().sum() == 2


def test_strided_queries_another_stream_and_negative_lengths():
    o, lse, q, cache, table, sl = wide_case([33, 70, 0] * 60, 2, 4, 128, 16, seed=16)
    fused = torch.zeros((180, 12, 128), device="cuda").bfloat16()
    fused[:, 2:10] = q
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        again = kda.attn_decode(fused[:, 2:10], cache, table.cuda(), (sl - 5 * (sl == 0)).int())
    st.synchronize()
    assert torch.equal(again, o)


@pytest.mark.parametrize("D,P,Hq,Hk", [(64, 16, 4, 2), (128, 64, 16, 1), (128, 16, 8, 8)])
@pytest.mark.parametrize("lens", [[1], [500, 0, 33, 70], [100] * 300])
def test_after_waits_that_gave_up(lens, D, P, Hq, Hk):
    """A limit of zero polls: every piece's later units are NaN too, empty sequences stay zero, and the
    next call is right."""
    o, lse, q, cache, table, sl = wide_case(lens, Hk, Hq // Hk, D, P, seed=17)
    dt = table.cuda()
    kda.device_status()
    kda.set_wait_limit(0)
    try:
        bad, bad_lse = kda.attn_decode(q, cache, dt, sl, return_lse=True)
        with pytest.raises(kda.KDAError) as e:
            kda.device_status()
        assert "attention" in str(e.value)
    finally:
        kda.set_wait_limit(None)
    some = sl > 0
    assert bad[some].isnan().all() and bad_lse[some].isnan().all()
    assert (bad[~some] == 0).all() and (bad_lse[~some] == float("-inf")).all()
    again = kda.attn_decode(q, cache, dt, sl, return_lse=True)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    kda.device_status()
