"""GPU tests of the decode's weights and sums over their whole range (kda_attn_decode): tokens far above
all others, whose values are zero.  Tolerances as in test_attn_decode_gpu.py: half a step of f16 of the
sum of p |v|, whatever the largest weight is."""
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


def attend(q, cache, table, lens, P, wide, **kw):
    """With the table as it is, or as wide as a server's (the cut form)."""
    if wide:
        table = torch.cat([table, torch.full((len(lens), 2048 // P), -1, dtype=torch.int32)], 1)
    o, lse = kda.attn_decode(q, cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), return_lse=True, **kw)
    torch.cuda.synchronize()
    return o, lse


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("at", [0, 37])
@pytest.mark.parametrize("nats", [6.0, 12.0, 15.0, 18.0, 22.0, 40.0])
@pytest.mark.parametrize("Hk,G,D,P", [(2, 4, 128, 16), (1, 1, 64, 64), (1, 16, 128, 32), (2, 12, 64, 16)])
def test_one_token_far_above_the_others(Hk, G, D, P, nats, at, wide):
    """A first (or a middle) token takes nearly all the weight and has a value of zero: the output is what
    the others make of it.  Every second query head sees it half as far above."""
    lens = [260, 64, 1000, 33][: 2 if at else 4]
    lens = [max(n, at + 3) for n in lens]
    table, pages = table_for(lens, P, 51)
    cache = filled_cache(pages, Hk, P, D, 51, (-4, -3))
    q = torch.full((len(lens), Hk * G, D), 1.0, device="cuda")
    q[:, 1::2] = 0.5
    # scores: D * (the channels' mean of code * scale) * D^-0.5; others' keys hardly reach one nat
    cache.k.copy_((torch.randn(cache.k.shape, generator=gen(52), device="cuda") * 8).to(torch.float8_e4m3fn))
    for n in range(len(lens)):
        page = int(table[n, at // P])
        code = nats * D ** -0.5 / cache.k_scale[page]  # one for each head
        cache.k[page, :, at % P] = code[:, None].expand(Hk, D).to(torch.float8_e4m3fn)
        cache.v[page, :, at % P] = torch.zeros((Hk, D), device="cuda").to(torch.float8_e4m3fn)
    q = q.bfloat16()
    o, lse = attend(q, cache, table, lens, P, wide, out_dtype=torch.float32)
    assert o.isfinite().all()
    verify(o, lse, q, cache, table, lens)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D,P,G", [(128, 64, 4), (64, 16, 16)])
def test_weights_of_every_size(D, P, G, wide):
    """Scores that fall by a fifth of a nat from token to token, from 100 nats down, and every value small
    where the weight is large: v grows as the weight falls, over 14 powers of two."""
    n, Hk = 500, 1
    table, pages = table_for([n], P, 53)
    cache = filled_cache(pages, Hk, P, D, 53, (-4, -3))
    cache.k.zero_()
    drop = torch.linspace(0, 1, n)
    codes = (100.0 * (1 - drop) * D ** 0.5 / 2 ** -4 / D)  # in every channel, the query being one
    for j in range(n):
        page, off = int(table[0, j // P]), j % P
        cache.k_scale[page], cache.v_scale[page] = 2.0 ** -4, 2.0 ** (4 * (j // P) * P // 128)
        cache.k[page, :, off] = codes[j].expand(Hk, D).cuda().to(torch.float8_e4m3fn)
    q = torch.full((1, Hk * G, D), 1.0, device="cuda").bfloat16() * torch.linspace(0.1, 1, Hk * G, device="cuda")[None, :, None]
    q = q.bfloat16()
    o, lse = attend(q, cache, table, [n], P, wide, out_dtype=torch.float32)
    assert o.isfinite().all()
    verify(o, lse, q, cache, table, [n])


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D,G", [(128, 4), (64, 12)])
def test_small_and_zero_values(D, G, wide):
    """Values that use little of the codes' range under a scale of one, values that are all zero, and
    both behind a token that takes the weight."""
    lens, Hk, P = [700, 700, 90], 2, 32
    table, pages = table_for(lens, P, 54)
    cache = filled_cache(pages, Hk, P, D, 54, (-4, -3))
    cache.v_scale.fill_(1.0)
    cache.v.copy_((0.02 * torch.randn(cache.v.shape, generator=gen(55), device="cuda")).to(torch.float8_e4m3fn))
    cache.v.view(torch.uint8)[table[1, : -(-lens[1] // P)].long().cuda()] = 0
    q = (3 * torch.randn((len(lens), Hk * G, D), generator=gen(56), device="cuda")).bfloat16()
    o, lse = attend(q, cache, table, lens, P, wide, out_dtype=torch.float32)
    verify(o, lse, q, cache, table, lens)
    assert (o[1] == 0).all()
    cache.v_scale[int(table[1, 3]), 1] = float("nan")  # zero codes under a scale that is no number
    o2, lse2 = attend(q, cache, table, lens, P, wide, out_dtype=torch.float32)
    assert o2[1, G:].isnan().all() and torch.equal(o2[1, :G], o[1, :G]) and torch.equal(o2[[0, 2]], o[[0, 2]])
    assert torch.equal(lse2[[0, 2]], lse[[0, 2]]) and torch.equal(lse2[1, :G], lse[1, :G])


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D,P,G", [(128, 16, 4), (64, 64, 16)])
@pytest.mark.parametrize("exp", [(-126, -110), (-120, -119), (-126, 119), (100, 119), (-75, -65)])
def test_value_scales_of_any_size(exp, D, P, G, wide):
    """Value scales from 2^-126 to 2^118, alike and mixed page by page: the weights' sum, and with it the
    log-sum-exp, does not depend on them."""
    lens, Hk = [900, 77, 1], 2
    table, pages = table_for(lens, P, 57)
    cache = filled_cache(pages, Hk, P, D, 57, (-6, -4))
    cache.v_scale.copy_(torch.exp2(torch.randint(*exp, cache.v_scale.shape, generator=gen(58), device="cuda").double()).float())
    assert (cache.v_scale > 0).all() and cache.v_scale.isfinite().all()
    q = torch.randn((len(lens), Hk * G, D), generator=gen(59), device="cuda").bfloat16()
    o, lse = attend(q, cache, table, lens, P, wide, out_dtype=torch.float32)
    assert o.isfinite().all()
    verify(o, lse, q, cache, table, lens)


@pytest.mark.parametrize("wide", [False, True])
def test_the_log_sum_of_a_head_whose_value_scale_is_no_number(wide):
    lens, Hk, G, D, P = [300, 60], 2, 4, 64, 16
    table, pages = table_for(lens, P, 60)
    cache = filled_cache(pages, Hk, P, D, 60)
    q = (2 * torch.randn((len(lens), Hk * G, D), generator=gen(61), device="cuda")).bfloat16()
    o, lse = attend(q, cache, table, lens, P, wide)
    cache.v_scale[int(table[0, 2]), 1] = float("nan")
    cache.v_scale[int(table[1, 0]), 0] = float("inf")
    o2, lse2 = attend(q, cache, table, lens, P, wide)
    assert o2[0, G:].isnan().all() and not o2[1, :G].isfinite().any()
    assert torch.equal(o2[0, :G], o[0, :G]) and torch.equal(o2[1, G:], o[1, G:])
    cache.v_scale.fill_(1.0)
    verify(attend(q, cache, table, lens, P, wide)[0], lse2, q, cache, table, lens)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hk,G,D,P", [(2, 4, 128, 16), (1, 12, 64, 64)])
@pytest.mark.parametrize("far", [12, 16, 20, 24])
def test_a_query_channel_far_above_the_others(Hk, G, D, P, far, wide):
    """One channel of each query 2^far above the others, where every key is zero: the scores are what the
    other channels make of them."""
    lens = [300, 40]
    table, pages = table_for(lens, P, 62)
    cache = filled_cache(pages, Hk, P, D, 62, (-5, -3))
    cache.k[..., 3] = torch.zeros(cache.k.shape[:3], device="cuda").to(torch.float8_e4m3fn)
    q = torch.randn((len(lens), Hk * G, D), generator=gen(63), device="cuda")
    q[..., 3] = 2.0 ** far
    q = q.bfloat16()
    o, lse = attend(q, cache, table, lens, P, wide, out_dtype=torch.float32)
    verify(o, lse, q, cache, table, lens)


@pytest.mark.parametrize("big", [2.0 ** 127, 3.3e38, 2.0 ** -120])
def test_queries_at_the_types_ends(big):
    """The largest bf16 numbers, and among the smallest normal ones."""
    lens, Hk, G, D, P = [200], 1, 4, 64, 16
    table, pages = table_for(lens, P, 64)
    cache = filled_cache(pages, Hk, P, D, 64)
    q = torch.randn((1, Hk * G, D), generator=gen(65), device="cuda").sign() * torch.rand((1, Hk * G, D), generator=gen(66), device="cuda")
    q[..., 0] = 1.0
    q = (q.double() * big).bfloat16()
    assert q.isfinite().all()
    scale = 0.1 / big if big > 1 else 2.0 ** 100
    o, lse = attend(q, cache, table, lens, P, False, out_dtype=torch.float32, scale=scale)
    verify(o, lse, q, cache, table, lens, scale)
