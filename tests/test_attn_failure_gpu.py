"""GPU tests of the attention kernels' failure detection, made to happen without a fault: their
first-line waits on copies get a bound of zero polls, so that each gives up at once while its
copy is still in flight.  The kernel lets the copies land, writes NaN into the rows it was
responsible for and counts the event; the next call is right again.  No test here faults,
traps or hangs the GPU."""
import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda

pytestmark = pytest.mark.gpu
TIMEOUT = 4


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


def run_with_zero_limit(call):
    call()  # loaded and right
    kda.device_status()
    kda.set_wait_limit(0)
    try:
        out = call()
        with pytest.raises(kda.KDAError) as e:
            kda.device_status()
        assert e.value.status == TIMEOUT and "attention" in str(e.value)
        kda.device_status()  # counted once
    finally:
        kda.set_wait_limit(None)
    return out


@pytest.mark.parametrize("D,DV,Hq,Hk", [(64, 64, 4, 2), (128, 128, 3, 3), (192, 128, 8, 1)])
@pytest.mark.parametrize("lens", [[1], [700], [130, 0, 1000, 5], [40] * 200])
def test_prompt(lens, D, DV, Hq, Hk):
    """One tile, several items a CTA, an idle second tile, a row block that ends early."""
    g = torch.Generator(device="cuda").manual_seed(1)
    T = sum(lens)
    q, k, v = (torch.randn((T, h, d), generator=g, device="cuda").bfloat16() for h, d in ((Hq, D), (Hk, D), (Hk, DV)))
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    call = lambda: kda.attn_prompt(q, k, v, cu_seqlens=cu, return_lse=True)
    want = call()
    o, lse = run_with_zero_limit(call)
    assert torch.isnan(o).all() and torch.isnan(lse).all()
    got = call()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("D,P,Hq,Hk", [(64, 16, 4, 2), (128, 64, 16, 1), (128, 16, 8, 8)])
@pytest.mark.parametrize("lens", [[1], [3000], [500, 0, 33, 70], [100] * 300])
def test_decode(lens, D, P, Hq, Hk):
    """One step, a sequence in many pieces, several units a CTA; an empty sequence stays zero."""
    g = torch.Generator(device="cuda").manual_seed(2)
    need = [-(-n // P) for n in lens]
    pages = max(1, sum(need))
    cache = kda.kv_cache(pages, Hk, D, P)
    for codes in (cache.k, cache.v):
        codes.copy_(torch.randn(codes.shape, generator=g, device="cuda").to(torch.float8_e4m3fn))
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    table, at = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32), 0
    for n, w in enumerate(need):
        table[n, :w] = torch.arange(at, at + w, dtype=torch.int32)
        at += w
    table = table.cuda()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn((len(lens), Hq, D), generator=g, device="cuda").bfloat16()
    call = lambda: kda.attn_decode(q, cache, table, sl, return_lse=True)
    want = call()
    o, lse = run_with_zero_limit(call)
    some = sl > 0
    assert torch.isnan(o[some]).all() and torch.isnan(lse[some]).all()
    assert (o[~some] == 0).all() and (lse[~some] == float("-inf")).all()
    got = call()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
