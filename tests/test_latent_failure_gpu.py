"""GPU tests of the latent-attention kernels' failure detection, made to happen without a fault: their
first-line waits on copies get a bound of zero polls, so that each gives up at once while its copy is
still in flight.  The kernels let the copies land, write NaN into the rows they were responsible for and
count the event; the next call is right again.  No test here faults, traps or hangs the GPU."""
import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda

pytestmark = pytest.mark.gpu
TIMEOUT = 4


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


def run_with_zero_limit(call, what):
    call()  # loaded and right
    kda.device_status()
    kda.set_wait_limit(0)
    try:
        out = call()
        with pytest.raises(kda.KDAError) as e:
            kda.device_status()
        assert e.value.status == TIMEOUT and what in str(e.value)
        kda.device_status()  # counted once
    finally:
        kda.set_wait_limit(None)
    return out


@pytest.mark.parametrize("H,P", [(16, 16), (64, 64), (128, 128)])
@pytest.mark.parametrize("lens", [[1], [3000], [500, 33, 70], [100] * 300])
def test_attention(lens, H, P):
    """One step, a sequence in many pieces, several units a CTA."""
    g = torch.Generator(device="cuda").manual_seed(2)
    need = [-(-n // P) for n in lens]
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = torch.arange(at, at + n)
        at += n
    cache = torch.randn((at, P, 576), generator=g, device="cuda").bfloat16()
    q = torch.randn((len(lens), H, 576), generator=g, device="cuda").bfloat16()
    table, sl = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    call = lambda: kda.attn_latent(q, cache, table, sl, return_lse=True)
    want = call()
    o, lse = run_with_zero_limit(call, "attention")
    assert torch.isnan(o).all() and torch.isnan(lse).all()
    got = call()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T,H", [(1, 2), (300, 40)])
def test_products(T, H):
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    q, o, x, w = r(T, H, 192), r(T, H, 512), r(T, 576), r(H, 256, 512)
    for call in (lambda: (kda.latent_queries(q, w)[..., :512],), lambda: (kda.latent_values(o, w),), lambda: kda.latent_expand(x, w)):
        want = call()
        bad = run_with_zero_limit(call, "latent-product")
        assert all(torch.isnan(t).all() for t in bad)
        assert all(torch.equal(a, b) for a, b in zip(call(), want))


def test_expansion_of_many_tokens():
    """Pairs of CTAs: both give up together."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((1100, 576), generator=g, device="cuda").bfloat16()
    w = torch.randn((40, 256, 512), generator=g, device="cuda").bfloat16()
    call = lambda: kda.latent_expand(x, w)
    want = call()
    bad = run_with_zero_limit(call, "latent-product")
    assert all(torch.isnan(t).all() for t in bad)
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
