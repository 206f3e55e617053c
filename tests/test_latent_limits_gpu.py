"""GPU tests of the latent-attention kernels under small limits of their first-line waits: some copies
arrive in time and some do not, so that a kernel gives up in the middle of its work, a part of its warps behind
products that still come through.  Every call ends, what is not NaN is what the call without a limit gives, and NaN
and the status come together.  Which copies are late depends on the memory's load (a copy of 1 GB runs beside the
calls), so either outcome is taken.  No test here faults, traps or hangs the GPU."""
import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda
from tests.test_kv_append_gpu import gen, table_for

pytestmark = pytest.mark.gpu
TIMEOUT = 4
LIMITS = [1, 2, 4, 8, 12, 16, 16, 20, 24, 28, 32, 48]


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


def under_limits(call):
    """Pairs of (results, whether a wait gave up) for each limit."""
    a = torch.zeros(1 << 29, dtype=torch.uint8, device="cuda")
    b, beside = torch.empty_like(a), torch.cuda.Stream()
    kda.device_status()
    for limit in LIMITS:
        torch.cuda.synchronize()
        with torch.cuda.stream(beside):
            b.copy_(a)
        kda.set_wait_limit(limit)
        try:
            out, late = call(), False
            try:
                kda.device_status()
            except kda.KDAError as e:
                assert e.status == TIMEOUT
                late = True
        finally:
            kda.set_wait_limit(None)
        yield out, late


@pytest.mark.parametrize("lens,new", [([100] * 300, None), ([4000, 33, 70] * 20, None), ([200] * 100, [5] * 100), ([60000], None)])
@pytest.mark.parametrize("H,P", [(16, 16), (96, 128)])
def test_attention(lens, new, H, P):
    g = gen(sum(lens))
    table, pages = table_for(lens, P, 1)
    T = len(lens) if new is None else sum(new)
    cache = torch.randn((pages, P, 576), generator=g, device="cuda").bfloat16()
    q = torch.randn((T, H, 576), generator=g, device="cuda").bfloat16()
    table, sl = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = None if new is None else torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    call = lambda: kda.attn_latent(q, cache, table, sl, cu_seqlens=cu, return_lse=True)
    want, want_lse = call()
    assert want.isfinite().all()
    for (o, lse), late in under_limits(call):
        lost = lse.isnan()
        assert torch.equal(o.isnan(), lost[..., None].expand_as(o)) and bool(lost.any()) == late
        assert torch.equal(o[~lost], want[~lost]) and torch.equal(lse[~lost], want_lse[~lost])
    o, lse = call()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("T,H", [(3, 4), (700, 32), (1500, 48)])
def test_products(T, H):
    g = gen(T)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    q, o, x, w = r(T, H, 192), r(T, H, 512), r(T, 576), r(H, 256, 512)
    for call in (lambda: (kda.latent_queries(q, w),), lambda: (kda.latent_values(o, w),), lambda: kda.latent_expand(x, w)):
        want = call()
        for out, late in under_limits(call):
            lost = [t.isnan() for t in out]
            assert any(bool(n.any()) for n in lost) == late
            assert all(torch.equal(a[~n], b[~n]) for a, b, n in zip(out, want, lost))
        assert all(torch.equal(a, b) for a, b in zip(call(), want))
