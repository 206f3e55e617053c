"""GPU tests of an append's positions (kda_kv_append) where cu_seqlens leaves the rows and where places
pass 2^31: keys and queries of one token turn by the same angle."""
import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


def rows(T, H, D, seed):
    return torch.randn((T, H, D), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def turned(x, pos, f, mag):
    want = ref.rotary(ref.f64(x), pos, f.cpu(), mag)
    return want, ref.HALF_BF16 * want.abs() + ref.ROTARY_ROUNDINGS * ref.HALF_F32 * ref.rotary_size(ref.f64(x), 2 * f.numel(), mag, "half")


@pytest.mark.parametrize("Hq,T", [(4, 21), (64, 9000)])  # the second with the queries in a launch of their own
@pytest.mark.parametrize("cu", [[-5, 10 ** 6], [-(2 ** 31), 8, 2 ** 31 - 1], [-7, -3, 5, 10 ** 6]])
def test_bounds_are_clamped_for_keys_and_queries(cu, Hq, T):
    Hk, D, P = 1, 64, 16
    N, ctx = len(cu) - 1, [3, 100, 40][: len(cu) - 1]
    lo = [min(max(c, 0), T) for c in cu]
    pos = torch.cat([torch.arange(c, c + b - a) for c, a, b in zip(ctx, lo[:-1], lo[1:])])
    assert pos.numel() == T
    need = [-(-(c + b - a) // P) for c, a, b in zip(ctx, lo[:-1], lo[1:])]
    table = torch.full((N, max(need)), -1, dtype=torch.int32)
    at = 0
    for n, m in enumerate(need):
        table[n, :m] = torch.arange(at, at + m, dtype=torch.int32)
        at += m
    q, k = rows(T, Hq, D, 81), rows(T, Hk, D, 82)
    f, mag = kda.rotary_inv_freq(D)
    cache = kda.kv_cache(at, Hk, D, P)
    qr, kr = kda.kv_append(k, k, cache, table.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                           cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), inv_freq=f, magnitude=mag, q=q,
                           return_k=True)
    for got, x in ((qr, q), (kr, k)):
        ref.check("rotated", got, *turned(x, pos, f, mag))


@pytest.mark.parametrize("Hq,T", [(2, 6), (64, 9000)])
@pytest.mark.parametrize("ctx", [2 ** 31 - 1, 2 ** 31 - 4])
def test_places_that_pass_2_to_the_31(ctx, Hq, T):
    """A sequence's places behind the table are not stored, but its keys and queries are turned by their
    place all the same, which an int32 does not hold from 2^31 on."""
    Hk, D, P = 1, 64, 16
    q, k = rows(T, Hq, D, 83), rows(T, Hk, D, 84)
    f, mag = kda.rotary_inv_freq(D, base=1e6)
    cache = kda.kv_cache(1, Hk, D, P)
    qr, kr = kda.kv_append(k, k, cache, torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                           torch.tensor([ctx], dtype=torch.int32, device="cuda"),
                           cu_seqlens=torch.tensor([0, T], dtype=torch.int32, device="cuda"), inv_freq=f, magnitude=mag, q=q,
                           return_k=True)
    pos = torch.arange(ctx, ctx + T)
    for got, x in ((qr, q), (kr, k)):
        ref.check("rotated", got, *turned(x, pos, f, mag))
    assert (cache.k.view(torch.uint8) == 0).all() and (cache.k_scale == 1).all()


def test_a_long_append_captured_and_on_two_streams():
    """The form with a launch of its own for the queries, whose CTAs begin beside the last runs: replayed
    with new rows, and two at once; what follows in the stream sees both launches' results."""
    T, Hk, Hq, D, P = 3000, 2, 16, 128, 32
    f, mag = kda.rotary_inv_freq(D)
    pages = -(-T // P)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    zero, cu = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, T], dtype=torch.int32, device="cuda")
    sets = [(rows(T, Hq, D, 90 + i), rows(T, Hk, D, 95 + i)) for i in range(3)]

    def call(q, k, cache):
        before = kda.launch_count()
        qr, kr = kda.kv_append(k, k, cache, table, zero, cu_seqlens=cu, inv_freq=f, magnitude=mag, q=q, return_k=True)
        assert kda.launch_count() == before + 2
        return [qr.clone(), kr.clone(), *(t.view(torch.uint8).clone() for t in cache)]  # copies behind it in the stream

    want = [call(q, k, kda.kv_cache(pages, Hk, D, P)) for q, k in sets]
    ref.check("queries", want[0][0], *turned(sets[0][0], torch.arange(T), f, mag))
    q, k = (t.clone() for t in sets[0])
    cache = kda.kv_cache(pages, Hk, D, P)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call(q, k, cache)
    for s, w in zip(sets, want):
        q.copy_(s[0])
        k.copy_(s[1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, w))
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    caches = [kda.kv_cache(pages, Hk, D, P) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(call(*sets[i], caches[i]))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        assert all(torch.equal(a, b) for r in runs for a, b in zip(r, w))
