"""GPU tests of rotary positions where numbers are not finite, angles small or positions large
(kda_rotary, kda_kv_append), against the 64-bit formula.  Tolerances as in test_rotary_gpu.py."""
import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


def make(T, H, D, dtype, seed):
    return torch.randn((T, H, D), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def same_kind(got, want):
    """Infinities of the same sign, NaN and finite numbers in the same places."""
    got, want = ref.f64(got), ref.f64(want)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.isinf(), want.isinf()) and (got[want.isinf()] == want[want.isinf()]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("inverse", [False, True])
def test_infinities_turn_by_the_formula(dtype, layout, inverse):
    """An infinity in either channel of a pair, of either sign, in both, and a NaN; position 0 among
    them (infinity times sin 0 is NaN)."""
    R, inf = 32, float("inf")
    x = make(12, 3, 64, dtype, 71)
    a, b = ((5, 5 + R // 2) if layout == "half" else (10, 11))
    for t, (u, w) in enumerate([(inf, 1.0), (-inf, 1.0), (1.0, inf), (1.0, -inf), (inf, inf), (inf, -inf), (float("nan"), 2.0),
                                (inf, 0.0), (0.0, -inf)]):
        x[t, 1, a], x[t, 1, b] = u, w
    x[9], x[10, 2, a], x[11, 0, 50] = make(1, 3, 64, dtype, 72)[0], inf, -inf
    pos = torch.tensor([3, 1, 2, 1000, 7, 9, 4, 5, 6, 8, 0, 77], dtype=torch.int32, device="cuda")
    f, mag = kda.rotary_inv_freq(R)
    y = kda.rotary(x, pos, f, magnitude=mag, layout=layout, inverse=inverse)
    want = ref.rotary(ref.f64(x), pos.cpu(), f.cpu(), mag, layout, inverse)
    same_kind(y, want)
    ok = want.isfinite()
    tol = ref.ROTARY_ROUNDINGS * ref.HALF_F32 * ref.rotary_size(ref.f64(x).nan_to_num(0.0, 0.0, 0.0), R, mag, layout)
    tol = tol + (ref.HALF_BF16 * want.abs() if dtype == torch.bfloat16 else 0.0)
    ref.check("finite channels", torch.where(ok, ref.f64(y), 0.0), torch.where(ok, want, 0.0), torch.where(ok, tol, 0.0))


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_infinities_in_an_append(step, layout):
    """Rotated keys and queries as the formula has them; in the cache what is not finite is NaN."""
    T, Hk, D, P, inf = 6, 2, 64, 16, float("inf")
    x = make(T, Hk, D, torch.bfloat16, 73)
    a, b = ((5, 5 + D // 2) if layout == "half" else (10, 11))
    for t, (u, w) in enumerate([(inf, 1.0), (1.0, inf), (1.0, -inf), (inf, -inf), (float("nan"), 0.0)]):
        x[t, 1, a], x[t, 1, b] = u, w
    f, mag = kda.rotary_inv_freq(D)
    if step:
        ctx, cu, table = torch.arange(3, 3 + T), None, torch.arange(T)[:, None]
    else:
        ctx, cu, table = torch.tensor([3]), torch.tensor([0, T], dtype=torch.int32, device="cuda"), torch.zeros((1, 1))
    cache = kda.kv_cache(T, Hk, D, P)
    q, k = kda.kv_append(x, x, cache, table.int().cuda(), ctx.int().cuda(), cu_seqlens=cu, inv_freq=f, magnitude=mag,
                         layout=layout, q=x, return_k=True)
    want = ref.rotary(ref.f64(x), torch.arange(3, 3 + T), f.cpu(), mag, layout)
    same_kind(q, want)
    same_kind(k, want)
    for t in range(T):
        code = cache.k[t if step else 0, :, 3 + t].float().cpu()
        assert torch.equal(code.isnan(), ~want[t].isfinite())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("base,scaling", [(1e6, None), (1e4, "linear"), (1e9, "yarn")])
def test_the_sine_of_a_small_angle(base, scaling, layout):
    """Pairs whose second channel is zero: the second output is a sine alone, and is held to fp32's own
    precision however slowly the pair turns."""
    R = 128
    f, mag = kda.rotary_inv_freq(R, base=base, scaling=scaling, factor=32.0)
    pos = torch.tensor([1, 2, 3, 7, 100, 4097, -1, -5], dtype=torch.int32, device="cuda")
    x = make(pos.numel(), 2, R, torch.float32, 74)
    second = slice(R // 2, R) if layout == "half" else slice(1, R, 2)
    x[..., second] = 0
    y = kda.rotary(x, pos, f, magnitude=mag, layout=layout)
    want = ref.rotary(ref.f64(x), pos.cpu(), f.cpu(), mag, layout)
    # the angle's turn per position is cut at 2^-64 turns; the rest are roundings relative to the sine
    cut = 2.0 ** -64 * 2 * torch.pi * pos.cpu().double().abs()[:, None, None] * 8
    tol = ref.ROTARY_ROUNDINGS * ref.HALF_F32 * want.abs() + cut
    ref.check("sines", y[..., second], want[..., second], tol[..., second])
