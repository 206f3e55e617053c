"""GPU tests of the shared channels' rotation over the whole range of int32 positions and of places in a sequence,
against angles reduced exactly (fractions).  Tolerance: that of tests/test_rotary_gpu.py, and the angle's own error of
|position| * 2^-64 turns (2^31 * 2^-64 * 2 pi < 2^-30) of the pair's size."""
import math
from fractions import Fraction

import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda
from tests import attn_reference as ref
from tests.test_kv_append_gpu import gen
from tests.test_latent_rows_gpu import C, ROW, cum, weights

pytestmark = pytest.mark.gpu
TURN = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494")
TOP = (1 << 31) - 1


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


def turned(x, positions, f, mag, layout):
    """x [T, H, 64] float64."""
    x, n = x.clone(), 2 * f.numel()
    for i, w in enumerate(f.tolist()):
        a, b = (i, i + n // 2) if layout == "half" else (2 * i, 2 * i + 1)
        angle = [float(Fraction(p) * Fraction(w) % TURN) for p in positions]
        c, s = (torch.tensor([fn(t) * mag for t in angle], dtype=torch.float64)[:, None] for fn in (math.cos, math.sin))
        xa, xb = x[..., a].clone(), x[..., b].clone()
        x[..., a], x[..., b] = xa * c - xb * s, xa * s + xb * c
    return x


def verify(name, got, x, positions, f, mag, layout):
    x, n = ref.f64(x), 2 * f.numel()
    want = turned(x, positions, f.cpu(), mag, layout)
    tol = ref.HALF_BF16 * want.abs() + (ref.ROTARY_ROUNDINGS * ref.HALF_F32 + 2.0 ** -30) * ref.rotary_size(x, n, mag, layout)
    tol[..., n:] = 0
    ref.check(name, got, want, tol)


@pytest.mark.parametrize("n,layout", [(64, "half"), (64, "interleaved"), (16, "half"), (48, "interleaved")])
def test_queries(n, layout):
    g = gen(n)
    pos = [0, 1, -1, TOP, TOP - 1, -TOP, -TOP - 1, 1 << 30, (1 << 30) + 1]
    pos += torch.randint(-1 << 31, 1 << 31, (31,), generator=torch.Generator().manual_seed(n)).tolist()
    assert min(pos) < -1 << 30 and sum(p > 1 << 30 for p in pos) > 5
    q = torch.randn((len(pos), 3, 192), generator=g, device="cuda").bfloat16()
    f, mag = kda.rotary_inv_freq(n, scaling="yarn", factor=8.0)
    out = kda.latent_queries(q, weights(3, 1), positions=torch.tensor(pos, dtype=torch.int32, device="cuda"), inv_freq=f,
                             magnitude=mag, layout=layout)
    verify("shared", out[..., C:], q[..., 128:], pos, f, mag, layout)


@pytest.mark.parametrize("n,layout", [(64, "half"), (64, "interleaved"), (32, "half")])
def test_appended_rows(n, layout):
    """Rows that are wanted densely, of tokens whose places lie far behind the table."""
    new, ctx = [4, 1, 30], [(1 << 30) - 2, TOP, TOP - 40]
    x = torch.randn((sum(new), ROW), generator=gen(n + 1), device="cuda").bfloat16()
    cache = kda.latent_cache(2, 16)
    f, mag = kda.rotary_inv_freq(n)
    rows = kda.latent_append(x, cache, torch.zeros((3, 1), dtype=torch.int32, device="cuda"),
                             torch.tensor(ctx, dtype=torch.int32, device="cuda"), cu_seqlens=cum(new), inv_freq=f,
                             magnitude=mag, layout=layout, return_rows=True)
    assert (cache == 0).all()  # none of them has a page
    places = [c + i for m, c in zip(new, ctx) for i in range(m)]
    verify("rows", rows[:, None, C:], x[:, None, C:], places, f, mag, layout)
