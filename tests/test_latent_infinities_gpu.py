"""GPU tests of attention over latent rows that hold infinities, against the formula in 64 bits.  A row with an
infinite channel gets the score +inf, -inf or NaN.  +inf and NaN make all of a seeing token's output NaN; with -inf the
row's weight is 0, so that the output is that of the other rows but NaN (0 times infinity) in the row's infinite
channels.  This has to hold wherever the row lies: among the tokens that the call's other tokens do not all see, before
them, and in sequences that are cut.  Tolerances as in tests/test_attn_latent_gpu.py."""
import math

import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda
from tests import attn_reference as ref
from tests.test_attn_latent_gpu import C, cum, make, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


def look(o, lse, q, rows, seen):
    """One token's heads."""
    scale = 192 ** -0.5
    o, lse, k, qs = o.cpu(), lse.cpu(), rows[:seen].cpu(), ref.f64(q).cpu()
    # (as a sum of products, one by one: a library product may not carry infinities through)
    z = torch.stack([(qs[h] * k).sum(1) for h in range(qs.shape[0])]) * scale
    lost = (z.isnan() | (z == math.inf)).any(1)
    assert o[lost].isnan().all() and lse[lost].isnan().all()
    odd = ~k[:, :C].isfinite().all(0)  # channels
    for h in (~lost).nonzero().flatten().tolist():
        keep = z[h] > -math.inf
        assert keep.any()
        f, x = k[keep], z[h][keep]
        wl = torch.logsumexp(x, 0)
        p = torch.exp(x - wl)
        want, av = p @ f[:, :C], p @ f[:, :C].abs()
        moved = 2.0 ** -17 * (f.abs() @ qs[h].abs()).amax() * scale + 2.0 ** -19 + (32 + seen / 64) * 2.0 ** -24
        tol = (ref.HALF_BF16 + 2 * moved + (seen / 16 + 1) * 2.0 ** -23) * av
        tol = tol + (ref.HALF_BF16 if o.dtype == torch.bfloat16 else 2.0 ** -20) * want.abs()
        assert torch.equal(o[h].isnan(), odd)
        ref.check(f"head {h}", o[h][~odd], want[~odd], tol[~odd])
        ref.check(f"lse {h}", lse[h], wl, moved + 2.0 ** -22 * wl.abs())
    return int((~lost).sum())


# (length, rows of the call, place of the odd row from the end), and the channels that are infinite
CASES = [((70, 6, 3), [3]), ((70, 6, 3), [300, 511]), ((70, 6, 5), [570]), ((129, 4, 2), [128, 570]), ((64, 64, 40), [7]), ((66, 5, 4), [0]),
         ((300, 3, 200), [256]), ((20000, 6, 3), [5]), ((20000, 4, 4), [130]), ((90, 40, 1), [200]), ((10, 10, 10), [1])]


@pytest.mark.parametrize("at,channels", CASES)
@pytest.mark.parametrize("H,P,out", [(16, 16, torch.bfloat16), (3, 64, torch.float32), (72, 128, torch.bfloat16)])
def test_infinite_rows(at, channels, H, P, out):
    length, m, back = at
    lens, new = [40, length, 17], [2, m, 1]
    q, cache, table, sl = make(lens, H, P, length + m, sum(new))
    call = lambda: kda.attn_latent(q, cache, table.cuda(), sl, cu_seqlens=cum(new), return_lse=True, out_dtype=out)
    o, lse = call()
    place = length - back
    spot = cache[int(table[1, place // P]), place % P]
    spot[channels] = torch.tensor([math.inf, -math.inf][:len(channels)], device="cuda").bfloat16()
    if place > 20:  # and a second one that all tokens see, with other channels
        cache[int(table[1, 10 // P]), 10 % P, 77] = -math.inf
    o2, lse2 = call()
    kda.device_status()
    mine = torch.zeros(sum(new), dtype=torch.bool, device="cuda")
    mine[2:2 + m] = True
    assert torch.equal(o2[~mine], o[~mine]) and torch.equal(lse2[~mine], lse[~mine])
    rows = rows_of(cache, table, 1, length)
    kept = 0
    for i in sorted({0, m - 1, m // 2, max(m - back, 0), max(m - back - 1, 0)}):
        seen = length - m + i + 1
        if seen > 1:  # (a token whose only row scores -inf has no weights to speak of)
            kept += look(o2[2 + i], lse2[2 + i], q[2 + i], rows, seen)
    assert kept > 0  # some scores were -inf


def test_the_same_alone_and_beside_others():
    """A token gets the same NaN whether the call has it alone or behind others that do not see the row."""
    H, P, L, m = 16, 32, 70, 6
    q, cache, table, sl = make([L], H, P, 3, m)
    cache[int(table[0, 66 // P]), 66 % P, 9] = math.inf
    dt = table.cuda()
    o, lse = kda.attn_latent(q, cache, dt, sl, cu_seqlens=cum([m]), return_lse=True)
    for i in range(m):
        a, b = kda.attn_latent(q[i:i + 1], cache, dt, sl - (m - 1 - i), return_lse=True)
        assert torch.equal(a[0].isnan(), o[i].isnan()) and torch.equal(b[0].isnan(), lse[i].isnan())
    assert not o[:2].isnan().any() and o[2:, :, 9].isnan().all() and o[2:].isfinite().any()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L", [1, 3, 200, 9000])
def test_all_scores_minus_infinity(L, out):
    """Every row is infinite where the first head's query is negative (its scores are -inf) and the second's is positive."""
    P, m = 64, min(L, 2)
    q, cache, table, sl = make([L], 2, P, L, m)
    cache[..., 20] = math.inf
    q[:, 0, 20], q[:, 1, 20] = -1.0, 1.0
    o, lse = kda.attn_latent(q, cache, table.cuda(), sl, cu_seqlens=cum([m]), return_lse=True, out_dtype=out)
    assert (lse[:, 0] == -math.inf).all() and lse[:, 1].isnan().all() and o[:, 1].isnan().all()
    assert o[:, 0, 20].isnan().all() and (o[:, 0, :20] == 0).all() and (o[:, 0, 21:] == 0).all()
