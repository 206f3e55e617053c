"""GPU tests of the latent rows' append (kda_latent_append) and of the products between heads and latent
(kda_latent_queries, kda_latent_values, kda_latent_expand) against their formulas in 64 bits, and of a
layer's prompt and steps in both forms.

Tolerances.  Append: one rounding to bf16; the norm's sum of 512 squares in 21 steps, its root and
reciprocal, three products: below 2^-18.  Turned channels as tests/test_rotary_gpu.py.  Products: one
rounding to bf16, and an fp32 sum of K products in K / 16 steps, each losing at most two units of 2^-24
of the running size: below 2^-17 of sum |a||b|."""
import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda
from tests import attn_reference as ref
from tests.test_kv_append_gpu import gen, table_for

pytestmark = pytest.mark.gpu
C, R, ROW = 512, 64, 576
SUM = 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


def cum(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def weights(H, seed):
    return (torch.randn((H, 256, C), generator=gen(seed), device="cuda") * C ** -0.5).bfloat16()


def want_rows(x, places, norm_w, eps, f, mag, layout):
    """(rows, tolerance) in 64 bits."""
    c, r = ref.f64(x[:, :C]), ref.f64(x[:, C:])[:, None]
    ct = torch.zeros_like(c)
    if norm_w is not None:
        c = c / torch.sqrt((c * c).mean(1, keepdim=True) + eps) * ref.f64(norm_w)
        ct = (ref.HALF_BF16 + 2.0 ** -18) * c.abs() + 2.0 ** -133  # (bf16's smallest step)
    rt = torch.zeros_like(r)
    if f is not None:
        n = 2 * f.numel()
        rt = ref.rotary_size(r, n, mag, layout) * ref.ROTARY_ROUNDINGS * ref.HALF_F32
        r = ref.rotary(r, places, f.cpu(), mag, layout)
        rt = rt + ref.HALF_BF16 * r.abs()
        rt[..., n:] = 0
    return torch.cat([c, r[:, 0]], 1), torch.cat([ct, rt[:, 0]], 1)


def append_case(new, ctx, P, *, norm=True, turned=64, layout="half", seed=0, one=False, beside=0, eps=1e-5, scale=1.0):
    g = gen(seed)
    T = sum(new)
    table, pages = table_for([a + b for a, b in zip(new, ctx)], P, seed)
    cache = torch.randn((pages, P, ROW), generator=g, device="cuda").bfloat16()
    old = cache.clone()
    x = (scale * torch.randn((T, beside + ROW), generator=g, device="cuda")).bfloat16()[:, beside:]
    w = 1 + 0.1 * torch.randn(C, generator=g, device="cuda") if norm else None
    f, mag = kda.rotary_inv_freq(turned, scaling="yarn", factor=4.0) if turned else (None, 1.0)
    rows = kda.latent_append(x, cache, table.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                             cu_seqlens=None if one else cum(new), norm_w=w, eps=eps, inv_freq=f, magnitude=mag, layout=layout,
                             return_rows=True)
    places = torch.cat([torch.arange(c, c + n) for n, c in zip(new, ctx)])
    want, tol = want_rows(x, places, w, eps, f, mag, layout)
    ref.check("rows", rows, want, tol)
    flat, t = old.view(-1, ROW), 0
    for n, (a, c) in enumerate(zip(new, ctx)):
        for j in range(c, c + a):
            flat[int(table[n, j // P]) * P + j % P] = rows[t]
            t += 1
    assert torch.equal(cache, old)  # the same rows, and nothing else written
    return x, rows, cache, table


@pytest.mark.parametrize("new,ctx", [([1], [0]), ([5, 0, 17], [0, 3, 15]), ([64, 65, 1], [0, 63, 128]), ([300], [1]),
                                     ([1] * 70, list(range(70)))])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_append(new, ctx, P):
    append_case(new, ctx, P, seed=sum(new))


@pytest.mark.parametrize("turned", [0, 16, 32, 48, 64])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", [False, True])
def test_append_forms(turned, layout, norm):
    append_case([7, 40], [90000, 0], 16, norm=norm, turned=turned, layout=layout, seed=turned, beside=24)


def test_append_one_token_each():
    append_case([1] * 300, [(7 * i) % 100 for i in range(300)], 64, one=True, seed=1)


@pytest.mark.parametrize("scale,eps", [(1e25, 1e-5), (1e-25, 1e-5), (1e-20, 1e-30), (1e-3, 0.7), (1e-25, 3.0), (1e18, 1e-5)])
def test_append_sizes(scale, eps):
    """Squares beyond fp32's range, and eps of any size."""
    append_case([20], [5], 16, turned=0, scale=scale, eps=eps, seed=2)


def test_append_zero_and_not_finite():
    g = gen(3)
    x = torch.randn((6, ROW), generator=g, device="cuda").bfloat16()
    x[0] = 0
    x[1, 7], x[2, 7], x[3, 570] = float("nan"), float("inf"), float("-inf")
    cache = kda.latent_cache(1, 16)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = kda.latent_append(x, cache, table, z, cu_seqlens=cum([6]), norm_w=torch.ones(C, device="cuda"), return_rows=True)
    assert (rows[0] == 0).all() and rows[1, :C].isnan().all() and torch.equal(rows[1, C:], x[1, C:])
    assert rows[2, 7].isnan() and (rows[2, :7] == 0).all() and (rows[2, 8:C] == 0).all()
    assert torch.equal(rows[3, C:], x[3, C:]) and rows[3, :C].isfinite().all()
    f, _ = kda.rotary_inv_freq(16)
    turned = kda.latent_append(x, cache, table, z, cu_seqlens=cum([6]), inv_freq=f, return_rows=True)
    assert torch.equal(turned[1:3, :C].view(torch.int16), x[1:3, :C].view(torch.int16))  # not normalised: bit for bit
    assert torch.equal(turned[:, C + 16:].view(torch.int16), x[:, C + 16:].view(torch.int16))


def test_append_padding_and_rows_of_no_sequence():
    """Negative, too large and missing pages are not stored (the rows come all the same); rows before the
    first and behind the last sequence stay as they are."""
    g = gen(4)
    x = torch.randn((10, ROW), generator=g, device="cuda").bfloat16()
    cache = torch.full((3, 16, ROW), 5.0, device="cuda").bfloat16()
    table = torch.tensor([[-1, 1], [3, 0], [2, 1 << 30]], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([15, 2, 31], dtype=torch.int32, device="cuda")
    cu = torch.tensor([1, 3, 5, 8], dtype=torch.int32, device="cuda")
    out = torch.full((10, ROW), 9.0, device="cuda").bfloat16()
    kda.latent_append(x, cache, table, ctx, cu_seqlens=cu, rows_out=out)
    assert (out[0] == 9).all() and (out[8:] == 9).all() and torch.equal(out[1:8], x[1:8])
    want = torch.full((3, 16, ROW), 5.0, device="cuda").bfloat16()
    want[1, 0] = x[2]  # place 16 of sequence 0; its place 15, sequence 1 (page 3) and sequence 2 (behind the table) are not
    assert torch.equal(cache, want)


def test_append_captured():
    x, rows, cache, table = append_case([3, 30], [10, 0], 16, turned=0, norm=False, seed=5)
    dt, cu = table.cuda(), cum([3, 30])
    ctx = torch.zeros(2, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.latent_append(x, cache, dt, ctx, cu_seqlens=cu)
    cache.zero_()
    ctx.copy_(torch.tensor([10, 0], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache.view(-1, ROW)[int(table[0, 0]) * 16 + 10], x[0])


TOKENS_HEADS = [(1, 1), (8, 32), (127, 3), (128, 2), (129, 5), (300, 16), (40, 160), (1000, 1)]


@pytest.mark.parametrize("T,H", TOKENS_HEADS)
@pytest.mark.parametrize("turned,layout", [(0, "half"), (64, "half"), (64, "interleaved"), (32, "half"), (48, "interleaved")])
def test_queries(T, H, turned, layout):
    g = gen(T + H)
    fused = torch.randn((T, H + 2, 192), generator=g, device="cuda").bfloat16()
    q, w = fused[:, 1:H + 1], weights(H, T)
    f, mag = kda.rotary_inv_freq(turned, scaling="yarn", factor=8.0) if turned else (None, 1.0)
    pos = torch.randint(0, 1 << 31 - 1, (T,), generator=g, device="cuda").int() if turned else None
    out = kda.latent_queries(q, w, positions=pos, inv_freq=f, magnitude=mag, layout=layout)
    kda.device_status()
    qn, wk = ref.f64(q[..., :128]), ref.f64(w[:, :128])
    want = torch.einsum("thn,hnc->thc", qn, wk)
    tol = ref.HALF_BF16 * want.abs() + SUM * torch.einsum("thn,hnc->thc", qn.abs(), wk.abs())
    ref.check("latent", out[..., :C], want, tol)
    r = ref.f64(q[..., 128:])
    if not turned:
        assert torch.equal(out[..., C:], q[..., 128:])
        return
    size = ref.rotary_size(r, turned, mag, layout)
    want = ref.rotary(r, pos.cpu(), f.cpu(), mag, layout)
    # (positions go up to 2^31, where an angle is off by up to 2^-29 turns' worth beside the roundings)
    tol = ref.HALF_BF16 * want.abs() + (ref.ROTARY_ROUNDINGS * ref.HALF_F32 + 2.0 ** -24) * size
    tol[..., turned:] = 0
    ref.check("shared", out[..., C:], want, tol)


@pytest.mark.parametrize("T,H", TOKENS_HEADS)
def test_values(T, H):
    g = gen(T * H)
    o = torch.randn((T, H + 1, C), generator=g, device="cuda").bfloat16()[:, :H]
    w = weights(H, T + 1)
    out = kda.latent_values(o, w.flatten(0, 1))  # the projection's weight as it lies
    kda.device_status()
    a, b = ref.f64(o), ref.f64(w[:, 128:])
    want = torch.einsum("thc,hnc->thn", a, b)
    ref.check("values", out, want, ref.HALF_BF16 * want.abs() + SUM * torch.einsum("thc,hnc->thn", a.abs(), b.abs()))


@pytest.mark.parametrize("T,H", TOKENS_HEADS)
def test_expand(T, H):
    g = gen(T * H + 1)
    x = torch.randn((T, 32 + ROW), generator=g, device="cuda").bfloat16()[:, 32:]
    w = weights(H, T + 2)
    k, v = kda.latent_expand(x, w)
    kda.device_status()
    a, b = ref.f64(x[:, :C]), ref.f64(w).flatten(0, 1)
    want = (a @ b.T).view(T, H, 256)
    tol = ref.HALF_BF16 * want.abs() + SUM * (a.abs() @ b.abs().T).view(T, H, 256)
    ref.check("keys", k[..., :128], want[..., :128], tol[..., :128])
    ref.check("values", v, want[..., 128:], tol[..., 128:])
    assert torch.equal(k[..., 128:], x[:, None, C:].expand(T, H, R))


def test_products_of_nothing_write_nothing():
    w = weights(3, 1)
    e = lambda *s: torch.zeros(s, device="cuda").bfloat16()
    assert kda.latent_queries(e(0, 3, 192), w).shape == (0, 3, ROW) and kda.latent_values(e(0, 3, C), w).shape == (0, 3, 128)
    k, v = kda.latent_expand(e(0, ROW), w)
    assert k.shape == (0, 3, 192) and v.shape == (0, 3, 128)


def test_products_write_only_their_rows():
    """Outputs that are slices of larger buffers: what lies around them stays."""
    T, H = 77, 5
    w = weights(H, 2)
    g = gen(6)
    q = torch.randn((T, H, 192), generator=g, device="cuda").bfloat16()
    for call, width in ((lambda out: kda.latent_queries(q, w, out=out), ROW),
                        (lambda out: kda.latent_values(torch.randn((T, H, C), generator=g, device="cuda").bfloat16(), w, out=out), 128)):
        big = torch.full((T + 2, H, width), 3.0, device="cuda").bfloat16()
        call(big[1:T + 1])
        assert (big[0] == 3).all() and (big[-1] == 3).all() and not (big[1:-1] == 3).all()


def test_host_tensors():
    T, H = 9, 4
    w, g = weights(H, 3), gen(7)
    q, x = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((T, H, 192), (T, ROW)))
    assert torch.equal(kda.latent_queries(q.cpu(), w.cpu()), kda.latent_queries(q, w).cpu())
    o = torch.randn((T, H, C), generator=g, device="cuda").bfloat16()
    assert torch.equal(kda.latent_values(o.cpu(), w), kda.latent_values(o, w).cpu())
    for a, b in zip(kda.latent_expand(x.cpu(), w), kda.latent_expand(x, w)):
        assert torch.equal(a, b.cpu())


def test_a_layer_in_both_forms():
    """A prompt in the expanded form and in the absorbed one, then a few steps, as a layer runs them, against
    attention of each head on its own keys and values in 64 bits.  Beside the attention's own
    tolerances, scores and values carry the roundings to bf16 of what the form hands on: the
    absorbed queries and outputs, or the expanded keys and values."""
    H, P, lens, steps = 6, 16, [70, 1, 130], 3
    T, N = sum(lens), len(lens)
    g = gen(8)
    w, norm = weights(H, 9), 1 + 0.1 * torch.randn(C, generator=g, device="cuda")
    f, mag = kda.rotary_inv_freq(R, scaling="yarn", factor=4.0)
    table, pages = table_for([n + steps for n in lens], P, 10)
    table, cache = table.cuda(), kda.latent_cache(pages, P)
    x = lambda n: torch.randn((n, ROW), generator=g, device="cuda").bfloat16()
    q = lambda n: torch.randn((n, H, 192), generator=g, device="cuda").bfloat16()
    ctx = torch.zeros(N, dtype=torch.int32, device="cuda")
    cu = cum(lens)
    x0, q0 = x(T), q(T)
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    rows = kda.latent_append(x0, cache, table, ctx, cu_seqlens=cu, norm_w=norm, inv_freq=f, magnitude=mag, return_rows=True)
    ctx = ctx + cu[1:] - cu[:-1]
    # expanded: the queries' shared channels turned by the same call that the absorbed form uses
    lq = kda.latent_queries(q0, w, positions=pos, inv_freq=f, magnitude=mag)
    k, v = kda.latent_expand(rows, w)
    whole = kda.attn_prompt(torch.cat([q0[..., :128], lq[..., C:]], -1), k, v, cu_seqlens=cu)
    absorbed = kda.latent_values(kda.attn_latent(lq, cache, table, ctx, cu_seqlens=cu), w)

    def check(name, got, qn, at, rows_n, seen):
        """One token's heads: qn [H, 192] with its shared channels turned, rows_n the sequence's rows."""
        r, wd = ref.f64(rows_n), ref.f64(w)
        for h in range(H):
            kk = torch.cat([r[:, :C] @ wd[h, :128].T, r[:, C:]], 1)
            vv = r[:, :C] @ wd[h, 128:].T
            want, _, av, size = ref.attend(ref.f64(qn[h:h + 1]), kk, vv, 192 ** -0.5, [seen])
            lat = (ref.f64(qn[h:h + 1, :128]).abs() @ wd[h, :128].abs() @ r[:seen, :C].abs().T).max() * 192 ** -0.5
            moved = 2 * (ref.HALF_BF16 + 2.0 ** -17) * (size + lat)  # scores off by a rounding of queries or keys
            vabs = (r[:seen, :C].abs() @ wd[h, 128:].abs().T).amax(0)
            tol = (torch.exp(moved) - 1)[:, None] * av + 4 * ref.HALF_BF16 * (av + vabs) + ref.HALF_BF16 * want.abs()
            ref.check(f"{name} {at} head {h}", got[h:h + 1], want, tol)

    all_rows = list(rows.split(lens))
    for n in range(N):
        for i in {0, lens[n] // 2, lens[n] - 1}:
            t = int(cu[n]) + i
            qn = torch.cat([q0[t, :, :128], lq[t, :, C:]], -1)
            check("expanded", whole[t], qn, t, all_rows[n], i + 1)
            check("absorbed", absorbed[t], qn, t, all_rows[n], i + 1)
    for _ in range(steps):
        x1, q1 = x(N), q(N)
        r1 = kda.latent_append(x1, cache, table, ctx, norm_w=norm, inv_freq=f, magnitude=mag, return_rows=True)
        lq = kda.latent_queries(q1, w, positions=ctx, inv_freq=f, magnitude=mag)
        ctx = ctx + 1
        o = kda.latent_values(kda.attn_latent(lq, cache, table, ctx), w)
        for n in range(N):
            all_rows[n] = torch.cat([all_rows[n], r1[n:n + 1]])
            check("step", o[n], torch.cat([q1[n, :, :128], lq[n, :, C:]], -1), n, all_rows[n], all_rows[n].shape[0])
    y = kda.o_proj(o.flatten(1).contiguous(), torch.randn((128, H * 128), generator=g, device="cuda").bfloat16())
    assert y.shape == (N, 128) and y.isfinite().all()


def test_refusals():
    w = weights(2, 1)
    z = lambda *s: torch.zeros(s, device="cuda").bfloat16()
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    f, _ = kda.rotary_inv_freq(64)
    wide, _ = kda.rotary_inv_freq(128)
    cache = kda.latent_cache(2, 16)
    for call, err in [
            (lambda: kda.latent_append(z(1, 512), cache, i(1, 1), i(1)), ValueError),
            (lambda: kda.latent_append(z(1, ROW).float(), cache, i(1, 1), i(1)), TypeError),
            (lambda: kda.latent_append(z(1, ROW).cpu(), cache, i(1, 1), i(1)), ValueError),
            (lambda: kda.latent_append(z(2, ROW), cache, i(1, 1), i(1)), kda.KDAError),
            (lambda: kda.latent_append(z(1, ROW), cache, i(1, 1), i(2)), ValueError),
            (lambda: kda.latent_append(z(1, ROW), cache, i(1, 1), i(1), norm_w=torch.ones(64, device="cuda")), ValueError),
            (lambda: kda.latent_append(z(1, ROW), cache, i(1, 1), i(1), norm_w=torch.ones(C, device="cuda"), eps=0.0), kda.KDAError),
            (lambda: kda.latent_append(z(1, ROW), cache, i(1, 1), i(1), inv_freq=wide), kda.KDAError),
            (lambda: kda.latent_append(z(1, ROW), cache, i(1, 1), i(1), layout="x"), ValueError),
            (lambda: kda.latent_append(z(1, ROW), cache, i(1, 1), i(1), rows_out=z(2, ROW)), ValueError),
            (lambda: kda.latent_append(cache[0, :1], cache, i(1, 1), i(1)), kda.KDAError),  # the cache's own rows
            (lambda: kda.latent_queries(z(1, 2, 128), w), ValueError), (lambda: kda.latent_queries(z(1, 3, 192), w), ValueError),
            (lambda: kda.latent_queries(z(1, 2, 192), w, positions=i(1)), ValueError),
            (lambda: kda.latent_queries(z(1, 2, 192), w, positions=i(2), inv_freq=f), ValueError),
            (lambda: kda.latent_queries(z(1, 2, 192), w.float()), TypeError),
            (lambda: kda.latent_queries(z(1, 2, 192), w[:, :128]), ValueError),
            (lambda: kda.latent_values(z(1, 2, 128), w), ValueError),
            (lambda: kda.latent_values(z(1, 2, C), w, out=z(1, 2, C)), ValueError),
            (lambda: kda.latent_expand(z(1, C), w), ValueError), (lambda: kda.latent_expand(z(1, ROW).float(), w), TypeError)]:
        with pytest.raises(err):
            call()
