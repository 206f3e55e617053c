"""GPU tests of the prompt's causal attention (kda_attn_prompt) against 64-bit attention.  Tolerance
per output: the weights' rounding to bf16 (half a step, relative to sum p |v|), one rounding to the
output's type, and the scores' fp32 accumulation, whose error moves every weight: at most 2^-20 of
the largest sum |q||k| * scale (192 products, each accumulation step losing at most two units of
2^-24 of the running size; the exponential's argument is held to 2^-22 of the score).  Where the keys
are divided, the sums of at most 32 parts are joined in fp32: a factor within 2^-22 and 33 roundings,
37 * 2^-24 of sum p |v|."""
import math

import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu

DIMS = [(64, 64), (128, 128), (192, 128)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def cum(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")


def make(Tq, Tk, Hq, Hk, D, DV, seed, sharp=1.0):
    g = gen(seed)
    r = lambda n, h, d, s=1.0: (s * torch.randn((n, h, d), generator=g, device="cuda")).bfloat16()
    return r(Tq, Hq, D, sharp), r(Tk, Hk, D), r(Tk, Hk, DV)


def verify(o, lse, q, k, v, nq, nk, scale=None, heads=None, rows=None):
    """heads / rows: what is looked at (default everything)."""
    Hq, Hk, D = q.shape[1], k.shape[1], q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    G, q0, k0 = Hq // Hk, 0, 0
    for n, (a, b) in enumerate(zip(nq, nk)):
        at = torch.arange(a) if rows is None else torch.tensor(sorted({r for r in rows if r < a}), dtype=torch.long)
        for h in range(Hq) if heads is None else heads:
            sel = (q0 + at).cuda()
            want, wl, av, size = ref.attend(ref.f64(q[sel, h]), ref.f64(k[k0:k0 + b, h // G]), ref.f64(v[k0:k0 + b, h // G]),
                                            scale, (at + 1 + b - a).tolist())
            moved = 2.0 ** -20 * size + 2.0 ** -20
            moved = moved + 37 * 2.0 ** -24
            tol = (ref.HALF_BF16 + 2 * moved)[:, None] * av
            tol = tol + (ref.HALF_BF16 if o.dtype == torch.bfloat16 else 2.0 ** -20) * want.abs()
            ref.check(f"o[{n}, head {h}]", o[sel, h], want, tol)
            if lse is not None:
                ref.check(f"lse[{n}, head {h}]", lse[sel, h], wl, moved + 2.0 ** -22 * wl.abs().nan_to_num(posinf=0.0))
        q0, k0 = q0 + a, k0 + b


def case(nq, nk, Hq, Hk, D, DV, seed=0, out=torch.bfloat16, scale=None, sharp=1.0, **look):
    q, k, v = make(sum(nq), sum(nk), Hq, Hk, D, DV, seed, sharp)
    o, lse = kda.attn_prompt(q, k, v, cu_seqlens=cum(nq), cu_seqlens_k=None if nq == nk else cum(nk), return_lse=True,
                             out_dtype=out, scale=scale)
    kda.device_status()
    verify(o, lse, q, k, v, nq, nk, scale, **look)
    return o, lse, q, k, v


@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [129], [255, 1, 256], [257, 0, 100], [0, 3, 0], [385],
                                  [5, 130, 64, 1, 300]])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (4, 2), (3, 1)])
@pytest.mark.parametrize("D,DV", DIMS)
def test_lengths(lens, Hq, Hk, D, DV):
    case(lens, lens, Hq, Hk, D, DV, seed=sum(lens))


@pytest.mark.parametrize("nq,nk", [([1], [500]), ([100], [228]), ([130, 7], [131, 400]), ([200], [72]),
                                   ([300, 10, 4], [20, 0, 4]), ([256], [384]), ([129, 129], [1, 1000])])
@pytest.mark.parametrize("Hq,Hk,D,DV", [(2, 1, 128, 128), (1, 1, 64, 64), (2, 2, 192, 128)])
def test_contexts_and_rows_that_see_nothing(nq, nk, Hq, Hk, D, DV):
    """More keys than queries (a continued context), and fewer (leading rows see nothing)."""
    o, lse, *_ = case(nq, nk, Hq, Hk, D, DV, seed=sum(nk))
    q0 = 0
    for a, b in zip(nq, nk):
        blind = max(0, a - b)
        assert (o[q0:q0 + blind] == 0).all() and (lse[q0:q0 + blind] == -math.inf).all()
        q0 += a


def test_no_keys_at_all():
    q, k, v = make(5, 0, 2, 1, 64, 64, 1)
    o, lse = kda.attn_prompt(q, k, v, return_lse=True)
    assert (o == 0).all() and (lse == -math.inf).all()
    assert kda.attn_prompt(q[:0], k, v).shape == (0, 2, 64)


@pytest.mark.parametrize("D,DV", DIMS)
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_long(D, DV, out):
    """Many key blocks, so that every ring goes round many times; rows sampled."""
    rows = list(range(0, 2500, 173)) + [2499, 2498, 127, 128, 1151, 1152]
    case([2500, 700], [2500, 1500], 4, 2, D, DV, seed=3, out=out, rows=rows, heads=[0, 3])


@pytest.mark.parametrize("Hq,Hk", [(8, 1), (12, 4), (10, 2), (7, 7), (64, 1)])
def test_groups(Hq, Hk):
    case([150, 37], [150, 37], Hq, Hk, 64, 64, seed=Hq)


def test_many_sequences():
    """More sequences than lanes of a warp, in no order of length."""
    lens = [(i * 37) % 90 for i in range(75)]
    case(lens, lens, 2, 1, 64, 64, seed=5)


@pytest.mark.parametrize("D,DV", DIMS)
def test_rising_and_sharp_scores(D, DV):
    """Scores of several hundred; keys that grow along the sequence, so that the reference maximum is
    set anew in block after block; negative and tiny scales."""
    case([400], [400], 2, 1, D, DV, seed=6, sharp=25.0)
    q, k, v = make(600, 600, 2, 1, D, DV, 7)
    q = q.abs()
    k = (k.abs().float() * torch.linspace(0.1, 4, 600, device="cuda")[:, None, None]).bfloat16()
    for scale in (None, -0.2, 1e-12):
        for ws in ("auto", None):
            o, lse = kda.attn_prompt(q, k, v, return_lse=True, scale=scale, workspace=ws)
            verify(o, lse, q, k, v, [600], [600], scale, rows=list(range(0, 600, 41)) + [599])


@pytest.mark.parametrize("D,DV", DIMS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_nothing_masked_enters(D, DV, bad):
    """Rows of another sequence and later tokens of the same one hold NaN or infinities: what does not
    see them keeps its value to the bit, what sees them does not."""
    nq = nk = [200, 90]
    q, k, v = make(290, 290, 2, 1, D, DV, 8)
    o, lse = kda.attn_prompt(q, k, v, cu_seqlens=cum(nq), return_lse=True)
    k2, v2 = k.clone(), v.clone()
    k2[200:], v2[200:] = bad, bad  # the second sequence
    o2, lse2 = kda.attn_prompt(q, k2, v2, cu_seqlens=cum(nq), return_lse=True)
    assert torch.equal(o2[:200], o[:200]) and torch.equal(lse2[:200], lse[:200])
    v3 = v.clone()
    v3[70, 0, 5] = bad  # seen from row 70 on
    o3, lse3 = kda.attn_prompt(q, k, v3, cu_seqlens=cum(nq), return_lse=True)
    verify(o3[:70], None, q[:70], k[:70], v[:70], [70], [70])
    assert torch.equal(lse3, lse) and not o3[70:200, :, 5].isfinite().any()
    assert torch.equal(o3[128:200, :, :5], o[128:200, :, :5]) and torch.equal(o3[200:], o[200:])
    k4 = k.clone()
    k4[70, 0, 5] = bad
    o4, _ = kda.attn_prompt(q, k4, v, cu_seqlens=cum(nq), return_lse=True)
    assert torch.equal(o4[:70], o[:70]) and torch.equal(o4[200:], o[200:])


def test_rows_of_no_sequence_are_left_alone():
    q, k, v = make(100, 100, 2, 1, 64, 64, 9)
    o = torch.full((100, 2, 64), 7.0, device="cuda").bfloat16()
    cu = torch.tensor([3, 40, 77], dtype=torch.int32, device="cuda")
    kda.attn_prompt(q, k, v, cu_seqlens=cu, o=o)
    assert (o[:3] == 7).all() and (o[77:] == 7).all()
    verify(o[3:77], None, q[3:77], k[3:77], v[3:77], [37, 37], [37, 37])
    wild = torch.tensor([-50, 40, 10 ** 6], dtype=torch.int32, device="cuda")  # clamped to the tensors
    verify(kda.attn_prompt(q, k, v, cu_seqlens=wild), None, q, k, v, [40, 60], [40, 60])


def test_strided_rows_dense_batch_and_host():
    Hq, Hk, D = 4, 2, 128
    fused = torch.randn((2, 70, (Hq + 2 * Hk) * D), generator=gen(10), device="cuda").bfloat16()
    q, k, v = (t.unflatten(-1, (-1, D)) for t in fused.split([Hq * D, Hk * D, Hk * D], -1))
    o = kda.attn_prompt(q, k, v)
    assert o.shape == (2, 70, Hq, D)
    flat = [t.flatten(0, 1).contiguous() for t in (q, k, v)]
    assert torch.equal(o.flatten(0, 1), kda.attn_prompt(*flat, cu_seqlens=cum([70, 70])))
    verify(o.flatten(0, 1), None, *flat, [70, 70], [70, 70])
    assert torch.equal(kda.attn_prompt(*(t.cpu() for t in (q, k, v))), o.cpu())
    one = kda.attn_prompt(q[1], k[1], v[1])
    assert torch.equal(one, o[1])


def test_same_bits_again_on_another_stream_and_from_a_graph():
    q, k, v = make(1000, 1000, 4, 2, 128, 128, 11)
    o = kda.attn_prompt(q, k, v)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        again = [kda.attn_prompt(q, k, v) for _ in range(3)]
    st.synchronize()
    assert all(torch.equal(x, o) for x in again)
    out, cu = torch.empty_like(o), cum([400, 600])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.attn_prompt(q, k, v, cu_seqlens=cu, o=out)
    cu.copy_(cum([0, 1000]))
    graph.replay()
    torch.cuda.synchronize()
    # (how the keys are divided goes by the number of sequences, so the eager call is one of two as well)
    assert torch.equal(out, kda.attn_prompt(q, k, v, cu_seqlens=cu))
    whole = kda.attn_prompt(q, k, v, cu_seqlens=cu, workspace=None)
    assert torch.equal(whole, kda.attn_prompt(q, k, v, workspace=None))


@pytest.mark.parametrize("Hq,Hk", [(2, 1), (1, 1)])
def test_more_than_128_sequences(Hq, Hk):
    """More sequences than a warp holds at once (128), with and without tokens, the longest one last."""
    lens = [(7 * n * n + 3 * n) % 61 for n in range(300)] + [0, 700]
    q, k, v = make(sum(lens), sum(lens), Hq, Hk, 64, 64, 16)
    for ws in ("auto", None):
        o, lse = kda.attn_prompt(q, k, v, cu_seqlens=cum(lens), return_lse=True, workspace=ws)
        verify(o, lse, q, k, v, lens, lens, rows=[0, 1, 7, 20, 39, 60, 127, 128, 255, 256, 600, 699])


def test_two_calls_at_once():
    """Two streams at the same time, and the KDA prefill beside them."""
    from kimi_delta_attention_gated_gb300.inputs import make_inputs
    x, y = make(900, 900, 4, 2, 64, 64, 14), make(1500, 1500, 2, 2, 192, 128, 15)
    want = [kda.attn_prompt(*x), kda.attn_prompt(*y)]
    d = make_inputs("prefill", device="cuda", T=200, H=2)
    kd = lambda: kda.chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], scale=d["scale"])[0]
    want.append(kd())
    calls = [lambda: kda.attn_prompt(*x), lambda: kda.attn_prompt(*y), kd]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    outs = [[] for _ in calls]
    for _ in range(8):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(calls[i]())
    torch.cuda.synchronize()
    kda.device_status()
    for w, got in zip(want, outs):
        assert all(torch.equal(g, w) for g in got)


def test_equal_lengths_without_cu_seqlens_and_more_keys():
    """Dense batches: q [B, T, ..] with k, v [B, S, ..], S more and less than T."""
    for B, T, S in ((3, 130, 300), (2, 200, 50), (40, 3, 3)):
        q, k, v = make(B * T, B * S, 2, 1, 128, 128, B)
        o, lse = kda.attn_prompt(q.unflatten(0, (B, T)), k.unflatten(0, (B, S)), v.unflatten(0, (B, S)), return_lse=True)
        verify(o.flatten(0, 1), lse.flatten(0, 1), q, k, v, [T] * B, [S] * B)


def test_the_prompt_and_the_decode_agree():
    """The last row of a prompt against one decode step over the appended cache: the same attention but
    for the cache's 8 bits."""
    T, Hk, G, D, P = 333, 2, 4, 128, 32
    g = gen(12)
    r = lambda h: torch.randn((T, h, D), generator=g, device="cuda").bfloat16()
    q, k, v = r(Hk * G), r(Hk), r(Hk)
    f, _ = kda.rotary_inv_freq(D)
    pages = -(-T // P)
    cache = kda.kv_cache(pages, Hk, D, P)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).int()[None].cuda()
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    qr, kr = kda.kv_append(k, v, cache, table, zero, cu_seqlens=cum([T]), inv_freq=f, q=q, return_k=True)
    o = kda.attn_prompt(qr, kr, v, out_dtype=torch.float32)
    d = kda.attn_decode(qr[-1:], cache, table, zero + T, out_dtype=torch.float32)
    for h in range(Hk):
        hs = slice(h * G, (h + 1) * G)
        _, _, av, size = ref.attend(ref.f64(qr[-1, hs]), ref.f64(kr[:, h]), ref.f64(v[:, h]), D ** -0.5, [T] * G)
        off = (ref.HALF_E4M3 + ref.HALF_BF16) * size
        ref.check(f"head {h}", d[0, hs], ref.f64(o[-1, hs]),
                  ((torch.exp(2 * off) - 1)[:, None] + ref.HALF_E4M3 + 2 * ref.HALF_BF16) * av)


def test_refusals():
    q, k, v = make(10, 10, 4, 2, 64, 64, 13)
    cu = cum([10])
    bad = [(dict(q=q.float()), TypeError), (dict(k=k[:, :1]), ValueError), (dict(v=v[:5]), ValueError),
           (dict(cu_seqlens=cu.long()), TypeError), (dict(cu_seqlens=cu.cpu()), ValueError),
           (dict(cu_seqlens_k=cu), ValueError), (dict(scale=0.0), kda.KDAError), (dict(scale=float("inf")), kda.KDAError),
           (dict(q=q[:, :3].contiguous()), kda.KDAError), (dict(v=v[..., :32].contiguous()), kda.KDAError),
           (dict(out_dtype=torch.float16), TypeError), (dict(q=q[:7], cu_seqlens=cum([7])), kda.KDAError),
           (dict(q=q[None]), ValueError)]
    for over, err in bad:
        a = dict(q=q, k=k, v=v)
        a.update(over)
        with pytest.raises(err):
            kda.attn_prompt(a.pop("q"), a.pop("k"), a.pop("v"), **a)
    with pytest.raises(kda.KDAError):
        kda.attn_prompt(q, k, v, o=q)  # o over q
