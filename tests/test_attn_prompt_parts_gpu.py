"""GPU tests of the prompt's attention where it divides each row's keys among several CTAs (few rows and
heads): against 64-bit attention, with the tolerance of the form in one go plus the joining's."""
import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda
from tests import attn_reference as ref
from tests.test_attn_prompt_gpu import DIMS, cum, make, verify

pytestmark = pytest.mark.gpu
EDGES = [0, 1, 127, 128, 129, 255, 256, 257, 500, 511, 512, 640, 999, 1000, 1023, 1407, 2000, 2047, 2999, 4095]


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


def size(q, k, v, n=1):
    return kda.attn_prompt_workspace_size(q.shape[0], k.shape[0], q.shape[1], k.shape[1], v.shape[2], n)


def test_where_it_divides():
    few = kda.attn_prompt_workspace_size(4096, 4096, 2, 1, 128)
    assert few > 0 and few % (256 * 130 * 4) == 0 and few < 128 << 20
    assert kda.attn_prompt_workspace_size(256, 8192, 8, 8, 128) > 0      # a chunk behind a long context
    assert kda.attn_prompt_workspace_size(8192, 8192, 32, 8, 128) == 0   # work items enough
    assert kda.attn_prompt_workspace_size(100, 100, 1, 1, 64) == 0       # one block of keys


@pytest.mark.parametrize("D,DV", DIMS)
@pytest.mark.parametrize("Hq,Hk", [(2, 1), (1, 1), (3, 3)])
@pytest.mark.parametrize("T", [300, 1000, 4096])
def test_one_prompt(D, DV, Hq, Hk, T):
    q, k, v = make(T, T, Hq, Hk, D, DV, T + Hq)
    assert (size(q, k, v) > 0) == (T > 300)  # three blocks of keys are not worth a second launch
    o, lse = kda.attn_prompt(q, k, v, return_lse=True)
    verify(o, lse, q, k, v, [T], [T], rows=EDGES)
    whole, wl = kda.attn_prompt(q, k, v, return_lse=True, workspace=None)
    verify(whole, wl, q, k, v, [T], [T], rows=EDGES)
    again = kda.attn_prompt(q, k, v)
    assert torch.equal(again, o)  # the parts are joined in their order


@pytest.mark.parametrize("D,DV", DIMS)
@pytest.mark.parametrize("nq,nk", [(1, 5000), (17, 3000), (200, 2177), (129, 129), (700, 300)])
def test_a_chunk_behind_a_context(D, DV, nq, nk):
    """Few queries and many keys; more queries than keys: rows that see nothing."""
    q, k, v = make(nq, nk, 4, 2, D, DV, nq + nk)
    o, lse = kda.attn_prompt(q, k, v, cu_seqlens=cum([nq]), cu_seqlens_k=cum([nk]), return_lse=True)
    verify(o, lse, q, k, v, [nq], [nk], rows=EDGES + [nq - 1])


@pytest.mark.parametrize("D,DV", DIMS)
@pytest.mark.parametrize("long,divides", [(1000, False), (4000, True)])
def test_ragged_batches(D, DV, long, divides):
    """Lengths far from their mean, empty sequences, more parts than a sequence has key blocks."""
    nq, nk = [long, 0, 3, 129, 500, 40], [long, 7, 2000, 129, 450, 40]
    q, k, v = make(sum(nq) + 9, sum(nk), 2, 2, D, DV, 5)
    assert (size(q, k, v, len(nq)) > 0) == divides
    o = torch.full((q.shape[0], 2, DV), 5.0, dtype=torch.bfloat16, device="cuda")
    o, lse = kda.attn_prompt(q, k, v, cu_seqlens=cum(nq), cu_seqlens_k=cum(nk), o=o, return_lse=True)
    assert (o[sum(nq):] == 5).all()  # rows of no sequence
    verify(o, lse, q, k, v, nq, nk, rows=EDGES)


def test_fp32_outputs_and_large_scores():
    """Scores of some hundreds: the parts' maxima lie far apart."""
    q, k, v = make(1500, 1500, 2, 1, 128, 128, 6, sharp=40.0)
    o, lse = kda.attn_prompt(q, k, v, out_dtype=torch.float32, return_lse=True)
    verify(o, lse, q, k, v, [1500], [1500], rows=EDGES)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_what_a_row_does_not_see(bad):
    """A value that is not finite, in the middle of a block: rows before it stay right, those behind it
    are NaN or infinite, whichever part sees it."""
    T, at = 2000, 900
    q, k, v = make(T, T, 2, 1, 64, 64, 7)
    assert size(q, k, v) > 0
    clean = v.clone()
    v[at, 0, 3] = bad
    o = kda.attn_prompt(q, k, v)
    verify(o[:at], None, q[:at], k[:at], clean[:at], [at], [at], rows=[0, 500, 767, 768, 769, 895, 896, 897, 899])
    assert not torch.isfinite(o[at:, :, 3]).any()
    k[at, 0, 3] = bad  # a key: its scores' rows are NaN where they see it
    o = kda.attn_prompt(q, k, clean)
    verify(o[:at], None, q[:at], k[:at], clean[:at], [at], [at], rows=[0, 500, 767, 768, 769, 895, 896, 897, 899])
    if bad != bad:
        assert torch.isnan(o[at:]).all()


def test_captured_with_its_workspace_and_on_two_streams():
    x, y = make(3000, 3000, 2, 1, 128, 128, 8), make(1111, 1111, 1, 1, 192, 128, 9)
    want = [kda.attn_prompt(*x), kda.attn_prompt(*y)]
    graphs, outs = [], []
    for a in (x, y, x):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(kda.attn_prompt(*a))
        graphs.append(g)
    given = torch.empty(size(*x), dtype=torch.uint8, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, i in zip(streams, (0, 1)):
            with torch.cuda.stream(st):
                graphs[i].replay()
        with torch.cuda.stream(streams[0]):
            mine = kda.attn_prompt(*x, workspace=given)
            graphs[2].replay()
    torch.cuda.synchronize()
    for o, w in zip((*outs, mine), (want[0], want[1], want[0], want[0])):
        assert torch.equal(o, w)


def test_refusals():
    q, k, v = make(1000, 1000, 2, 1, 64, 64, 10)
    need = size(q, k, v)
    with pytest.raises(kda.KDAError):
        kda.attn_prompt(q, k, v, workspace=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        kda.attn_prompt(q, k, v, workspace=torch.empty(need, dtype=torch.uint8))
    with pytest.raises(ValueError):
        kda.attn_prompt(q, k, v, workspace="mine")
    raw = torch.empty(q.numel() * 2 + need, dtype=torch.uint8, device="cuda")
    o = raw[:q.numel() * 2].view(torch.bfloat16).view(q.shape)
    with pytest.raises(kda.KDAError):  # the workspace begins within o
        kda.attn_prompt(q, k, v, o=o, workspace=raw[q.numel() * 2 - 1024:][:need])


def test_after_a_wait_that_gave_up():
    q, k, v = make(2000, 2000, 2, 1, 128, 128, 11)
    want = kda.attn_prompt(q, k, v)
    kda.device_status()
    kda.set_wait_limit(0)
    try:
        o, lse = kda.attn_prompt(q, k, v, return_lse=True)
        with pytest.raises(kda.KDAError):
            kda.device_status()
    finally:
        kda.set_wait_limit(None)
    assert torch.isnan(o).all() and torch.isnan(lse).all()
    assert torch.equal(kda.attn_prompt(q, k, v), want)
