"""GPU tests of masked values that are not finite in the prompt's attention (kda_attn_prompt): they spoil
the products of the rows in whose blocks they lie, which are then computed alone.  Tolerances as in
test_attn_prompt_gpu.py."""
import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda
from tests.test_attn_prompt_gpu import DIMS, cum, make, verify

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


@pytest.mark.parametrize("workspace", ["auto", None])
@pytest.mark.parametrize("bad", [float("nan"), float("-inf")])
@pytest.mark.parametrize("Hq,Hk,D,DV", [(2, 1, 64, 64), (1, 1, 128, 128), (4, 2, 192, 128)])
def test_rows_of_a_long_context(Hq, Hk, D, DV, bad, workspace):
    """Rows that see 60000 keys each, beside finite sequences: no wait of any warp runs out meanwhile, and
    what does not see the value keeps its bits."""
    nq, nk = [40, 200, 30], [40, 60000, 400]
    q, k, v = make(sum(nq), sum(nk), Hq, Hk, D, DV, 41)
    call = lambda x: kda.attn_prompt(q, k, x, cu_seqlens=cum(nq), cu_seqlens_k=cum(nk), return_lse=True, workspace=workspace)
    o, lse = call(v)
    at = nk[0] + nk[1] - 3  # the long sequence's third last key: only its last three queries see it
    v2 = v.clone()
    v2[at, Hk - 1, 7] = bad
    o2, lse2 = call(v2)
    kda.device_status()
    assert torch.equal(lse2, lse)
    G, end = Hq // Hk, nq[0] + nq[1]
    sees = torch.zeros_like(o, dtype=torch.bool)
    sees[end - 3:end, Hq - G:, 7] = True
    assert not o2[sees].isfinite().any()
    same = ~sees
    same[nq[0]:end, Hq - G:, 7] = False  # computed alone
    assert torch.equal(o2[same], o[same])
    verify(o2[nq[0]:end - 3], lse2[nq[0]:end - 3], q[nq[0]:end - 3], k[nk[0]:at], v[nk[0]:at], [nq[1] - 3], [nk[1] - 3],
           rows=[0, 1, 71, 72, 100, 195, 196], heads=[Hq - 1])


@pytest.mark.parametrize("D,DV", DIMS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_padded_sequence(D, DV, bad):
    """Every value behind the valid part: the rows before it stand, those behind it see one."""
    T, valid = 4000, 2100
    q, k, v = make(2 * T, 2 * T, 8, 4, D, DV, 42)
    split = lambda t: t.unflatten(0, (2, T))
    o, lse = kda.attn_prompt(split(q), split(k), split(v), return_lse=True)
    v2 = v.clone()
    v2[valid:T] = bad
    o2, lse2 = kda.attn_prompt(split(q), split(k), split(v2), return_lse=True)
    kda.device_status()
    assert torch.equal(lse2, lse) and torch.equal(o2[1], o[1]) and torch.equal(o2[0, :2048], o[0, :2048])
    assert not o2[0, valid:].isfinite().any()
    verify(o2[0, :valid], None, q[:valid], k[:valid], v[:valid], [valid], [valid], rows=[2047, 2048, 2049, 2099], heads=[0, 7])


def test_several_values_in_the_tile_and_rows_that_see_none():
    """Values of both infinities and NaN on both sides of a row; more queries than keys, so that the
    first rows see nothing and are zero."""
    nq, nk = 300, 200
    q, k, v = make(nq, nk, 2, 1, 64, 64, 43)
    v[10, 0, 0], v[50, 0, 0], v[60, 0, 1], v[199, 0, 2] = float("inf"), float("-inf"), float("nan"), float("inf")
    for ws in ("auto", None):
        o = kda.attn_prompt(q, k, v, cu_seqlens=cum([nq]), cu_seqlens_k=cum([nk]), workspace=ws).float()
        assert (o[:100] == 0).all()
        assert o[100:110].isfinite().all()
        assert (o[110:150, :, 0] == float("inf")).all() and o[150:, :, 0].isnan().all()
        assert o[:160, :, 1].isfinite().all() and o[160:, :, 1].isnan().all()
        assert o[:299, :, 2].isfinite().all() and (o[299, :, 2] == float("inf")).all()
        clean = v.nan_to_num(0.0, 0.0, 0.0)
        verify(o[:110].bfloat16(), None, q[:110], k[:10], clean[:10], [110], [10])
        assert o[..., 3:].isfinite().all()


@pytest.mark.parametrize("scale", [None, -0.3])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_scales_and_types(scale, out):
    """Rows computed alone with a negative scale and fp32 outputs, whole and in parts."""
    T, at = 700, 650
    q, k, v = make(T, T, 2, 1, 128, 128, 44)
    clean = v.clone()
    v[at, 0, 100] = float("nan")
    for ws in ("auto", None):
        o, lse = kda.attn_prompt(q, k, v, return_lse=True, scale=scale, out_dtype=out, workspace=ws)
        verify(o[:at], lse[:at], q[:at], k[:at], clean[:at], [at], [at], scale, rows=[0, 511, 512, 513, 600, 639, 640, 649])
        assert o[at:, :, 100].isnan().all() and o[at:, :, :100].isfinite().all()
    kda.device_status()
