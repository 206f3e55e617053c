"""GPU tests of single-token attention in the form that cuts the sequences' steps into pieces and
joins them (kda_attn_decode with a block table that holds many tokens), which needs a workspace.
Tolerances as in test_attn_decode_gpu.py."""
import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda
from tests.test_attn_decode_gpu import gen, verify
from tests.test_kv_append_gpu import filled_cache, table_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


@pytest.mark.parametrize("P", [16, 32, 128])
@pytest.mark.parametrize("D,Hk,G", [(128, 2, 4), (64, 1, 16)])
def test_each_step_takes_its_own_pages_scales(D, Hk, G, P):
    """Pages' scales are powers of two apart, so a step that read another step's scales would be off
    by far more than a rounding.  The same bits every time."""
    lens = [1000, 33, 16 * 37 + 1]
    table, pages = table_for(lens, P, 31)
    cache = filled_cache(pages, Hk, P, D, 31, (-12, -4))
    q = torch.randn((len(lens), Hk * G, D), generator=gen(32), device="cuda").bfloat16()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    dt = table.cuda()
    assert kda.attn_decode_workspace_size(len(lens), Hk * G, Hk, D, dt.shape[1] * P) > 0
    o, lse = kda.attn_decode(q, cache, dt, sl, return_lse=True)
    verify(o, lse, q, cache, table, lens)
    for _ in range(20):
        again = kda.attn_decode(q, cache, dt, sl, return_lse=True)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
