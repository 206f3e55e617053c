"""GPU tests of the latent rows' norm at the upper end of bf16, where the squares' sum overflows fp32 unless the row is
scaled far enough.  Tolerance: as in tests/test_latent_rows_gpu.py."""
import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda
from tests.test_latent_rows_gpu import C, ROW, append_case, cum, want_rows
from tests import attn_reference as ref
from tests.test_kv_append_gpu import gen

pytestmark = pytest.mark.gpu
MOST = torch.finfo(torch.bfloat16).max


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


@pytest.mark.parametrize("scale", [1e35, 5e36, 2e37, 7e37])
@pytest.mark.parametrize("eps", [1e-5, 1.0, 1e30])
def test_large_rows(scale, eps):
    append_case([20], [5], 16, turned=0, scale=scale, eps=eps, seed=2)


@pytest.mark.parametrize("width", [1, 2, 3, 8, 100, C])
def test_rows_of_the_largest_value(width):
    """`width` channels at bf16's largest, the others from nothing to far below."""
    g = gen(width)
    x = torch.zeros((4, ROW), device="cuda")
    x[1:, :C] = torch.randn((3, C), generator=g, device="cuda") * torch.tensor([1.0, 1e20, 1e34], device="cuda")[:, None]
    x[:, torch.randperm(C, generator=g, device="cuda")[:width]] = MOST
    x = x.bfloat16()
    w = 1 + 0.1 * torch.randn(C, generator=g, device="cuda")
    rows = kda.latent_append(x, kda.latent_cache(1, 16), torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                             torch.zeros(1, dtype=torch.int32, device="cuda"), cu_seqlens=cum([4]), norm_w=w, return_rows=True)
    want, tol = want_rows(x, torch.arange(4), w, 1e-5, None, 1.0, "half")
    ref.check("rows", rows, want, tol)
