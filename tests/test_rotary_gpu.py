"""GPU tests of the rotary positions (kda_rotary) against the 64-bit rotation.  Tolerance: the
fp32 roundings of the rotation (ROTARY_ROUNDINGS half steps of |a| + |b|) plus, for bf16, one
rounding of the result."""
import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda
from tests import attn_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


def make(T, H, D, dtype, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((T, H, D), generator=g, device="cuda").to(dtype)


def verify(y, x, pos, f, mag, layout, inverse):
    want = ref.rotary(ref.f64(x), pos.cpu(), f.cpu(), mag, layout, inverse)
    R = 2 * f.numel()
    tol = ref.ROTARY_ROUNDINGS * ref.HALF_F32 * ref.rotary_size(ref.f64(x), R, abs(mag), layout)
    if x.dtype == torch.bfloat16:
        tol = tol + ref.HALF_BF16 * want.abs()
    ref.check("rotary", y, want, tol)
    assert torch.equal(y[..., R:], x[..., R:])


@pytest.mark.parametrize("T,H,D,R", [(1, 1, 64, 64), (1, 96, 128, 128), (7, 3, 64, 32), (33, 5, 192, 64),
                                     (130, 2, 256, 256), (257, 12, 64, 16), (19, 4, 40, 16), (300, 33, 128, 96)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_shapes(T, H, D, R, layout, dtype):
    x = make(T, H, D, dtype)
    f, mag = kda.rotary_inv_freq(R)
    pos = (torch.arange(T, device="cuda") * 37 % 5003).int()
    verify(kda.rotary(x, pos, f, magnitude=mag, layout=layout), x, pos, f, mag, layout, False)


@pytest.mark.parametrize("scaling", [None, "linear", "ntk", "yarn"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions(scaling, layout):
    """Positions up to 2^31 - 1 and negative ones.  The double frequency's own rounding moves the
    angle by position * frequency * 2^-52 at most, 1e-6 at 2^31; at 2^20 nothing shows."""
    pos = torch.tensor([0, 1, 1048575, 1048576, 999983, -1, -70001], dtype=torch.int32, device="cuda")
    x = make(pos.numel(), 2, 128, torch.float32, 1)
    f, mag = kda.rotary_inv_freq(128, scaling=scaling, factor=8.0)
    verify(kda.rotary(x, pos, f, magnitude=mag, layout=layout), x, pos, f, mag, layout, False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_inverse_strides_and_in_place(dtype):
    """A slice of a fused projection, turned in place and back; its neighbours stay as they are."""
    T, H, D, R = 45, 4, 128, 64
    fused = make(T, H + 3, D, dtype, 2).view(T, (H + 3) * D)
    before = fused.clone()
    x = fused[:, D:(H + 1) * D].unflatten(1, (H, D))
    pos = torch.randint(0, 100000, (T,), dtype=torch.int32, device="cuda")
    f, _ = kda.rotary_inv_freq(R)
    y = kda.rotary(x, pos, f, out=x)
    assert y.data_ptr() == x.data_ptr()
    orig = before[:, D:(H + 1) * D].unflatten(1, (H, D))
    verify(x, orig, pos, f, 1.0, "half", False)
    assert torch.equal(fused[:, :D], before[:, :D]) and torch.equal(fused[:, (H + 1) * D:], before[:, (H + 1) * D:])
    back = kda.rotary(orig, pos, f, inverse=True, magnitude=1.5)
    verify(back, orig, pos, f, 1.5, "half", True)


def test_the_inverse_is_the_gradient():
    """sum(rotate(x) * w) changes along a direction by sum(inverse(w) * direction)."""
    x, w, d = (make(9, 2, 64, torch.float32, s) for s in (3, 4, 5))
    pos = torch.randint(0, 5000, (9,), dtype=torch.int32, device="cuda")
    f, _ = kda.rotary_inv_freq(64)
    turn = lambda t, **k: kda.rotary(t, pos, f, magnitude=1.25, **k).double()
    want = ((turn(x + d) - turn(x - d)) / 2 * w.double()).sum()  # the map is linear
    got = (turn(w, inverse=True) * d.double()).sum()
    size = (w.double().abs() * d.double().abs()).sum() * 2 * 1.25
    assert abs(got - want) <= 4 * ref.ROTARY_ROUNDINGS * ref.HALF_F32 * size


def test_nan_and_infinity_stay_in_their_pair():
    x = make(3, 2, 64, torch.float32, 6)
    x[1, 0, 3] = float("nan")
    x[2, 1, 40] = float("inf")
    f, _ = kda.rotary_inv_freq(64)
    pos = torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")
    y = kda.rotary(x, pos, f)
    touched = torch.zeros_like(x, dtype=torch.bool)
    touched[1, 0, [3, 35]] = True
    touched[2, 1, [8, 40]] = True
    assert y[~touched].isfinite().all() and not y[touched].isfinite().any()


def test_no_tokens_and_host_tensors():
    f, _ = kda.rotary_inv_freq(64)
    assert kda.rotary(make(0, 2, 64, torch.float32), torch.zeros(0, dtype=torch.int32, device="cuda"), f).shape == (0, 2, 64)
    x = make(5, 2, 64, torch.float32, 7)
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    y = kda.rotary(x.cpu(), pos.cpu(), f.cpu())
    assert y.device.type == "cpu" and torch.equal(y, kda.rotary(x, pos, f).cpu())


def test_graph_replay_reads_the_new_inputs():
    x = make(17, 4, 128, torch.bfloat16, 8)
    pos = torch.arange(17, dtype=torch.int32, device="cuda")
    f, _ = kda.rotary_inv_freq(128)
    out = torch.empty_like(x)
    kda.rotary(x, pos, f, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.rotary(x, pos, f, out=out)
    x.copy_(make(17, 4, 128, torch.bfloat16, 9))
    pos.add_(1000)
    graph.replay()
    torch.cuda.synchronize()
    verify(out, x, pos, f, 1.0, "half", False)


def test_refusals():
    f, _ = kda.rotary_inv_freq(64)
    x, pos = make(4, 2, 64, torch.float32), torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        kda.rotary(x, pos[:3], f)
    with pytest.raises(ValueError):
        kda.rotary(x, pos, f, layout="pairs")
    with pytest.raises(TypeError):
        kda.rotary(x.half(), pos, f)
    with pytest.raises(TypeError):
        kda.rotary(x, pos.long(), f)
    with pytest.raises(TypeError):
        kda.rotary(x, pos, f.float())
    with pytest.raises(kda.KDAError):
        kda.rotary(x, pos, torch.cat([f, f]))  # more channels than the head has
    with pytest.raises(kda.KDAError):
        kda.rotary(x, pos, f[:5].contiguous())  # not a multiple of 16 channels
    with pytest.raises(kda.KDAError):
        kda.rotary(x[:3], pos[:3], f, out=x[1:])  # a partial overlap
