"""Plain 64-bit references of the full-attention operators, on the host: rotary positions, the
paged 8-bit cache and attention.  Loops over sequences and tokens, no code of the library."""
import math

import numpy as np
import torch

HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2  # a rounding's largest relative error
HALF_F16 = torch.finfo(torch.float16).eps / 2
HALF_F32 = torch.finfo(torch.float32).eps / 2
HALF_E4M3 = torch.finfo(torch.float8_e4m3fn).eps / 2


def f64(t):
    return t.detach().to("cpu").double() if not t.dtype.itemsize == 1 else t.detach().to("cpu").float().double()


def rotary(x, positions, inv_freq, magnitude=1.0, layout="half", inverse=False):
    """x [T, H, D] float64; pair by pair."""
    x = x.clone()
    R = 2 * inv_freq.numel()
    for i in range(R // 2):
        a, b = (i, i + R // 2) if layout == "half" else (2 * i, 2 * i + 1)
        w = positions.double() * inv_freq[i].double()
        c, s = (torch.cos(w) * magnitude)[:, None], (torch.sin(w) * magnitude)[:, None]
        if inverse:
            s = -s
        xa, xb = x[..., a].clone(), x[..., b].clone()
        x[..., a], x[..., b] = xa * c - xb * s, xa * s + xb * c
    return x


def rotary_size(x, R, magnitude, layout):
    """|a| + |b| of each channel's pair times the magnitude (the channel's own size where it is not
    rotated): what the rotation's rounding errors are relative to."""
    y = x.abs().clone()
    h = R // 2
    if layout == "half":
        s = (y[..., :h] + y[..., h:R]) * magnitude
        y[..., :h], y[..., h:R] = s, s
    else:
        s = (y[..., 0:R:2] + y[..., 1:R:2]) * magnitude
        y[..., 0:R:2], y[..., 1:R:2] = s, s
    return y


# cos and sin: the angle's two roundings (pi / 4 * 2 halves), about two in the series; one for the
# magnitude; one and a half in the difference of products
ROTARY_ROUNDINGS = 8


def to_e4m3(x):
    """Nearest e4m3 value of x (|x| <= 448), ties to even."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(x)
    step = np.exp2(np.maximum(e - 4, -9).astype(np.float64))
    return np.round(x / step) * step


def attend(q, k, v, scale, seen):
    """q [n, D], k [L, D], v [L, DV], row i sees the first seen[i] keys (none: zero, lse -inf).
    Returns (o, lse, weighted |v|, largest sum |q||k| * scale of a row's scores)."""
    n, L = q.shape[0], k.shape[0]
    o = torch.zeros((n, v.shape[1]), dtype=torch.float64)
    av, lse = o.clone(), torch.full((n,), -math.inf, dtype=torch.float64)
    size = torch.zeros(n, dtype=torch.float64)
    for i in range(n):
        m = int(min(max(int(seen[i]), 0), L))
        if m == 0:
            continue
        s = (k[:m] @ q[i]) * scale
        lse[i] = torch.logsumexp(s, 0)
        p = torch.exp(s - lse[i])
        o[i], av[i] = p @ v[:m], p @ v[:m].abs()
        size[i] = (k[:m].abs() @ q[i].abs()).max() * abs(scale)
    return o, lse, av, size


def check(name, got, want, tol):
    got = f64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    bad = ~(((got - want).abs() <= tol) | ((got == want)) | (got.isnan() & want.isnan()))
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {got[i].item()!r}, "
                             f"want {want[i].item()!r}, tolerance {torch.as_tensor(tol).expand_as(want)[i].item()!r}")
