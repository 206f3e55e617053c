"""CPU checks of the full-attention entry points of the C ABI: bad arguments are refused on the host
with a defined status before anything is launched.  The device pointers are fake aligned
addresses that validation never dereferences."""
import ctypes
import math

import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 2
BF16, F32 = 0, 1
FAKE = 0x10000000
SPAN = 1 << 26  # fake tensors of one call lie this far apart


def fake(i):
    return FAKE + i * SPAN


@pytest.fixture(scope="module")
def lib():
    from kimi_delta_attention_gated_gb300 import build as b
    b.build()
    from kimi_delta_attention_gated_gb300 import _load
    return _load()


def rotary(lib, **over):
    a = dict(x=fake(0), dt=BF16, xs=512, pos=fake(1), f=fake(2), mag=1.0, R=64, lay=0, inv=0, out=fake(3), os=512, T=8,
             H=4, D=128)
    a.update(over)
    return lib.kda_rotary(*(a[k] for k in ("x", "dt", "xs", "pos", "f", "mag", "R", "lay", "inv", "out", "os", "T", "H",
                                           "D")), None)


@pytest.mark.parametrize("over,code", [
    (dict(x=None), INVALID), (dict(pos=None), INVALID), (dict(out=None), INVALID), (dict(f=None), INVALID),
    (dict(dt=5), UNSUPPORTED), (dict(D=132, xs=528, os=528), UNSUPPORTED), (dict(D=264, xs=1056, os=1056), UNSUPPORTED),
    (dict(R=0), INVALID), (dict(R=24), UNSUPPORTED), (dict(R=144), INVALID), (dict(lay=2), INVALID), (dict(inv=2), INVALID),
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(xs=511), INVALID), (dict(xs=516), INVALID), (dict(os=100), INVALID),
    (dict(x=fake(0) + 8), INVALID), (dict(pos=fake(1) + 2), INVALID), (dict(f=fake(2) + 4), INVALID),
    (dict(mag=float("inf")), INVALID), (dict(out=fake(0) + 1024), INVALID), (dict(out=fake(0), os=1024), INVALID),
    (dict(out=fake(2)), INVALID), (dict(T=1 << 32), UNSUPPORTED),
])
def test_rotary_refuses(lib, over, code):
    assert rotary(lib, **over) == code
    assert lib.kda_last_error()


def test_no_tokens_launch_nothing(lib):
    before = lib.kda_launch_count()
    assert rotary(lib, T=0, x=None, out=None, pos=None) == OK
    assert append(lib, T=0, N=0, k=None, v=None) == OK
    assert decode(lib, N=0, q=None, o=None) == OK
    assert prompt(lib, Tq=0, Tk=0, N=0, q=None, k=None, v=None, o=None) == OK
    assert lib.kda_launch_count() == before


def append(lib, **over):
    a = dict(k=fake(0), ks=256, v=fake(1), vs=256, T=6, Hk=2, D=128, kc=fake(2), vc=fake(3), kscale=fake(4),
             vscale=fake(5), pages=10, P=16, bt=fake(6), mb=4, ctx=fake(7), cu=fake(8), N=3, f=fake(9), mag=1.0, R=128,
             lay=0, q=None, qs=0, Hq=0, qo=None, ko=None)
    a.update(over)
    return lib.kda_kv_append(*(a[k] for k in ("k", "ks", "v", "vs", "T", "Hk", "D", "kc", "vc", "kscale", "vscale", "pages",
                                              "P", "bt", "mb", "ctx", "cu", "N", "f", "mag", "R", "lay", "q", "qs", "Hq",
                                              "qo", "ko")), None)


@pytest.mark.parametrize("over,code", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(kc=None), INVALID), (dict(vscale=None), INVALID),
    (dict(bt=None), INVALID), (dict(ctx=None), INVALID), (dict(D=96, ks=192, vs=192), UNSUPPORTED), (dict(P=24), UNSUPPORTED),
    (dict(P=256), UNSUPPORTED), (dict(Hk=0), INVALID), (dict(pages=0), INVALID), (dict(mb=0), INVALID), (dict(T=-1), INVALID),
    (dict(cu=None), INVALID),                              # one token per sequence needs tokens == n_seqs
    (dict(N=0), INVALID), (dict(N=70000), UNSUPPORTED), (dict(ks=200), INVALID), (dict(vs=257), INVALID),
    (dict(f=None), INVALID), (dict(R=0), INVALID), (dict(R=130), INVALID), (dict(R=40), UNSUPPORTED),
    (dict(q=fake(10)), INVALID),                           # q without q_out
    (dict(q=fake(10), qo=fake(11), Hq=0, qs=256), INVALID), (dict(q=fake(10), qo=fake(11), Hq=3, qs=384), INVALID),
    (dict(q=fake(10), qo=fake(11), Hq=4, qs=500), INVALID), (dict(kc=fake(2) + 8), INVALID), (dict(bt=fake(6) + 2), INVALID),
    (dict(ko=fake(0)), INVALID), (dict(kc=fake(1)), INVALID), (dict(kc=fake(3) + 4096), INVALID), (dict(kscale=fake(7)), INVALID),
    (dict(pages=1 << 30, P=128), UNSUPPORTED), (dict(mb=1 << 30), INVALID),
])
def test_append_refuses(lib, over, code):
    assert append(lib, **over) == code
    assert lib.kda_last_error()


def decode(lib, **over):
    a = dict(q=fake(0), qs=512, kc=fake(1), vc=fake(2), ks=fake(3), vs=fake(4), pages=10, P=64, bt=fake(5), mb=40, lens=fake(6),
             N=2, Hq=4, Hk=2, D=128, scale=0.1, o=fake(7), dt=BF16, lse=fake(8), ws=fake(9), wsb=1 << 25)
    a.update(over)
    return lib.kda_attn_decode(*(a[k] for k in ("q", "qs", "kc", "vc", "ks", "vs", "pages", "P", "bt", "mb", "lens", "N", "Hq",
                                                "Hk", "D", "scale", "o", "dt", "lse", "ws", "wsb")), None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(kc=None), INVALID), (dict(lens=None), INVALID),
    (dict(D=192, qs=768), UNSUPPORTED), (dict(P=8), UNSUPPORTED), (dict(Hq=5, qs=640), INVALID), (dict(Hq=0), INVALID),
    (dict(dt=4), UNSUPPORTED), (dict(scale=float("nan")), INVALID), (dict(qs=100), INVALID), (dict(q=fake(0) + 4), INVALID),
    (dict(lse=fake(8) + 1), INVALID), (dict(ws=None), INVALID), (dict(ws=fake(9) + 8), INVALID), (dict(o=fake(0)), INVALID),
    (dict(lse=fake(7)), INVALID), (dict(ws=fake(1)), INVALID), (dict(N=-1), INVALID), (dict(pages=1 << 28, P=128), UNSUPPORTED),
])
def test_decode_refuses(lib, over, code):
    assert decode(lib, **over) == code
    assert lib.kda_last_error()


def test_decode_workspace(lib):
    size = lib.kda_attn_decode_workspace_size
    assert size(0, 4, 2, 128, 100) == 0 and size(2, 5, 2, 128, 100) == 0 and size(2, 4, 2, 96, 100) == 0
    assert size(-1, 4, 2, 128, 100) == 0 and size(2, 4, 2, 128, -1) == 0
    assert size(1, 4, 2, 128, 64) == 0               # few tokens: nothing is joined
    large = size(64, 4, 2, 128, 100000)
    assert large > 0
    assert size(1000, 4, 2, 128, 1000000) == size(2000, 4, 2, 128, 1000000)  # as many pieces as the GPU holds at once
    need = size(2, 4, 2, 128, 100 * 64)
    assert decode(lib, mb=100, wsb=need - 1) == INVALID


def prompt(lib, **over):
    a = dict(q=fake(0), qs=512, k=fake(1), ks=256, v=fake(2), vs=256, Tq=8, Tk=8, Hq=4, Hk=2, D=128, DV=128, cu=fake(3),
             cuk=None, N=2, scale=0.1, o=fake(4), dt=BF16, lse=fake(5), ws=None, wsb=0)
    a.update(over)
    return lib.kda_attn_prompt(*(a[k] for k in ("q", "qs", "k", "ks", "v", "vs", "Tq", "Tk", "Hq", "Hk", "D", "DV", "cu", "cuk",
                                                "N", "scale", "o", "dt", "lse", "ws", "wsb")), None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(o=None), INVALID),
    (dict(ws=fake(7) + 4), INVALID),
    (dict(D=192), INVALID),                                # 192/128 is built; the strides do not fit it
    (dict(D=64), UNSUPPORTED), (dict(DV=64), UNSUPPORTED), (dict(D=96, DV=96), UNSUPPORTED), (dict(Hq=3), INVALID),
    (dict(Hq=0), INVALID), (dict(Tq=-1), INVALID), (dict(Tk=9), INVALID), (dict(cu=None, cuk=fake(6)), INVALID),
    (dict(cu=None, N=3), INVALID), (dict(N=0), INVALID), (dict(N=20000), UNSUPPORTED), (dict(scale=0.0), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(dt=3), UNSUPPORTED), (dict(qs=511), INVALID), (dict(vs=100), INVALID),
    (dict(k=fake(1) + 2), INVALID), (dict(cu=fake(3) + 1), INVALID), (dict(o=fake(2)), INVALID), (dict(lse=fake(4)), INVALID),
    (dict(Tq=1 << 31, Tk=1 << 31), UNSUPPORTED),
])
def test_prompt_refuses(lib, over, code):
    assert prompt(lib, **over) == code
    assert lib.kda_last_error()


def test_prompt_workspace(lib):
    size = lib.kda_attn_prompt_workspace_size
    for bad in ((0, 8, 4, 2, 128, 1), (8, -1, 4, 2, 128, 1), (8, 8, 5, 2, 128, 1), (8, 8, 4, 2, 96, 1), (8, 8, 4, 2, 128, 0)):
        assert size(*bad) == 0
    assert size(100, 100, 8, 2, 64, 1) == 0          # one block of keys
    assert size(8192, 8192, 32, 8, 128, 1) == 0      # work items enough
    assert size(5, 5, 1, 1, 64, 10) == 0             # fewer rows than sequences


def test_inv_freq_scalings():
    """Against the formulas, number by number."""
    from kimi_delta_attention_gated_gb300 import rotary_inv_freq
    R, s = 64, 8.0
    base = [10000.0 ** (-2 * i / R) for i in range(R // 2)]
    f, m = rotary_inv_freq(R, device="cpu")
    assert m == 1.0 and torch.allclose(f, torch.tensor(base, dtype=torch.float64), rtol=1e-15)
    f, m = rotary_inv_freq(R, scaling="linear", factor=s, device="cpu")
    assert m == 1.0 and torch.allclose(f, torch.tensor([b / s for b in base], dtype=torch.float64), rtol=1e-15)
    f, m = rotary_inv_freq(R, scaling="ntk", factor=s, device="cpu")
    assert math.isclose(f[-1].item(), base[-1] / s, rel_tol=1e-12) and f[0] == 1.0
    f, m = rotary_inv_freq(R, scaling="yarn", factor=s, original_max_position=4096, device="cpu")
    assert math.isclose(m, 0.1 * math.log(s) + 1)
    for i, b in enumerate(base):
        turns = 4096 * b / (2 * math.pi)
        want = b if turns >= 32 else b / s if turns <= 1 else b * (turns - 1) / 31 + b / s * (1 - (turns - 1) / 31)
        assert math.isclose(f[i].item(), want, rel_tol=1e-12)
    for bad in (dict(rotary_dim=63), dict(rotary_dim=0), dict(rotary_dim=64, factor=0.5), dict(rotary_dim=64, scaling="x"),
                dict(rotary_dim=64, scaling="yarn", beta_fast=1.0, beta_slow=1.0)):
        with pytest.raises(ValueError):
            rotary_inv_freq(device="cpu", **bad)


def test_python_refuses_host_caches():
    import kimi_delta_attention_gated_gb300 as kda
    cache = kda.kv_cache(2, 1, 64, 16, device="cpu")
    x = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.kv_append(x, x, cache, i[None], i)
    with pytest.raises(ValueError):
        kda.attn_decode(x, cache, i[None], i)
