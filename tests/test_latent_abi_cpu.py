"""CPU checks of the latent-attention entry points of the C ABI: bad arguments are refused on the host with a
defined status before anything is launched.  The device pointers are fake aligned addresses that
validation never dereferences."""
import pytest
import torch

from tests.test_attn_abi_cpu import BF16, F32, INVALID, OK, UNSUPPORTED, fake, lib  # noqa: F401


def append(lib, **over):
    a = dict(x=fake(0), xs=576, T=6, c=fake(1), pages=10, P=16, bt=fake(2), mb=4, ctx=fake(3), cu=fake(4), N=3, w=fake(5),
             eps=1e-5, f=fake(6), mag=1.0, R=64, lay=0, out=fake(7))
    a.update(over)
    return lib.kda_latent_append(*(a[k] for k in ("x", "xs", "T", "c", "pages", "P", "bt", "mb", "ctx", "cu", "N", "w", "eps",
                                                  "f", "mag", "R", "lay", "out")), None)


@pytest.mark.parametrize("over,code", [
    (dict(x=None), INVALID), (dict(c=None), INVALID), (dict(bt=None), INVALID), (dict(ctx=None), INVALID),
    (dict(xs=575), INVALID), (dict(xs=580), INVALID), (dict(T=-1), INVALID), (dict(T=(1 << 30) + 1), UNSUPPORTED),
    (dict(cu=None), INVALID),                              # one token per sequence needs tokens == n_seqs
    (dict(N=0), INVALID), (dict(N=-1), INVALID), (dict(N=70000), UNSUPPORTED), (dict(P=8), UNSUPPORTED),
    (dict(P=256), UNSUPPORTED), (dict(pages=0), INVALID), (dict(mb=0), INVALID), (dict(pages=1 << 28), UNSUPPORTED),
    (dict(mb=1 << 28), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(eps=1e-31), INVALID), (dict(f=None), INVALID), (dict(R=0), INVALID),
    (dict(R=80), INVALID), (dict(R=24), UNSUPPORTED), (dict(lay=2), INVALID), (dict(mag=float("nan")), INVALID),
    (dict(x=fake(0) + 8), INVALID), (dict(c=fake(1) + 2), INVALID), (dict(bt=fake(2) + 2), INVALID),
    (dict(cu=fake(4) + 1), INVALID), (dict(w=fake(5) + 2), INVALID), (dict(f=fake(6) + 4), INVALID),
    (dict(out=fake(7) + 8), INVALID), (dict(out=fake(0)), INVALID), (dict(c=fake(0) + 1152), INVALID),
    (dict(out=fake(1) + 1152), INVALID), (dict(c=fake(5)), INVALID), (dict(out=fake(3)), INVALID),
])
def test_append_refuses(lib, over, code):  # noqa: F811
    assert append(lib, **over) == code
    assert lib.kda_last_error()


def product(lib, what, **over):
    width = {"queries": 192, "values": 512, "expand": 576}[what]
    a = dict(x=fake(0), xs=width * (1 if what == "expand" else 4), T=8, H=4, w=fake(1), pos=fake(2), f=fake(3), mag=1.0, R=64, lay=0,
             out=fake(4), out2=fake(5))
    a.update(over)
    names = {"queries": ("x", "xs", "T", "H", "w", "pos", "f", "mag", "R", "lay", "out"), "values": ("x", "xs", "T", "H", "w", "out"),
             "expand": ("x", "xs", "T", "H", "w", "out", "out2")}[what]
    return getattr(lib, "kda_latent_" + what)(*(a[k] for k in names), None)


@pytest.mark.parametrize("what", ["queries", "values", "expand"])
@pytest.mark.parametrize("over,code", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(out=None), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID),
    (dict(H=5000, xs=1 << 22), UNSUPPORTED), (dict(T=(1 << 30) + 1), UNSUPPORTED), (dict(xs=100), INVALID),
    (dict(xs=(1 << 20) + 4), INVALID), (dict(x=fake(0) + 8), INVALID), (dict(w=fake(1) + 8), INVALID),
    (dict(out=fake(4) + 8), INVALID), (dict(out=fake(0)), INVALID), (dict(out=fake(1) + 16), INVALID),
])
def test_products_refuse(lib, what, over, code):  # noqa: F811
    assert product(lib, what, **over) == code
    assert lib.kda_last_error()


@pytest.mark.parametrize("over,code", [
    (dict(pos=None), INVALID), (dict(f=None), INVALID), (dict(R=0), INVALID), (dict(R=0, f=None), INVALID),
    (dict(R=128), INVALID), (dict(R=8), UNSUPPORTED), (dict(lay=-1), INVALID), (dict(pos=fake(2) + 2), INVALID),
    (dict(out=fake(2)), INVALID), (dict(out=fake(3)), INVALID),
])
def test_queries_refuse_positions(lib, over, code):  # noqa: F811
    assert product(lib, "queries", **over) == code
    assert lib.kda_last_error()


@pytest.mark.parametrize("over", [dict(out2=None), dict(out2=fake(5) + 4), dict(out2=fake(4) + 1024), dict(out2=fake(0))])
def test_expand_refuses_values(lib, over):  # noqa: F811
    assert product(lib, "expand", **over) == INVALID


def attn(lib, **over):
    a = dict(q=fake(0), qs=4 * 576, T=6, H=4, c=fake(1), pages=10, P=64, bt=fake(2), mb=40, lens=fake(3), cu=fake(4), N=3, scale=0.1,
             o=fake(5), dt=BF16, lse=fake(6), ws=fake(7), wsb=1 << 25)
    a.update(over)
    return lib.kda_attn_latent(*(a[k] for k in ("q", "qs", "T", "H", "c", "pages", "P", "bt", "mb", "lens", "cu", "N", "scale", "o",
                                                "dt", "lse", "ws", "wsb")), None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(c=None), INVALID), (dict(bt=None), INVALID), (dict(lens=None), INVALID),
    (dict(cu=None), INVALID), (dict(N=0), INVALID), (dict(N=70000), UNSUPPORTED), (dict(T=-1), INVALID),
    (dict(T=(1 << 24) + 1), UNSUPPORTED), (dict(H=0), INVALID), (dict(H=5000, qs=5000 * 576), UNSUPPORTED), (dict(P=24), UNSUPPORTED),
    (dict(pages=0), INVALID), (dict(mb=0), INVALID), (dict(pages=1 << 26), UNSUPPORTED), (dict(mb=1 << 26), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=1e31), INVALID),
    (dict(dt=3), UNSUPPORTED), (dict(qs=2303), INVALID), (dict(qs=2308), INVALID), (dict(q=fake(0) + 8), INVALID),
    (dict(c=fake(1) + 8), INVALID), (dict(lse=fake(6) + 2), INVALID), (dict(ws=fake(7) + 8), INVALID), (dict(ws=None), INVALID),
    (dict(wsb=16), INVALID), (dict(o=fake(0)), INVALID), (dict(o=fake(1)), INVALID), (dict(lse=fake(5)), INVALID),
    (dict(ws=fake(1)), INVALID), (dict(ws=fake(5)), INVALID), (dict(lse=fake(3)), INVALID),
])
def test_attn_refuses(lib, over, code):  # noqa: F811
    assert attn(lib, **over) == code
    assert lib.kda_last_error()


def test_no_tokens_launch_nothing(lib):  # noqa: F811
    before = lib.kda_launch_count()
    assert append(lib, T=0, N=0, x=None, out=None) == OK and append(lib, T=0, x=None) == OK
    assert product(lib, "queries", T=0, x=None, out=None, pos=None) == OK
    assert product(lib, "values", T=0, x=None, out=None) == OK
    assert product(lib, "expand", T=0, x=None, out=None, out2=None) == OK
    assert attn(lib, T=0, N=0, q=None, o=None, ws=None) == OK and attn(lib, T=0, q=None, o=None, ws=None) == OK
    assert lib.kda_launch_count() == before


def test_workspace(lib):  # noqa: F811
    size = lib.kda_attn_latent_workspace_size
    for bad in ((0, 1, 4, 100), (1, 0, 4, 100), (1, 1, 0, 100), (1, 1, 4, -1), (70000, 1, 4, 100), (1, 1 << 25, 4, 100),
                (1, 1, 5000, 100), (1, 1, 4, 1 << 31)):
        assert size(*bad) == 0
    need = size(2, 2, 16, 100 * 64)
    assert need > 0 and need % 16 == 0
    assert attn(lib, N=2, T=2, H=16, qs=16 * 576, mb=100, wsb=need - 1) == INVALID
    # as many pieces as the GPU holds at once: more tokens in the table need no more
    assert size(64, 64, 32, 100000) == size(64, 64, 32, 1000000)


def test_python_refuses():
    import kimi_delta_attention_gated_gb300 as kda
    cache = kda.latent_cache(2, 16, device="cpu")
    assert cache.shape == (2, 16, 576) and cache.dtype == torch.bfloat16
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.latent_append(torch.zeros((1, 576), dtype=torch.bfloat16), cache, i[None], i)
    with pytest.raises(ValueError):
        kda.attn_latent(torch.zeros((1, 2, 576), dtype=torch.bfloat16), cache, i[None], i)
