"""GPU tests of latent attention as a server calls it: single steps beside prompts and drafts (the two ways to
split the work), many heads, captured layers, graphs and streams side by side, padded batches, caches and
outputs behind 4 GB, offsets that do not ascend.  Results are held against the same rows in 64 bits
(tolerances in tests/test_attn_latent_gpu.py and tests/test_latent_rows_gpu.py), or, where only the manner of the
call differs, against the plain call's bits."""
import pytest
import torch

import kimi_delta_attention_gated_gb300 as kda
from tests import attn_reference as ref
from tests.test_attn_latent_gpu import case, cum, make, verify
from tests.test_kv_append_gpu import gen
from tests.test_latent_rows_gpu import SUM, weights

pytestmark = pytest.mark.gpu
C, R, ROW = 512, 64, 576


@pytest.fixture(scope="module", autouse=True)
def built():
    from kimi_delta_attention_gated_gb300 import build
    build.build()


@pytest.mark.parametrize("lens,new,H", [
    ([900] * 19 + [700], [1] * 19 + [300], 32),      # single tokens beside a prompt: a sequence's tiles apart
    ([700] * 6, [5] * 6, 64),                        # as many rows each: its tiles together
    ([700] * 6, [9] * 6, 64),
    ([2100, 40, 2100], [6, 6, 6], 40),
    ([1500] * 3, [4] * 3, 192),                      # several tiles of a token
    ([2000, 1, 600], None, 192),
    ([3000, 70], None, 320),
    ([3000, 70], [2, 1], 520),
    ([5000], [200], 16),
    ([300, 0, 2000, 5], [0, 3, 70, 1], 24),
])
def test_mixed_batches(lens, new, H):
    case(lens, H, 64, new, seed=H + len(lens), heads=sorted({0, H // 2, H - 1}), tokens=[0, 1, 4, 8, 63, 69, 130, 299])


def test_many_sequences_in_both_ways():
    """More sequences than threads of a CTA, with a few longer ones among them."""
    new = [1] * 500
    new[3], new[499], new[200] = 40, 7, 0
    case([130 + i % 70 for i in range(500)], 16, 16, new, seed=31, heads=[0, 15], tokens=[0, 6, 39])
    case([90] * 450, 64, 16, [3] * 450, seed=32, heads=[63], tokens=[0, 2])


def test_padded_batch():
    """Empty sequences and rows behind the last one, as a batch padded to a captured size has them."""
    lens, new = [300, 0, 90, 0, 0], [2, 0, 1, 0, 0]
    q, cache, table, sl = make(lens, 32, 64, 33, 8)
    cu = cum(new)
    o = torch.full((8, 32, C), 7.0, device="cuda").bfloat16()
    _, lse = kda.attn_latent(q, cache, table.cuda(), sl, cu_seqlens=cu, o=o, return_lse=True)
    kda.device_status()
    verify(o, lse, q, cache, table, lens, new)
    assert (o[3:] == 7).all()


@pytest.mark.parametrize("N,H,L", [(2, 16, 2000), (4, 64, 9000), (40, 16, 70)])
def test_offsets_that_do_not_ascend(N, H, L):
    """Offsets that go back count rows twice: the outputs are nobody's, but nothing beside them is written, and the
    next call is right."""
    T = 40
    q, cache, table, sl = make([L] * N, H, 64, 34, T)
    dt = table.cuda()
    cu = torch.tensor(([0, T] * N)[:N + 1], dtype=torch.int32, device="cuda")
    need = kda.attn_latent_workspace_size(N, T, H, dt.shape[1] * 64)
    ws = torch.full((need + 4096,), 165, dtype=torch.uint8, device="cuda")
    o = torch.full((T + 2, H, C), 7.0, device="cuda").bfloat16()
    kda.attn_latent(q, cache, dt, sl, cu_seqlens=cu, o=o[1:-1], workspace=ws[:need])
    kda.device_status()
    assert (ws[need:] == 165).all() and (o[0] == 7).all() and (o[-1] == 7).all()
    right = cum([T] + [0] * (N - 1))
    got, lse = kda.attn_latent(q, cache, dt, sl, cu_seqlens=right, workspace=ws[:need], return_lse=True)
    verify(got, lse, q, cache, table, [L] * N, [T] + [0] * (N - 1), heads=[0], tokens=[0, 39])


class Layer:
    """The calls of one step, from fixed buffers, and the buffers."""

    def __init__(self, N, H, L, P, seed, new=1):
        g = gen(seed)
        self.T = N * new
        _, self.cache, table, _ = make([L] * N, 1, P, seed, 1)
        self.w, self.norm = weights(H, seed), 1 + 0.1 * torch.randn(C, generator=g, device="cuda")
        self.x = torch.randn((self.T, ROW), generator=g, device="cuda").bfloat16()
        self.q = torch.randn((self.T, H, 192), generator=g, device="cuda").bfloat16()
        self.table, self.cu = table.cuda(), cum([new] * N) if new > 1 else None
        self.ctx = torch.randint(L // 2, L - new, (N,), generator=g, device="cuda").int()
        self.f, self.mag = kda.rotary_inv_freq(R)
        self.new = new
        self.out = torch.zeros((self.T, H, 128), device="cuda").bfloat16()
        self.lq = torch.zeros((self.T, H, ROW), device="cuda").bfloat16()
        self.o = torch.zeros((self.T, H, C), device="cuda").bfloat16()
        self.rows = torch.zeros((self.T, ROW), device="cuda").bfloat16()
        self.kv = torch.zeros((self.T, H, 192), device="cuda").bfloat16(), torch.zeros((self.T, H, 128), device="cuda").bfloat16()
        need = kda.attn_latent_workspace_size(N, self.T, H, self.table.shape[1] * P)
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def __call__(self):
        kda.latent_append(self.x, self.cache, self.table, self.ctx, cu_seqlens=self.cu, norm_w=self.norm, inv_freq=self.f,
                          magnitude=self.mag, rows_out=self.rows)
        pos = (self.ctx[:, None] + torch.arange(self.new, device="cuda", dtype=torch.int32)).flatten()
        kda.latent_queries(self.q, self.w, positions=pos, inv_freq=self.f, magnitude=self.mag, out=self.lq)
        kda.attn_latent(self.lq, self.cache, self.table, self.ctx + self.new, cu_seqlens=self.cu, o=self.o, workspace=self.ws)
        kda.latent_values(self.o, self.w, out=self.out)
        kda.latent_expand(self.rows, self.w, k_out=self.kv[0], v_out=self.kv[1])

    def results(self):
        return [t.clone() for t in (self.out, self.lq, self.o, self.rows, self.cache, *self.kv)]

    def capture(self):
        self()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self()
        return g


@pytest.mark.parametrize("N,H,new", [(3, 16, 1), (2, 128, 1), (5, 32, 4), (130, 160, 1)])
def test_captured_layer(N, H, new):
    """A whole step captured and replayed with other inputs gives the eager calls' bits."""
    layer = Layer(N, H, 400, 32, 40 + N, new)
    graph = layer.capture()
    g = gen(50)
    for _ in range(2):
        layer.x.copy_(torch.randn(layer.x.shape, generator=g, device="cuda"))
        layer.q.copy_(torch.randn(layer.q.shape, generator=g, device="cuda"))
        layer.ctx.copy_(torch.randint(0, 400 - new, (N,), generator=g, device="cuda"))
        graph.replay()
        got = layer.results()
        layer()
        assert all(torch.equal(a, b) for a, b in zip(got, layer.results()))
    kda.device_status()


def test_two_graphs_at_once():
    """Two captured layers, each with its own workspace, replayed on two streams at the same time."""
    layers = [Layer(4, 32, 3000, 64, 60), Layer(3, 64, 2000, 16, 61, 3)]
    graphs = [x.capture() for x in layers]
    want = []
    for x in layers:
        x()
        want.append(x.results())
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for x, w in zip(layers, want):
        assert all(torch.equal(a, b) for a, b in zip(x.results(), w))
    kda.device_status()


def test_steps_without_a_pause():
    """Calls whose launches overlap each other's ends: each reads what the one before wrote."""
    layer = Layer(7, 48, 500, 64, 62)
    start = layer.ctx.clone()

    def steps(wait):
        layer.ctx.copy_(start)
        layer.cache.zero_()
        for _ in range(12):
            layer()
            layer.q[:, :, :128] = layer.out
            layer.ctx += 1
            if wait:
                torch.cuda.synchronize()
        return layer.results()

    q = layer.q.clone()
    a = steps(False)
    layer.q.copy_(q)
    b = steps(True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_cache_behind_4_gb():
    """Pages whose bytes lie behind 2^32, and elements behind 2^31."""
    P, pages = 128, 33000  # 4.9 GB
    cache = torch.empty((pages, P, ROW), device="cuda", dtype=torch.bfloat16)
    table = torch.tensor([[pages - 1, 0, 29200], [14564, pages - 2, 31000]], dtype=torch.int32)
    lens, H, g = [300, 384], 16, gen(70)
    x = torch.randn((sum(lens), ROW), generator=g, device="cuda").bfloat16()
    rows = kda.latent_append(x, cache, table.cuda(), torch.zeros(2, dtype=torch.int32, device="cuda"), cu_seqlens=cum(lens),
                             return_rows=True)
    assert torch.equal(rows, x)
    assert torch.equal(cache[pages - 1], x[:128]) and torch.equal(cache[31000], x[556:684])
    q = torch.randn((2, H, ROW), generator=g, device="cuda").bfloat16()
    o, lse = kda.attn_latent(q, cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), return_lse=True)
    kda.device_status()
    verify(o, lse, q, cache, table, lens)


def test_products_behind_4_gb():
    """Outputs and inputs of more than 2^31 elements, looked at near both ends."""
    T, H = 60000, 64
    w, g = weights(H, 71), gen(72)
    look = [0, 1, T // 2, T - 129, T - 1]
    q = torch.randn((T, H, 192), generator=g, device="cuda", dtype=torch.bfloat16)
    lq = kda.latent_queries(q, w)
    qn, wk = ref.f64(q[look, :, :128]), ref.f64(w[:, :128])
    want, size = torch.einsum("thn,hnc->thc", qn, wk), torch.einsum("thn,hnc->thc", qn.abs(), wk.abs())
    ref.check("queries", lq[look][..., :C], want, ref.HALF_BF16 * want.abs() + SUM * size)
    assert torch.equal(lq[..., C:], q[..., 128:])
    v = kda.latent_values(lq[..., :C].contiguous(), w)
    a, b = ref.f64(lq[look][..., :C]), ref.f64(w[:, 128:])
    want, size = torch.einsum("thc,hnc->thn", a, b), torch.einsum("thc,hnc->thn", a.abs(), b.abs())
    ref.check("values", v[look], want, ref.HALF_BF16 * want.abs() + SUM * size)
    del lq, v, q
    T = 190000
    look = [0, T // 2, T - 129, T - 1]
    x = torch.randn((T, ROW), generator=g, device="cuda", dtype=torch.bfloat16)
    k, v = kda.latent_expand(x, w)
    kda.device_status()
    a, b = ref.f64(x[look, :C]), ref.f64(w).flatten(0, 1)
    want, size = (a @ b.T).view(-1, H, 256), (a.abs() @ b.abs().T).view(-1, H, 256)
    tol = ref.HALF_BF16 * want.abs() + SUM * size
    ref.check("keys", k[look][..., :128], want[..., :128], tol[..., :128])
    ref.check("expanded values", v[look], want[..., 128:], tol[..., 128:])
    assert all(torch.equal(k[t, :, 128:], x[t, C:].expand(H, R)) for t in look)


def test_products_on_another_stream():
    layer = Layer(9, 24, 300, 16, 73)
    layer()
    want = layer.results()
    for t in (layer.out, layer.lq, layer.o, layer.rows, *layer.kv):
        t.zero_()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        layer()
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, layer.results()))


@pytest.mark.parametrize("T,H", [(300, 152), (513, 110), (1024, 80), (2305, 33), (8192, 10), (257, 160), (20000, 4)])
def test_expansion_of_many_tokens(T, H):
    """Tiles that end inside a pair's 256 tokens or inside the first half of them, runs that begin inside a head."""
    g = gen(T + H)
    x = torch.randn((T, 64 + ROW), generator=g, device="cuda").bfloat16()[:, 64:]
    w = weights(H, T + 3)
    big = torch.full((T + 2, H, 192), 3.0, device="cuda").bfloat16(), torch.full((T + 2, H, 128), 3.0, device="cuda").bfloat16()
    k, v = kda.latent_expand(x, w, k_out=big[0][1:-1], v_out=big[1][1:-1])
    kda.device_status()
    a, b = ref.f64(x[:, :C]), ref.f64(w).flatten(0, 1)
    want = (a @ b.T).view(T, H, 256)
    tol = ref.HALF_BF16 * want.abs() + SUM * (a.abs() @ b.abs().T).view(T, H, 256)
    ref.check("keys", k[..., :128], want[..., :128], tol[..., :128])
    ref.check("values", v, want[..., 128:], tol[..., 128:])
    assert torch.equal(k[..., 128:], x[:, None, C:].expand(T, H, R))
    assert all((y[0] == 3).all() and (y[-1] == 3).all() for y in big)


@pytest.mark.parametrize("lens,new,H", [
    ([1000] * 64, [4] * 64, 32),                                # units whole, a few a piece
    ([1000] * 64, [4] * 60 + [7, 0, 1, 9], 32),
    ([900 + 3 * i % 200 for i in range(256)], None, 64),
    ([260 + 7 * i % 90 for i in range(170)] + [0] * 10, None, 16),
    ([300] * 170 + [9000], None, 16),                           # one sequence far longer: cut
    ([300] * 100 + [700] * 100, [1, 2] * 100, 128),
])
def test_units_left_whole(lens, new, H):
    """About as many units as pieces, of equal and of unequal lengths."""
    case(lens, H, 64, new, seed=H + len(lens), heads=[0, H - 1], tokens=[0, 1, 3, 6, 8])


@pytest.mark.parametrize("H", [1, 2, 3, 5, 7, 12, 20, 50, 70, 100, 193])
@pytest.mark.parametrize("lens,new", [([700, 130], [81, 5]), ([3000, 40, 66], [3, 2, 1]), ([90], None), ([5000, 12], None)])
def test_tiles_of_any_heads(H, lens, new):
    """Heads that fill a tile's rows unevenly: tokens that begin anywhere in it."""
    case(lens, H, 32, new, seed=H, heads=sorted({0, H // 2, H - 1}), tokens=[0, 1, 2, 4, 11, 12, 31, 33, 64, 80])
