"""The operators together, as a layer runs them: permute -> linear (swiglu) -> linear ->
combine and the four gradients in reverse, on the routes of beam_moe_route."""
import pytest
import torch

import sparse_moe_layer_beam_b200 as bm

pytestmark = pytest.mark.gpu

H, I, E, G, Gk, K = 256, 128, 16, 4, 2, 4


class Layer:
    """Buffers of one layer call; forward() and backward() make the library's calls."""

    def __init__(self, x, ids, w, w13, w2, dout):
        T = x.shape[0]
        A = T * K
        new = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
        self.x, self.ids, self.w, self.w13, self.w2, self.dout = x, ids, w, w13, w2, dout
        self.rows = bm.rows_cfg(H, E, K)
        self.up = bm.linear_cfg(H, I, E, "swiglu")
        self.down = bm.linear_cfg(I, H, E, out_fp32=False)
        self.xp, self.z, self.h, self.y = new(A, H), new(A, 2 * I), new(A, I), new(A, H)
        self.pos, self.off = new(T, K, t=torch.int32), new(E + 1, t=torch.int32)
        self.out = new(T, H)
        self.dy, self.dw = new(A, H), new(T, K, t=torch.float32)
        self.dh, self.dw2 = new(A, I), new(E, H, I)
        self.dxp, self.dw13, self.dx = new(A, H), new(E, 2 * I, H), new(T, H)
        size = max(bm.beam_moe_permute_workspace_size(self.rows, T),
                   bm.beam_moe_linear_workspace_size(self.up, A, True),
                   bm.beam_moe_linear_workspace_size(self.down, A, True))
        self.ws = new(size, t=torch.uint8)

    def forward(self):
        bm.beam_moe_permute(self.rows, self.x, self.ids, self.xp, self.pos, self.off, self.ws)
        bm.beam_moe_linear(self.up, self.xp, self.w13, self.h, self.ws, offsets=self.off, z=self.z)
        bm.beam_moe_linear(self.down, self.h, self.w2, self.y, self.ws, offsets=self.off)
        bm.beam_moe_combine(self.rows, self.y, self.pos, self.w, self.out)

    def backward(self):
        bm.beam_moe_combine_backward(self.rows, self.dout, self.y, self.pos, self.w, self.dy,
                                     self.dw)
        bm.beam_moe_linear_backward(self.down, self.dy, self.h, self.w2, self.ws, dx=self.dh,
                                    dw=self.dw2, offsets=self.off)
        bm.beam_moe_linear_backward(self.up, self.dh, self.xp, self.w13, self.ws, dx=self.dxp,
                                    dw=self.dw13, z=self.z, offsets=self.off)
        bm.beam_moe_permute_backward(self.rows, self.dxp, self.pos, self.dx)

    def results(self):
        return {k: getattr(self, k).clone()
                for k in ("out", "dx", "dw", "dw13", "dw2", "z", "h", "y")}


def make(T, seed, dropped=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = n(T, H).bfloat16()
    wr, w13, w2 = n(E, H) / 16, (n(E, 2 * I, H) / 16).bfloat16(), (n(E, H, I) / 11).bfloat16()
    ids = torch.empty((T, K), dtype=torch.int32, device="cuda")
    w = torch.empty((T, K), device="cuda")
    cfg = bm.beam_cfg(H, I, E, G, Gk, K)
    ws = torch.empty(bm.beam_moe_workspace_size(cfg, T, bm.OP_ROUTE), dtype=torch.uint8,
                     device="cuda")
    bm.beam_moe_route(cfg, x, wr, None, ids, w, None, ws)
    if dropped:
        ids[T - dropped:] = -1
    return Layer(x, ids, w, w13, w2, n(T, H).bfloat16()), cfg


def exact(L):
    """The layer and its gradients by autograd in 64 bits, token by slot."""
    x, w, w13, w2 = (t.double().requires_grad_() for t in (L.x, L.w, L.w13, L.w2))
    out = torch.zeros(L.out.shape, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, k = (L.ids == e).nonzero(as_tuple=True)
        z = x[t] @ w13[e].T
        h = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
        out = out.index_add(0, t, w[t, k][:, None] * (h @ w2[e].T))
    out.backward(L.dout.double())
    return {"out": out.detach(), "dx": x.grad, "dw": w.grad, "dw13": w13.grad, "dw2": w2.grad}


def rel(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("T,dropped", [(1, 0), (70, 9), (700, 0)])
def test_the_layer_and_its_gradients(T, dropped):
    L, _ = make(T, T, dropped)
    L.forward()
    L.backward()
    got = L.results()
    # relative RMS: every 16-bit tensor on the way (h, y, out; dy, dh, dZ and the result) adds
    # at most half a step of each element, 2^-8 at most and independent: the worst path holds six
    # (h, y's, dy, dh, dZ, z's slope, the result): sqrt(6) 2^-8 < 0.01
    for k, want in exact(L).items():
        assert rel(got[k], want) <= 0.01, (k, rel(got[k], want))


def test_the_layer_is_the_fused_block():
    """beam_moe_forward_routed on the same routes keeps y in FP32; its h is the layer's h, its
    output the layer's up to y's rounding to bf16 (2^-8 of each of K terms) and out's own."""
    L, cfg = make(333, 5)
    L.forward()
    out = torch.empty_like(L.out)
    ws = torch.empty(bm.beam_moe_workspace_size(cfg, 333), dtype=torch.uint8, device="cuda")
    bm.beam_moe_forward_routed(cfg, L.x, L.ids, L.w, L.w13, L.w2, out, ws)
    assert bm.beam_moe_check(ws) == 0
    terms = (L.w[..., None] * L.y[L.pos.long()].float()).abs().sum(1).double()
    err = (out.double() - L.out.double()).abs()
    # + h: where the two kernels' FP32 sums lie on either side of a rounding, 2^-7 of an h
    assert bool((err <= 2 * 2.0 ** -8 * terms + 2 * 2.0 ** -8 * out.double().abs() + 0.02).all())
    assert rel(L.out, out.double()) <= 0.006


def test_captured_layer_replays_and_repeats():
    """The whole step in a CUDA graph, replayed on other inputs, equals eager calls bit for bit;
    an eager run between replays and a second captured graph with its own buffers change
    nothing."""
    L, _ = make(130, 6)
    M, _ = make(130, 7)
    want = {}
    for name, layer in (("L", L), ("M", M)):
        layer.forward()
        layer.backward()
        want[name] = layer.results()
    torch.cuda.synchronize()
    graphs = []
    for layer in (L, M):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
            layer.forward()
            layer.backward()
        graphs.append(graph)
    for _ in range(2):
        for name, layer, graph in (("L", L, graphs[0]), ("M", M, graphs[1])):
            layer.out.fill_(5)
            layer.dx.fill_(5)
            graph.replay()
            M.forward()
            torch.cuda.synchronize()
            for k, v in layer.results().items():
                assert torch.equal(v, want[name][k]), (name, k)
    # the first graph on the second layer's tokens and routes
    for k in ("x", "ids", "w", "w13", "w2", "dout"):
        getattr(L, k).copy_(getattr(M, k))
    graphs[0].replay()
    torch.cuda.synchronize()
    for k, v in L.results().items():
        assert torch.equal(v, want["M"][k]), k


def test_two_streams_at_once():
    """Two layers on two streams, each with its own workspace."""
    layers = [make(500, 8)[0], make(90, 9)[0]]
    want = []
    for layer in layers:
        layer.forward()
        layer.backward()
        want.append(layer.results())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        for layer, s in zip(layers, streams):
            with torch.cuda.stream(s):
                layer.forward()
                layer.backward()
    torch.cuda.synchronize()
    for layer, w in zip(layers, want):
        for k, v in layer.results().items():
            assert torch.equal(v, w[k]), k
