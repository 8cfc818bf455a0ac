"""The row and linear operators where element offsets pass 32 bits, and where the first call of
a process is captured into a CUDA graph."""
import subprocess
import sys

import pytest
import torch

import sparse_moe_layer_beam_b200 as bm

pytestmark = pytest.mark.gpu


def test_rows_beyond_2_31_elements():
    """65536 tokens x 8 experts x 5120: 2.7e9 elements of sorted rows."""
    T, K, H, E = 65536, 8, 5120, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    ids = torch.rand((T, E), generator=g, device="cuda").topk(K, dim=1).indices.int()
    cfg = bm.rows_cfg(H, E, K)
    xp = torch.empty((T * K, H), dtype=torch.bfloat16, device="cuda")
    pos = torch.empty((T, K), dtype=torch.int32, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(bm.beam_moe_permute_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    bm.beam_moe_permute(cfg, x, ids, xp, pos, off, ws)
    assert off.tolist()[-1] == T * K
    assert torch.equal(off.diff().long(), torch.bincount(ids.flatten().long(), minlength=E))
    assert torch.equal(pos.flatten().sort().values.long(), torch.arange(T * K, device="cuda"))
    for k in range(K):
        assert torch.equal(xp[pos[:, k].long()], x)
    # the sum of a token's K copies is K x, exactly
    out = torch.empty_like(x)
    bm.beam_moe_combine(cfg, xp, pos, None, out)
    assert torch.equal(out, x * 8)
    w = torch.full((T, K), 0.25, device="cuda")
    dw = torch.empty_like(w)
    one = torch.ones_like(x)
    bm.beam_moe_combine_backward(cfg, one, xp, pos, w, xp, None)  # dy over y: dy alone reads no y
    assert bool((xp[-1] == 0.25).all()) and bool((xp[T * K // 2] == 0.25).all())
    bm.beam_moe_combine_backward(cfg, one, xp, pos, w, None, dw)
    assert bool((dw == 0.25 * H).all())


@pytest.mark.parametrize("n_in,n_out", [(64, 5128), (5128, 64)])
def test_linear_beyond_2_31_elements(n_in, n_out):
    """430000 rows: 2.2e9 elements on the wide side. Small whole numbers, so that every sum is
    exact in FP32 and equal to a product in another order."""
    R, E = 430_000, 3
    g = torch.Generator(device="cuda").manual_seed(2)
    small = lambda *s: torch.randint(-1, 2, s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, w, dy = small(R, n_in), small(E, n_out, n_in), small(R, n_out)
    off = torch.tensor([0, 5, 214_999, R], dtype=torch.int32, device="cuda")
    cfg = bm.linear_cfg(n_in, n_out, E)
    ws = torch.empty(bm.beam_moe_linear_workspace_size(cfg, R, True), dtype=torch.uint8,
                     device="cuda")
    y, dx = torch.zeros_like(dy), torch.zeros_like(x)
    dw = torch.empty_like(w)
    db = torch.empty((E, n_out), device="cuda")
    bm.beam_moe_linear(cfg, x, w, y, ws, offsets=off)
    assert bm.beam_moe_check(ws) == 0
    bm.beam_moe_linear_backward(cfg, dy, x, w, ws, dx=dx, dw=dw, dbias=db, offsets=off)
    assert bm.beam_moe_check(ws) == 0
    for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        pick = torch.tensor(sorted({a, a + 1, (a + b) // 2, b - 2, b - 1}), device="cuda")
        assert torch.equal(y[pick], (x[pick].float() @ w[e].float().T).bfloat16())
        assert torch.equal(dx[pick], (dy[pick].float() @ w[e].float()).bfloat16())
        want = torch.zeros((n_out, n_in), device="cuda")
        for i in range(a, b, 50_000):  # whole numbers below 2^24: exact
            j = min(b, i + 50_000)
            want += dy[i:j].float().T @ x[i:j].float()
        assert torch.equal(dw[e], want.bfloat16())
        assert torch.equal(db[e], dy[a:b].float().sum(0))


CAPTURE = """
import sys
sys.path.insert(0, %r)
import torch
import sparse_moe_layer_beam_b200 as bm
torch.cuda.init()
s = torch.cuda.Stream()
rows = []
for R, K, N, E in ((1, 512, 512, 1), (700, 1024, 2048, 2), (1500, 2048, 2560, 1)):
    cfg = bm.linear_cfg(K, N, E, "silu")
    x = torch.ones((R, K), device="cuda").bfloat16()
    w = torch.full((E, N, K), 2.0 ** -10, device="cuda").bfloat16()
    off = torch.tensor([0] + [R] * E, dtype=torch.int32, device="cuda") if E > 1 else None
    y, z = (torch.zeros((R, N), device="cuda").bfloat16() for _ in range(2))
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    db = torch.zeros((E, N), device="cuda")
    ws = torch.empty(bm.beam_moe_linear_workspace_size(cfg, R, True), dtype=torch.uint8,
                     device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        bm.beam_moe_linear(cfg, x, w, y, ws, offsets=off, z=z)
        bm.beam_moe_linear_backward(cfg, y, x, w, ws, dx=dx, dw=dw, dbias=db, z=z, offsets=off)
    graph.replay()
    torch.cuda.synchronize()
    assert bm.beam_moe_check(ws) == 0
    want = K * 2.0 ** -10
    assert bool((z == want).all()), z
    assert bool(dw[0].ne(0).all()) and bool(dx.ne(0).all()) and bool(db[0].ne(0).all())
print("captured")
"""


def test_first_call_of_a_process_may_be_captured():
    root = __file__.rsplit("/", 2)[0]
    r = subprocess.run([sys.executable, "-c", CAPTURE % root], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
