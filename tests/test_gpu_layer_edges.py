"""The row and linear operators on the GPU at the limits of what their documentation allows.

Inputs are small whole numbers unless stated, so that every FP32 sum is exact whatever its order
and results equal the 64-bit ones rounded once, bit for bit.
"""
import pytest
import torch

import sparse_moe_layer_beam_b200 as bm
from tests import _layer_ops as ref
from tests.test_layer_ops_limits import offset_vectors

pytestmark = pytest.mark.gpu
LEFT = 7.0
BF = torch.bfloat16


def whole(shape, seed, t=BF):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=g).to(t)


# rows, experts, n_in, n_out: the few-row form, split tiles, 128- and 256-column tiles, CTA pairs
SHAPES = [(3, 40, 64, 72), (100, 512, 64, 64), (130, 4, 72, 136), (700, 60, 320, 328),
          (1417, 10, 256, 2600), (3000, 3, 1032, 1288)]


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("R,E,n_in,n_out", SHAPES)
def test_offsets_that_do_not_ascend(R, E, n_in, n_out, act):
    """No row has two experts, and nothing is written outside the buffers: the workspace is the
    front of a larger one with a pattern behind it."""
    cfg = bm.linear_cfg(n_in, n_out, E, act)
    x, w, dy = whole((R, n_in), 1), whole((E, n_out, n_in), 2), whole((R, n_out), 3)
    z = whole((R, n_out), 4)
    xd, wd, dyd, zd = x.cuda(), w.cuda(), dy.cuda(), z.cuda()
    need = bm.beam_moe_linear_workspace_size(cfg, R, True)
    big = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    ws = big[:need]
    for i, off in enumerate(offset_vectors(E, R, R)):
        if 4 <= i < 38:  # eight of the 42
            continue
        offd = torch.tensor(off, dtype=torch.int32, device="cuda")
        y = torch.full((R, n_out), LEFT, dtype=BF, device="cuda")
        dx = torch.full((R, n_in), LEFT, dtype=BF, device="cuda")
        dw = torch.full((E, n_out, n_in), LEFT, dtype=BF, device="cuda")
        db = torch.full((E, n_out), LEFT, device="cuda")
        bm.beam_moe_linear(cfg, xd, wd, y, ws, offsets=offd)
        assert bm.beam_moe_check(ws) == 0
        bm.beam_moe_linear_backward(cfg, dyd, xd, wd, ws, dx=dx, dw=dw, dbias=db, offsets=offd,
                                    z=zd if act == "relu" else None)
        assert bm.beam_moe_check(ws) == 0
        assert bool((big[need:] == 0xA5).all())
        wy, wdx = torch.full((R, n_out), LEFT, dtype=BF), torch.full((R, n_in), LEFT, dtype=BF)
        wdw, wdb = torch.zeros((E, n_out, n_in)), torch.zeros((E, n_out))
        dz = torch.where(z > 0, dy, 0.0) if act == "relu" else dy
        for e, (a, b) in enumerate(ref.segments(off, R)):
            if a == b:
                continue
            wy[a:b] = ref.act(x[a:b].float() @ w[e].float().T, act).to(BF)
            wdx[a:b] = (dz[a:b].float() @ w[e].float()).to(BF)
            wdw[e] = dz[a:b].float().T @ x[a:b].float()
            wdb[e] = dz[a:b].float().sum(0)
        assert torch.equal(y.cpu(), wy) and torch.equal(dx.cpu(), wdx)
        assert torch.equal(dw.cpu(), wdw.to(BF)) and torch.equal(db.cpu(), wdb)


@pytest.mark.parametrize("H,dtype", [(5120, "bf16"), (33, "fp32"), (1002, "fp16")])
def test_tokens_without_any_row(H, dtype):
    """A rank that has none of the experts: rows = 0, every pos is -1 (or points at no row), and
    an empty tensor has no address. The sums over no rows are zeros."""
    t = {"bf16": BF, "fp16": torch.float16, "fp32": torch.float32}[dtype]
    T, K = 37, 3
    cfg = bm.rows_cfg(H, 16, K, dtype)
    pos = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    pos[1, 2] = 0
    none = torch.empty((0, H), dtype=t, device="cuda")
    w = torch.full((T, K), float("nan"), device="cuda")
    out = torch.full((T, H), LEFT, dtype=t, device="cuda")
    bm.beam_moe_combine(cfg, none, pos, w, out)
    assert not out.any()
    out.fill_(LEFT)
    bm.beam_moe_combine(cfg, torch.empty((0, H), device="cuda"), pos, None, out)
    assert not out.any()
    dx = torch.full((T, H), LEFT, dtype=t, device="cuda")
    bm.beam_moe_permute_backward(cfg, none, pos, dx)
    assert not dx.any()
    dout = torch.full((T, H), float("nan"), dtype=t, device="cuda")
    for y in (none, None):
        dw = torch.full((T, K), LEFT, device="cuda")
        bm.beam_moe_combine_backward(cfg, dout, y, pos, w, none, dw)
        assert not dw.any()
    bm.beam_moe_combine_backward(cfg, dout, none, pos, w, none, None)
    e = torch.empty((0, K), dtype=torch.int32, device="cuda")
    bm.beam_moe_combine_backward(cfg, none, none, e, None, none, None)


@pytest.mark.parametrize("which", ["dx", "dw", "dbias"])
def test_each_gradient_alone_without_rows(which):
    cfg = bm.linear_cfg(64, 72, 2, "silu")
    e = lambda n: torch.empty((0, n), dtype=BF, device="cuda")  # noqa: E731
    out = {"dx": e(64), "dw": torch.ones((2, 72, 64), dtype=BF, device="cuda"),
           "dbias": torch.ones((2, 72), device="cuda")}[which]
    ws = torch.empty(bm.beam_moe_linear_workspace_size(cfg, 0, True), dtype=torch.uint8,
                     device="cuda")
    w = torch.ones((2, 72, 64), dtype=BF, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    bm.beam_moe_linear_backward(cfg, e(72), e(64), w, ws, z=e(72), offsets=off, **{which: out})
    assert not out.any()


@pytest.mark.parametrize("backward", [False, True])
def test_status_of_a_call_without_rows(backward):
    """The status word of a workspace that held anything reports the call, not what was there."""
    cfg = bm.linear_cfg(64, 72)
    e = lambda n: torch.empty((0, n), dtype=BF, device="cuda")  # noqa: E731
    w = torch.ones((1, 72, 64), dtype=BF, device="cuda")
    ws = torch.full((bm.beam_moe_linear_workspace_size(cfg, 0, True),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    if backward:
        bm.beam_moe_linear_backward(cfg, e(72), e(64), w, ws, dw=torch.empty_like(w))
    else:
        bm.beam_moe_linear(cfg, e(64), w, e(72), ws)
    assert bm.beam_moe_check(ws) == 0


def test_threads_at_once():
    """Four threads, each on a stream, with tensors and a workspace of its own."""
    import threading
    R, n_in, n_out = (5, 90, 700, 1500), 1032, 1288
    w = whole((1, n_out, n_in), 5)
    wd, wrong, start = w.cuda(), [], threading.Barrier(len(R))
    torch.cuda.synchronize()

    def work(i):
        x, dy = whole((R[i], n_in), 10 + i), whole((R[i], n_out), 20 + i)
        cfg = bm.linear_cfg(n_in, n_out)
        with torch.cuda.stream(torch.cuda.Stream()):
            xd, dyd = x.cuda(), dy.cuda()
            ws = torch.empty(bm.beam_moe_linear_workspace_size(cfg, R[i], True),
                             dtype=torch.uint8, device="cuda")
            start.wait(60)
            for _ in range(20):
                y, dx, dw = torch.empty_like(dyd), torch.empty_like(xd), torch.empty_like(wd)
                bm.beam_moe_linear(cfg, xd, wd, y, ws)
                bm.beam_moe_linear_backward(cfg, dyd, xd, wd, ws, dx=dx, dw=dw)
            status = bm.beam_moe_check(ws)
            same = (torch.equal(y.cpu(), (x.float() @ w[0].float().T).to(BF))
                    and torch.equal(dx.cpu(), (dy.float() @ w[0].float()).to(BF))
                    and torch.equal(dw.cpu()[0], (dy.float().T @ x.float()).to(BF)))
        if status or not same:
            wrong.append((i, status, same))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(R))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu", "swiglu"])
def test_gradients_far_out(act):
    """dZ where squares and cubes of Z, or products of dY and Z, leave FP32: finite, and the
    formula's. One row, so that the bias's gradient is dZ in FP32; within 2^-18 of the terms that
    dZ adds up. Where a sigmoid or a cdf lies below FP32's normal numbers, 2^-126, it may be zero:
    a slope is at most |z| 2a'(z) times that there, 90 for silu (z < -87), 227 for gelu_tanh
    (z < -9.9) and 15 for gelu, and |z| e^z only falls behind; so dZ is off by 256 2^-126 |dy up|
    at most."""
    z = torch.tensor([s * v for v in (1e2, 1e4, 1e10, 2e18, 2e19, 1e30, 3e38, 0.5)
                      for s in (1, -1)])
    dy = torch.full((z.numel(),), 4.0)
    if act == "swiglu":
        up = torch.tensor([1e-30, 3e38])
        z = torch.cat((z.repeat(2), up.repeat_interleave(z.numel())))
        dy = torch.cat((dy, torch.full_like(dy, 2.0 ** -10)))
    z, dy = z[None].to(BF), dy[None].to(BF)
    N, n_out = z.shape[1], dy.shape[1]
    cfg = bm.linear_cfg(8, n_out, 1, act)
    ws = torch.empty(bm.beam_moe_linear_workspace_size(cfg, 1, True), dtype=torch.uint8,
                     device="cuda")
    db = torch.full((1, N), LEFT, device="cuda")
    bm.beam_moe_linear_backward(cfg, dy.cuda(), None, None, ws, dbias=db, z=z.cuda())
    want = ref.act_grad(dy.double(), z.double(), act)
    terms = ref.act_grad_terms(dy.double(), z.double(), act)
    # a result beyond FP32 is infinite
    want = torch.where(want.abs() > torch.finfo(torch.float32).max, want.sign() * torch.inf, want)
    got = db.cpu().double()
    scale = dy.double().abs()
    if act == "swiglu":
        scale = (scale * z.double().chunk(2, -1)[1].abs().clamp(min=1)).repeat(1, 2)
    fine = (got == want) | ((got - want).abs() <= 2.0 ** -18 * terms + 2.0 ** -118 * scale)
    assert bool(fine.all()), list(zip(z[0].tolist(), got[0].tolist(), want[0].tolist()))


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "swiglu"])
@pytest.mark.parametrize("R,E,n_in,n_out", [(1, 1, 8, 64)] + SHAPES)
def test_fp32_outputs_keep_fp32(R, E, n_in, n_out, act):
    """One product a sum, so Z is exact and what is left is the activation's own error.

    e^-z: 2^-22 from the exponential, 2^-24 from the product behind it; 1 + e 2^-24; the quotient
    2^-22; swiglu's factor 2^-24: 3 2^-22 in all. gelu_tanh's argument 2a takes six roundings,
    6 2^-24 |2a| of the gate. gelu: erfc within 2^-21, its argument's two roundings, which move
    it by 2 2^-24 (1 + z^2) at most, and the product's. Below z = -80 (-9 gelu_tanh, -12 gelu) FP32 runs out: within
    256 2^-126 of the other half there."""
    N = n_out * (2 if act == "swiglu" else 1)
    g = torch.Generator().manual_seed(R + n_out)
    x, w = torch.zeros((R, n_in), dtype=BF), torch.zeros((E, N, n_in), dtype=BF)
    x[:, 0] = (torch.randn(R, generator=g).exp()).to(BF)
    w[:, :, 0] = (torch.randn((E, N), generator=g) * 12).to(BF)
    lo = [min(R, e * (R // E + 1)) for e in range(E + 1)]
    cfg = bm.linear_cfg(n_in, n_out, E, act, out_fp32=True)
    y = torch.full((R, n_out), LEFT, device="cuda")
    ws = torch.empty(bm.beam_moe_linear_workspace_size(cfg, R), dtype=torch.uint8, device="cuda")
    bm.beam_moe_linear(cfg, x.cuda(), w.cuda(), y, ws,
                       offsets=torch.tensor(lo, dtype=torch.int32, device="cuda"))
    z = torch.cat([x[a:b, :1].double() * w[e, :, 0].double()
                   for e, (a, b) in enumerate(zip(lo, lo[1:]))])
    gate = z[:, :n_out]
    if act == "gelu":
        gate_of = 0.5 * torch.special.erfc(gate * -0.5 ** 0.5)
    elif act == "gelu_tanh":
        gate_of = torch.special.expit((8 / torch.pi) ** 0.5 * (gate + 0.044715 * gate ** 3))
    else:
        gate_of = torch.special.expit(gate)
    other = z[:, n_out:] if act == "swiglu" else torch.ones_like(gate)
    want = gate * gate_of * other
    rel = {"gelu": 2.0 ** -21 + 2.0 ** -23 * (1 + gate ** 2) + 2.0 ** -24,
           "gelu_tanh": 3 * 2.0 ** -22 + 6 * 2.0 ** -24 * (
               (8 / torch.pi) ** 0.5 * (gate + 0.044715 * gate ** 3)).abs()
           }.get(act, torch.full_like(gate, 3 * 2.0 ** -22))
    deep = gate < {"gelu": -12, "gelu_tanh": -9}.get(act, -80)
    tol = torch.where(deep, 2.0 ** -24 * want.abs(), rel * want.abs()) + (
        2.0 ** -118 * other.abs().clamp(min=1))
    tol = torch.where(deep, want.abs() + tol, tol)
    err = (y.cpu().double() - want).abs()
    assert bool((err <= tol).all()), (err / want.abs())[(err > tol)].max()


# rows, offsets, n_in, n_out: tiles split over a cluster; 128- and 256-column tiles; CTA pairs; a
# dense layer, and experts whose segments end inside a step
LONG = [(1 << 20, None, 64, 64), ((1 << 20) + 37, (0, 5, 40_000, (1 << 20) + 30), 72, 136),
        ((1 << 20) + 5, None, 1024, 1024), ((1 << 19) + 3, None, 4096, 1152),
        ((1 << 19) + 77, (0, 32_769, 32_769, (1 << 19) + 70), 1032, 2600)]


@pytest.mark.parametrize("R,off,n_in,n_out", LONG)
def test_long_sums_of_one_sign(R, off, n_in, n_out):
    """dW over half a million rows and more, fp16, every term positive: half a step, 2^-11; what
    the tensor cores cut off, at most a step of the sum, 2^-23, for each 16 of the 16384 rows
    between drains; and one FP32 addition a drain."""
    E = len(off) - 1 if off else 1
    g = torch.Generator(device="cuda").manual_seed(R)
    x = (0.5 + torch.rand((R, n_in), generator=g, device="cuda", dtype=torch.float16))
    dy = (0.5 + torch.rand((R, n_out), generator=g, device="cuda", dtype=torch.float16)) / 1024
    cfg = bm.linear_cfg(n_in, n_out, E, dtype="fp16")
    ws = torch.empty(bm.beam_moe_linear_workspace_size(cfg, R, True), dtype=torch.uint8,
                     device="cuda")
    dw = torch.full((E, n_out, n_in), LEFT, dtype=torch.float16, device="cuda")
    bm.beam_moe_linear_backward(
        cfg, dy, x, None, ws, dw=dw,
        offsets=torch.tensor(off, dtype=torch.int32, device="cuda") if off else None)
    assert bm.beam_moe_check(ws) == 0
    for e, (a, b) in enumerate(zip(off or (0,), off[1:] if off else (R,))):
        want = torch.zeros((n_out, n_in), dtype=torch.float64, device="cuda")
        for i in range(a, b, 1 << 16):
            j = min(b, i + (1 << 16))
            want += dy[i:j].double().T @ x[i:j].double()
        err = (dw[e].double() - want).abs()
        tol = (2.0 ** -11 + 1024 * 2.0 ** -23 + (R >> 14) * 2.0 ** -24) * want
        assert bool((err <= tol).all()), (e, (err / want).max().item())


@pytest.mark.parametrize("off", [None, (0, 3, 20_003, 49_990)])
def test_long_sums_beside_the_other_gradients(off):
    """All three gradients of 50000 narrow rows: both products and the biases' sums in one launch,
    dW's sums drained on the way. Whole numbers: exact."""
    R, n_in, n_out = 50_000, 64, 72
    E = len(off) - 1 if off else 1
    x, w, dy = whole((R, n_in), 1), whole((E, n_out, n_in), 2), whole((R, n_out), 3)
    cfg = bm.linear_cfg(n_in, n_out, E)
    ws = torch.empty(bm.beam_moe_linear_workspace_size(cfg, R, True), dtype=torch.uint8,
                     device="cuda")
    dx = torch.full((R, n_in), LEFT, dtype=BF, device="cuda")
    dw = torch.full((E, n_out, n_in), LEFT, dtype=BF, device="cuda")
    db = torch.full((E, n_out), LEFT, device="cuda")
    bm.beam_moe_linear_backward(
        cfg, dy.cuda(), x.cuda(), w.cuda(), ws, dx=dx, dw=dw, dbias=db,
        offsets=torch.tensor(off, dtype=torch.int32, device="cuda") if off else None)
    assert bm.beam_moe_check(ws) == 0
    wdx = torch.full((R, n_in), LEFT, dtype=BF)
    for e, (a, b) in enumerate(zip(off or (0,), off[1:] if off else (R,))):
        wdx[a:b] = (dy[a:b].float() @ w[e].float()).to(BF)
        assert torch.equal(dw[e].cpu(), (dy[a:b].float().T @ x[a:b].float()).to(BF))
        assert torch.equal(db[e].cpu(), dy[a:b].float().sum(0))
    assert torch.equal(dx.cpu(), wdx)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
def test_each_bias_gradient_is_its_difference(act):
    """Every element of dbias against the central difference of its own column's loss, step
    h = 2^-6. Z is whole numbers and quarters below 64, which bf16 holds exactly, so the backward
    sees the forward's Z. A difference is off by h^2/6 max|act'''| of the sum of |dY| (silu''' and
    gelu''' below 0.8; swiglu 0.5 |up|, as the other half stands still) and by 2^-20 (|Z| + |Y|) / h
    of |dY| for the two outputs' errors; dbias itself by 2^-18 of its terms."""
    counts, n_in, n_out, h = [40, 0, 90], 64, 72, 2.0 ** -6
    R, E, N = sum(counts), len(counts), n_out * (2 if act == "swiglu" else 1)
    x, w = whole((R, n_in), 1), whole((E, N, n_in), 2)
    bias = (torch.randint(0, 4, (E, N), generator=torch.Generator().manual_seed(3)) + 0.5) / 4
    if act != "relu":  # relu: an eighth keeps Z away from the corner
        bias = bias - 0.125
    dy = torch.randn((R, n_out), generator=torch.Generator().manual_seed(4)).to(BF)
    off = torch.tensor([0, 40, 40, 130], dtype=torch.int32, device="cuda")
    cfg, wide = bm.linear_cfg(n_in, n_out, E, act), bm.linear_cfg(n_in, n_out, E, act, out_fp32=True)
    ws = torch.empty(bm.beam_moe_linear_workspace_size(cfg, R, True), dtype=torch.uint8,
                     device="cuda")
    xd, wd = x.cuda(), w.cuda()

    def forward(b):
        y = torch.empty((R, n_out), device="cuda")
        z = torch.empty((R, N), dtype=BF, device="cuda")
        bm.beam_moe_linear(wide, xd, wd, y, ws, bias=b.cuda(), offsets=off, z=z)
        return y.cpu().double(), z

    y, zd = forward(bias)
    db = torch.empty((E, N), device="cuda")
    bm.beam_moe_linear_backward(cfg, dy.cuda(), None, None, ws, dbias=db, offsets=off,
                                z=None if act == "none" else zd)
    z, dyd, db = zd.cpu().double(), dy.double(), db.cpu().double()
    terms = ref.act_grad_terms(dyd, z, act).abs()
    for half in range(N // n_out):
        step = torch.zeros((E, N))
        step[:, half * n_out:(half + 1) * n_out] = h
        diff = (forward(bias + step)[0] - forward(bias - step)[0]) / (2 * h) * dyd
        third = 0.0 if act in ("none", "relu") else 0.8
        if act == "swiglu":
            third = 0.5 * z[:, n_out:].abs() if half == 0 else 0.0
        each = dyd.abs() * (h * h / 6 * third
                            + 2.0 ** -20 * (z.abs().reshape(R, -1, n_out).amax(1) + y.abs() + 1) / h)
        for e, (a, b) in enumerate(((0, 40), (40, 40), (40, 130))):
            cols = slice(half * n_out, (half + 1) * n_out)
            tol = each[a:b].sum(0) + 2.0 ** -18 * terms[a:b, cols].sum(0)
            assert bool(((diff[a:b].sum(0) - db[e, cols]).abs() <= tol).all()), (act, half, e)


@pytest.mark.parametrize("R", [2, 9, 64, 512, 3000])
def test_many_experts_at_full_width(R):
    """A batch over 256 experts of the block's own width, 5120 -> 2 x 2560 and back, decode to a
    small prefill: one row an expert or none, and a few. x has one value per row and 64 columns,
    so that Z is exact (a product of two bf16 numbers sums to one term per row) and each row shows
    which weights it met."""
    E, H, I = 256, 5120, 2560
    g = torch.Generator(device="cuda").manual_seed(R)
    w = (torch.randint(1, 128, (E, 2 * I, 1), generator=g, device="cuda").float() / 64).to(BF)
    w13 = w * torch.ones((1, 1, H), device="cuda", dtype=BF)
    pick = torch.randint(0, E, (R,), generator=g, device="cuda").sort().values
    off = torch.searchsorted(pick, torch.arange(E + 1, device="cuda")).int()
    x = torch.zeros((R, H), dtype=BF, device="cuda")
    at = torch.randint(0, H, (R,), generator=g, device="cuda")
    v = (torch.randint(-64, 65, (R,), generator=g, device="cuda").float() / 16).to(BF)
    x[torch.arange(R), at] = v
    cfg = bm.linear_cfg(H, I, E, "swiglu")
    ws = torch.empty(bm.beam_moe_linear_workspace_size(cfg, R, True), dtype=torch.uint8,
                     device="cuda")
    h = torch.full((R, I), LEFT, dtype=BF, device="cuda")
    z = torch.full((R, 2 * I), LEFT, dtype=BF, device="cuda")
    bm.beam_moe_linear(cfg, x, w13, h, ws, offsets=off, z=z)
    assert bm.beam_moe_check(ws) == 0
    want = v.double()[:, None] * w[pick, :, 0].double()
    assert torch.equal(z, want.to(BF))
    act = ref.act(want, "swiglu")
    # half a step, and 2^-18 for the FP32 arithmetic before it
    assert bool(((h.double() - act).abs() <= (2.0 ** -8 + 2.0 ** -18) * act.abs()).all())
    # dX: one row of W_e at a time comes back; dW: every expert's own outer products
    dz = torch.zeros((R, 2 * I), dtype=BF, device="cuda")
    col = torch.randint(0, 2 * I, (R,), generator=g, device="cuda")
    dz[torch.arange(R), col] = 2.0
    plain = bm.linear_cfg(H, 2 * I, E)
    dx = torch.full((R, H), LEFT, dtype=BF, device="cuda")
    dw = torch.full((E, 2 * I, H), LEFT, dtype=BF, device="cuda")
    ws = torch.empty(bm.beam_moe_linear_workspace_size(plain, R, True), dtype=torch.uint8,
                     device="cuda")
    bm.beam_moe_linear_backward(plain, dz, x, w13, ws, dx=dx, dw=dw, offsets=off)
    assert bm.beam_moe_check(ws) == 0
    assert torch.equal(dx, (2 * w13[pick, col].float()).to(BF))
    wdw = torch.zeros((E, 2 * I, H), dtype=torch.float32, device="cuda")
    wdw.index_put_((pick, col, at), 2 * v.float(), accumulate=True)
    assert torch.equal(dw, wdw.to(BF))


def test_tensors_without_a_dimension_are_refused():
    c, lc = bm.rows_cfg(16, 4, 2), bm.linear_cfg(16, 8)
    bad = torch.zeros((), dtype=BF, device="cuda")
    x = torch.zeros((3, 16), dtype=BF, device="cuda")
    pos = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    w = torch.zeros((1, 8, 16), dtype=BF, device="cuda")
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    for call in (lambda: bm.beam_moe_permute(c, bad, pos, x, pos, off, ws),
                 lambda: bm.beam_moe_permute_backward(c, bad, pos, x),
                 lambda: bm.beam_moe_permute_backward(c, x, pos, bad),
                 lambda: bm.beam_moe_permute_backward(c, None, pos, x),
                 lambda: bm.beam_moe_combine(c, bad, pos, None, x),
                 lambda: bm.beam_moe_combine(c, x, pos, None, bad),
                 lambda: bm.beam_moe_combine_backward(c, x, bad, pos, None, x, None),
                 lambda: bm.beam_moe_combine_backward(c, x, None, pos, None, None, None),
                 lambda: bm.beam_moe_linear(lc, bad, w, x, ws),
                 lambda: bm.beam_moe_linear_backward(lc, bad, x, w, ws, dx=x)):
        with pytest.raises(ValueError):
            call()
