"""permute, combine and their gradients on the GPU against their definitions in 64 bits.

Tolerances. Copies and places are exact. A combine is a chain of K FP32 FMAs: each rounds the
running sum once, so it is off by at most K 2^-24 sum|w y|, then half a step of the output's
type. dy is one FP32 product (2^-24 of it) and half a step. dw is an FP32 sum of H products in
per-thread chains of at most H/128 + 8 of them, joined by eight more additions: at most
(H/128 + 16) 2^-24 sum|dout y|.
"""
import numpy as np
import pytest
import torch

import sparse_moe_layer_beam_b200 as bm
from tests import _layer_ops as ref

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LEFT = 7.0  # what untouched rows hold


def routes(T, E, K, seed, dropped=0.0, same=False, skew=0.0):
    rng = np.random.default_rng(seed)
    score = rng.standard_normal((T, E)) + skew * (np.arange(E) < max(1, E // 16))
    ids = np.argsort(-score, axis=1)[:, :K].astype(np.int32)
    if same:  # experts that occur several times in a token's ids
        ids = rng.integers(0, max(1, E // 3), (T, K)).astype(np.int32)
    ids[rng.random((T, K)) < dropped] = -1
    return ids


def run_permute(x, ids, E, dtype):
    T, K = ids.shape
    cfg = bm.rows_cfg(x.shape[1], E, K, dtype)
    xp = torch.full((T * K, x.shape[1]), LEFT, dtype=x.dtype, device="cuda")
    pos = torch.full((T, K), -9, dtype=torch.int32, device="cuda")
    off = torch.full((E + 1,), -9, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(256, bm.beam_moe_permute_workspace_size(cfg, T)), dtype=torch.uint8,
                     device="cuda")
    bm.beam_moe_permute(cfg, x, torch.from_numpy(ids).cuda(), xp, pos, off, ws)
    return xp, pos, off


# one launch (at most 8192 assignments) and three; every copy unit; one expert; 512 experts
CASES = [
    # T, H, E, K, dtype, dropped, same, skew
    (1, 8, 1, 1, "bf16", 0.0, False, 0.0),
    (1, 5120, 256, 8, "bf16", 0.0, False, 0.0),
    (3, 1, 2, 2, "fp16", 0.0, False, 0.0),
    (7, 1003, 24, 3, "bf16", 0.2, False, 0.0),
    (64, 5120, 256, 8, "bf16", 0.0, False, 0.0),
    (33, 17, 512, 32, "fp32", 0.1, True, 0.0),
    (100, 130, 5, 4, "fp16", 1.0, False, 0.0),  # no assignment names an expert
    (1024, 64, 256, 8, "bf16", 0.0, False, 2.0),   # the last one-launch size
    (1025, 64, 256, 8, "bf16", 0.1, False, 2.0),   # the first three-launch size
    (2500, 33, 512, 7, "fp32", 0.3, True, 0.0),
    (9000, 24, 1, 1, "fp16", 0.0, False, 0.0),
    (4097, 258, 96, 6, "bf16", 0.0, False, 3.0),
    (3000, 16, 7, 32, "bf16", 0.05, True, 0.0),
]


@pytest.mark.parametrize("T,H,E,K,dtype,dropped,same,skew", CASES)
def test_permute_and_its_backward(T, H, E, K, dtype, dropped, same, skew):
    ids = routes(T, E, K, T + H, dropped, same, skew)
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, H), generator=g).to(TYPES[dtype])
    xp, pos, off = run_permute(x.cuda(), ids, E, dtype)
    want_pos, want_off, src = ref.places(ids, E)
    assert np.array_equal(pos.cpu().numpy(), want_pos)
    assert np.array_equal(off.cpu().numpy(), want_off)
    got, n = xp.cpu(), src.size
    assert torch.equal(got[:n], x[src // K])
    assert bool((got[n:] == LEFT).all())  # rows behind the last expert's

    dxp = torch.randn((T * K, H), generator=g).to(TYPES[dtype])
    dxp[n:] = float("nan")  # rows that no assignment has
    dx = torch.full((T, H), LEFT, dtype=TYPES[dtype], device="cuda")
    bm.beam_moe_permute_backward(bm.rows_cfg(H, E, K, dtype), dxp.cuda(), pos, dx)
    want, mag = ref.combine(dxp, want_pos, None)
    tol = K * 2.0 ** -24 * mag + ref.HALF_STEP[dx.dtype] * want.abs() * 1.01 + ref.TINY[dx.dtype]
    assert bool(((dx.cpu().double() - want).abs() <= tol).all())


@pytest.mark.parametrize("y_dtype", ["same", "fp32"])
@pytest.mark.parametrize("T,H,E,K,dtype,dropped,same,skew", CASES)
def test_combine_and_its_backward(T, H, E, K, dtype, dropped, same, skew, y_dtype):
    y_type = torch.float32 if y_dtype == "fp32" else TYPES[dtype]
    ids = routes(T, E, K, T + H + 1, dropped, same, skew)
    if T > 5:
        ids[T - T // 5:] = -1  # a batch padded at its end
    pos, _, src = ref.places(ids, E)
    rows = src.size + 3  # three rows that no slot names
    g = torch.Generator().manual_seed(T + 2)
    y = torch.randn((rows, H), generator=g).to(y_type)
    y[src.size:] = float("nan")
    w = torch.rand((T, K), generator=g) * 2 - 0.5
    w[torch.from_numpy(pos < 0)] = float("nan")  # weights of slots without a row
    dout = torch.randn((T, H), generator=g).to(TYPES[dtype])
    cfg = bm.rows_cfg(H, E, K, dtype)
    dpos = torch.from_numpy(pos.astype(np.int32)).cuda()
    out = torch.full((T, H), LEFT, dtype=TYPES[dtype], device="cuda")
    bm.beam_moe_combine(cfg, y.cuda(), dpos, w.cuda(), out)
    want, mag = ref.combine(y, pos, w)
    tol = K * 2.0 ** -24 * mag + ref.HALF_STEP[out.dtype] * want.abs() * 1.01 + ref.TINY[out.dtype]
    assert bool(((out.cpu().double() - want).abs() <= tol).all())

    dy = torch.full((rows, H), LEFT, dtype=y_type, device="cuda")
    dw = torch.full((T, K), LEFT, dtype=torch.float32, device="cuda")
    bm.beam_moe_combine_backward(cfg, dout.cuda(), y.cuda(), dpos, w.cuda(), dy, dw)
    got = dy.cpu()
    assert bool((got[src.size:] == LEFT).all())
    want = w.double().reshape(-1)[src][:, None] * dout.double()[src // K]
    tol = (ref.HALF_STEP[y_type] + 2.0 ** -23) * want.abs() + ref.TINY[y_type]
    assert bool(((got[:src.size].double() - want).abs() <= tol).all())
    prod = dout.double()[src // K] * y.double()[:src.size]
    want, mag = torch.zeros(T * K, dtype=torch.float64), torch.zeros(T * K, dtype=torch.float64)
    want[src], mag[src] = prod.sum(1), prod.abs().sum(1)
    tol = (H / 128 + 16) * 2.0 ** -24 * mag
    assert bool(((dw.cpu().double().reshape(-1) - want).abs() <= tol).all())

    one = torch.full_like(dy, LEFT)  # each gradient alone is the same
    bm.beam_moe_combine_backward(cfg, dout.cuda(), None, dpos, w.cuda(), one, None)
    assert torch.equal(one, dy)
    alone = torch.empty_like(dw)
    bm.beam_moe_combine_backward(cfg, dout.cuda(), y.cuda(), dpos, w.cuda(), None, alone)
    assert torch.equal(alone, dw)


def test_combine_without_weights_and_with_rows_out_of_range():
    T, H, E, K = 50, 96, 8, 4
    pos, _, src = ref.places(routes(T, E, K, 5), E)
    y = torch.randn((T * K - 20, H)).bfloat16()  # the last 20 rows do not exist
    cfg = bm.rows_cfg(H, E, K)
    bad = torch.from_numpy(pos.astype(np.int32))
    bad[0, 0], bad[1, 1] = 2 ** 31 - 1, -2 ** 31
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    bm.beam_moe_combine(cfg, y.cuda(), bad.cuda(), None, out)
    want, mag = ref.combine(y, bad.numpy().astype(np.int64), None)
    tol = K * 2.0 ** -24 * mag + 2.0 ** -8 * want.abs() * 1.01
    assert bool(((out.cpu().double() - want).abs() <= tol).all())
    dy = torch.full((T * K - 20, H), LEFT, dtype=torch.bfloat16, device="cuda")
    dw = torch.empty((T, K), device="cuda")
    dout = torch.ones((T, H), dtype=torch.bfloat16, device="cuda")
    bm.beam_moe_combine_backward(cfg, dout, y.cuda(), bad.cuda(), None, dy, dw)
    there = (bad >= 0) & (bad < y.shape[0])
    assert bool((dw.cpu()[~there] == 0).all())
    named = torch.zeros(y.shape[0], dtype=torch.bool)
    named[bad[there].long()] = True
    assert bool((dy.cpu()[named] == 1).all()) and bool((dy.cpu()[~named] == LEFT).all())


def test_combine_gradients_are_the_differences():
    """The combine is linear in y and in w: with FP32 rows its differences are its gradients
    up to the rounding of the three sums (1e-4 of their magnitude is over 1000 roundings)."""
    T, H, E, K = 40, 72, 6, 3
    pos, _, src = ref.places(routes(T, E, K, 6, 0.2), E)
    g = torch.Generator().manual_seed(8)
    cfg = bm.rows_cfg(H, E, K, "fp32")
    y, dy_dir = (torch.randn((T * K, H), generator=g).cuda() for _ in range(2))
    w, w_dir = (torch.randn((T, K), generator=g).cuda() for _ in range(2))
    dout = torch.randn((T, H), generator=g).cuda()
    dpos = torch.from_numpy(pos.astype(np.int32)).cuda()

    def loss(yy, ww):
        out = torch.empty((T, H), device="cuda")
        bm.beam_moe_combine(cfg, yy, dpos, ww, out)
        return (out.double() * dout.double()).sum().item()

    dy, dw = torch.zeros_like(y), torch.empty_like(w)
    bm.beam_moe_combine_backward(cfg, dout, y, dpos, w, dy, dw)
    base = loss(y, w)
    for diff, grad in ((loss(y + dy_dir, w) - base, (dy.double() * dy_dir.double()).sum().item()),
                       (loss(y, w + w_dir) - base, (dw.double() * w_dir.double()).sum().item())):
        assert abs(diff - grad) <= 1e-4 * (abs(base) + abs(grad) + 100)


def test_no_tokens():
    cfg = bm.rows_cfg(64, 5, 2)
    off = torch.full((6,), -3, dtype=torch.int32, device="cuda")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    i = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    bm.beam_moe_permute(cfg, e, i, e, i, off, ws)
    assert off.tolist() == [0] * 6
    bm.beam_moe_combine(cfg, e, i, None, e)
    bm.beam_moe_permute_backward(cfg, e, i, e)
    torch.cuda.synchronize()
