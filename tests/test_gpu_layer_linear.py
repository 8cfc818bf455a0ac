"""linear and its gradients on the GPU against their formulas in 64 bits.

Tolerances, beyond half a step of each 16-bit output. The tensor cores sum n exact products in
FP32 with n additions that lose at most one step, 2^-23 of the sum of magnitudes S each: n 2^-23
S. An activation passes an error of z on times its largest slope (1.13; swiglu: the other half's
size times 1.1) and is itself computed within 2^-20 of |z| + |act|. dX and dW are products of
the dZ that the kernel rounds to 16 bits: their elements' roundings are independent and at most
half a step, so the error's RMS over an output is at most that of one half step of each term
plus that of the output's own rounding, eps/2 each of the output's RMS for products of
independent terms; the sum is held to eps. Each element is held to the sum of its terms' half
steps.
"""
import pytest
import torch

import sparse_moe_layer_beam_b200 as bm
from tests import _layer_ops as ref

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
LEFT = 7.0


def offsets_of(counts):
    return torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32)


def make(counts, tail, n_in, n_out, act, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    E, R = len(counts), sum(counts) + tail
    N = n_out * (2 if act == "swiglu" else 1)
    t = TYPES[dtype]
    d = {"x": torch.randn((R, n_in), generator=g).to(t),
         "w": (torch.randn((E, N, n_in), generator=g) / n_in ** 0.5).to(t),
         "bias": torch.randn((E, N), generator=g) * 0.2,
         "z": (torch.randn((R, N), generator=g) * 1.5).to(t),
         "dy": torch.randn((R, n_out), generator=g).to(t),
         "off": offsets_of(counts)}
    return d, E, R, N


def segments(off):
    return [(e, int(off[e]), int(off[e + 1])) for e in range(len(off) - 1)]


def forward_ref(d, act, residual):
    """(z, y, slack of z, slack of y) in 64 bits; rows outside the segments NaN."""
    R, N = d["x"].shape[0], d["w"].shape[1]
    n_in = d["x"].shape[1]
    z = torch.full((R, N), float("nan"), dtype=torch.float64)
    sz = torch.zeros_like(z)
    for e, a, b in segments(d["off"]):
        x, w = d["x"][a:b].double(), d["w"][e].double()
        z[a:b] = x @ w.T
        sz[a:b] = (n_in + 1) * 2.0 ** -23 * (x.abs() @ w.abs().T)
        if d.get("use_bias"):
            z[a:b] += d["bias"][e].double()
            sz[a:b] += 2.0 ** -23 * z[a:b].abs()
    y = ref.act(z, act)
    if act == "swiglu":
        (g, u), (sg, su) = z.chunk(2, -1), sz.chunk(2, -1)
        sy = 1.1 * u.abs() * sg + (g.abs() + 0.3) * su + 2.0 ** -20 * (y.abs() + g.abs())
    else:
        sy = 1.13 * sz + 2.0 ** -20 * (z.abs() + y.abs())
    if residual is not None:
        y = y + residual.double()
        sy = sy + 2.0 ** -23 * y.abs()
    return z, y, sz, sy


def run_forward(d, E, act, dtype, n_in, n_out, residual=None, out32=False, want_z=True, bias=True):
    R, N = d["x"].shape[0], d["w"].shape[1]
    cfg = bm.linear_cfg(n_in, n_out, E, act, dtype, out32)
    out_t = torch.float32 if out32 else TYPES[dtype]
    y = torch.full((R, n_out), LEFT, dtype=out_t, device="cuda")
    z = torch.full((R, N), LEFT, dtype=TYPES[dtype], device="cuda") if want_z else None
    ws = torch.empty(bm.beam_moe_linear_workspace_size(cfg, R), dtype=torch.uint8, device="cuda")
    bm.beam_moe_linear(cfg, d["x"].cuda(), d["w"].cuda(), y, ws,
                       bias=d["bias"].cuda() if bias else None,
                       residual=None if residual is None else residual.cuda(),
                       offsets=d["off"].cuda() if E > 1 else None, z=z)
    assert bm.beam_moe_check(ws) == 0
    return y.cpu(), None if z is None else z.cpu()


# counts per expert, rows behind them, n_in, n_out, act, dtype: single rows and tokens (the
# contraction split over clusters), ragged row blocks, empty experts, widths that are no
# multiple of a tile or of 64, enough tiles for 128- and 256-column tiles
CASES = [
    ([1], 0, 8, 8, "none", "bf16"),
    ([1], 0, 5120, 640, "gelu", "bf16"),
    ([3], 0, 1000, 264, "relu", "fp16"),
    ([4], 0, 2056, 40, "swiglu", "bf16"),
    ([0, 1, 0, 2, 0], 1, 328, 72, "gelu", "bf16"),  # up to four rows in all: one row at a time
    ([0] * 40 + [1, 1], 2, 136, 200, "swiglu", "fp16"),
    ([1] + [0] * 510 + [2], 0, 64, 72, "silu", "bf16"),
    ([0] * 200 + [1] + [0] * 112, 1, 72, 64, "none", "fp16"),
    ([5], 0, 5120, 264, "swiglu", "bf16"),
    ([129], 0, 72, 136, "silu", "bf16"),
    ([300], 0, 520, 1320, "gelu_tanh", "fp16"),
    ([1, 0, 5, 130], 7, 200, 72, "swiglu", "bf16"),
    ([0, 0, 64, 1, 257, 0], 3, 128, 264, "none", "fp16"),
    ([0, 0, 0], 5, 64, 64, "gelu", "bf16"),
    ([2] * 60 + [0] * 4 + [40], 0, 320, 328, "swiglu", "bf16"),  # 128-column tiles
    ([100] * 9 + [517], 1, 256, 2600, "silu", "bf16"),           # 256-column tiles
    ([700, 0, 2300], 0, 1032, 1288, "swiglu", "fp16"),           # CTA pairs from here on
    ([129, 300, 0, 513], 2, 1032, 5128, "gelu", "bf16"),
    ([1400], 0, 1096, 3208, "none", "fp16"),
    ([400, 100, 1, 900], 0, 2312, 1672, "swiglu", "bf16"),
]


@pytest.mark.parametrize("out32", [False, True])
@pytest.mark.parametrize("counts,tail,n_in,n_out,act,dtype", CASES)
def test_forward(counts, tail, n_in, n_out, act, dtype, out32):
    d, E, R, N = make(counts, tail, n_in, n_out, act, dtype, n_in + n_out)
    d["use_bias"] = True
    res = torch.randn((R, n_out), generator=torch.Generator().manual_seed(1))
    res = res if out32 else res.to(TYPES[dtype])
    y, z = run_forward(d, E, act, dtype, n_in, n_out, res, out32)
    wz, wy, sz, sy = forward_ref(d, act, res)
    n = sum(counts)
    half = ref.HALF_STEP[TYPES[dtype]]
    tiny = ref.TINY[TYPES[dtype]]
    assert bool(((z[:n].double() - wz[:n]).abs() <= sz[:n] * 1.01 + half * wz[:n].abs() * 1.01
                 + tiny).all())
    half = 2.0 ** -24 if out32 else half
    assert bool(((y[:n].double() - wy[:n]).abs() <= sy[:n] * 1.01 + half * wy[:n].abs() * 1.01
                 + tiny).all())
    assert bool((y[n:] == LEFT).all()) and bool((z[n:] == LEFT).all())  # behind the last expert
    # without bias, residual and z: the plain product, activated
    d["use_bias"] = False
    y, _ = run_forward(d, E, act, dtype, n_in, n_out, None, out32, False, False)
    _, wy, _, sy = forward_ref(d, act, None)
    assert bool(((y[:n].double() - wy[:n]).abs() <= sy[:n] * 1.01 + half * wy[:n].abs() * 1.01
                 + tiny).all())


def run_backward(d, E, act, dtype, n_in, n_out, which=("dx", "dw", "dbias")):
    R, N = d["x"].shape[0], d["w"].shape[1]
    cfg = bm.linear_cfg(n_in, n_out, E, act, dtype)
    t = TYPES[dtype]
    got = {"dx": torch.full((R, n_in), LEFT, dtype=t, device="cuda"),
           "dw": torch.full((E, N, n_in), LEFT, dtype=t, device="cuda"),
           "dbias": torch.full((E, N), LEFT, device="cuda")}
    got = {k: v for k, v in got.items() if k in which}
    ws = torch.empty(bm.beam_moe_linear_workspace_size(cfg, R, True), dtype=torch.uint8,
                     device="cuda")
    bm.beam_moe_linear_backward(cfg, d["dy"].cuda(), d["x"].cuda() if "dw" in which else None,
                                d["w"].cuda() if "dx" in which else None, ws, **got,
                                z=None if act == "none" else d["z"].cuda(),
                                offsets=d["off"].cuda() if E > 1 else None)
    assert bm.beam_moe_check(ws) == 0
    return {k: v.cpu() for k, v in got.items()}


def check_product(got, a, b, half_a, n, dtype, name, more):
    """got = a b: a's elements rounded within half_a relative, n products a sum, `more` from
    a's own error before its rounding."""
    want, mag = a @ b, a.abs() @ b.abs()
    half = ref.HALF_STEP[TYPES[dtype]]
    err = (got.double() - want).abs()
    # where a is below the type's normal numbers its rounding is half its smallest step instead
    if half_a:
        more = more + 0.5 * ref.TINY[TYPES[dtype]] * b.abs().sum(0)
    tol = ((half_a + n * 2.0 ** -23) * mag + half * want.abs() + more) * 1.01 + ref.TINY[TYPES[dtype]]
    assert bool((err <= tol).all()), (name, (err - tol).max())
    if want.numel() > 1000:
        rms = lambda v: v.square().mean().sqrt().item()  # noqa: E731
        assert rms(err) <= 2 * half * rms(want), (name, rms(err) / rms(want))


@pytest.mark.parametrize("counts,tail,n_in,n_out,act,dtype", CASES)
def test_backward(counts, tail, n_in, n_out, act, dtype):
    d, E, R, N = make(counts, tail, n_in, n_out, act, dtype, n_in + n_out + 1)
    n = sum(counts)
    for k in ("x", "dy", "z"):
        d[k][n:] = float("nan")  # rows that belong to no expert
    got = run_backward(d, E, act, dtype, n_in, n_out)
    dz = ref.act_grad(d["dy"].double(), d["z"].double(), act)
    # dZ in FP32 before its rounding: some ten operations of 2^-24 and an exponential within
    # 2^-20 on terms that may cancel (every slope but relu's crosses zero)
    off = torch.zeros_like(dz) if act == "none" else 2.0 ** -18 * ref.act_grad_terms(
        d["dy"].double(), d["z"].double(), act)
    half = 0.0 if act == "none" else ref.HALF_STEP[TYPES[dtype]]
    for e, a, b in segments(d["off"]):
        w, x = d["w"][e].double(), d["x"][a:b].double()
        check_product(got["dx"][a:b], dz[a:b], w, half, N, dtype, "dx", off[a:b] @ w.abs())
        check_product(got["dw"][e], dz[a:b].T, x, half, b - a, dtype, "dw", off[a:b].T @ x.abs())
        # FP32 chains of at most 16 rows, then 8, then the blocks: under 64 + rows/1024 additions
        want, mag = dz[a:b].sum(0), dz[a:b].abs().sum(0)
        tol = (64 + (b - a) / 1024) * 2.0 ** -24 * mag + off[a:b].sum(0) + 1e-30
        assert bool(((got["dbias"][e].double() - want).abs() <= tol).all())
    assert bool((got["dx"][n:] == LEFT).all())
    for k in got:  # each gradient alone is the same, bit for bit
        assert torch.equal(run_backward(d, E, act, dtype, n_in, n_out, (k,))[k], got[k]), k


def test_experts_do_not_touch_each_other():
    """NaN in one expert's rows, weights and bias stays there: row blocks, contraction tails
    (n_out no multiple of 64) and the rows of a step behind a segment belong to others."""
    counts, n_in, n_out = [70, 31, 5, 200], 200, 136
    for act in ("none", "swiglu"):
        d, E, R, N = make(counts, 0, n_in, n_out, act, "bf16", 3)
        clean = run_forward(d, E, act, "bf16", n_in, n_out)
        clean_b = run_backward(d, E, act, "bf16", n_in, n_out)
        for bad in range(E):
            a, b = int(d["off"][bad]), int(d["off"][bad + 1])
            dirty = {k: v.clone() for k, v in d.items()}
            for k in ("x", "dy", "z"):
                dirty[k][a:b] = float("nan")
            dirty["w"][bad] = float("inf")
            dirty["bias"][bad] = float("nan")
            y, z = run_forward(dirty, E, act, "bf16", n_in, n_out)
            got = run_backward(dirty, E, act, "bf16", n_in, n_out)
            rows = torch.ones(R, dtype=torch.bool)
            rows[a:b] = False
            exp = torch.arange(E) != bad
            assert torch.equal(y[rows], clean[0][rows]) and torch.equal(z[rows], clean[1][rows])
            assert bool(y[a:b].isnan().all())
            assert torch.equal(got["dx"][rows], clean_b["dx"][rows])
            assert torch.equal(got["dw"][exp], clean_b["dw"][exp])
            assert torch.equal(got["dbias"][exp], clean_b["dbias"][exp])


def test_bias_gradient_is_the_difference():
    """Central differences of FP32 outputs along a direction of the biases, step h = 2^-5: off
    by h^2/6 |act'''| <= 2e-4 of the sum of |dy direction| and the outputs' rounding
    2^-23 / h of their magnitude; held to 1e-3 of the sum of magnitudes."""
    counts, n_in, n_out = [40, 0, 90], 64, 72
    for act in ("silu", "gelu", "gelu_tanh", "swiglu", "none"):
        d, E, R, N = make(counts, 0, n_in, n_out, act, "bf16", 4)
        direction = torch.randn((E, N), generator=torch.Generator().manual_seed(5))

        def loss(b):
            y, z = run_forward({**d, "bias": b}, E, act, "bf16", n_in, n_out, out32=True)
            return (y.double() * d["dy"].double()), z
        (up, _), (down, _), (_, z) = (loss(d["bias"] + 2.0 ** -5 * direction),
                                      loss(d["bias"] - 2.0 ** -5 * direction), loss(d["bias"]))
        diff = (up - down).sum().item() / 2.0 ** -4
        got = run_backward({**d, "z": z}, E, act, "bf16", n_in, n_out, ("dbias",))["dbias"]
        grad = (got.double() * direction.double()).sum().item()
        scale = (got.double() * direction.double()).abs().sum().item() + R * 3
        # z comes back rounded to bf16: |act''| <= 0.8 times half a step of |z| ~ 3, averaged out
        assert abs(diff - grad) <= 3e-3 * scale, (act, diff, grad, scale)


def test_residual_in_place_and_no_rows():
    d, E, R, N = make([37], 0, 72, 80, "none", "bf16", 6)
    res = torch.randn((R, 80)).bfloat16()
    want, _ = run_forward(d, 1, "none", "bf16", 72, 80, res)
    cfg = bm.linear_cfg(72, 80)
    y = res.cuda()
    ws = torch.empty(bm.beam_moe_linear_workspace_size(cfg, R), dtype=torch.uint8, device="cuda")
    bm.beam_moe_linear(cfg, d["x"].cuda(), d["w"].cuda(), y, ws, bias=d["bias"].cuda(), residual=y)
    assert torch.equal(y.cpu(), want)
    e = lambda n: torch.empty((0, n), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    dw = torch.ones((1, 80, 72), dtype=torch.bfloat16, device="cuda")
    db = torch.ones((1, 80), device="cuda")
    bm.beam_moe_linear(cfg, e(72), d["w"].cuda(), e(80), ws)
    bm.beam_moe_linear_backward(cfg, e(80), e(72), d["w"].cuda(), ws, dx=e(72), dw=dw, dbias=db)
    assert not dw.any() and not db.any()


def test_offsets_are_cut_off_at_the_rows():
    """Offsets that point outside [0, rows] or run backwards: what they cut off is no row."""
    d, E, R, N = make([50, 50], 0, 64, 72, "none", "bf16", 7)
    d["use_bias"] = True
    d["off"] = torch.tensor([-5, 60, 1000], dtype=torch.int32)
    y, _ = run_forward(d, 2, "none", "bf16", 64, 72)
    d["off"] = torch.tensor([0, 60, 100], dtype=torch.int32)
    want, _ = run_forward(d, 2, "none", "bf16", 64, 72)
    assert torch.equal(y, want)
    d["off"] = torch.tensor([80, 30, 90], dtype=torch.int32)  # expert 0: none, expert 1: 30..89
    y, _ = run_forward(d, 2, "none", "bf16", 64, 72)
    assert bool((y[:30] == LEFT).all()) and bool((y[90:] == LEFT).all())
    d["off"] = torch.tensor([0, 30, 90], dtype=torch.int32)
    want, _ = run_forward(d, 2, "none", "bf16", 64, 72)
    assert torch.equal(y[30:90], want[30:90])
    d["off"] = torch.tensor([80, 30, 90], dtype=torch.int32)
    assert not run_backward(d, 2, "none", "bf16", 64, 72)["dw"][0].any()
