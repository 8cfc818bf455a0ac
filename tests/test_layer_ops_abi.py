"""The row and linear operators on the host: sizes, refusals before any CUDA call, and the
64-bit formulas the GPU tests use against numerical differences (no GPU needed)."""
import ctypes

import pytest
import torch

import sparse_moe_layer_beam_b200 as bm
from tests import _layer_ops as ref

OK, INVALID, UNSUPPORTED, ALIGN, WS_SMALL = 0, 1, 2, 3, 4
A = 1 << 20  # aligned, never dereferenced: every call below is refused first


def rows_ws(c, T):
    n = ctypes.c_size_t(0)
    return bm.lib().beam_moe_permute_workspace_size(ctypes.byref(c), T, ctypes.byref(n)), n.value


def lin_ws(c, rows, backward=0):
    n = ctypes.c_size_t(0)
    return (bm.lib().beam_moe_linear_workspace_size(ctypes.byref(c), rows, backward,
                                                    ctypes.byref(n)), n.value)


@pytest.mark.parametrize("field,value,code", [
    ("width", 0, INVALID), ("width", 65537, UNSUPPORTED), ("n_experts", 0, INVALID),
    ("n_experts", 513, UNSUPPORTED), ("top_k", 0, INVALID), ("top_k", 33, UNSUPPORTED),
    ("dtype", 3, INVALID), ("dtype", -1, INVALID)])
def test_bad_rows_configuration(field, value, code):
    c = bm.rows_cfg(1024, 16, 4)
    assert rows_ws(c, 64)[0] == OK
    setattr(c, field, value)
    assert rows_ws(c, 64)[0] == code
    L = bm.lib()
    assert L.beam_moe_permute(ctypes.byref(c), 64, A, A, A, A, A, A, 1 << 30, None) == code
    assert L.beam_moe_permute_backward(ctypes.byref(c), 64, 9, A, A, A, None) == code
    assert L.beam_moe_combine(ctypes.byref(c), 64, 9, A, 0, A, A, A, None) == code
    assert L.beam_moe_combine_backward(ctypes.byref(c), 64, 9, A, A, 0, A, A, A, A, None) == code


def test_row_calls_refuse_bad_arguments():
    c = bm.rows_cfg(1024, 16, 4)
    L, r = bm.lib(), ctypes.byref(c)
    T = 5000  # 20000 assignments: sorted through the workspace
    st, need = rows_ws(c, T)
    assert st == OK and need >= 2 * T * 4
    assert rows_ws(c, -1)[0] == INVALID and rows_ws(c, 1 << 29)[0] == UNSUPPORTED
    good = [A, A, A, A, A, A]
    for i in range(6):
        bad = list(good)
        bad[i] = None
        assert L.beam_moe_permute(r, T, *bad, need, None) == INVALID
        bad[i] = A + 8
        assert L.beam_moe_permute(r, T, *bad, need, None) == ALIGN
    assert L.beam_moe_permute(r, T, *good, need - 1, None) == WS_SMALL
    assert L.beam_moe_permute(r, 0, None, None, None, None, None, None, 0, None) == INVALID
    assert L.beam_moe_permute_backward(r, 0, 0, None, None, None, None) == OK
    assert L.beam_moe_permute_backward(r, T, -1, A, A, A, None) == INVALID
    assert L.beam_moe_permute_backward(r, T, 9, A, A, None, None) == INVALID
    assert L.beam_moe_combine(r, 0, 0, None, 0, None, None, None, None) == OK
    assert L.beam_moe_combine(r, T, 9, A, 1, A, A, A, None) == INVALID  # fp16 rows of a bf16 layer
    assert L.beam_moe_combine(r, T, 9, A, 2, A, A + 4, A, None) == ALIGN
    assert L.beam_moe_combine(r, T, 9, None, 2, A, A, A, None) == INVALID
    assert L.beam_moe_combine_backward(r, T, 9, A, A, 0, A, A, None, None, None) == INVALID
    assert L.beam_moe_combine_backward(r, T, 9, A, None, 0, A, A, None, A, None) == INVALID
    assert L.beam_moe_combine_backward(r, T, 9, A, A, 0, A, A, A + 2, A, None) == ALIGN


@pytest.mark.parametrize("field,value,code", [
    ("n_in", 0, INVALID), ("n_in", 60, UNSUPPORTED), ("n_in", 65544, UNSUPPORTED),
    ("n_out", -8, INVALID), ("n_out", 100, UNSUPPORTED), ("n_experts", 0, INVALID),
    ("n_experts", 513, UNSUPPORTED), ("act", 6, INVALID), ("act", -1, INVALID),
    ("dtype", 2, INVALID), ("out_fp32", 2, INVALID)])
def test_bad_linear_configuration(field, value, code):
    c = bm.linear_cfg(64, 128, 4, "silu")
    assert lin_ws(c, 10)[0] == OK
    setattr(c, field, value)
    assert lin_ws(c, 10)[0] == code
    L = bm.lib()
    assert L.beam_moe_linear(ctypes.byref(c), 10, A, A, A, A, A, A, A, A, 1 << 30, None) == code
    assert L.beam_moe_linear_backward(ctypes.byref(c), 10, A, A, A, A, A, A, A, A, A, 1 << 30,
                                      None) == code


def test_linear_calls_refuse_bad_arguments():
    L = bm.lib()
    c = bm.linear_cfg(64, 128, 4, "swiglu")
    r = ctypes.byref(c)
    st, need = lin_ws(c, 1000)
    stb, needb = lin_ws(c, 1000, 1)
    assert st == stb == OK and needb >= need + 1000 * 256 * 2
    assert lin_ws(c, -1)[0] == INVALID and lin_ws(c, (1 << 22) + 1)[0] == UNSUPPORTED
    assert lin_ws(c, 1000, 2)[0] == INVALID
    f, b = L.beam_moe_linear, L.beam_moe_linear_backward
    assert f(r, 0, None, None, None, None, None, None, None, None, 0, None) == OK
    # x, w, bias, residual, offsets, y, z, ws
    good = [A] * 8
    for i, needed in enumerate((1, 1, 0, 0, 1, 1, 0, 1)):
        bad = list(good)
        if needed:
            bad[i] = None
            assert f(r, 1000, *bad, need, None) == INVALID, i
        bad[i] = A + 4
        assert f(r, 1000, *bad, need, None) == ALIGN, i
    assert f(r, 1000, *good, need - 1, None) == WS_SMALL
    # dy, x, w, z, offsets, dx, dw, dbias, ws
    good = [A] * 9
    for i, needed in enumerate((1, 1, 1, 1, 1, 0, 0, 0, 1)):
        bad = list(good)
        if needed:
            bad[i] = None
            assert b(r, 1000, *bad, needb, None) == INVALID, i
        bad[i] = A + 4
        assert b(r, 1000, *bad, needb, None) == ALIGN, i
    assert b(r, 1000, *good, needb - 1, None) == WS_SMALL
    assert b(r, 1000, A, A, A, A, A, None, None, None, A, needb, None) == INVALID


def test_the_binding_checks_its_tensors():
    c = bm.rows_cfg(16, 4, 2)
    x = torch.zeros((3, 16), dtype=torch.bfloat16)
    ids = torch.zeros((3, 2), dtype=torch.int32)
    xp = torch.zeros((6, 16), dtype=torch.bfloat16)
    off = torch.zeros(5, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    for bad in (dict(x=x.float()), dict(x=None), dict(x=torch.zeros((3, 32))[:, ::2].bfloat16().T),
                dict(topk_ids=ids.long()), dict(xp=xp[:5]), dict(offsets=off[:4]),
                dict(pos=ids.T), dict(x=torch.zeros((3, 32), dtype=torch.bfloat16)[:, :16])):
        args = dict(x=x, topk_ids=ids, xp=xp, pos=ids, offsets=off, ws=ws)
        args.update(bad)
        with pytest.raises(ValueError):
            bm.beam_moe_permute(c, **args)
    lc = bm.linear_cfg(16, 8)
    w = torch.zeros((1, 8, 16), dtype=torch.bfloat16)
    y = torch.zeros((3, 8), dtype=torch.bfloat16)
    for bad in (dict(w=w[0]), dict(y=y.float()), dict(bias=torch.zeros(8)), dict(y=None),
                dict(offsets=torch.zeros(2)), dict(z=y.float()), dict(ws=None)):
        args = dict(x=x, w=w, y=y, ws=ws)
        args.update(bad)
        with pytest.raises(ValueError):
            bm.beam_moe_linear(lc, **args)


@pytest.mark.parametrize("name", bm.ACTS)
def test_activation_gradients_are_the_differences(name):
    """Central differences of step h are off by h^2/6 max|act'''| (< 3 |dy| max(1, |up|) here)
    plus rounding 2^-52 |act| / h."""
    g = torch.Generator().manual_seed(3)
    z = torch.randn((50, 64), generator=g, dtype=torch.float64) * 2
    if name == "relu":
        z = torch.where(z.abs() < 1e-3, 1.0, z)  # away from the corner
    dy = torch.randn((50, 32 if name == "swiglu" else 64), generator=g, dtype=torch.float64)
    got = ref.act_grad(dy, z, name)
    h = 1e-5
    for j in (0, 13, 32, 63):
        d = torch.zeros_like(z)
        d[:, j] = h
        diff = ((ref.act(z + d, name) - ref.act(z - d, name)) / (2 * h) * dy).sum(1)
        assert (diff - got[:, j]).abs().max() < 1e-8
