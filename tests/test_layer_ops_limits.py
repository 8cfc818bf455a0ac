"""The row and linear operators at the limits of what their documentation allows, on the host:
offsets that do not ascend, sizes, first use by several threads (no GPU needed)."""
import random
import sys

import pytest

import sparse_moe_layer_beam_b200 as bm
from tests import _layer_ops as ref


def offset_vectors(E, rows, seed):
    """Offsets that break every promise: each second expert has all rows, descending ones, and
    random ones that point outside [0, rows], too."""
    rng = random.Random(seed)
    yield [rows * (e % 2) for e in range(E + 1)]
    yield [rows - e * rows // E for e in range(E + 1)]
    for _ in range(20):
        yield [rng.randint(-rows, 2 * rows) for _ in range(E + 1)]
        yield [rng.choice((0, rows, 2 ** 31 - 1, -2 ** 31)) for _ in range(E + 1)]


@pytest.mark.parametrize("E,rows,n_out", [(512, 100, 64), (4, 1000, 520), (32, 16384, 2560),
                                          (3, 7, 8), (200, 40000, 1024)])
def test_any_offsets_fit_the_workspace(E, rows, n_out):
    """Segments lie one behind the other, so a backward's partial sums (a row of n_out floats per
    block of 32 rows, or of 128 where there are enough of those) fit what it asks for."""
    have = bm.beam_moe_linear_workspace_size(bm.linear_cfg(64, n_out, E), rows, True)
    block = 32 if rows // 128 * -(-n_out // 256) < 512 else 128
    for off in offset_vectors(E, rows, E + rows):
        seg = ref.segments(off, rows)
        assert all(0 <= a <= b <= rows for a, b in seg)
        full = [s for s in seg if s[0] < s[1]]
        assert all(p[1] <= q[0] for p, q in zip(full, full[1:]))
        blocks = sum(-(-(b - a) // block) for a, b in seg)
        assert blocks <= rows // block + min(E, rows)
        assert 256 + blocks * n_out * 4 <= have


def test_nothing_to_do_is_no_error():
    """Empty outputs may have no address: no tokens, or no rows with only their gradient asked."""
    L, a = bm.lib(), 1 << 20
    c = bm.rows_cfg(64, 8, 2)
    assert L.beam_moe_combine_backward(c, 0, 0, None, None, 0, None, None, None, None, None) == 0
    assert L.beam_moe_combine_backward(c, 5, 0, a, None, 0, a, a, None, None, None) == 0
    lc = bm.linear_cfg(64, 128)
    assert L.beam_moe_linear_backward(lc, 0, None, None, a, None, None, None, None, None, None,
                                      0, None) == 0


@pytest.mark.parametrize("E,n_out,act", [(1, 5120, "none"), (32, 2560, "swiglu"), (512, 64, "gelu"),
                                         (3, 8, "relu"), (256, 65536, "none"), (7, 520, "silu")])
def test_a_workspace_serves_fewer_rows(E, n_out, act):
    """A program keeps one workspace, sized for its largest batch: no smaller one asks for more.
    (Row blocks of the backward change from 32 to 128 rows where rows // 128 * ceil(n_out / 256)
    reaches 512.)"""
    c = bm.linear_cfg(64, n_out, E, act)
    switch = -(-512 // -(-n_out // 256)) * 128
    rows = sorted({r for s in (1, switch, 4 * switch) for r in range(max(0, s - 300), s + 300)}
                  | {2 ** i + d for i in range(22) for d in (-1, 0, 1)})
    sizes = [bm.beam_moe_linear_workspace_size(c, r, True) for r in rows]
    assert sizes == sorted(sizes)
    assert all(bm.beam_moe_linear_workspace_size(c, r) <= s for r, s in zip(rows, sizes))
    r = bm.rows_cfg(64, 512, 8)
    sizes = [bm.beam_moe_permute_workspace_size(r, t) for t in range(900, 1200)]
    assert sizes == sorted(sizes)


def test_first_use_by_several_threads(monkeypatch):
    """A call takes the binding as ready once _types is there: at no line of its set-up may
    another thread find that and not the rest."""
    for name in ("_types", "_device", "_raw_stream"):
        monkeypatch.setattr(bm, name, None)
    half_ready = []

    def trace(frame, event, arg):
        if frame.f_code is not bm._bind_torch.__code__:
            return None
        if bm._types is not None and (bm._device is None or bm._raw_stream is None):
            half_ready.append(frame.f_lineno)
        return trace

    old = sys.gettrace()
    sys.settrace(trace)
    try:
        bm._bind_torch()
    finally:
        sys.settrace(old)
    assert bm._types and bm._device and bm._raw_stream and not half_ready


@pytest.mark.parametrize("T", [(1 << 28) + 1, 1 << 58, 1 << 60, (1 << 60) + 1, 1 << 62,
                               (1 << 63) - 1])
def test_more_tokens_than_are_supported(T):
    """T * top_k beyond 2^30, where the product leaves 64 bits too."""
    a, L = 1 << 20, bm.lib()
    for K in (4, 16, 32):
        c = bm.rows_cfg(64, 40, K)
        with pytest.raises(bm.BeamMoeError) as e:
            bm.beam_moe_permute_workspace_size(c, T)
        assert e.value.status == 2
        assert L.beam_moe_permute(c, T, a, a, a, a, a, a, 1 << 62, None) == 2
        assert L.beam_moe_combine(c, T, 9, a, 0, a, a, a, None) == 2
        assert L.beam_moe_combine_backward(c, T, 9, a, a, 0, a, a, a, a, None) == 2
    assert bm.beam_moe_permute_workspace_size(bm.rows_cfg(64, 40, 4), 1 << 28) > 1 << 31
    lc = bm.linear_cfg(64, 64)
    with pytest.raises(bm.BeamMoeError) as e:
        bm.beam_moe_linear_workspace_size(lc, T)
    assert e.value.status == 2
