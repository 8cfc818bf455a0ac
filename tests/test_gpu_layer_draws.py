"""The row and linear operators over the ranges they are measured on: drawn cases (odd widths,
dropped assignments, uneven experts, every type and activation) against the 64-bit results.

Tolerances, on the 2-norm of the difference over that of the result: a 16-bit result holds at
most two roundings of half a step each on the way (its own, and dZ's or none), so it is within
one step, 2 x 2^-8 (bf16) or 2 x 2^-11 (fp16). FP32 results hold sums of up to 5120 products:
the tensor cores' accumulation was measured at 3.0e-6 for 2560 and grows with the length, so
2e-5 is three times what 5120 gives.
"""
import random

import pytest
import torch

from perf import operators as ops

pytestmark = pytest.mark.gpu
BOUND = {torch.bfloat16: 2.0 ** -7, torch.float16: 2.0 ** -10, torch.float32: 2e-5}


def leaves(v, path="out"):
    if isinstance(v, dict):
        for k in sorted(v):
            yield from leaves(v[k], f"{path}.{k}")
    elif v is not None:
        yield path, v


@pytest.fixture
def own():
    ops.own = True
    yield
    ops.own = False


def check(case, seed):
    got = dict(leaves(ops.run(ops.prepare(case, seed))))
    for path, want in leaves(ops.exact(case, seed)):
        have = got[path]
        assert have.shape == want.shape
        norm = want.norm().item()
        off = (have.double() - want).norm().item()
        assert off <= BOUND[have.dtype] * norm, (case, path, off / max(norm, 1e-300))
    if case["op"] == "permute":  # the places, whole numbers, against the plain form's
        s = ops.prepare(case, seed)
        _, pos, offsets = ops._places(s["ids"], case["E"])
        assert torch.equal(got["out.pos"], pos) and torch.equal(got["out.offsets"], offsets)


@pytest.mark.parametrize("seed", range(40))
def test_drawn_cases(seed, own):
    check(ops.draw(random.Random(seed)), seed)
