"""The row and linear operators from their definitions, in 64 bits on the CPU, and their
gradients (tests only; nothing here calls the library)."""
import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# smallest steps of the types near zero (subnormals)
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


def places(ids, E):
    """(pos, offsets, src): the stable sort by expert, written as a loop over experts."""
    flat = np.asarray(ids).reshape(-1)
    pos = np.full(flat.size, -1, np.int64)
    offsets, src = [0], []
    for e in range(E):
        mine = np.nonzero(flat == e)[0]
        pos[mine] = len(src) + np.arange(mine.size)
        src.extend(mine.tolist())
        offsets.append(len(src))
    return pos.reshape(np.asarray(ids).shape), np.array(offsets), np.array(src, np.int64)


def segments(offsets, rows):
    """[(lo, hi)] of every expert: its rows of [offsets[e], offsets[e + 1]), cut off at [0, rows],
    that lie behind every expert's before it."""
    o = [min(max(int(v), 0), rows) for v in offsets]
    got, end = [], 0
    for a, b in zip(o, o[1:]):
        lo = max(a, end)
        got.append((lo, max(b, lo)))
        if b > a:
            end = max(end, b)
    return got


def combine(y, pos, w):
    """(sum_k w y[pos], sum_k |w y[pos]|) in 64 bits."""
    T, K = pos.shape
    out = torch.zeros((T, y.shape[1]), dtype=torch.float64)
    mag = torch.zeros_like(out)
    for k in range(K):
        p = torch.as_tensor(pos[:, k])
        ok = (p >= 0) & (p < y.shape[0])
        part = y.double()[p[ok]]
        if w is not None:
            part = part * w.double()[ok, k][:, None]
        out[ok] += part
        mag[ok] += part.abs()
    return out, mag


def act(z, name):
    """act(z) in 64 bits; swiglu: z is [gate | up]."""
    if name == "none":
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.special.erf(z / 2 ** 0.5))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * torch.special.expit(z)
    g, u = z.chunk(2, -1)
    return g * torch.special.expit(g) * u


def act_grad(dy, z, name):
    """dZ = dY act'(Z) by the derivatives' formulas, in 64 bits."""
    if name == "none":
        return dy
    if name == "relu":
        return torch.where(z > 0, dy, 0.0)
    if name == "gelu":
        pdf = torch.exp(-0.5 * z * z) / (2 * torch.pi) ** 0.5
        return dy * (0.5 * (1 + torch.special.erf(z / 2 ** 0.5)) + z * pdf)
    if name == "gelu_tanh":
        a = (2 / torch.pi) ** 0.5
        t = torch.tanh(a * (z + 0.044715 * z ** 3))
        return dy * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z))
    if name == "silu":
        s = torch.special.expit(z)
        return dy * (s + z * s * (1 - s))
    g, u = z.chunk(2, -1)
    s = torch.special.expit(g)
    return torch.cat((dy * u * (s + g * s * (1 - s)), dy * g * s), -1)


def act_grad_terms(dy, z, name):
    """Sum of the magnitudes of the terms that dZ adds up (slopes cross zero between them)."""
    dy = dy.abs()
    if name in ("none", "relu"):
        return act_grad(dy, z, name)
    if name == "swiglu":
        g, u = z.chunk(2, -1)
        s = torch.special.expit(g)
        return torch.cat((dy * u.abs() * (s + g.abs() * s * (1 - s)), dy * g.abs() * s), -1)
    up = act_grad(dy, z, name)  # cdf + z pdf and the like: the first term is the gate itself
    gate = torch.where(z == 0, 0.5, act(z, name) / torch.where(z == 0, 1.0, z)) * dy
    return gate + (up - gate).abs()
