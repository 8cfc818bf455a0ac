"""What the row and linear operators of the library compute, and cases to measure them on.

The operators are the parts of a mixture-of-experts layer around the router: token rows
sorted by expert (permute) and back with the routing weights applied (combine), the product
of each expert's rows with that expert's weights with bias, activation and residual in its
epilogue (linear), and the gradients of all three. run() computes a pass in a plain form out
of elementary torch operations in 32 bits, or, where `own` is true, makes the library's
calls. exact() gives the same results in 64 bits, from the definitions.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
ROW_OPS = ("permute", "permute_backward", "combine", "combine_backward")


# ---------------------------------------------------------------------- cases

def _rows(name, op, T, H, E, K, dtype, y_dtype=None, hot=0, dropped=0.0, padded=0):
    """A case of the row operators: T tokens of width H, K of E experts each. `hot` experts
    are chosen more often; a share `dropped` of the assignments names no expert (-1, as
    where another rank has it), and the last `padded` tokens of the batch name none."""
    return {"name": name, "op": op, "T": T, "H": H, "E": E, "K": K, "dtype": dtype,
            "y_dtype": y_dtype or dtype, "hot": hot, "dropped": dropped, "padded": padded}


def _linear(name, op, rows, n_in, n_out, E, act, dtype, bias, residual=False, out32=False,
            skew=0.0, tail=0):
    """A case of the linear operators: `rows` rows sorted by E experts (one expert: a dense
    layer), `tail` more rows behind the last expert's, `skew` the spread of the experts'
    popularity (the standard deviation of its logarithm)."""
    return {"name": name, "op": op, "rows": rows, "n_in": n_in, "n_out": n_out, "E": E,
            "act": act, "dtype": dtype, "bias": bias, "residual": residual, "out32": out32,
            "skew": skew, "tail": tail}


def listed():
    return [
        # one decode step of a serving batch: latency counts
        _rows("permute decode", "permute", 64, 5120, 256, 8, "bf16"),
        # a long prefill chunk with a few experts far more popular than the others
        _rows("permute skewed", "permute", 16384, 5120, 256, 8, "bf16", hot=16),
        # the gradient of a training micro-batch, some assignments on other ranks
        _rows("permute_backward dropped", "permute_backward", 4096, 5120, 256, 8, "fp16",
              dropped=0.25),
        # a small odd layer: the width is no multiple of a vector
        _rows("permute_backward odd", "permute_backward", 333, 1003, 24, 3, "bf16"),
        # the end of a decode step: fp32 rows of the down product, bf16 out
        _rows("combine decode", "combine", 64, 5120, 256, 8, "bf16", y_dtype="fp32"),
        # a prefill batch padded at its end
        _rows("combine padded", "combine", 4096, 5120, 256, 8, "bf16", padded=300),
        # a training micro-batch
        _rows("combine_backward batch", "combine_backward", 4096, 5120, 256, 8, "bf16"),
        # a small odd layer in 32 bits
        _rows("combine_backward odd", "combine_backward", 129, 255, 96, 6, "fp32",
              dropped=0.1),
        # one token through a dense projection onto the residual stream: the weights stream
        _linear("linear one token", "linear", 1, 5120, 5120, 1, "none", "bf16", True,
                residual=True),
        # gate/up of a prefill batch over experts of unlike popularity
        _linear("linear experts swiglu", "linear", 8192, 5120, 2560, 32, "swiglu", "bf16",
                False, skew=0.7),
        # a small dense layer's training step, ragged sizes
        _linear("linear_backward dense", "linear_backward", 1000, 520, 1320, 1, "gelu", "fp16",
                True),
        # gate/up of a training micro-batch
        _linear("linear_backward experts", "linear_backward", 16384, 5120, 2560, 32, "swiglu",
                "bf16", True, skew=0.5, tail=128),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    if rng.random() < 0.55:
        op = rng.choice(ROW_OPS)
        K = rng.randint(1, 10)
        E = _spread(rng, max(K, 4), 512)
        T = _spread(rng, 1, 16384)
        H = _spread(rng, 64, 8192) // rng.choice((1, 2, 8, 64))
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        y_dtype = dtype if op.startswith("permute") or rng.random() < 0.6 else "fp32"
        H = max(8, H) if H % 2 else max(8, H // 8 * 8)
        most = (16384 if op == "permute" else 4096) * 8 * 5120 * 2
        T = max(1, min(T, most // (K * H * BYTES[y_dtype])))
        case = _rows("", op, T, H, E, K, dtype, y_dtype, hot=rng.choice((0, 0, 1, E // 8)),
                     dropped=rng.choice((0.0, 0.0, 0.1, 0.5)),
                     padded=rng.choice((0, 0, T // 3)))
    else:
        op = rng.choice(("linear", "linear_backward"))
        n_in = 8 * _spread(rng, 8, 640)
        n_out = 8 * _spread(rng, 8, 640)
        E = rng.choice((1, _spread(rng, 2, 32)))
        rows = _spread(rng, 1, 16384)
        act = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"))
        most = (8192 if op == "linear" else 16384) * 5120 * 5120
        rows = max(1, min(rows, most // (n_in * n_out * (2 if act == "swiglu" else 1))))
        forward = op == "linear"
        case = _linear("", op, rows, n_in, n_out, E, act, rng.choice(("bf16", "fp16")),
                       rng.random() < 0.5, residual=forward and rng.random() < 0.5,
                       out32=forward and rng.random() < 0.3, skew=rng.choice((0.0, 0.5, 1.0)),
                       tail=rng.choice((0, 0, 5)) if E > 1 else 0)
    del case["name"]
    return case


# --------------------------------------------------------------------- inputs

def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _routes(g, c):
    """Routes as a router makes them: each token's K best of E noisy expert scores, which
    favour the `hot` experts, and positive weights that sum to 2.5."""
    T, E, K = c["T"], c["E"], c["K"]
    score = torch.randn((T, E), generator=g, device="cuda")
    score[:, :c["hot"]] += 2.0
    ids = score.topk(K, dim=1).indices.to(torch.int32)
    w = torch.rand((T, K), generator=g, device="cuda") + 0.1
    w = 2.5 * w / w.sum(1, keepdim=True)
    if c["dropped"]:
        ids[torch.rand((T, K), generator=g, device="cuda") < c["dropped"]] = -1
    if c["padded"]:
        ids[T - c["padded"]:] = -1
    return ids, w


def _places(ids, E):
    """(pos, offsets) of the stable sort of the assignments by expert."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=ids.device))
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=ids.device)
    pos = torch.where(key < E, row, -1)
    return order, pos.reshape(ids.shape).to(torch.int32), offsets.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"c": case}
    dtype = DTYPES[case["dtype"]]
    if case["op"] in ROW_OPS:
        T, H, E, K = case["T"], case["H"], case["E"], case["K"]
        y_dtype = DTYPES[case["y_dtype"]]
        ids, w = _routes(g, case)
        s["ids"], s["w"] = ids, w
        _, s["pos"], s["offsets"] = _places(ids, E)
        if case["op"] == "permute":
            s["x"] = _normal(g, (T, H), dtype)
            s["xp"] = torch.zeros((T * K, H), dtype=dtype, device="cuda")
        elif case["op"] == "permute_backward":
            s["dxp"] = _normal(g, (T * K, H), dtype)
            s["dx"] = torch.empty((T, H), dtype=dtype, device="cuda")
        else:
            s["y"] = _normal(g, (T * K, H), y_dtype, 0.1)
            if case["op"] == "combine":
                s["out"] = torch.empty((T, H), dtype=dtype, device="cuda")
            else:
                s["dout"] = _normal(g, (T, H), dtype)
                s["dy"] = torch.zeros((T * K, H), dtype=y_dtype, device="cuda")
                s["dw"] = torch.empty((T, K), dtype=torch.float32, device="cuda")
    else:
        R, n_in, n_out, E = case["rows"], case["n_in"], case["n_out"], case["E"]
        n_w = n_out * (2 if case["act"] == "swiglu" else 1)
        every = R + case["tail"]
        p = torch.exp(case["skew"] * torch.randn(E, generator=g, device="cuda"))
        e = torch.multinomial(p, R, replacement=True, generator=g)
        counts = torch.zeros(E, dtype=torch.int64, device="cuda")
        counts.index_add_(0, e, torch.ones_like(e))
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = counts.cumsum(0)
        s["offsets"] = offsets if E > 1 else None
        s["most"] = int(counts.max())  # rows of the busiest expert
        s["x"] = _normal(g, (every, n_in), dtype)
        s["w"] = _normal(g, (E, n_w, n_in), dtype, n_in ** -0.5)
        s["bias"] = _normal(g, (E, n_w), torch.float32, 0.1) if case["bias"] else None
        out_dtype = torch.float32 if case["out32"] else dtype
        if case["op"] == "linear":
            s["residual"] = _normal(g, (every, n_out), out_dtype) if case["residual"] else None
            s["y"] = torch.zeros((every, n_out), dtype=out_dtype, device="cuda")
        else:
            s["dy"] = _normal(g, (every, n_out), dtype)
            s["z"] = _normal(g, (every, n_w), dtype) if case["act"] != "none" else None
            s["dx"] = torch.zeros((every, n_in), dtype=dtype, device="cuda")
            s["dw"] = torch.empty((E, n_w, n_in), dtype=dtype, device="cuda")
            s["dbias"] = (torch.empty((E, n_w), dtype=torch.float32, device="cuda")
                          if case["bias"] else None)
    if own:  # the configuration and workspace that a program keeps beside its buffers
        import sparse_moe_layer_beam_b200 as bm
        s["bm"] = bm
        if case["op"] in ROW_OPS:
            s["cfg"] = bm.rows_cfg(case["H"], case["E"], case["K"], case["dtype"])
            n = bm.beam_moe_permute_workspace_size(s["cfg"], case["T"])
        else:
            s["cfg"] = bm.linear_cfg(case["n_in"], case["n_out"], case["E"], case["act"],
                                     case["dtype"], case["out32"])
            n = bm.beam_moe_linear_workspace_size(s["cfg"], case["rows"] + case["tail"],
                                                  case["op"] == "linear_backward")
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms

def _plain_permute(s):
    c, x = s["c"], s["x"]
    order, pos, offsets = _places(s["ids"], c["E"])
    row = torch.arange(order.numel(), device=x.device)
    xp = torch.where((row < offsets[-1])[:, None], x[order // c["K"]], s["xp"])
    return {"xp": xp, "pos": pos, "offsets": offsets}


def _plain_sum(rows, pos, w, dtype):
    """sum over k of w[t, k] rows[pos[t, k]], assignments without a row left out."""
    got = rows[pos.clamp(min=0).long()].float()
    if w is not None:
        got = got * w[..., None]
    return torch.where((pos >= 0)[..., None], got, 0.0).sum(1).to(dtype)


def _plain_combine_backward(s):
    c, pos, dout = s["c"], s["pos"], s["dout"]
    A = pos.numel()
    d = dout.float()
    there = pos >= 0
    dw = (d[:, None, :] * s["y"][pos.clamp(min=0).long()].float()).sum(-1)
    dw = torch.where(there, dw, 0.0)
    src = torch.full((A + 1,), -1, dtype=torch.int64, device=pos.device)
    src[torch.where(there, pos, A).reshape(-1).long()] = torch.arange(A, device=pos.device)
    src = src[:A]
    at = src.clamp(min=0)
    dy = s["w"].reshape(-1)[at][:, None] * d[at // c["K"]]
    return {"dy": torch.where((src >= 0)[:, None], dy.to(s["dy"].dtype), s["dy"]), "dw": dw}


def _silu(z):
    return z / (1.0 + torch.exp(-z))


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return _silu(z)
    if act == "swiglu":
        gate, up = z.chunk(2, -1)
        return _silu(gate) * up
    return z


def _act_backward(dy, z, act):
    if act == "relu":
        return torch.where(z > 0, dy, 0.0)
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return dy * (cdf + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2 * math.pi)))
    if act == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return dy * (0.5 * (1.0 + t)
                     + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * z * z))
    if act in ("silu", "swiglu"):
        gate, up = z.chunk(2, -1) if act == "swiglu" else (z, None)
        sig = 1.0 / (1.0 + torch.exp(-gate))
        slope = sig * (1.0 + gate * (1.0 - sig))
        if up is None:
            return dy * slope
        return torch.cat((dy * up * slope, dy * gate * sig), -1)
    return dy


class _Segments:
    """Each expert's rows as one row block of the same height, padded with zeros."""

    def __init__(self, s):
        E, every = s["c"]["E"], s["x"].shape[0]
        dev = s["x"].device
        off = s["offsets"]
        if off is None:
            off = torch.tensor([0, every], device=dev)
        off = off.long()
        at = off[:-1, None] + torch.arange(max(1, s["most"]), device=dev)
        self.at, self.there = at.clamp(max=every - 1), (at < off[1:, None])[..., None]
        row = torch.arange(every, device=dev)
        self.e = torch.searchsorted(off[1:], row, right=True).clamp(max=E - 1)
        self.i = (row - off[self.e]).clamp(max=max(1, s["most"]) - 1)
        self.mine = (row < off[-1])[:, None]

    def blocks(self, rows):
        return torch.where(self.there, rows[self.at].float(), 0.0)

    def back(self, blocks, into):
        return torch.where(self.mine, blocks[self.e, self.i].to(into.dtype), into)


def _plain_linear(s):
    seg = _Segments(s)
    z = torch.bmm(seg.blocks(s["x"]), s["w"].float().transpose(1, 2))
    if s["bias"] is not None:
        z = z + s["bias"][:, None, :]
    y = _act(z, s["c"]["act"])
    if s["residual"] is not None:
        y = y + seg.blocks(s["residual"])
    return seg.back(y, s["y"])


def _plain_linear_backward(s):
    seg = _Segments(s)
    dz = seg.blocks(s["dy"])
    if s["z"] is not None:
        dz = _act_backward(dz, seg.blocks(s["z"]), s["c"]["act"])
    got = {"dx": seg.back(torch.bmm(dz, s["w"].float()), s["dx"]),
           "dw": torch.bmm(dz.transpose(1, 2), seg.blocks(s["x"])).to(s["dw"].dtype)}
    if s["dbias"] is not None:
        got["dbias"] = dz.sum(1)
    return got


def _plain(s):
    op = s["c"]["op"]
    if op == "permute":
        return _plain_permute(s)
    if op == "permute_backward":
        return _plain_sum(s["dxp"], s["pos"], None, s["dx"].dtype)
    if op == "combine":
        return _plain_sum(s["y"], s["pos"], s["w"], s["out"].dtype)
    if op == "combine_backward":
        return _plain_combine_backward(s)
    return _plain_linear(s) if op == "linear" else _plain_linear_backward(s)


# ----------------------------------------------------------- the library's calls

def _own(s):
    bm, cfg, op = s["bm"], s["cfg"], s["c"]["op"]
    if op == "permute":
        bm.beam_moe_permute(cfg, s["x"], s["ids"], s["xp"], s["pos"], s["offsets"], s["ws"])
        return {"xp": s["xp"], "pos": s["pos"], "offsets": s["offsets"]}
    if op == "permute_backward":
        bm.beam_moe_permute_backward(cfg, s["dxp"], s["pos"], s["dx"])
        return s["dx"]
    if op == "combine":
        bm.beam_moe_combine(cfg, s["y"], s["pos"], s["w"], s["out"])
        return s["out"]
    if op == "combine_backward":
        bm.beam_moe_combine_backward(cfg, s["dout"], s["y"], s["pos"], s["w"], s["dy"], s["dw"])
        return {"dy": s["dy"], "dw": s["dw"]}
    if op == "linear":
        bm.beam_moe_linear(cfg, s["x"], s["w"], s["y"], s["ws"], bias=s["bias"],
                           residual=s["residual"], offsets=s["offsets"])
        return s["y"]
    bm.beam_moe_linear_backward(cfg, s["dy"], s["x"], s["w"], s["ws"], dx=s["dx"], dw=s["dw"],
                                dbias=s["dbias"], z=s["z"], offsets=s["offsets"])
    got = {"dx": s["dx"], "dw": s["dw"]}
    if s["dbias"] is not None:
        got["dbias"] = s["dbias"]
    return got


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------- work and exact results

def work(case):
    c = case
    if c["op"] in ROW_OPS:
        A = round((c["T"] - c["padded"]) * c["K"] * (1 - c["dropped"]))
        T, H = c["T"], c["H"]
        b, by = BYTES[c["dtype"]], BYTES[c["y_dtype"]]
        ids = 4 * T * c["K"]
        if c["op"] == "permute":  # x and ids in, rows and places out
            return {"bytes": T * H * b + ids + A * H * b + ids + 4 * (c["E"] + 1), "flops": 0}
        if c["op"] == "permute_backward":
            return {"bytes": A * H * b + ids + T * H * b, "flops": A * H}
        if c["op"] == "combine":
            return {"bytes": A * H * by + 2 * ids + T * H * b, "flops": 2 * A * H}
        return {"bytes": T * H * b + 2 * A * H * by + 3 * ids, "flops": 3 * A * H}
    R, n_in, n_out, E = c["rows"], c["n_in"], c["n_out"], c["E"]
    n_w = n_out * (2 if c["act"] == "swiglu" else 1)
    b, bo = BYTES[c["dtype"]], 4 if c["out32"] else BYTES[c["dtype"]]
    touched = min(E, R) * n_w * n_in * b  # weights of the experts with rows
    bias = 4 * E * n_w if c["bias"] else 0
    if c["op"] == "linear":
        out = R * n_out * bo * (2 if c["residual"] else 1)
        return {"bytes": R * n_in * b + touched + bias + out, "flops": 2 * R * n_in * n_w}
    z = 0 if c["act"] == "none" else R * n_w * b
    return {"bytes": R * (n_out + 2 * n_in) * b + z + touched + E * n_w * n_in * b + bias,
            "flops": 4 * R * n_in * n_w}


def _exact_rows(s):
    """Token by token and slot by slot from the definition: the rows of expert 0 first, then
    expert 1's, each in the order of the flattened assignments."""
    c = s["c"]
    T, E, K = c["T"], c["E"], c["K"]
    flat = s["ids"].reshape(-1).cpu().numpy()
    valid = (flat >= 0) & (flat < E)
    places = [i for _, i in sorted((int(e), i) for i, e in enumerate(flat) if valid[i])]
    at = torch.tensor(places, dtype=torch.int64, device="cuda")  # assignment of each row
    n = at.numel()
    if c["op"] == "permute":
        xp = s["xp"].double()
        xp[:n] = s["x"].double()[torch.div(at, K, rounding_mode="floor")]
        return {"xp": xp, "pos": None, "offsets": None}
    rows = s["dxp" if c["op"] == "permute_backward" else "y"]
    tok = torch.div(at, K, rounding_mode="floor")
    w = s["w"].double().reshape(-1)[at]
    if c["op"] == "combine_backward":
        d = s["dout"].double()[tok]
        dy = s["dy"].double()
        dy[:n] = d * w[:, None]
        dw = torch.zeros(T * K, dtype=torch.float64, device="cuda")
        dw[at] = torch.einsum("rh,rh->r", d, rows[:n].double())
        return {"dy": dy, "dw": dw.reshape(T, K)}
    part = rows[:n].double() * (w[:, None] if c["op"] == "combine" else 1.0)
    return torch.zeros((T, c["H"]), dtype=torch.float64, device="cuda").index_add_(0, tok, part)


def _gate(z, act):
    """The activation in 64 bits from torch's functions, differentiable."""
    f = torch.nn.functional
    if act == "swiglu":
        half = z.shape[-1] // 2
        return f.silu(z[:, :half]) * z[:, half:]
    return {"none": lambda v: v, "relu": f.relu, "gelu": f.gelu, "silu": f.silu,
            "gelu_tanh": lambda v: f.gelu(v, approximate="tanh")}[act](z)


def _exact_linear(s):
    c = s["c"]
    off = [0, s["x"].shape[0]] if s["offsets"] is None else s["offsets"].tolist()
    forward = c["op"] == "linear"
    y = s["y"].double() if forward else None
    got = None if forward else {
        "dx": s["dx"].double(), "dw": torch.zeros(s["dw"].shape, dtype=torch.float64, device="cuda")}
    if not forward and s["dbias"] is not None:
        got["dbias"] = torch.zeros(s["dbias"].shape, dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        x, w = s["x"][lo:hi].double(), s["w"][e].double()
        if forward:
            z = x @ w.T
            if s["bias"] is not None:
                z += s["bias"][e].double()
            y[lo:hi] = _gate(z, c["act"])
            if s["residual"] is not None:
                y[lo:hi] += s["residual"][lo:hi].double()
            continue
        dz = s["dy"][lo:hi].double()
        if s["z"] is not None:
            with torch.enable_grad():
                z = s["z"][lo:hi].double().requires_grad_()
                dz, = torch.autograd.grad(_gate(z, c["act"]), z, dz)
        got["dx"][lo:hi] = dz @ w
        got["dw"][e] = dz.T @ x
        if s["dbias"] is not None:
            got["dbias"][e] = dz.sum(0)
    return y if forward else got


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rows(s) if case["op"] in ROW_OPS else _exact_linear(s)
