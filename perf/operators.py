"""The microscaled 4-bit (MXFP4) operators: what they compute, over which sizes, and how a user calls them.

A row of K values is held in blocks of 32: 4-bit floats (1 sign, 2 exponent, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
negatives), two per byte with the earlier element in the low nibble, and one scale byte c per block that stands for 2^(c - 127).  A
row is stored in whole blocks: ceil(K / 32) * 16 bytes of codes and ceil(K / 32) scale bytes.

Operators (case["op"]):
  round    values to MXFP4 and back: what a program does that looks at what the format costs, and the two halves of storing a tensor
           in the format and reading it back;
  matmul   y = x W^T for one MXFP4 matrix W [rows, K] and rows x that are f32, bf16 or MXFP4 themselves;
  grouped  the same for a stack of matrices, where rows offsets[e] .. offsets[e + 1] of the output belong to matrix e; the rows of x
           may be gathered through a list of (token, choice) pairs as a router's worklist holds them;
  layer    the routed feed-forward layer out[t] = sum_j w[t, j] down_e(silu(gate_e x_t) * (up_e x_t)), e = ids[t, j], with MXFP4
           experts.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32
# magnitudes of the eight 4-bit codes without the sign
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one token's activations on their way into the format: a decode step, latency only
        {"name": "round_token", "op": "round", "x": "bf16", "rows": 1, "cols": 4096, "pad": 0},
        # eight experts' matrices of the 4096 / 1536 layer converted from an f32 checkpoint
        {"name": "round_weights", "op": "round", "x": "f32", "rows": 12288, "cols": 4096, "pad": 0},
        # activations of an odd width inside a wider buffer
        {"name": "round_odd", "op": "round", "x": "bf16", "rows": 4093, "cols": 1535, "pad": 9},
        # a projection of one token at decode
        {"name": "matmul_token", "op": "matmul", "x": "f32", "batch": 1, "rows": 4096, "cols": 4096, "y": "f32"},
        # a prompt's rows with both operands in the format
        {"name": "matmul_mx", "op": "matmul", "x": "mx", "batch": 2048, "rows": 4096, "cols": 4096, "y": "bf16"},
        # the up projection of a decode step over many sequences: 64 tokens, 8 choices each, gathered by the worklist's pairs
        {"name": "grouped_decode", "op": "grouped", "x": "bf16", "tokens": 64, "k": 8, "experts": 128, "rows": 1536, "cols": 4096,
         "skew": 0.25, "y": "f32"},
        # odd widths and ragged groups, several of them empty, f32 rows in group order
        {"name": "grouped_odd", "op": "grouped", "x": "f32", "tokens": 1001, "k": 1, "experts": 24, "rows": 777, "cols": 1001,
         "skew": 2.0, "y": "f32"},
        # a prefill chunk with both operands in the format
        {"name": "grouped_mx", "op": "grouped", "x": "mx", "tokens": 2048, "k": 8, "experts": 128, "rows": 1536, "cols": 4096,
         "skew": 0.25, "y": "bf16"},
        # one token, f32 activations: the latency of a decode step
        {"name": "layer_token", "op": "layer", "x": "f32", "tokens": 1, "k": 8, "experts": 128, "hidden": 4096, "inter": 1536,
         "skew": 0.25},
        # a small decode batch
        {"name": "layer_batch16", "op": "layer", "x": "bf16", "tokens": 16, "k": 8, "experts": 128, "hidden": 4096, "inter": 1536,
         "skew": 0.25},
        # a larger decode batch in f32
        {"name": "layer_batch64", "op": "layer", "x": "f32", "tokens": 64, "k": 8, "experts": 128, "hidden": 4096, "inter": 1536,
         "skew": 0.25},
        # a prompt
        {"name": "layer_prompt", "op": "layer", "x": "bf16", "tokens": 8192, "k": 8, "experts": 128, "hidden": 4096, "inter": 1536,
         "skew": 0.25},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of lo .. hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: half the time a multiple of 64, else any number."""
    n = _log(rng, lo, hi)
    return max(64, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(("round", "matmul", "grouped", "layer"))
    if op == "round":
        cols = _width(rng, 33, 6144)
        return {"op": op, "x": rng.choice(("f32", "bf16")), "rows": _log(rng, 1, max(1, 40_000_000 // cols)), "cols": cols,
                "pad": rng.choice((0, 0, 1, 8))}
    if op == "matmul":
        return {"op": op, "x": rng.choice(("f32", "bf16", "mx")), "batch": _log(rng, 1, 4096), "rows": _width(rng, 33, 6144),
                "cols": _width(rng, 33, 6144), "y": rng.choice(("f32", "bf16"))}
    k = rng.choice((1, 2, 4, 8))
    experts = rng.choice((8, 16, 64, 128))
    tokens = _log(rng, 1, 4096)
    if op == "grouped":
        return {"op": op, "x": rng.choice(("f32", "bf16", "mx")), "tokens": tokens, "k": k, "experts": experts,
                "rows": _width(rng, 33, 2048), "cols": _width(rng, 33, 4096), "skew": rng.choice((0.0, 0.25, 1.0)),
                "y": rng.choice(("f32", "bf16"))}
    return {"op": op, "x": rng.choice(("f32", "bf16")), "tokens": tokens, "k": k, "experts": experts,
            "hidden": _width(rng, 64, 4096), "inter": _width(rng, 33, 1536), "skew": rng.choice((0.0, 0.25, 1.0))}


def _blocks(cols):
    return (cols + BLOCK - 1) // BLOCK


def _mx_bytes(rows, cols):
    """Codes and scale bytes of `rows` rows."""
    return rows * _blocks(cols) * 17


def _row_bytes(kind, cols):
    return _mx_bytes(1, cols) if kind == "mx" else cols * (4 if kind == "f32" else 2)


def _touched(experts, pairs):
    """Experts that `pairs` random picks reach on average."""
    return experts * (1.0 - (1.0 - 1.0 / experts) ** pairs)


def work(case):
    op = case["op"]
    if op == "round":
        n = case["rows"] * case["cols"]
        moved = 2 * n * (4 if case["x"] == "f32" else 2) + 2 * _mx_bytes(case["rows"], case["cols"])
        return {"bytes": moved, "flops": 2 * n}
    if op == "matmul":
        b, o, i = case["batch"], case["rows"], case["cols"]
        return {"bytes": _mx_bytes(o, i) + b * _row_bytes(case["x"], i) + b * _row_bytes(case["y"], o), "flops": 2 * b * o * i}
    n = case["tokens"] * case["k"]
    live = _touched(case["experts"], n)
    if op == "grouped":
        o, i = case["rows"], case["cols"]
        return {"bytes": live * _mx_bytes(o, i) + case["tokens"] * _row_bytes(case["x"], i) + n * _row_bytes(case["y"], o),
                "flops": 2 * n * o * i}
    h, f = case["hidden"], case["inter"]
    return {"bytes": live * (2 * _mx_bytes(f, h) + _mx_bytes(h, f)) + 2 * case["tokens"] * _row_bytes(case["x"], h) + 8 * n,
            "flops": 6 * n * h * f}


# ----------------------------------------------------------------- inputs ---

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _activations(g, rows, cols):
    """Normal rows, each of a size of its own, with a few large channels, as the hidden states of a language model have."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device=DEV))
    big = torch.rand(1, cols, generator=g, device=DEV) < 0.01
    return torch.where(big, 8.0 * x, x)


def _codes(g, shape, cols, near):
    """Packed codes and scales as a converted checkpoint holds them: any code, scales within four powers of two of each other, the
    elements past the row's end zero."""
    nb = _blocks(cols)
    q = torch.randint(0, 256, (*shape, nb * 16), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.randint(near, near + 4, (*shape, nb), generator=g, device=DEV, dtype=torch.uint8)
    last = cols - (nb - 1) * BLOCK
    q[..., (nb - 1) * 16 + (last + 1) // 2:] = 0
    if last % 2:
        q[..., (nb - 1) * 16 + last // 2] &= 15
    return q, s


def _near(cols):
    """The scale byte for which a sum over `cols` unit inputs comes out near one."""
    return 127 - 5 - round(math.log2(cols) / 2)


def _routing(g, case):
    """Router logits with some experts liked better than others (`skew`), the k largest of each token and their softmax."""
    t, e, k = case["tokens"], case["experts"], case["k"]
    logits = torch.randn(t, e, generator=g, device=DEV) + case["skew"] * torch.randn(1, e, generator=g, device=DEV)
    top = logits.topk(k, dim=1)
    return top.indices.to(torch.int32), torch.softmax(top.values, 1)


def _worklist(ids, experts):
    """The (token, choice) pairs sorted by expert and where each expert's begin."""
    flat = ids.reshape(-1).long()
    pairs = torch.sort(flat, stable=True).indices.to(torch.int32)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.bincount(flat, minlength=experts).cumsum(0).to(torch.int32)
    return pairs, offsets


def prepare(case, seed):
    g = _generator(seed)
    op, kind = case["op"], case["x"]
    state = {"case": case}
    if op == "round":
        wide = _activations(g, case["rows"], case["cols"] + case["pad"]).to(DTYPES[kind])
        state["x"] = wide[:, :case["cols"]]
        return state
    if op == "layer":
        h, f, e = case["hidden"], case["inter"], case["experts"]
        state["x"] = _activations(g, case["tokens"], h).to(DTYPES[kind])
        state["ids"], state["w"] = _routing(g, case)
        state["pairs"], state["offsets"] = _worklist(state["ids"], e)
        for name, rows, cols in (("gate", f, h), ("up", f, h), ("down", h, f)):
            state[name] = _codes(g, (e, rows), cols, _near(cols))
    else:
        o, i = case["rows"], case["cols"]
        n = case["batch"] if op == "matmul" else case["tokens"]
        if kind == "mx":
            state["x"], state["x_s"] = _codes(g, (n,), i, 124)
        else:
            state["x"], state["x_s"] = _activations(g, n, i).to(DTYPES[kind]), None
        if op == "matmul":
            state["w"] = _codes(g, (o,), i, _near(i))
        else:
            state["w"] = _codes(g, (case["experts"], o), i, _near(i))
            state["pairs"], state["offsets"] = _worklist(_routing(g, case)[0], case["experts"])
    if "offsets" in state:
        # the largest group, which a program without ragged products pads every group to
        state["most"] = int((state["offsets"][1:] - state["offsets"][:-1]).max())
    if own:
        import grouped_int4_expert_amd as qm
        if op == "layer":
            state["layer"] = qm.MxLayer(*(qm.MxMat(*state[m], cols) for m, cols in (("gate", case["hidden"]), ("up", case["hidden"]),
                                                                                  ("down", case["inter"]))))
        else:
            state["mat"] = qm.MxMat(*state["w"], case["cols"])
    return state


# ------------------------------------------------------------- plain form ---

def _to_mx(x):
    """f32 rows -> (codes as magnitudes with sign, scale bytes), both by block."""
    rows, cols = x.shape
    nb = _blocks(cols)
    b = torch.zeros(rows, nb * BLOCK, device=x.device)
    b[:, :cols] = x
    b = b.view(rows, nb, BLOCK)
    # the exponent of the block's largest magnitude, less two: that element then lies in [4, 8)
    field = (b.abs().amax(2).view(torch.int32) >> 23) & 255
    scale = (field - 2).clamp(min=0)
    a = torch.ldexp(b.abs(), (127 - scale)[:, :, None])
    # nearest value, a tie to the even code, 6 at most
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code | torch.where(torch.signbit(b), 8, 0)
    return code.view(rows, nb, 16, 2), scale


def _pack(code, scale):
    rows, nb = scale.shape
    return (code[..., 0] | (code[..., 1] << 4)).to(torch.uint8).view(rows, nb * 16), scale.to(torch.uint8)


def _from_mx(q, s, cols):
    """Packed rows [..., nb * 16] and scale bytes [..., nb] -> f32 [..., cols]."""
    table = torch.tensor(VALUES + tuple(-v for v in VALUES), device=q.device)
    pairs = torch.stack((table.repeat(16), table.repeat_interleave(16)), 1)
    v = pairs[q.int()].view(*s.shape, BLOCK)
    v = torch.ldexp(v, (s.int() - 127)[..., None])
    return v.view(*s.shape[:-1], s.shape[-1] * BLOCK)[..., :cols]


def _ragged(x, w, offsets, most):
    """y[r] = W_e x[r] for the rows r of every group e (x in group order, f32)."""
    q, s = w
    experts, cols, n = q.shape[0], x.shape[1], x.shape[0]
    row = torch.arange(n, device=x.device)
    group = torch.searchsorted(offsets[1:].long(), row, right=True)
    if n <= experts:
        return torch.bmm(_from_mx(q[group], s[group], cols), x[:, :, None])[:, :, 0]
    place = row - offsets.long()[group]
    padded = torch.zeros(experts, most, cols, device=x.device)
    padded[group, place] = x
    return torch.bmm(padded, _from_mx(q, s, cols).transpose(1, 2))[group, place]


def _plain(state):
    case, op = state["case"], state["case"]["op"]
    if op == "round":
        x = state["x"]
        return _from_mx(*_pack(*_to_mx(x.float())), case["cols"]).to(x.dtype)
    if op == "layer":
        token = state["pairs"].long() // case["k"]
        x = state["x"].float()[token]
        gate = _ragged(x, state["gate"], state["offsets"], state["most"])
        up = _ragged(x, state["up"], state["offsets"], state["most"])
        y = _ragged(gate / (1.0 + torch.exp(-gate)) * up, state["down"], state["offsets"], state["most"])
        y = y * state["w"].reshape(-1)[state["pairs"].long()][:, None]
        back = torch.empty_like(y)
        back[state["pairs"].long()] = y
        return back.view(case["tokens"], case["k"], -1).sum(1).to(state["x"].dtype)
    x = _from_mx(state["x"], state["x_s"], case["cols"]) if case["x"] == "mx" else state["x"].float()
    if op == "matmul":
        y = x @ _from_mx(*state["w"], case["cols"]).t()
    else:
        y = _ragged(x[state["pairs"].long() // case["k"]], state["w"], state["offsets"], state["most"])
    return y.to(DTYPES[case["y"]])


def run(state):
    if not own:
        return _plain(state)
    import grouped_int4_expert_amd as qm
    case, op = state["case"], state["case"]["op"]
    if op == "round":
        q, s = qm.qmoe_mx_quantize(state["x"])
        return qm.qmoe_mx_dequantize(q, s, case["cols"], dtype=state["x"].dtype)
    if op == "layer":
        return qm.qmoe_mx_layer(state["layer"], state["x"], state["ids"], state["w"])
    if op == "matmul":
        return qm.qmoe_mx_matmul(state["mat"], state["x"], x_s=state["x_s"], out_dtype=DTYPES[case["y"]])
    return qm.qmoe_mx_grouped(state["mat"], state["x"], state["offsets"], pairs=state["pairs"], k=case["k"], x_s=state["x_s"],
                              out_dtype=DTYPES[case["y"]])


# ---------------------------------------------------------------- exactly ---

def _exact_values(q, s, cols):
    """What packed rows stand for, in 64 bits, from the fields of each code: (-1)^sign * 2^(e - 1) * (1 + m / 2), or m / 2 for e = 0."""
    lo, hi = q & 15, q >> 4
    c = torch.stack((lo, hi), -1).flatten(-2).to(torch.int64)
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e > 0, torch.exp2(e.double() - 1) * (1 + m / 2), m / 2)
    v = torch.where(c >= 8, -v, v)
    return (v * torch.exp2(s.double() - 127).repeat_interleave(BLOCK, -1))[..., :cols]


def _exact_groups(x, w, offsets, cols):
    ends = offsets.tolist()
    out = torch.zeros(x.shape[0], w[0].shape[1], dtype=torch.float64, device=x.device)
    for e in range(w[0].shape[0]):
        a, b = ends[e], ends[e + 1]
        if b > a:
            out[a:b] = x[a:b] @ _exact_values(w[0][e], w[1][e], cols).t().contiguous()
    return out


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "round":
        x = state["x"].double()
        nb = _blocks(case["cols"])
        b = torch.nn.functional.pad(x, (0, nb * BLOCK - case["cols"])).view(-1, nb, BLOCK)
        most = b.abs().amax(2, keepdim=True)
        exponent = torch.where(most > 0, torch.frexp(most).exponent.double() - 3, torch.full_like(most, -127.0)).clamp(-127, 127)
        v = b / torch.exp2(exponent)
        # a step of the grid is 1/2 below 2, 1 below 4, 2 above; rounding half to even in steps is what the codes' parity asks for
        step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).double()
        v = (torch.round(v / step) * step).clamp(-6, 6) * torch.exp2(exponent)
        return v.reshape(x.shape[0], -1)[:, :case["cols"]]
    if op == "layer":
        t, k = case["tokens"], case["k"]
        pairs = state["pairs"].long()
        x = state["x"].double()[pairs // k]
        gate = _exact_groups(x, state["gate"], state["offsets"], case["hidden"])
        up = _exact_groups(x, state["up"], state["offsets"], case["hidden"])
        y = _exact_groups(torch.nn.functional.silu(gate) * up, state["down"], state["offsets"], case["inter"])
        y = y * state["w"].double().reshape(-1)[pairs][:, None]
        out = torch.zeros(t, case["hidden"], dtype=torch.float64, device=y.device)
        return out.index_add_(0, pairs // k, y)
    cols = case["cols"]
    x = _exact_values(state["x"], state["x_s"], cols) if case["x"] == "mx" else state["x"].double()
    if op == "matmul":
        return x @ _exact_values(*state["w"], cols).t().contiguous()
    return _exact_groups(x[state["pairs"].long() // case["k"]], state["w"], state["offsets"], cols)
