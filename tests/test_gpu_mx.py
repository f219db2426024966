"""The MXFP4 entry points on the GPU against 64-bit references: rounding to
the format and back bit for bit, the products and the routed layer within
bounds that follow each rounded quantity (mx_ref)."""
import ctypes

import numpy as np
import pytest
import torch

import grouped_int4_expert_amd as qm
import mx_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def np64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def same_bits(a, b):
    return np.array_equal(np.asarray(a), np.asarray(b))


# ---------------------------------------------------------------- rounding ---

@pytest.mark.parametrize("rows,cols,ld", [(1, 1, 1), (3, 31, 31), (2, 32, 32), (5, 33, 40), (7, 257, 257),
                                          (64, 4096, 4096), (33, 1535, 1544), (1000, 96, 96)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_quantize_and_back(kind, rows, cols, ld):
    say(f"mx round {kind} {rows}x{cols} ld {ld}")
    g = gen(rows * 7 + cols)
    wide = torch.randn(rows, ld, generator=g) * torch.exp(4 * torch.randn(rows, 1, generator=g))
    x = wide.to(TYPES[kind])[:, :cols]
    rq, rs = ref.quantize(np64(x))
    xd = wide.to(TYPES[kind]).to(DEV)[:, :cols]
    q, s = qm.qmoe_mx_quantize(xd)
    assert same_bits(s.cpu(), rs)
    assert same_bits(q.cpu(), rq)
    for t in (torch.float32, torch.bfloat16):
        back = torch.full((rows, ld), 7.0, dtype=t, device=DEV)
        qm.qmoe_mx_dequantize(q, s, cols, out=back[:, :cols])
        assert same_bits(np64(back[:, :cols]), ref.decode(rq, rs, cols))   # exact in bf16 too
        assert (back[:, cols:] == 7.0).all()


def test_quantize_borders_and_extremes():
    # every multiple of 1/16 up to 8 and its neighbours, in blocks led by 4, 6 and 7.5
    v = np.arange(-128, 129) / 16.0
    near = np.concatenate([np.nextafter(np.float32(v), np.float32(9)), np.nextafter(np.float32(v), np.float32(-9)),
                           np.float32(v)]).astype(np.float64)
    rows = []
    for lead in (4.0, 6.0, 7.5):
        for e in (-127, -126, -120, -3, 0, 60, 125):
            some = near[np.abs(near) <= 7.75]
            pad = np.zeros((-len(some)) % 31)
            body = np.concatenate([some, pad]).reshape(-1, 31)
            rows.append(np.ldexp(np.concatenate([np.full((len(body), 1), lead), body], 1), e))
    x = torch.from_numpy(np.concatenate(rows)).to(torch.float32)
    say(f"mx borders {tuple(x.shape)}")
    rq, rs = ref.quantize(np64(x))
    q, s = qm.qmoe_mx_quantize(x.to(DEV))
    assert same_bits(s.cpu(), rs)
    assert same_bits(q.cpu(), rq)
    # zeros, signed zeros, the smallest and largest numbers, NaN and infinities
    y = torch.zeros(9, 64)
    y[1, 3] = -0.0
    y[2, 5] = 2.0 ** -149
    y[3, 5] = 2.0 ** -126
    y[4, 40] = torch.finfo(torch.float32).max
    y[5, 7] = float("nan")
    y[6, 33] = float("inf")
    y[7, 33] = -float("inf")
    y[8, 0], y[8, 1] = 1.0, 2.0 ** -30
    rq, rs = ref.quantize(np64(y))
    q, s = qm.qmoe_mx_quantize(y.to(DEV))
    assert same_bits(s.cpu(), rs) and same_bits(q.cpu(), rq)
    back = np64(qm.qmoe_mx_dequantize(q, s, 64))
    assert np.array_equal(back, ref.decode(rq, rs, 64), equal_nan=True)
    assert np.isnan(back[5, :32]).all() and (back[5, 32:] == 0).all()
    # every code under every scale
    q = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    s = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16)
    back = np64(qm.qmoe_mx_dequantize(q.to(DEV), s.to(DEV), 512))
    want = ref.decode(q, s, 512)
    with np.errstate(invalid="ignore"):
        want = np.where(np.abs(want) >= 2.0 ** 128, np.sign(want) * np.inf, want)
    assert np.array_equal(back, want, equal_nan=True)


# ---------------------------------------------------------------- products ---

def rows_of(kind, g, n, cols):
    """(device operand, device scales or None, float64 values)."""
    if kind == "mx":
        q, s = ref.rand_mx(g, (n,), cols, 124)
        return q.to(DEV), s.to(DEV), ref.decode(q, s, cols)
    x = (torch.randn(n, cols, generator=g) * torch.exp(torch.randn(n, 1, generator=g))).to(TYPES[kind])
    return x.to(DEV), None, np64(x)


def parts(kind):
    return 3 if kind == "f32" else 1


def check(got, want, bound, out_type, what):
    got = np64(got)
    if out_type == torch.bfloat16:
        bound = bound + ref.UB * (np.abs(want) + bound)
    else:
        bound = bound + ref.U * (np.abs(want) + bound)
    worst = float((np.abs(got - want) / np.maximum(bound, 1e-300)).max()) if got.size else 0.0
    norm = np.linalg.norm(want)
    rel = float(np.linalg.norm(got - want) / norm) if norm else 0.0
    say(f"  {what}: rel {rel:.2e}, worst |err| / bound {worst:.3f}")
    assert np.isfinite(got).all() and worst <= 1.0
    # independent roundings: a random walk of one step of 2 U per addition
    assert rel <= 2.0 ** -8 if out_type == torch.bfloat16 else rel <= 2.0 ** -20


@pytest.mark.parametrize("batch,rows,cols", [(1, 1, 1), (1, 256, 1024), (3, 33, 31), (16, 48, 96), (17, 130, 257),
                                             (5, 64, 4096), (33, 77, 1001), (70, 300, 160), (129, 256, 513),
                                             (200, 515, 512), (300, 96, 64)])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_matmul(kind, out, batch, rows, cols):
    say(f"mx matmul {kind} -> {out} {batch}x{cols} by {rows}")
    g = gen(batch + rows * 3 + cols)
    q, s = ref.rand_mx(g, (rows,), cols)
    x, x_s, xv = rows_of(kind, g, batch, cols)
    y = qm.qmoe_mx_matmul(qm.MxMat(q.to(DEV), s.to(DEV), cols), x, x_s=x_s, out_dtype=TYPES[out])
    want, m = ref.product(ref.decode(q, s, cols), xv)
    check(y, want, ref.sum_bound(cols, parts(kind)) * m, TYPES[out], "matmul")


# Products large enough for the tiles' kernels (rows x outputs counts, not inputs): whole and partial
# tiles, odd widths on every side.
@pytest.mark.parametrize("batch,rows,cols", [(2100, 1000, 64), (2049, 1021, 257), (1300, 2304, 96), (3001, 900, 33),
                                             (1030, 3000, 1001)])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_matmul_tiles(kind, out, batch, rows, cols):
    test_matmul(kind, out, batch, rows, cols)


@pytest.mark.parametrize("per", [20, 50, 150, 400])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_tiles(kind, gather, per):
    """Ragged groups of `per` rows on average, one of them empty, for each size of tile."""
    say(f"mx grouped tiles {kind} per={per} gather={gather}")
    g = gen(per + gather)
    experts, rows, cols = (70, 1300, 160) if per < 100 else (9, 2060, 321)
    c = torch.randint(per // 2, per * 3 // 2, (experts,), generator=g)
    c[3] = 0
    used = int(c.sum())
    n = used + 3
    offsets = torch.zeros(experts + 1, dtype=torch.int32)
    offsets[1:] = c.cumsum(0).to(torch.int32)
    q, s = ref.rand_mx(g, (experts, rows), cols)
    tokens = n // 2 + 1
    x, x_s, xv = rows_of(kind, g, tokens if gather else n, cols)
    pairs = torch.randint(0, tokens * 2, (n,), generator=g).to(torch.int32) if gather else None
    if gather:
        pairs[5] = -1
    out = torch.full((n, rows), 9.0, device=DEV)
    qm.qmoe_mx_grouped(qm.MxMat(q.to(DEV), s.to(DEV), cols), x, offsets.to(DEV),
                       pairs=None if pairs is None else pairs.to(DEV), k=2 if gather else 1, x_s=x_s, out=out)
    src = pairs.numpy() // 2 if gather else np.arange(n)
    want, m = np.zeros((used, rows)), np.zeros((used, rows))
    for e in range(experts):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b > a:
            want[a:b], m[a:b] = ref.product(ref.decode(q[e], s[e], cols), xv[src[a:b]])
    if gather:
        assert (out[5] == 0).all()
        want[5] = 0
    check(out[:used], want, ref.sum_bound(cols, parts(kind)) * m, torch.float32, "grouped tiles")
    assert (out[used:] == 9.0).all()


def group_sizes(kind, experts, g):
    if kind == "few":
        c = torch.randint(0, 4, (experts,), generator=g)
    elif kind == "some":
        c = torch.randint(0, 50, (experts,), generator=g)
    else:
        c = torch.randint(0, 200, (experts,), generator=g)
        c[::3] = 0
        c[1] = 300
    return c


@pytest.mark.parametrize("sizes,experts,rows,cols", [("few", 9, 40, 96), ("few", 130, 64, 256), ("some", 7, 100, 257),
                                                     ("many", 5, 260, 512), ("many", 6, 77, 1001)])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped(kind, gather, sizes, experts, rows, cols):
    say(f"mx grouped {kind} {sizes} E={experts} {rows}x{cols} gather={gather}")
    g = gen(experts * 11 + cols + gather)
    c = group_sizes(sizes, experts, g)
    used = int(c.sum())
    n = used + 5                                   # rows behind the last group
    offsets = torch.zeros(experts + 1, dtype=torch.int32)
    offsets[1:] = c.cumsum(0).to(torch.int32)
    q, s = ref.rand_mx(g, (experts, rows), cols)
    k = 3
    tokens = max(1, n // k + 2)
    x, x_s, xv = rows_of(kind, g, tokens if gather else n, cols)
    pairs = torch.randint(0, tokens * k, (n,), generator=g).to(torch.int32) if gather else None
    out = torch.full((n, rows + 3), 9.0, device=DEV)
    qm.qmoe_mx_grouped(qm.MxMat(q.to(DEV), s.to(DEV), cols), x, offsets.to(DEV),
                       pairs=None if pairs is None else pairs.to(DEV), k=k if gather else 1, x_s=x_s,
                       out=out[:, :rows])
    src = pairs.numpy() // k if gather else np.arange(n)
    wv = ref.decode(q, s, cols)
    want, m = np.zeros((used, rows)), np.zeros((used, rows))
    for e in range(experts):
        a, b = int(offsets[e]), int(offsets[e + 1])
        want[a:b], m[a:b] = ref.product(wv[e], xv[src[a:b]])
    check(out[:used, :rows], want, ref.sum_bound(cols, parts(kind)) * m, torch.float32, "grouped")
    assert (out[used:] == 9.0).all() and (out[:, rows:] == 9.0).all()


def test_grouped_bad_pairs_and_offsets():
    say("mx grouped bad pairs and offsets")
    g = gen(3)
    E, O, K, T = 4, 64, 128, 6
    for n in (20, 200):
        q, s = ref.rand_mx(g, (E, O), K)
        W = qm.MxMat(q.to(DEV), s.to(DEV), K)
        for kind in ("f32", "bf16", "mx"):
            x, x_s, xv = rows_of(kind, g, T, K)
            pairs = torch.arange(n, dtype=torch.int32) % (2 * T)
            pairs[3], pairs[7], pairs[11] = -1, 2 * T, 2 ** 31 - 1
            offsets = torch.tensor([0, n // 2, n // 2, n, n], dtype=torch.int32)
            y = qm.qmoe_mx_grouped(W, x, offsets.to(DEV), pairs=pairs.to(DEV), k=2, x_s=x_s,
                                   out_dtype=torch.float32)
            assert (y[[3, 7, 11]] == 0).all()
            p = pairs.numpy()
            good = (p >= 0) & (p < 2 * T)
            e = np.where(np.arange(n) < n // 2, 0, 2)
            wv = ref.decode(q, s, K)
            want = np.stack([wv[e[r]] @ xv[p[r] // 2] if good[r] else np.zeros(O) for r in range(n)])
            m = np.stack([np.abs(wv[e[r]]) @ np.abs(xv[p[r] // 2]) if good[r] else np.zeros(O) for r in range(n)])
            check(y, want, ref.sum_bound(K, parts(kind)) * m, torch.float32, f"bad pairs {kind} n={n}")
            # offsets outside [0, n] are clamped, decreasing ones give empty groups
            wild = torch.tensor([-5, n // 2, 3, 2 ** 31 - 1, 7], dtype=torch.int32)
            out = torch.full((n + 8, O), 9.0, device=DEV)
            qm.qmoe_mx_grouped(W, x, wild.to(DEV), pairs=pairs.to(DEV), k=2, x_s=x_s, out=out[:n])
            torch.cuda.synchronize()
            assert (out[n:] == 9.0).all()


@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("batch", [2, 100])
def test_non_finite_values_reach_their_outputs(kind, batch):
    say(f"mx non-finite {kind} batch {batch}")
    g = gen(8)
    O, K = 70, 224
    q, s = ref.rand_mx(g, (O,), K)
    q[q == 0] = 0x22                                # no zero pairs: inf * 0 would be NaN either way
    s[5, 3] = 255
    x, x_s, xv = rows_of(kind, g, batch, K)
    if kind == "mx":
        x_s[1, 2] = 255
        xv[1, 64:96] = np.nan
    else:
        x[1, 70] = float("nan")
        x[0, 5] = float("inf")
        xv[1, 70], xv[0, 5] = np.nan, np.inf
    y = np64(qm.qmoe_mx_matmul(qm.MxMat(q.to(DEV), s.to(DEV), K), x, x_s=x_s, out_dtype=torch.float32))
    wv = ref.decode(q, s, K)
    with np.errstate(invalid="ignore"):
        want = xv @ wv.T
    assert np.array_equal(np.isnan(y), np.isnan(want))
    assert np.array_equal(np.isinf(y), np.isinf(want))
    assert np.array_equal(np.sign(y[np.isinf(y)]), np.sign(want[np.isinf(want)]))


def test_f32_rows_keep_their_bits():
    # one-hot rows: y is W's column times x exactly, whatever x's magnitude
    say("mx one-hot f32")
    g = gen(9)
    O, K = 40, 96
    q, s = ref.rand_mx(g, (O,), K)
    for batch in (8, 120):
        x = torch.zeros(batch, K)
        at = torch.randint(0, K, (batch,), generator=g)
        v = torch.randn(batch, generator=g) * torch.exp2(torch.randint(-90, 90, (batch,), generator=g).float())
        x[torch.arange(batch), at] = v
        y = np64(qm.qmoe_mx_matmul(qm.MxMat(q.to(DEV), s.to(DEV), K), x.to(DEV)))
        want = np64(v)[:, None] * ref.decode(q, s, K).T[at.numpy()]
        # a product of 24 and 2 significant bits rounds once
        assert (np.abs(y - want) <= ref.U * np.abs(want)).all()


# ------------------------------------------------------------------- layer ---

def make_layer(g, E, H, F):
    m = [ref.rand_mx(g, (E, F), H), ref.rand_mx(g, (E, F), H), ref.rand_mx(g, (E, H), F)]
    dev = qm.MxLayer(*(qm.MxMat(q.to(DEV), s.to(DEV), c) for (q, s), c in zip(m, (H, H, F))))
    return dev, [ref.decode(q, s, c) for (q, s), c in zip(m, (H, H, F))]


def routing(g, T, E, k):
    logits = torch.randn(T, E, generator=g) + torch.randn(1, E, generator=g)
    top = logits.topk(k, 1)
    return top.indices.to(torch.int32), torch.softmax(top.values, 1)


def check_layer(got, want, bound, kind, what):
    got = np64(got)
    worst = float((np.abs(got - want) / np.maximum(bound, 1e-300)).max())
    rel = float(np.linalg.norm(got - want) / np.linalg.norm(want))
    say(f"  {what}: rel {rel:.2e}, worst |err| / bound {worst:.3f}")
    assert worst <= 1.0
    # bf16: h and out each round once, half a step at most
    assert rel <= (2.0 ** -7 if kind == "bf16" else 2.0 ** -18)


@pytest.mark.parametrize("T,E,H,F,k", [(1, 8, 128, 64, 2), (1, 128, 256, 96, 8), (3, 4, 100, 45, 4), (16, 16, 256, 128, 4),
                                       (17, 16, 128, 130, 2), (70, 4, 257, 65, 2), (130, 3, 384, 200, 1),
                                       (300, 5, 96, 160, 3)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_layer(kind, T, E, H, F, k):
    say(f"mx layer {kind} T={T} E={E} {H}/{F} k={k}")
    g = gen(T + E + H + F)
    dev, (gate, up, down) = make_layer(g, E, H, F)
    x = torch.randn(T, H, generator=g).to(TYPES[kind])
    ids, w = routing(g, T, E, k)
    want, bound = ref.layer(gate, up, down, np64(x), ids.numpy(), np64(w), parts(kind), kind == "bf16")
    got = qm.qmoe_mx_layer(dev, x.to(DEV), ids.to(DEV), w.to(DEV))
    assert got.dtype == x.dtype
    check_layer(got, want, bound, kind, "layer")
    assert torch.equal(got, qm.qmoe_mx_layer(dev, x.to(DEV), ids.to(DEV), w.to(DEV)))


@pytest.mark.parametrize("T,E,H,F,k", [(700, 6, 1030, 420, 4), (900, 40, 512, 610, 2), (2500, 5, 384, 333, 1)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_layer_tiles(kind, T, E, H, F, k):
    test_layer(kind, T, E, H, F, k)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("T", [2, 12, 60])
def test_layer_dropped_and_repeated_ids(kind, T):
    say(f"mx layer dropped and repeated ids {kind} T={T}")
    g = gen(31)
    E, H, F, k = 6, 128, 96, 4
    dev, (gate, up, down) = make_layer(g, E, H, F)
    x = torch.randn(T, H, generator=g).to(TYPES[kind])
    ids, w = routing(g, T, E, k)
    ids[0] = torch.tensor([-1, E, 2 ** 31 - 1, -(2 ** 31)])      # a token no expert takes
    ids[1] = torch.tensor([2, 2, 2, 5])                          # one expert three times
    want, bound = ref.layer(gate, up, down, np64(x), ids.numpy(), np64(w), parts(kind), kind == "bf16")
    out = torch.full((T, H), 9.0, dtype=x.dtype, device=DEV)
    got = qm.qmoe_mx_layer(dev, x.to(DEV), ids.to(DEV), w.to(DEV), out=out)
    assert got is out and (got[0] == 0).all()
    check_layer(got, want, bound, kind, "layer")


def test_layer_empty():
    g = gen(32)
    dev, _ = make_layer(g, 4, 128, 64)
    x = torch.empty(0, 128, device=DEV)
    out = qm.qmoe_mx_layer(dev, x, torch.empty(0, 2, dtype=torch.int32, device=DEV), torch.empty(0, 2, device=DEV))
    assert out.shape == (0, 128)
    y = qm.qmoe_mx_matmul(qm.MxMat(dev.gate.q[0], dev.gate.s[0], 128), x)
    assert y.shape == (0, 64)
    q, s = qm.qmoe_mx_quantize(x)
    assert q.shape == (0, 64) and s.shape == (0, 4)


# --------------------------------------------------------------- used together

@pytest.mark.parametrize("T", [4, 40, 300])
def test_quantize_route_group_and_layer_together(T):
    """Weights rounded to the format on the device; router, worklist, grouped
    products and the layer on them: the layer equals its parts."""
    say(f"mx pipeline T={T}")
    g = gen(50 + T)
    E, H, F, k = 8, 256, 128, 2
    dense = [torch.randn(E * r, c, generator=g) / c ** 0.5 for r, c in ((F, H), (F, H), (H, F))]
    mats = []
    for d, r, c in zip(dense, (F, F, H), (H, H, F)):
        q, s = qm.qmoe_mx_quantize(d.to(DEV))
        mats.append(qm.MxMat(q.view(E, r, -1), s.view(E, r, -1), c))
    layer = qm.MxLayer(*mats)
    x = torch.randn(T, H, generator=g)
    ids, w = qm.qmoe_route(torch.randn(T, E, generator=g).to(DEV), k)
    out = qm.qmoe_mx_layer(layer, x.to(DEV), ids, w)
    wl = qm.qmoe_worklist(ids, E)
    a = qm.qmoe_mx_grouped(mats[0], x.to(DEV), wl["offsets"], pairs=wl["pairs"], k=k)
    u = qm.qmoe_mx_grouped(mats[1], x.to(DEV), wl["offsets"], pairs=wl["pairs"], k=k)
    y = qm.qmoe_mx_grouped(mats[2], torch.nn.functional.silu(a) * u, wl["offsets"])
    p = wl["pairs"].long()
    again = torch.zeros(T, H, device=DEV).index_add_(0, p // k, y * w.reshape(-1)[p][:, None])
    vals = [ref.decode(m.q.cpu(), m.s.cpu(), m.cols) for m in mats]
    for d, m, v in zip(dense, mats, vals):
        assert same_bits(ref.quantize(np64(d))[0], m.q.cpu().view(-1, m.q.shape[-1]))
    want, bound = ref.layer(*vals, np64(x), ids.cpu().numpy(), np64(w), 3, False)
    check_layer(out, want, bound, "f32", "layer")
    check_layer(again, want, bound, "f32", "parts")
    # MXFP4 rows: the same numbers as their values
    xq, xs = qm.qmoe_mx_quantize(x.to(DEV))
    a4 = qm.qmoe_mx_grouped(mats[0], xq, wl["offsets"], pairs=wl["pairs"], k=k, x_s=xs)
    av = qm.qmoe_mx_grouped(mats[0], qm.qmoe_mx_dequantize(xq, xs, H), wl["offsets"], pairs=wl["pairs"], k=k)
    assert float((a4 - av).norm() / av.norm()) <= 2.0 ** -20


# Passes of two column tiles (2048 inputs and more, a block per compute unit): full passes, a last one of
# one tile, groups of uneven sizes with empty and single-row ones among them.
@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("batch,rows,cols", [(130, 4100, 2049), (257, 4100, 2080), (300, 4100, 2177)])
def test_matmul_wide_passes(kind, batch, rows, cols):
    test_matmul(kind, "f32", batch, rows, cols)


@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
def test_grouped_wide_passes(kind):
    say(f"mx grouped wide passes {kind}")
    g = gen(8)
    E, O, K = 9, 2060, 2048
    off = torch.tensor([0, 0, 1, 150, 37, 17, 16, 130, 0, 90]).cumsum(0).to(torch.int32)
    n = int(off[-1])
    q, s = ref.rand_mx(g, (E, O), K)
    x, x_s, xv = rows_of(kind, g, n, K)
    y = qm.qmoe_mx_grouped(qm.MxMat(q.to(DEV), s.to(DEV), K), x, off.to(DEV), x_s=x_s)
    want, m = np.zeros((n, O)), np.zeros((n, O))
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        want[a:b], m[a:b] = ref.product(ref.decode(q[e], s[e], K), xv[a:b])
    check(y, want, ref.sum_bound(K, parts(kind)) * m, y.dtype, "grouped wide passes")     # bf16 of bf16 rows


# ------------------------------------------------- streams, graphs, large stacks

def calls(T, seed=77, E=12, H=384, F=224, k=3):
    """Every entry point once on one set of inputs: a list of functions without arguments."""
    g = gen(seed + T)
    layer, _ = make_layer(g, E, H, F)
    x = torch.randn(T, H, generator=g)
    ids, w = routing(g, T, E, k)
    xd, xb, ids, w = x.to(DEV), x.bfloat16().to(DEV), ids.to(DEV), w.to(DEV)
    wl = qm.qmoe_worklist(ids, E)
    q, s = qm.qmoe_mx_quantize(xd)
    one = qm.MxMat(layer.gate.q[1], layer.gate.s[1], H)
    return [lambda **kw: qm.qmoe_mx_quantize(xb, **kw)[0],
            lambda **kw: qm.qmoe_mx_dequantize(q, s, H, **kw),
            lambda **kw: qm.qmoe_mx_matmul(one, xd, **kw),
            lambda **kw: qm.qmoe_mx_matmul(one, q, x_s=s, **kw),
            lambda **kw: qm.qmoe_mx_grouped(layer.up, xd, wl["offsets"], pairs=wl["pairs"], k=k, **kw),
            lambda **kw: qm.qmoe_mx_grouped(layer.up, xb, wl["offsets"], pairs=wl["pairs"], k=k, **kw),
            lambda **kw: qm.qmoe_mx_grouped(layer.up, q, wl["offsets"], pairs=wl["pairs"], k=k, x_s=s, **kw),
            lambda **kw: qm.qmoe_mx_layer(layer, xd, ids, w, **kw),
            lambda **kw: qm.qmoe_mx_layer(layer, xb, ids, w, **kw)], (xd, xb)


@pytest.mark.parametrize("T", [1, 7, 60, 3000])
def test_replayed_graphs(T):
    """Two captured graphs of the same calls (each with workspaces of its own), replayed in turn with eager
    work between: every replay gives the eager results of the inputs as they are then."""
    say(f"mx graphs T={T}")
    fs, (xd, xb) = calls(T)
    for f in fs:
        f()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = [f() for f in fs]
        graphs.append((gr, outs))
    for r in range(4):
        xd.mul_(1.25)
        xb.mul_(-1.0)
        want = [f() for f in fs]
        gr, outs = graphs[r & 1]
        for o in outs:
            o.zero_()
        gr.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), (T, r, i)


@pytest.mark.parametrize("T", [2, 90])
def test_streams(T):
    """Calls on two streams at once, each given by argument, equal the same calls on the current one."""
    say(f"mx streams T={T}")
    fs, keep = calls(T)
    want = [f() for f in fs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [[f(stream=st) for f in fs] for st in streams]
        torch.cuda.synchronize()
        for outs in got:
            for i, (a, b) in enumerate(zip(outs, want)):
                assert torch.equal(a, b), (T, i)


def test_views_and_given_buffers():
    say("mx views")
    g = gen(5)
    O, K = 96, 256
    q, s = ref.rand_mx(g, (O,), K)
    W = qm.MxMat(q.to(DEV), s.to(DEV), K)
    wide = torch.randn(40, K + 24, generator=g).to(DEV)
    for t in (torch.float32, torch.bfloat16):
        x = wide.to(t)[:, 8:8 + K]
        want = qm.qmoe_mx_matmul(W, x.contiguous())
        out = torch.zeros(40, O + 8, dtype=t, device=DEV)
        if t == torch.float32:                  # 8 elements in: 32 bytes, aligned
            got = qm.qmoe_mx_matmul(W, x, out=out[:, :O])
            assert torch.equal(got, want) and (out[:, O:] == 0).all()
        one = qm.qmoe_mx_matmul(W, x[3])        # a single row
        assert torch.equal(one, qm.qmoe_mx_matmul(W, x[3:4].contiguous()))
    with pytest.raises(qm.QmoeError):
        qm.qmoe_mx_matmul(W, wide[:, 1:1 + K])                       # misaligned rows
    with pytest.raises(ValueError):
        qm.qmoe_mx_matmul(W, wide.t()[:K].t()[:, ::2])
    with pytest.raises(ValueError):
        qm.qmoe_mx_matmul(W, wide[:, :K], out=torch.empty(40, O + 1, device=DEV))
    with pytest.raises(ValueError):
        qm.qmoe_mx_layer(qm.MxLayer(*[qm.MxMat(W.q[None], W.s[None], K)] * 2,
                                    qm.MxMat(*[torch.zeros(1, K, n, dtype=torch.uint8, device=DEV) for n in (48, 3)], O)),
                         wide[:, :K].contiguous(), torch.zeros(40, 2, dtype=torch.int32, device=DEV),
                         torch.zeros(40, 1, device=DEV))


@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
def test_stack_past_four_gigabytes(kind):
    """Expert offsets beyond 32 bits: the last experts of a strided stack of 5 GB."""
    say(f"mx large stack {kind}")
    g = gen(6)
    E, O, K = 160, 64, 256
    stride = 5 * (1 << 30) // E // 16 * 16
    q, s = ref.rand_mx(g, (E, O), K)
    buf = torch.empty(E * stride, dtype=torch.uint8, device=DEV)
    big = buf.as_strided((E, O, K // 2), (stride, K // 2, 1))
    big.copy_(q.to(DEV))
    W = qm.MxMat.__new__(qm.MxMat)
    small = qm.MxMat(q.to(DEV), s.to(DEV), K)
    W.__dict__.update(small.__dict__)
    W.keep = buf
    W.desc = qm.qmoe_mxmat.from_buffer_copy(small.desc)
    W.desc.q, W.desc.q_expert_stride = big.data_ptr(), stride
    W.ref = ctypes.byref(W.desc)
    for per in (1, 40):
        n = E * per
        x, x_s, _ = rows_of(kind, g, n, K)
        offsets = torch.arange(0, n + 1, per, dtype=torch.int32, device=DEV)
        assert torch.equal(qm.qmoe_mx_grouped(W, x, offsets, x_s=x_s), qm.qmoe_mx_grouped(small, x, offsets, x_s=x_s))


@pytest.mark.parametrize("E,T,k", [(1024, 5, 64), (1024, 70, 16), (300, 40, 1), (1, 9, 1), (65, 3, 5)])
def test_layer_many_experts_and_choices(E, T, k):
    say(f"mx layer E={E} T={T} k={k}")
    g = gen(E + T)
    H, F = 64, 40
    dev, (gate, up, down) = make_layer(g, E, H, F)
    for kind in ("f32", "bf16"):
        x = torch.randn(T, H, generator=g).to(TYPES[kind])
        ids, w = routing(g, T, E, min(k, E))
        want, bound = ref.layer(gate, up, down, np64(x), ids.numpy(), np64(w), parts(kind), kind == "bf16")
        check_layer(qm.qmoe_mx_layer(dev, x.to(DEV), ids.to(DEV), w.to(DEV)), want, bound, kind, "layer")


@pytest.mark.parametrize("T,H,F", [(1, 16384, 64), (2, 20001, 70), (1, 64, 8192), (3, 100, 12000), (40, 9000, 48)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_layer_wide_sides(kind, T, H, F):
    """Sides whose rows need more than 64 KB of LDS in the decode kernels, or do not fit at all."""
    say(f"mx layer wide {kind} T={T} {H} / {F}")
    g = gen(H + F)
    dev, (gate, up, down) = make_layer(g, 3, H, F)
    x = torch.randn(T, H, generator=g).to(TYPES[kind])
    ids, w = routing(g, T, 3, 2)
    want, bound = ref.layer(gate, up, down, np64(x), ids.numpy(), np64(w), parts(kind), kind == "bf16")
    check_layer(qm.qmoe_mx_layer(dev, x.to(DEV), ids.to(DEV), w.to(DEV)), want, bound, kind, "layer")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_nonfinite_rows_in_tiles(kind):
    """A NaN or infinity stays in its own row where a tile holds it beside others."""
    say(f"mx non-finite rows {kind}")
    g = gen(12)
    E, O, K, n = 4, 700, 512, 2600
    q, s = ref.rand_mx(g, (E, O), K)
    off = torch.tensor([0, 900, 900, 1700, n], dtype=torch.int32, device=DEV)
    x = torch.randn(n, K, generator=g).to(TYPES[kind])
    bad = x.clone()
    rows = [3, 77, 901, 1699, 2599]
    for r, v in zip(rows, (float("nan"), float("inf"), -float("inf"), float("nan"), float("inf"))):
        bad[r, (r * 7) % K] = v
    W = qm.MxMat(q.to(DEV), s.to(DEV), K)
    a, b = (qm.qmoe_mx_grouped(W, t.to(DEV), off, out_dtype=torch.float32).cpu() for t in (x, bad))
    keep = torch.ones(n, dtype=torch.bool)
    keep[rows] = False
    assert torch.equal(a[keep], b[keep])
    assert not torch.isfinite(b[rows]).any()


# Calls that fill the GPU several times over, for the larger tiles: 64 and 128 rows of f32 and bf16, 128 and
# 256 of MXFP4.
@pytest.mark.parametrize("batch,rows,cols", [(1100, 4000, 1030), (2300, 4000, 1030), (4200, 4001, 1025)])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_matmul_large_tiles(kind, out, batch, rows, cols):
    test_matmul(kind, out, batch, rows, cols)


@pytest.mark.parametrize("kind", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_large_tiles(kind, gather):
    say(f"mx grouped large tiles {kind} gather={gather}")
    g = gen(31 + gather)
    E, O, K = 9, 4000, 1030
    off = torch.tensor([0, 700, 1, 0, 255, 1023, 640, 257, 129, 995]).cumsum(0).to(torch.int32)
    n = int(off[-1])
    q, s = ref.rand_mx(g, (E, O), K)
    x, x_s, xv = rows_of(kind, g, n // 2 if gather else n, K)
    pairs = torch.randint(0, n // 2 * 2, (n + 2,), generator=g).to(torch.int32) if gather else None
    y = torch.full((n + 2 if gather else n, O), 3.0, device=DEV)
    qm.qmoe_mx_grouped(qm.MxMat(q.to(DEV), s.to(DEV), K), x, off.to(DEV),
                       pairs=None if pairs is None else pairs.to(DEV), k=2 if gather else 1, x_s=x_s, out=y)
    src = pairs.numpy()[:n] // 2 if gather else np.arange(n)
    want, m = np.zeros((n, O)), np.zeros((n, O))
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        want[a:b], m[a:b] = ref.product(ref.decode(q[e], s[e], K), xv[src[a:b]])
    check(y[:n], want, ref.sum_bound(K, parts(kind)) * m, torch.float32, "grouped large tiles")
    assert (y[n:] == 3.0).all()


@pytest.mark.parametrize("T,E,H,F,k", [(700, 6, 1030, 1100, 4), (2000, 6, 1030, 1100, 4)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_layer_large_tiles(kind, T, E, H, F, k):
    test_layer(kind, T, E, H, F, k)
