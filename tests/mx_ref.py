"""MXFP4 in 64 bits, for the tests: decoding by the fields of each code,
rounding by distance to the eight magnitudes, and the products with the
magnitudes of their terms.  Shares nothing with the library."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24         # half a step of f32
UB = 2.0 ** -8         # half a step of bf16
MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def blocks(cols):
    return (cols + 31) // 32


def decode(q, s, cols):
    """uint8 [..., nb * 16], [..., nb] -> float64 [..., cols]."""
    q, s = np.asarray(q), np.asarray(s)
    c = np.stack([q & 15, q >> 4], -1).reshape(*s.shape, 32)
    v = MAGS[c & 7] * np.where(c & 8, -1.0, 1.0)
    sc = np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))
    return (v * sc[..., None]).reshape(*s.shape[:-1], -1)[..., :cols]


def quantize(x):
    """float64 [rows, cols] -> (codes, scale bytes).  The nearest magnitude by
    distance; of two equally near ones the one with the even code."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb = blocks(cols)
    b = np.zeros((rows, nb * 32))
    b[:, :cols] = x
    b = b.reshape(rows, nb, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    most = np.abs(b).max(-1)
    with np.errstate(divide="ignore"):
        e = np.where(most > 0, np.frexp(most)[1] - 3, -127)
    e = np.clip(e, -127, 127)
    a = np.abs(b) / np.ldexp(1.0, e)[..., None]
    d = np.abs(a[..., None] - MAGS)
    # even codes first among equals
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])
    code = order[np.argmin(d[..., order], -1)]
    code = code | np.where(np.signbit(b), 8, 0)
    code = np.where(bad[..., None], 0, code).reshape(rows, nb, 16, 2)
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    return (code[..., 0] | code[..., 1] << 4).astype(np.uint8).reshape(rows, nb * 16), s


def rand_mx(g, shape, cols, near=None):
    """Random codes with zeros past `cols`, scale bytes within four of each
    other, such that a sum over unit inputs is near one."""
    nb = blocks(cols)
    near = 122 - round(np.log2(max(cols, 1)) / 2) if near is None else near
    q = torch.randint(0, 256, (*shape, nb * 16), generator=g, dtype=torch.uint8)
    s = torch.randint(near, near + 4, (*shape, nb), generator=g, dtype=torch.uint8)
    last = cols - (nb - 1) * 32
    q[..., (nb - 1) * 16 + (last + 1) // 2:] = 0
    if last % 2:
        q[..., (nb - 1) * 16 + last // 2] &= 15
    return q, s


def product(w, x):
    """(y, M): x [n, K] times w [O, K] and the sums of the terms' magnitudes."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def sum_bound(K, parts):
    """Error of an f32 sum of `parts` exact products for each of K inputs,
    relative to the sum of the terms' magnitudes: every one of the parts * K
    additions inside the matrix instructions rounds or truncates once (at most
    2 U of a partial sum, which the magnitudes bound), as do the at most 64
    additions that join the pieces and the conversion."""
    return 2.0 * U * (parts * K + 64)


def silu(z):
    with np.errstate(over="ignore"):
        return z / (1.0 + np.exp(-z))


def layer(gate, up, down, x, ids, w, parts, bf16):
    """(out, bound) of the routed layer in 64 bits; the weights float64 [E, ..],
    x [T, H].  The bound follows each rounded quantity: gate and up sums, the
    SiLU (derivative at most 1.1; at most 8 roundings of its own) and the
    product, h's rounding to bf16 where x is bf16, the down sum, the routing
    weight and the k additions, and out's own rounding."""
    T, H = x.shape
    F = gate.shape[1]
    out, bound, top = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    for e in range(gate.shape[0]):
        t, j = np.nonzero(ids == e)
        if not len(t):
            continue
        a, am = product(gate[e], x[t])
        u, um = product(up[e], x[t])
        da, du = sum_bound(H, parts) * am, sum_bound(H, parts) * um
        h = silu(a) * u
        dh = 1.1 * da * np.abs(u) + np.abs(silu(a)) * du + 1.1 * da * du + 16 * U * np.abs(h)
        if bf16:
            dh = dh + UB * (np.abs(h) + dh)
        y, ym = product(down[e], h)
        far = dh @ np.abs(down[e]).T
        dy = far + sum_bound(F, parts) * (ym + far)
        wt = w[t, j][:, None]
        np.add.at(out, t, wt * y)
        np.add.at(bound, t, np.abs(wt) * (dy + 2 * U * np.abs(y)))
        np.add.at(top, t, np.abs(wt) * (np.abs(y) + dy))
    bound += 2 * U * ids.shape[1] * top
    return out, bound + (UB if bf16 else U) * (np.abs(out) + bound)
