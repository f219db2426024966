"""The MXFP4 entry points on a host without a GPU: sizes, and every refusal,
none of which launches anything; and the 64-bit reference of the GPU tests
against values written out by hand."""
import ctypes

import numpy as np
import pytest
import torch

import grouped_int4_expert_amd as q
import mx_ref as ref
from grouped_int4_expert_amd import qmoe_mx_layer_desc, qmoe_mxmat

A = 1 << 40      # 16-byte aligned addresses that are never dereferenced
GB = 1 << 30
OK, NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE, ALIAS, ABI = range(8)


@pytest.fixture(scope="module")
def lib():
    return q.load()


def mat(rows=64, cols=256, at=A, qs=None, ss=None, size=None):
    m = qmoe_mxmat()
    m.struct_size = ctypes.sizeof(qmoe_mxmat) if size is None else size
    m.rows, m.cols = rows, cols
    m.q, m.s = at, at + 16 * GB
    nb = (cols + 31) // 32
    m.q_expert_stride = rows * nb * 16 if qs is None else qs
    m.s_expert_stride = rows * nb if ss is None else ss
    return m


X, XS, Y, OFF, PAIRS, WS = (A + i * 64 * GB for i in range(1, 7))


def matmul(lib, m, dtype=q.QMOE_F32, x=X, x_s=None, batch=4, x_ld=256, y_dtype=q.QMOE_F32, y=Y, y_ld=64, ws=WS,
           ws_bytes=1 << 30):
    return lib.qmoe_mx_matmul(ctypes.byref(m) if m else None, dtype, x, x_s, batch, x_ld, y_dtype, y, y_ld, ws,
                              ws_bytes, None)


def grouped(lib, m, experts=8, dtype=q.QMOE_F32, x=X, x_s=None, x_rows=4, x_ld=256, offsets=OFF, pairs=PAIRS, k=2, n=8,
            y_dtype=q.QMOE_F32, y=Y, y_ld=64, ws=WS, ws_bytes=1 << 30):
    return lib.qmoe_mx_grouped(ctypes.byref(m) if m else None, experts, dtype, x, x_s, x_rows, x_ld, offsets, pairs, k,
                               n, y_dtype, y, y_ld, ws, ws_bytes, None)


def desc(E=8, H=256, F=64, **kw):
    d = qmoe_mx_layer_desc()
    d.struct_size = ctypes.sizeof(qmoe_mx_layer_desc)
    d.experts, d.hidden, d.inter = E, H, F
    d.gate, d.up, d.down = mat(F, H), mat(F, H, A + 20 * GB), mat(H, F, A + 40 * GB)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def layer(lib, d, dtype=q.QMOE_F32, x=X, tokens=4, ids=OFF, w=PAIRS, k=2, out=Y, ws=WS, ws_bytes=1 << 30):
    return lib.qmoe_mx_layer(ctypes.byref(d) if d else None, dtype, x, tokens, ids, w, k, out, ws, ws_bytes, None)


def test_sizes(lib):
    assert lib.qmoe_mx_code_bytes(3, 33) == 3 * 2 * 16
    assert lib.qmoe_mx_scale_bytes(3, 33) == 6
    assert lib.qmoe_mx_code_bytes(-1, 33) == lib.qmoe_mx_scale_bytes(1, -1) == 0
    assert lib.qmoe_mx_code_bytes(1 << 20, 1 << 15) == 1 << 34
    m = mat(64, 256)
    b = ctypes.byref(m)
    assert lib.qmoe_mx_workspace_bytes(b, q.QMOE_BF16, 5, 256) == 0
    assert lib.qmoe_mx_workspace_bytes(b, q.QMOE_BF16, 5, 257) >= 5 * 256 * 2
    assert lib.qmoe_mx_workspace_bytes(b, q.QMOE_F32, 5, 256) >= 5 * 256 * 6
    assert lib.qmoe_mx_workspace_bytes(b, q.QMOE_MXFP4, 5, 256) == 0
    assert lib.qmoe_mx_workspace_bytes(None, q.QMOE_F32, 5, 256) == 0
    d = desc()
    assert lib.qmoe_mx_layer_workspace_bytes(ctypes.byref(d), 4, 2, q.QMOE_F32) > 8 * (256 * 4 + 128 * 6)
    assert lib.qmoe_mx_layer_workspace_bytes(ctypes.byref(d), 4, 65, q.QMOE_F32) == 0
    assert lib.qmoe_mx_layer_workspace_bytes(ctypes.byref(d), 4, 2, q.QMOE_F32_DIGITS) == 0


def test_convert_refusals(lib):
    def quant(x=X, t=q.QMOE_F32, rows=4, cols=64, ld=64, codes=Y, scales=WS):
        return lib.qmoe_mx_quantize(x, t, rows, cols, ld, codes, scales, None)

    def back(codes=Y, scales=WS, rows=4, cols=64, y=X, t=q.QMOE_F32, ld=64):
        return lib.qmoe_mx_dequantize(codes, scales, rows, cols, y, t, ld, None)

    for f, v in ((quant, "x"), (back, "y")):
        assert f(rows=0) == OK and f(cols=0, ld=0) == OK
        assert f(**{v: None}) == NULL and f(codes=None) == NULL and f(scales=None) == NULL
        assert f(rows=-1) == SHAPE and f(cols=-1) == SHAPE and f(ld=63) == SHAPE and f(ld=1 << 31) == SHAPE
        assert f(t=q.QMOE_MXFP4) == UNSUPPORTED and f(t=q.QMOE_F32_DIGITS) == UNSUPPORTED
        assert f(**{v: X + 2}) == ALIGN and f(codes=Y + 4) == ALIGN
        assert f(codes=X + 64) == ALIAS and f(scales=X + 1023) == ALIAS and f(scales=Y + 127) == ALIAS
        assert f(scales=X + 1023, ld=4096) == ALIAS


def test_matmul_refusals(lib):
    m = mat()
    assert matmul(lib, m, batch=0) == OK
    assert matmul(lib, None) == NULL
    for kw in ({"x": None}, {"y": None}, {"dtype": q.QMOE_MXFP4, "x_s": None}):
        assert matmul(lib, m, **kw) == NULL
    assert matmul(lib, mat(size=8)) == ABI
    for kw in ({"batch": -1}, {"x_ld": 255}, {"y_ld": 63}, {"x_ld": 1 << 31}, {"y_ld": 1 << 31},
               {"batch": (1 << 30) + 1}):
        assert matmul(lib, m, **kw) == SHAPE, kw
    assert matmul(lib, mat(0)) == SHAPE and matmul(lib, mat(64, 0, qs=0, ss=0)) == SHAPE
    assert matmul(lib, m, dtype=q.QMOE_F32_DIGITS) == UNSUPPORTED and matmul(lib, m, y_dtype=3) == UNSUPPORTED
    assert matmul(lib, mat(1 << 20, 4096), y_ld=1 << 20, x_ld=4096) == UNSUPPORTED     # 2 GB of codes
    for kw in ({"x": X + 8}, {"y": Y + 8}, {"ws": WS + 8}, {"dtype": q.QMOE_MXFP4, "x_s": XS + 8}):
        assert matmul(lib, m, **kw) == ALIGN, kw
    assert matmul(lib, mat(at=A + 8)) == ALIGN
    need = lib.qmoe_mx_workspace_bytes(ctypes.byref(m), q.QMOE_F32, 4, 256)
    assert matmul(lib, m, ws_bytes=need - 1) == WORKSPACE and matmul(lib, m, ws=None) == WORKSPACE
    for kw in ({"y": X}, {"y": A}, {"y": A + 16 * GB}, {"y": WS}, {"ws": X}, {"ws": A},
               {"dtype": q.QMOE_MXFP4, "x_s": Y + 16}):
        assert matmul(lib, m, **kw) == ALIAS, kw


def test_grouped_refusals(lib):
    m = mat()
    assert grouped(lib, m, n=0) == OK
    assert grouped(lib, None) == NULL and grouped(lib, m, offsets=None) == NULL
    for kw in ({"experts": 0}, {"experts": 1025}, {"k": 0}, {"n": -1}, {"x_rows": 0}, {"pairs": None}, {"n": (1 << 30) + 1}):
        assert grouped(lib, m, **kw) == SHAPE, kw
    assert grouped(lib, mat(qs=64 * 8 * 16 - 16)) == SHAPE and grouped(lib, mat(ss=64 * 8 - 1)) == SHAPE
    assert grouped(lib, mat(qs=64 * 8 * 16 + 8)) == ALIGN
    assert grouped(lib, m, offsets=OFF + 2) == ALIGN and grouped(lib, m, pairs=PAIRS + 1) == ALIGN
    # a gather over 2 GB of operand rows
    assert grouped(lib, m, x_rows=(1 << 31) // 1536 + 1, ws_bytes=1 << 40) == UNSUPPORTED
    for kw in ({"y": OFF}, {"y": PAIRS + 16}, {"ws": OFF}, {"ws": PAIRS}, {"y": A + 7 * 64 * 8 * 16}):
        assert grouped(lib, m, **kw) == ALIAS, kw


def test_layer_refusals(lib):
    d = desc()
    assert layer(lib, d, tokens=0) == OK
    assert layer(lib, None) == NULL
    for kw in ({"x": None}, {"ids": None}, {"w": None}, {"out": None}):
        assert layer(lib, d, **kw) == NULL, kw
    assert layer(lib, desc(struct_size=4)) == ABI and layer(lib, desc(gate=mat(64, 256, size=4))) == ABI
    for bad in (desc(experts=0), desc(experts=1025), desc(hidden=128), desc(inter=32), desc(up=mat(96, 256)),
                desc(down=mat(256, 96))):
        assert layer(lib, bad) == SHAPE
    for kw in ({"tokens": -1}, {"k": 0}, {"k": 65}, {"tokens": (1 << 30) // 2 + 1}):
        assert layer(lib, d, **kw) == SHAPE, kw
    assert layer(lib, d, dtype=q.QMOE_F32_DIGITS) == UNSUPPORTED and layer(lib, d, dtype=q.QMOE_MXFP4) == UNSUPPORTED
    assert layer(lib, d, tokens=(1 << 31) // 1536 + 1, ws_bytes=1 << 50) == UNSUPPORTED
    for kw in ({"x": X + 4}, {"out": Y + 4}, {"ids": OFF + 2}, {"w": PAIRS + 2}, {"ws": WS + 8}):
        assert layer(lib, d, **kw) == ALIGN, kw
    need = lib.qmoe_mx_layer_workspace_bytes(ctypes.byref(d), 4, 2, q.QMOE_F32)
    assert layer(lib, d, ws_bytes=need - 1) == WORKSPACE and layer(lib, d, ws=None) == WORKSPACE
    for kw in ({"out": X}, {"out": OFF}, {"out": PAIRS}, {"out": WS + 64}, {"ws": X}, {"ws": A + 20 * GB},
               {"out": A + 40 * GB}):
        assert layer(lib, d, **kw) == ALIAS, kw


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64)
    with pytest.raises(TypeError):
        q.qmoe_mx_quantize(x)
    with pytest.raises(TypeError):
        q.MxMat(torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8), 64)


def test_reference_by_hand():
    x = np.zeros((2, 40))
    x[0, :9] = [6.0, -5.0, 2.5, 0.25, 0.75, 1.25, 1.75, 3.5, 7.9]
    x[1, 33] = -12.0
    codes, s = ref.quantize(x)
    assert s.tolist() == [[127, 0], [0, 128]]
    got = ref.decode(codes, s, 40)
    assert got[0, :9].tolist() == [6.0, -4.0, 2.0, 0.0, 1.0, 1.0, 2.0, 4.0, 6.0]
    assert got[1, 33] == -12.0 and (got[1, :33] == 0).all()
    assert codes[0, 0] == (7 | (8 | 6) << 4)
    y, m = ref.product(np.array([[1.0, -2.0]]), np.array([[3.0, 4.0]]))
    assert y[0, 0] == -5.0 and m[0, 0] == 11.0
    eye = np.eye(2)[None]
    out, bound = ref.layer(eye, eye, eye, np.array([[1.0, -2.0]]), np.array([[0, 7]]), np.array([[0.5, 0.5]]), 1, False)
    want = 0.5 * np.array([1 / (1 + np.exp(-1.0)), 4 / (1 + np.exp(2.0))])
    assert np.allclose(out[0], want, rtol=1e-14) and (bound > 0).all()


class OnDevice(torch.Tensor):
    """A host tensor that says it is on a device, for the checks before a launch."""
    is_cuda = property(lambda self: True)


def test_rows_of_views():
    wide = torch.zeros(6, 40).as_subclass(OnDevice)
    assert q._rows(wide, "x")[1:] == (6, 40)
    assert q._rows(wide[:, 8:24], "x")[1:] == (6, 40)
    assert q._rows(wide[::2, :8], "x")[1:] == (3, 80)
    assert q._rows(wide[2], "x")[1:] == (1, 40)
    assert q._rows(wide[:, 3:4], "x")[1:] == (6, 40)
    assert q._rows(wide[:1].expand(1, 40), "x")[1:] == (1, 40)
    for bad in (wide[:1].expand(6, 40), wide[0].expand(3, 40), wide.as_strided((5, 40), (8, 1)), wide[:, 3],
                wide.t(), wide[:, ::2], wide.reshape(2, 3, 40), wide[0, 0]):
        with pytest.raises(ValueError):
            q._rows(bad, "x")
