"""Refusals and sizes of the serving entry points, on the host: nothing here is launched."""
import ctypes

import numpy as np
import pytest
import torch

from dropless_mixture_experts_dmoe_b200 import binding as B
from dropless_mixture_experts_dmoe_b200 import build as build_mod

import serving_ref as R

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load()


def few(lib, d, mx4=False, **kw):
    a = dict(x=FAKE, logits=FAKE, w1=FAKE, w3=FAKE, w2=FAKE, top=FAKE, weights=FAKE, y=FAKE,
             status=FAKE, ws=FAKE, n=1 << 40)
    a.update(kw)
    if mx4:
        for w in ("w1", "w3", "w2"):
            v = a[w]
            a[w] = ctypes.byref(B.dmoe_mx4(*(v if isinstance(v, tuple) else (v, v)))) if v else None
    fn = lib.dmoe_mx4_forward_few if mx4 else lib.dmoe_forward_few
    return fn(ctypes.byref(d), a["x"], a["logits"], a["w1"], a["w3"], a["w2"], a["top"],
              a["weights"], a["y"], a["status"], a["ws"], a["n"], None)


@pytest.mark.parametrize("mx4", [False, True])
def test_few_refusals(lib, mx4):
    d = B.make_dims(128, 256, 128, 8, 2)
    for name in ("x", "w1", "w3", "w2", "top", "weights", "y", "status", "ws"):
        assert few(lib, d, mx4, **{name: None}) == -1, name
    for name in ("x", "logits", "w1", "w3", "w2", "top", "weights", "y", "ws"):
        assert few(lib, d, mx4, **{name: FAKE + 8}) == -5, name
    need = B.dmoe_workspace_bytes(d, B.WS_FEW)
    assert need >= 128 * 2 * 128 * 4
    assert few(lib, d, mx4, n=need - 1) == -4
    if mx4:
        assert few(lib, d, True, w3=(FAKE, 0)) == -1
        assert few(lib, d, True, w2=(FAKE, FAKE + 4)) == -5
    assert few(lib, B.make_dims(129, 256, 128, 8, 2), mx4) == -2
    assert few(lib, B.make_dims(16, 256, 128, 8, 2, flags=B.ROUTE_TOKEN_ROUNDING), mx4) == -2
    assert few(lib, B.make_dims(16, 200, 128, 8, 2), mx4) == -2
    assert few(lib, B.make_dims(16, 256, 128, 8, 9), mx4) == -2
    assert few(lib, B.make_dims(16, 256, 128, 2000, 2), mx4) == -3
    assert B.dmoe_workspace_bytes(B.make_dims(129, 256, 128, 8, 2), B.WS_FEW) == 0


def test_mx4_conversion_refusals(lib):
    m = B.dmoe_mx4(FAKE, FAKE)
    for rows, cols, code in ((0, 128, -2), (-1, 128, -2), (4, 0, -2), (4, 64, -2), (4, 200, -2),
                             (2 ** 41, 128, -8), (4, 2 ** 31, -8), (4, 2 ** 24, -8),
                             (2 ** 40, 2 ** 23, -8)):
        assert lib.dmoe_mx4_quantize(rows, cols, FAKE, ctypes.byref(m), None) == code
        assert lib.dmoe_mx4_dequantize(rows, cols, ctypes.byref(m), FAKE, None) == code
    for bad, code in ((None, -1), (B.dmoe_mx4(0, FAKE), -1), (B.dmoe_mx4(FAKE, 0), -1),
                      (B.dmoe_mx4(FAKE + 1, FAKE), -5), (B.dmoe_mx4(FAKE, FAKE + 8), -5)):
        p = ctypes.byref(bad) if bad else None
        assert lib.dmoe_mx4_quantize(4, 128, FAKE, p, None) == code
        assert lib.dmoe_mx4_dequantize(4, 128, p, FAKE, None) == code
    assert lib.dmoe_mx4_quantize(4, 128, None, ctypes.byref(m), None) == -1
    assert lib.dmoe_mx4_quantize(4, 128, FAKE + 2, ctypes.byref(m), None) == -5
    assert lib.dmoe_mx4_dequantize(4, 128, ctypes.byref(m), FAKE + 2, None) == -5


def test_mx4_forward_refusals(lib):
    d = B.make_dims(500, 256, 128, 8, 2)
    m = B.dmoe_map(*([FAKE] * len(B.MAP_FIELDS)))
    w = B.dmoe_mx4(FAKE, FAKE)
    n = B.dmoe_workspace_bytes(d, B.WS_MX4_FORWARD)
    P = B.dmoe_padded_rows_max(d)
    assert n >= P * 256 * 17 // 32 + P * 128 * 17 // 32 + P * 256 * 2 + P * 4 * 4

    def call(x=FAKE, w1=w, w3=w, w2=w, mm=m, y=FAKE, ws=FAKE, size=n, dims=d):
        r = lambda s: ctypes.byref(s) if s is not None else None
        return lib.dmoe_mx4_forward(ctypes.byref(dims), x, r(w1), r(w3), r(w2), r(mm), y, ws, size,
                                    None)

    for kw in (dict(x=None), dict(w1=None), dict(w2=B.dmoe_mx4(FAKE, 0)), dict(mm=None),
               dict(mm=B.dmoe_map()), dict(y=None), dict(ws=None)):
        assert call(**kw) == -1, kw
    for kw in (dict(x=FAKE + 4), dict(w3=B.dmoe_mx4(FAKE + 8, FAKE)), dict(y=FAKE + 8),
               dict(ws=FAKE + 8)):
        assert call(**kw) == -5, kw
    assert call(size=n - 1) == -4
    assert call(dims=B.make_dims(500, 256, 100, 8, 2)) == -2


def test_mx4_tensors_are_checked():
    u8 = dict(dtype=torch.uint8)
    assert B.Mx4.scales_shape(4, 256, 384) == (4, 2, 3, 32, 4, 4)
    assert B.Mx4.scales_shape(130, 128) == (2, 1, 32, 4, 4)
    for shape in ((4, 64), (0, 128), (2, 130, 128), (128, 200)):
        with pytest.raises(ValueError):
            B.Mx4.scales_shape(*shape)
    q = B.Mx4.empty(130, 256, device="cpu")
    assert q.shape == (130, 256) and q.codes.shape == (130, 128)
    with pytest.raises(ValueError):
        B.Mx4(torch.zeros(128, 64, **u8), torch.zeros(1, 1, 32, 4, 3, **u8))
    with pytest.raises(ValueError):
        B.Mx4(torch.zeros(128, 64), torch.zeros(1, 1, 32, 4, 4, **u8))
    with pytest.raises(ValueError):
        B.Mx4(torch.zeros(64, 128, **u8).t(), torch.zeros(1, 1, 32, 4, 4, **u8))
    with pytest.raises(B.DMoEError):
        B.FewBuffers(B.make_dims(129, 256, 128, 8, 2), device="cpu")


def test_reference_of_the_format():
    """The 64-bit definition on hand-worked blocks."""
    x = np.zeros((1, 64))
    x[0, :8] = [6, 5, 2.5, 3.5, -0.25, -0.75, 0.26, 7.9]
    x[0, 32:36] = [1.0, 0.5, -0.0625, 0.0625 * 1.01]
    q, e = R.mx4_blocks(x)
    assert e.tolist() == [[0.0, -2.0]]
    assert q[0, 0, :8].tolist() == [6, 4, 2, 4, -0.0, -1, 0.5, 6]
    assert q[0, 1, :4].tolist() == [4, 2, -0.0, 0.5]


def test_binding_checks_tensors_on_the_host():
    """Wrong device, type, shape or layout is a ValueError before the library is called."""
    d = B.make_dims(4, 256, 128, 8, 2)
    few = B.FewBuffers(d, device="cpu")
    bf = dict(dtype=torch.bfloat16)
    x, lg = torch.zeros(4, 256, **bf), torch.zeros(4, 8, **bf)
    w1, w2 = torch.zeros(8, 128, 256, **bf), torch.zeros(8, 256, 128, **bf)
    q1, q2 = B.Mx4.empty(8, 128, 256, device="cpu"), B.Mx4.empty(8, 256, 128, device="cpu")
    with pytest.raises(ValueError, match="x must be"):
        B.dmoe_forward_few(d, x, lg, w1, w1, w2, few, x)
    with pytest.raises(ValueError, match="x must be"):
        B.dmoe_forward_few(d, x.t(), lg, w1, w1, w2, few, x)
    with pytest.raises(ValueError, match="w1 must be"):
        B.dmoe_forward_few(d, FAKE, FAKE, w1, w1, w2, few, FAKE)
    with pytest.raises(ValueError, match="w1 must have"):
        B.dmoe_mx4_forward_few(d, FAKE, FAKE, q2, q1, q2, few, FAKE)
    with pytest.raises(ValueError, match="buffers"):
        B.dmoe_forward_few(B.make_dims(3, 256, 128, 8, 2), x, lg, w1, w1, w2, few, x)
    with pytest.raises(ValueError, match="src must be"):
        B.dmoe_mx4_quantize(w1, q1)
    with pytest.raises(ValueError, match="src must have"):
        B.dmoe_mx4_dequantize(q1, w1)


def test_buffers_of_the_serving_calls_are_fixed():
    """Their addresses are taken once: a replaced tensor or a changed size is refused."""
    d = B.make_dims(4, 256, 128, 8, 2)
    few = B.FewBuffers(d, device="cpu")
    for name in ("top_experts", "weights", "status", "ws"):
        with pytest.raises(AttributeError):
            setattr(few, name, getattr(few, name).clone())
    q = B.Mx4.empty(8, 128, 256, device="cpu")
    for name in ("codes", "scales"):
        with pytest.raises(AttributeError):
            setattr(q, name, getattr(q, name).clone())
    d.T = 5
    with pytest.raises(ValueError, match="buffers"):
        B.dmoe_forward_few(d, FAKE, FAKE, FAKE, FAKE, FAKE, few, FAKE)
    d.T = 4
    with pytest.raises(ValueError, match="the buffers must be on"):
        B.dmoe_forward_few(d, FAKE, FAKE, FAKE, FAKE, FAKE, few, FAKE)
    m = B.Mx4Buffers(d, device="cpu")
    w = (q, q, B.Mx4.empty(8, 256, 128, device="cpu"))
    with pytest.raises(ValueError, match="the map is"):
        B.dmoe_mx4_forward(B.make_dims(5, 256, 128, 8, 2), FAKE, *w, m.map, FAKE, m.ws)
    with pytest.raises(ValueError, match="smap.status"):
        B.dmoe_mx4_forward(d, FAKE, *w, m.map, FAKE, m.ws)


def test_weights_too_tall(lib):
    """Rows of the stacked weights past 31 bits."""
    d = B.make_dims(4, 2 ** 22, 128, 1024, 2)
    assert few(lib, d) == -8 and few(lib, d, True) == -8
    m = B.dmoe_map(*([FAKE] * len(B.MAP_FIELDS)))
    w = B.dmoe_mx4(FAKE, FAKE)
    r = ctypes.byref
    assert lib.dmoe_mx4_forward(r(d), FAKE, r(w), r(w), r(w), r(m), FAKE, FAKE, 1 << 60, None) == -8
