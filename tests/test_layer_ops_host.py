"""Layer operators without a GPU: refusals of the C ABI, workspace sizes, and
the references the GPU tests compare with (their gradients against
differences).

Every call below carries an argument that the host validation rejects, so
nothing here can reach a kernel.
"""
import ctypes

import numpy as np
import pytest

import additive_quantized_matmul_b200 as aq
import layer_ref as lr
from aq_inputs import LayerSpec, make_activations, make_layer

FAKE = 0x10000  # 16-byte aligned, never dereferenced
A = FAKE        # distinct fake arrays
X, Y, GY, GZ, GU, GX = (FAKE + 0x1000 * i for i in range(1, 7))
D = aq.LayerDesc.make(64, 256, 2, 8)
BIG = 1 << 40


def _ep(act=0, bias=None, residual=None):
    return aq.Epilogue(act, bias, residual)


def _fused(fn, d=D, packed=A, cb=A, s=A, x=X, n=8, ep=None, y=Y, ws=A, wsb=BIG):
    return getattr(aq.lib, fn)(ctypes.byref(d) if d is not None else None, packed, cb, s, x, n, ep, y, ws, wsb, None)


@pytest.mark.parametrize("fn", ["aq_gemv_fused", "aq_gemm_fused"])
def test_fused_refusals(fn):
    call = lambda **k: _fused(fn, **k)  # noqa: E731
    assert call(n=0) == 1 and call(n=-3) == 1 and call(n=17 if fn == "aq_gemv_fused" else (1 << 22) + 1) == 1
    assert call(d=None) == 1 and call(d=aq.LayerDesc.make(64, 256, 3, 8)) == 2
    assert call(packed=None) == 1 and call(cb=None) == 1 and call(x=None) == 1 and call(y=None) == 1
    assert call(x=Y) == 1
    assert call(packed=A + 8) == 3 and call(cb=A + 2) == 3 and call(x=X + 2) == 3 and call(y=Y + 8) == 3
    assert call(s=A + 1) == 3
    assert call(ep=_ep(5)) == 1 and call(ep=_ep(-1)) == 1
    assert call(ep=_ep(1, bias=A + 1)) == 3 and call(ep=_ep(1, residual=A + 8)) == 3
    assert call(ws=None) == 4 and call(wsb=8) == 4 and call(ws=A + 8) == 3


def test_input_grad_refusals():
    def call(d=D, packed=A, cb=A, s=A, gy=GY, T=8, gx=GX, ws=A, wsb=BIG):
        return aq.lib.aq_input_grad(ctypes.byref(d), packed, cb, s, gy, T, gx, ws, wsb, None)

    assert call(T=0) == 1 and call(T=(1 << 22) + 1) == 1
    assert call(gy=None) == 1 and call(gx=None) == 1 and call(gx=GY) == 1 and call(packed=None) == 1
    assert call(gy=GY + 2) == 3 and call(gx=GX + 2) == 3 and call(s=A + 1) == 3 and call(cb=A + 4) == 3
    assert call(ws=None) == 4 and call(wsb=4) == 4 and call(ws=A + 4) == 3
    assert call(d=aq.LayerDesc(64, 256, 4, 1, 16)) == 2


def test_fused_grad_refusals():
    def call(d=D, packed=A, cb=A, s=A, x=X, gy=GY, T=8, ep=None, gz=GZ, gb=A, gx=GX, ws=A, wsb=BIG):
        return aq.lib.aq_gemm_fused_grad(ctypes.byref(d), packed, cb, s, x, gy, T, ep, gz, gb, gx, ws, wsb, None)

    assert call(T=0) == 1 and call(T=(1 << 22) + 1) == 1
    assert call(x=None) == 1 and call(gy=None) == 1 and call(gz=None) == 1
    assert call(gz=X) == 1 and call(gz=GY) == 1 and call(gx=X) == 1 and call(gx=GY) == 1 and call(gx=GZ) == 1
    assert call(x=X + 2) == 3 and call(gy=GY + 4) == 3 and call(gz=GZ + 8) == 3 and call(gb=A + 4) == 3
    assert call(gx=GX + 2) == 3
    assert call(ep=_ep(7)) == 1 and call(ep=_ep(2, bias=A + 1)) == 3
    assert call(ws=None) == 4 and call(wsb=8) == 4 and call(ws=A + 8) == 3


@pytest.mark.parametrize("fn", ["aq_glu_gemv", "aq_glu_gemm"])
def test_glu_refusals(fn):
    def call(d=D, gate=(A, A, A), up=(A, A, A), x=X, n=8, act=4, y=Y, ws=A, wsb=BIG):
        return getattr(aq.lib, fn)(ctypes.byref(d), aq.Weights(*gate) if gate else None,
                                   aq.Weights(*up) if up else None, x, n, act, y, ws, wsb, None)

    assert call(n=0) == 1 and call(n=17 if fn == "aq_glu_gemv" else (1 << 22) + 1) == 1
    assert call(gate=None) == 1 and call(up=None) == 1 and call(x=None) == 1 and call(y=None) == 1 and call(x=Y) == 1
    assert call(gate=(None, A, A)) == 1 and call(up=(A, None, A)) == 1
    assert call(gate=(A + 8, A, A)) == 3 and call(up=(A, A + 2, A)) == 3 and call(up=(A, A, A + 1)) == 3
    assert call(act=5) == 1 and call(act=-1) == 1
    assert call(x=X + 8) == 3 and call(y=Y + 2) == 3
    assert call(ws=None) == 4 and call(wsb=8) == 4 and call(ws=A + 8) == 3


def test_glu_gemv_refuses_more_rows_than_counters():
    d = aq.LayerDesc.make(131080, 64, 1, 16)
    assert aq.aq_glu_gemv_workspace_bytes(d, 1) == 0
    w = aq.Weights(A, A, None)
    assert aq.lib.aq_glu_gemv(ctypes.byref(d), w, w, X, 1, 4, Y, A, BIG, None) == 1
    assert aq.aq_glu_gemv_workspace_bytes(aq.LayerDesc.make(131072, 64, 1, 16), 1) >= 16


def test_glu_grad_refusals():
    def call(d=D, gate=(A, A, A), up=(A, A, A), x=X, gy=GY, T=8, act=4, gg=GZ, gu=GU, gx=GX, ws=A, wsb=BIG):
        return aq.lib.aq_glu_grad(ctypes.byref(d), aq.Weights(*gate) if gate else None,
                                  aq.Weights(*up) if up else None, x, gy, T, act, gg, gu, gx, ws, wsb, None)

    assert call(T=0) == 1 and call(T=(1 << 22) + 1) == 1 and call(act=9) == 1
    assert call(gate=None) == 1 and call(up=None) == 1 and call(x=None) == 1 and call(gy=None) == 1
    assert call(gg=None) == 1 and call(gu=None) == 1
    for k, v in (("gg", X), ("gg", GY), ("gg", GU), ("gu", X), ("gu", GY), ("gx", X), ("gx", GY), ("gx", GZ), ("gx", GU)):
        assert call(**{k: v}) == 1, (k, v)
    assert call(gg=GZ + 2) == 3 and call(gu=GU + 8) == 3 and call(gx=GX + 4) == 3 and call(gy=GY + 2) == 3
    assert call(gate=(A, A, A + 1)) == 3
    assert call(ws=None) == 4 and call(wsb=8) == 4 and call(ws=A + 8) == 3


def test_workspace_sizes():
    bad = aq.LayerDesc.make(64, 256, 3, 8)
    for fn in (aq.aq_gemm_fused_workspace_bytes, aq.aq_input_grad_workspace_bytes,
               aq.aq_gemm_fused_grad_workspace_bytes, aq.aq_glu_gemm_workspace_bytes, aq.aq_glu_grad_workspace_bytes):
        assert fn(bad, 8) == 0 and fn(D, 0) == 0 and fn(D, (1 << 22) + 1) == 0
        for T in (1, 7, 8, 77, 2048, 1 << 22):
            assert fn(D, T) >= 16
    assert aq.aq_glu_gemv_workspace_bytes(D, 0) == 0 and aq.aq_glu_gemv_workspace_bytes(D, 17) == 0
    assert all(aq.aq_glu_gemv_workspace_bytes(D, b) >= 16 for b in range(1, 17))


def test_binding_raises():
    w = aq.Weights(A, A, A)
    with pytest.raises(aq.AQError):
        aq.aq_glu_gemv(D, w, w, X, 0, 4, Y, A, 1 << 30, stream=0)
    with pytest.raises(aq.AQError):
        aq.aq_gemm_fused(D, A, A, A, X, 8, Y, A, 1 << 30, stream=0, activation=11)


@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_reference_slopes_against_differences(kind):
    """Central differences of step h are off by h^2/6 times the third
    derivative (below 3 for each of these) and by 2 * 2^-53 |a| / h."""
    z = np.linspace(-6, 6, 4001) + 1e-3  # away from relu's corner
    h = 1e-4
    _, slope = lr.act(kind, z)
    diff = (lr.act(kind, z + h)[0] - lr.act(kind, z - h)[0]) / (2 * h)
    assert (np.abs(diff - slope) <= 3 * h * h / 6 + 2 * 2.0 ** -52 * (1 + np.abs(z)) / h).all()
    assert np.abs(slope).max() <= 1.13
    if kind not in ("none", "relu"):
        curve = (lr.act(kind, z + h)[1] - lr.act(kind, z - h)[1]) / (2 * h)
        assert np.abs(curve).max() <= 1.0


def test_reference_gradients_against_differences():
    """The gated block's and the fused product's reference gradients of
    L = sum(gy y) against central differences in x: their error is h^2/6
    times the third derivative along the direction and the rounding of L."""
    rng = np.random.default_rng(3)
    gate, up = (lr.Ref(make_layer(LayerSpec(24, 40, 2, 8, codebook_sigma=0.1), (5, i))) for i in range(2))
    x = rng.normal(size=(40, 6))
    gy = rng.normal(size=(24, 6))
    v = rng.normal(size=x.shape)
    h = 1e-5

    def glu_loss(xx):
        return (gy * lr.glu(gate, up, xx, "silu")[0]).sum()

    (gg, _), (gu, _) = lr.glu_grad(gate, up, x, gy, "silu")
    gx, _ = gate.back(gg, [(up, gu)])
    diff = (glu_loss(x + h * v) - glu_loss(x - h * v)) / (2 * h)
    assert abs(diff - (gx * v).sum()) <= 1e-6 * np.abs(gx * v).sum()

    bias = rng.normal(size=24)

    def fused_loss(xx, bb):
        return (gy * lr.fused(gate, xx, "gelu", bb)[0]).sum()

    (gz, _), (gb, _) = lr.fused_grad(gate, x, gy, "gelu", bias)
    gx, _ = gate.back(gz)
    diff = (fused_loss(x + h * v, bias) - fused_loss(x - h * v, bias)) / (2 * h)
    assert abs(diff - (gx * v).sum()) <= 1e-6 * np.abs(gx * v).sum()
    vb = rng.normal(size=24)
    diff = (fused_loss(x, bias + h * vb) - fused_loss(x, bias - h * vb)) / (2 * h)
    assert abs(diff - (gb * vb).sum()) <= 1e-6 * np.abs(gb * vb).sum()
