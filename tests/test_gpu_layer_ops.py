"""Layer operators on the GPU, through the binding, against 64-bit references
with derived tolerances (layer_ref.py): the product with bias, activation and
residual, the gated feed-forward block, the input gradient, and their
backward passes.

Every input lies between bands of NaN, every output between canaries, and
the status word of each workspace is read.
"""
import numpy as np
import pytest
import torch

import additive_quantized_matmul_b200 as aq
import layer_ref as lr
from aq_inputs import LayerSpec, make_activations, make_layer
from aqtest import DevLayer, dev, guarded, guards_intact, to_f16, workspace

pytestmark = pytest.mark.gpu

SCHEMES = [(1, 16), (2, 8), (1, 8), (2, 16), (8, 8)]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
FENCE = 2048  # binary16 elements of NaN before and after each input


def fenced(a):
    a = np.ascontiguousarray(a, dtype=np.float16)
    n = a.size
    pad = -n % 8  # keep the second band right behind the data
    full = torch.full((2 * FENCE + n + pad,), 0x7E00, dtype=torch.int16, device="cuda")
    full[FENCE:FENCE + n] = torch.from_numpy(a.view(np.int16).ravel()).cuda()
    return full[FENCE:FENCE + n]


def half(t, *shape):
    return to_f16(t).reshape(shape)


class Case:
    """Layers of one shape with their references; runs each operator."""

    def __init__(self, out, inp, K, B, seed, layers=1, sigma=0.05, scaled=True, scale=None):
        self.out, self.inp = out, inp
        self.layers = [make_layer(LayerSpec(out, inp, K, B, codebook_sigma=sigma), (seed, i)) for i in range(layers)]
        if scale is not None:
            for L in self.layers:
                L.scales[...] = (L.scales.view(np.float16).astype(np.float64) * scale).astype(np.float16).view(L.scales.dtype)
        self.refs = [lr.Ref(L, scaled) for L in self.layers]
        self.dls = [DevLayer(L) for L in self.layers]
        self.desc = self.dls[0].desc
        self.books = [fenced(L.codebooks.view(np.float16)) for L in self.layers]
        self.scales = [fenced(L.scales.view(np.float16)) if scaled else None for L in self.layers]
        self.weights = [aq.Weights.make(d.packed, c, s) for d, c, s in zip(self.dls, self.books, self.scales)]

    def w(self):
        return self.desc, self.dls[0].packed, self.books[0], self.scales[0]

    def fused(self, x, kind="none", bias=None, residual=None, gemm=None, ws=None):
        n = x.shape[1]
        gemm = n > 16 if gemm is None else gemm
        full, y = guarded(self.out * n)
        size = aq.aq_gemm_fused_workspace_bytes if gemm else aq.aq_gemv_workspace_bytes
        ws = workspace(size(self.desc, n)) if ws is None else ws
        (aq.aq_gemm_fused if gemm else aq.aq_gemv_fused)(
            *self.w(), fenced(x), n, y, ws, activation=aq.ACTIVATIONS[kind],
            bias=None if bias is None else fenced(bias), residual=None if residual is None else fenced(residual))
        assert aq.aq_workspace_status(ws) == 0
        assert guards_intact(full)
        return half(y, self.out, n)

    def fused_grad(self, x, gy, kind, bias=None, want_bias=True, want_x=True, ws=None):
        n = x.shape[1]
        fz, gz = guarded(self.out * n)
        fx, gx = guarded(self.inp * n)
        fb = torch.full((self.out + 64,), 7.25, dtype=torch.float32, device="cuda")
        ws = workspace(aq.aq_gemm_fused_grad_workspace_bytes(self.desc, n)) if ws is None else ws
        aq.aq_gemm_fused_grad(*self.w(), fenced(x), fenced(gy), n, gz, fb[32:] if want_bias else None,
                              gx if want_x else None, ws, activation=aq.ACTIVATIONS[kind],
                              bias=None if bias is None else fenced(bias))
        assert aq.aq_workspace_status(ws) == 0
        assert guards_intact(fz) and guards_intact(fx)
        assert bool((fb[:32] == 7.25).all()) and bool((fb[32 + self.out:] == 7.25).all())
        return half(gz, self.out, n), fb[32:32 + self.out].cpu().numpy(), half(gx, self.inp, n)

    def input_grad(self, gy, ws=None):
        n = gy.shape[1]
        full, gx = guarded(self.inp * n)
        ws = workspace(aq.aq_input_grad_workspace_bytes(self.desc, n)) if ws is None else ws
        aq.aq_input_grad(*self.w(), fenced(gy), n, gx, ws)
        assert aq.aq_workspace_status(ws) == 0
        assert guards_intact(full)
        return half(gx, self.inp, n)

    def glu(self, x, kind, gemm=None, ws=None):
        n = x.shape[1]
        gemm = n > 16 if gemm is None else gemm
        full, y = guarded(self.out * n)
        size = aq.aq_glu_gemm_workspace_bytes if gemm else aq.aq_glu_gemv_workspace_bytes
        ws = workspace(size(self.desc, n)) if ws is None else ws
        (aq.aq_glu_gemm if gemm else aq.aq_glu_gemv)(self.desc, *self.weights, fenced(x), n, aq.ACTIVATIONS[kind], y, ws)
        assert aq.aq_workspace_status(ws) == 0
        assert guards_intact(full)
        return half(y, self.out, n)

    def glu_grad(self, x, gy, kind, want_x=True, ws=None):
        n = x.shape[1]
        fg, gg = guarded(self.out * n)
        fu, gu = guarded(self.out * n)
        fx, gx = guarded(self.inp * n)
        ws = workspace(aq.aq_glu_grad_workspace_bytes(self.desc, n)) if ws is None else ws
        aq.aq_glu_grad(self.desc, *self.weights, fenced(x), fenced(gy), n, aq.ACTIVATIONS[kind], gg, gu,
                       gx if want_x else None, ws)
        assert aq.aq_workspace_status(ws) == 0
        assert guards_intact(fg) and guards_intact(fu) and guards_intact(fx)
        return half(gg, self.out, n), half(gu, self.out, n), half(gx, self.inp, n)


def acts(rows, n, seed, sigma=1.0):
    return (make_activations(rows, n, seed).view(np.float16).astype(np.float32) * sigma).astype(np.float16)


SHAPES = [(8, 8), (20, 520), (136, 264), (300, 1032)]


@pytest.mark.parametrize("K,B", SCHEMES)
@pytest.mark.parametrize("out,inp", SHAPES + [(1000, 2056)])
@pytest.mark.parametrize("n", [1, 2, 3, 8, 16])
def test_gemv_fused(K, B, out, inp, n):
    c = Case(out, inp, K, B, 11 * out + n)
    x, b, r = acts(inp, n, (1, n)), acts(out, 1, 2).ravel(), acts(out, n, (3, n))
    kind = ACTS[(n + K + B) % 5]
    lr.check(c.fused(x, kind, b, r), lr.fused(c.refs[0], x, kind, b, r), f"{kind} bias residual")
    lr.check(c.fused(x, "silu", None, None), lr.fused(c.refs[0], x, "silu"), "silu")
    lr.check(c.fused(x, "none", None, r), lr.fused(c.refs[0], x, "none", None, r), "residual")


@pytest.mark.parametrize("n", range(1, 17))
@pytest.mark.parametrize("K,B", [(1, 16), (2, 8)])
def test_gemv_fused_every_batch(K, B, n):
    c = Case(300, 1032, K, B, 77)
    x, b, r = acts(1032, n, (1, n)), acts(300, 1, 2).ravel(), acts(300, n, (3, n))
    lr.check(c.fused(x, "gelu", b, r), lr.fused(c.refs[0], x, "gelu", b, r), "gelu bias residual")


@pytest.mark.parametrize("K,B", SCHEMES)
@pytest.mark.parametrize("out,inp,T", [(8, 8, 1), (20, 520, 7), (136, 264, 8), (300, 1032, 77), (136, 2056, 520),
                                       (520, 264, 333), (1000, 1032, 1032)])
def test_gemm_fused(K, B, out, inp, T):
    c = Case(out, inp, K, B, out + T)
    x, b, r = acts(inp, T, (1, T)), acts(out, 1, 2).ravel(), acts(out, T, (3, T))
    kind = ACTS[(T + K + B) % 5]
    lr.check(c.fused(x, kind, b, r, gemm=True), lr.fused(c.refs[0], x, kind, b, r), f"{kind} bias residual")
    lr.check(c.fused(x, "silu", gemm=True), lr.fused(c.refs[0], x, "silu"), "silu")


@pytest.mark.parametrize("n", [5, 40, 45])
def test_fused_without_epilogue_is_the_plain_product(n):
    """ep = NULL (or all empty): the product itself, within its error."""
    c = Case(136, 264, 2, 8, 5)
    x = acts(264, n, 6)
    lr.check(c.fused(x), lr.fused(c.refs[0], x, "none"), "no epilogue")


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8), (8, 8)])
@pytest.mark.parametrize("n", [1, 4, 72, 75])
def test_residual_in_place_and_unit_scales(K, B, n):
    c = Case(200, 520, K, B, 8, scaled=False)
    x, r = acts(520, n, 1), acts(200, n, 2)
    full, y = guarded(200 * n)
    y.copy_(torch.from_numpy(r.view(np.int16).ravel()).cuda())
    gemm = n > 16
    ws = workspace((aq.aq_gemm_fused_workspace_bytes if gemm else aq.aq_gemv_workspace_bytes)(c.desc, n))
    (aq.aq_gemm_fused if gemm else aq.aq_gemv_fused)(*c.w(), fenced(x), n, y, ws, residual=y)
    torch.cuda.synchronize()
    assert guards_intact(full)
    lr.check(half(y, 200, n), lr.fused(c.refs[0], x, "none", None, r), "in place")


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8), (8, 8)])
@pytest.mark.parametrize("n", [1, 2, 8, 40])
def test_scales_and_bias_at_any_even_address(K, B, n):
    c = Case(520, 1032, K, B, 14, layers=2)
    x, b, gy = acts(1032, n, 1), acts(520, 1, 2).ravel(), acts(520, n, 3)

    def odd(t):
        full = torch.zeros(t.numel() + 8, dtype=torch.int16, device="cuda")
        full[3:3 + t.numel()] = t.view(torch.int16)
        return full[3:3 + t.numel()]

    c.scales = [odd(s) for s in c.scales]
    c.weights = [aq.Weights.make(d.packed, k, s) for d, k, s in zip(c.dls, c.books, c.scales)]
    full, y = guarded(520 * n)
    ws = workspace(max(aq.aq_gemm_fused_workspace_bytes(c.desc, n), aq.aq_gemv_workspace_bytes(c.desc, min(n, 16))))
    (aq.aq_gemm_fused if n > 16 else aq.aq_gemv_fused)(*c.w(), fenced(x), n, y, ws, activation=4,
                                                       bias=odd(fenced(b)))
    torch.cuda.synchronize()
    assert guards_intact(full)
    lr.check(half(y, 520, n), lr.fused(c.refs[0], x, "silu", b), "fused")
    lr.check(c.glu(x, "silu"), lr.glu(*c.refs, x, "silu"), "glu")
    lr.check(c.input_grad(gy), c.refs[0].back(gy), "input grad")


@pytest.mark.parametrize("K,B", SCHEMES)
@pytest.mark.parametrize("out,inp", SHAPES + [(1000, 2056)])
@pytest.mark.parametrize("n", [1, 2, 3, 8, 16])
def test_glu_gemv(K, B, out, inp, n):
    c = Case(out, inp, K, B, 13 * out + n, layers=2)
    x = acts(inp, n, (1, n))
    kind = ACTS[(n + K + B) % 5]
    lr.check(c.glu(x, kind), lr.glu(*c.refs, x, kind), kind)
    lr.check(c.glu(x, "silu"), lr.glu(*c.refs, x, "silu"), "silu")


@pytest.mark.parametrize("n", range(1, 17))
@pytest.mark.parametrize("K,B", [(1, 16), (2, 8)])
def test_glu_gemv_every_batch(K, B, n):
    c = Case(300, 1032, K, B, 78, layers=2)
    x = acts(1032, n, (1, n))
    lr.check(c.glu(x, "silu"), lr.glu(*c.refs, x, "silu"), "silu")


@pytest.mark.parametrize("K,B", SCHEMES)
@pytest.mark.parametrize("out,inp,T", [(8, 8, 1), (20, 520, 7), (72, 264, 8), (300, 1032, 77), (136, 2056, 520),
                                       (520, 264, 333), (1000, 1032, 1032)])
def test_glu_gemm(K, B, out, inp, T):
    c = Case(out, inp, K, B, out + T, layers=2)
    x = acts(inp, T, (1, T))
    kind = ACTS[(T + K + B) % 5]
    lr.check(c.glu(x, kind, gemm=True), lr.glu(*c.refs, x, kind), kind)
    lr.check(c.glu(x, "silu", gemm=True), lr.glu(*c.refs, x, "silu"), "silu")


@pytest.mark.parametrize("K,B", SCHEMES)
@pytest.mark.parametrize("out,inp,T", [(8, 8, 1), (20, 520, 7), (520, 136, 8), (300, 1032, 77), (2056, 136, 520),
                                       (264, 520, 333), (1032, 1000, 1032)])
def test_input_grad(K, B, out, inp, T):
    c = Case(out, inp, K, B, out + T)
    gy = acts(out, T, (4, T))
    lr.check(c.input_grad(gy), c.refs[0].back(gy), "input grad")


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8)])
@pytest.mark.parametrize("scale", [2.0 ** -12, 3e-3, 100.0, 20000.0])
def test_input_grad_scales_of_any_magnitude(K, B, scale):
    """Small scales lose no bits and large ones overflow no weight: 2^E
    follows the largest; gy is sized to keep gx finite."""
    c = Case(264, 136, K, B, 21, scale=scale)
    gy = acts(264, 40, 5, sigma=min(64.0, 0.1 / scale))
    lr.check(c.input_grad(gy), c.refs[0].back(gy), f"scales around {scale}")


def test_input_grad_zero_scales_and_one_row_dominating():
    c = Case(264, 136, 2, 8, 22)
    for spread in ("zero", "one"):
        s = np.zeros(264, np.float16)
        if spread == "one":
            s[:] = np.float16(2e-4)
            s[17] = np.float16(512.0)
        c.scales[0] = fenced(s)
        c.refs[0].s = s.astype(np.float64)
        gy = acts(264, 24, 6, sigma=0.05)
        lr.check(c.input_grad(gy), c.refs[0].back(gy), spread)


@pytest.mark.parametrize("K,B", SCHEMES)
@pytest.mark.parametrize("out,inp,T", [(8, 8, 1), (20, 520, 7), (136, 264, 40), (300, 1032, 77), (136, 2056, 520),
                                       (520, 264, 333)])
def test_fused_grad(K, B, out, inp, T):
    c = Case(out, inp, K, B, out + T)
    x, b, gy = acts(inp, T, (1, T)), acts(out, 1, 2).ravel(), acts(out, T, (3, T), 0.1)
    for kind in (ACTS[(T + K + B) % 5], "gelu_tanh"):
        gz, gb, gx = c.fused_grad(x, gy, kind, b)
        want_z, want_b = lr.fused_grad(c.refs[0], x, gy, kind, b)
        lr.check(gz, want_z, f"{kind} grad_z")
        lr.check(gb, want_b, f"{kind} grad_bias")
        lr.check(gx, c.refs[0].back(gz), f"{kind} grad_x")


def test_fused_grad_optional_outputs():
    c = Case(136, 264, 1, 16, 9)
    x, gy = acts(264, 48, 1), acts(136, 48, 2, 0.1)
    gz, gb, gx = c.fused_grad(x, gy, "silu", want_bias=False)
    assert (gb == 7.25).all()
    lr.check(gx, c.refs[0].back(gz), "grad_x alone")
    gz2, gb, gx = c.fused_grad(x, gy, "silu", want_x=False)
    assert np.array_equal(gz.view(np.uint16), gz2.view(np.uint16))
    assert (gx.view(np.uint16) == 0x7E5A).all()  # untouched
    lr.check(gb, lr.fused_grad(c.refs[0], x, gy, "silu")[1], "grad_bias alone")


@pytest.mark.parametrize("K,B", SCHEMES)
@pytest.mark.parametrize("out,inp,T", [(8, 8, 1), (20, 520, 7), (136, 264, 40), (300, 1032, 77), (136, 2056, 520),
                                       (520, 264, 333)])
def test_glu_grad(K, B, out, inp, T):
    c = Case(out, inp, K, B, out + T, layers=2)
    x, gy = acts(inp, T, (1, T)), acts(out, T, (3, T), 0.1)
    for kind in (ACTS[(T + K + B) % 5], "silu"):
        gg, gu, gx = c.glu_grad(x, gy, kind)
        want_g, want_u = lr.glu_grad(*c.refs, x, gy, kind)
        lr.check(gg, want_g, f"{kind} grad_gate")
        lr.check(gu, want_u, f"{kind} grad_up")
        lr.check(gx, c.refs[0].back(gg, [(c.refs[1], gu)]), f"{kind} grad_x")


def test_glu_grad_without_grad_x():
    c = Case(136, 264, 2, 8, 9, layers=2)
    x, gy = acts(264, 45, 1), acts(136, 45, 2, 0.1)
    full = c.glu_grad(x, gy, "silu")
    part = c.glu_grad(x, gy, "silu", want_x=False)
    assert np.array_equal(full[0].view(np.uint16), part[0].view(np.uint16))
    assert np.array_equal(full[1].view(np.uint16), part[1].view(np.uint16))
    assert (part[2].view(np.uint16) == 0x7E5A).all()


@pytest.mark.parametrize("n", [1, 6, 40])
@pytest.mark.parametrize("K,B", [(1, 16), (2, 8)])
def test_infinities_and_nan_stay_in_their_columns(K, B, n):
    """A NaN or infinity in one token's activations reaches that token's
    results only."""
    c = Case(72, 264, K, B, 31, layers=2)
    x = acts(264, n, 1)
    clean = (c.fused(x, "silu"), c.glu(x, "silu"))
    bad = x.copy()
    bad[5, n - 1] = np.float16(np.nan)
    bad[70, n - 1] = np.float16(np.inf)
    for got, want in zip((c.fused(bad, "silu"), c.glu(bad, "silu")), clean):
        assert np.isnan(got[:, n - 1].astype(np.float32)).all()
        assert np.array_equal(got[:, :n - 1].view(np.uint16), want[:, :n - 1].view(np.uint16))


def test_relu_keeps_nan_and_overflow_becomes_infinity():
    c = Case(72, 264, 1, 16, 32)
    x = acts(264, 24, 1)
    x[:, 3] = np.float16(np.nan)
    assert np.isnan(c.fused(x, "relu")[:, 3].astype(np.float32)).all()
    x = np.full((264, 24), 60000, np.float16)
    z, ez = c.refs[0].z(x)
    got = c.fused(x, "none").astype(np.float64)
    sure = np.abs(z) - ez > 65520
    assert sure.any() and np.array_equal(got[sure], np.sign(z[sure]) * np.inf)


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8)])
def test_gradient_against_differences_of_the_forward(K, B):
    """sum(gy y) along the gradient's signs in x, from aq_glu_gemm's own
    outputs: each y carries its error, the central difference the third
    derivative's share, taken from the 64-bit block as `curve`."""
    c = Case(72, 264, K, B, 41, layers=2, sigma=0.03)
    T = 24
    x = acts(264, T, 1)
    gy = acts(72, T, 3)
    g = gy.astype(np.float64)
    (gg, _), (gu, _) = lr.glu_grad(*c.refs, x, gy, "silu")
    want, _ = c.refs[0].back(gg, [(c.refs[1], gu)])
    step = (np.sign(want) * 2.0 ** -6).astype(np.float16)
    lo = (x - step).astype(np.float16)
    hi = (x + step).astype(np.float16)
    v = hi.astype(np.float64) - lo.astype(np.float64)  # the difference taken, exactly
    _, _, gx = c.glu_grad(x, gy, "silu")
    yh, yl = c.glu(hi, "silu", gemm=True).astype(np.float64), c.glu(lo, "silu", gemm=True).astype(np.float64)
    rh, rl = lr.glu(*c.refs, hi, "silu"), lr.glu(*c.refs, lo, "silu")
    curve = abs((g * (rh[0] - rl[0])).sum() - (want * v).sum())
    got_gg, got_gu, _ = c.glu_grad(x, gy, "silu")
    egx = c.refs[0].back(got_gg, [(c.refs[1], got_gu)])
    lim = curve + (np.abs(g) * (rh[1] + rl[1])).sum() + (np.abs(v) * (egx[1] + np.abs(egx[0] - want))).sum()
    diff = (g * (yh - yl)).sum()
    assert abs(diff - (gx.astype(np.float64) * v).sum()) <= lim
    assert lim < 0.05 * abs(diff)  # and the limit says something


def _block(K, B, T, seed, hidden=264, ffn=520):
    """A feed-forward block: gated block, down projection with residual."""
    ff = Case(ffn, hidden, K, B, seed, layers=2)
    down = Case(hidden, ffn, K, B, seed + 1)
    return ff, down


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8)])
@pytest.mark.parametrize("T", [1, 5, 40, 77, 136])
def test_feed_forward_block_forward_and_backward(K, B, T):
    """The operators as a block uses them, back to back on one stream with one
    workspace: h = glu(x), y = x + down(h); then gh = down^T gy, the gated
    block's gradients, and its parameter gradients.  Each step is held to its
    own error on the GPU values it was given."""
    ff, down = _block(K, B, T, 50 + T)
    x, gy = acts(264, T, 1), acts(264, T, 2, 0.1)
    gemm = T > 16
    sizes = [aq.aq_glu_gemm_workspace_bytes(ff.desc, T), aq.aq_gemm_fused_workspace_bytes(down.desc, T),
             aq.aq_glu_grad_workspace_bytes(ff.desc, T), aq.aq_input_grad_workspace_bytes(down.desc, T)]
    if not gemm:
        sizes += [aq.aq_glu_gemv_workspace_bytes(ff.desc, T), aq.aq_gemv_workspace_bytes(down.desc, T)]
    ws = workspace(max(sizes))
    stream = torch.cuda.Stream()
    xd, gyd = fenced(x), fenced(gy)
    h, y, gh, gg, gu, gx = (torch.empty(r * T, dtype=torch.int16, device="cuda")
                            for r in (520, 264, 520, 520, 520, 264))
    torch.cuda.synchronize()
    for _ in range(2):  # the second pass on the workspace the first one left
        (aq.aq_glu_gemm if gemm else aq.aq_glu_gemv)(ff.desc, *ff.weights, xd, T, 4, h, ws, stream=stream)
        (aq.aq_gemm_fused if gemm else aq.aq_gemv_fused)(*down.w(), h, T, y, ws, stream=stream, residual=xd)
        aq.aq_input_grad(*down.w(), gyd, T, gh, ws, stream=stream)
        aq.aq_glu_grad(ff.desc, *ff.weights, xd, gh, T, 4, gg, gu, gx, ws, stream=stream)
    stream.synchronize()
    assert aq.aq_workspace_status(ws, stream=stream) == 0
    H = half(h, 520, T)
    lr.check(H, lr.glu(*ff.refs, x, "silu"), "h")
    lr.check(half(y, 264, T), lr.fused(down.refs[0], H, "none", None, x), "y")
    GH = half(gh, 520, T)
    lr.check(GH, down.refs[0].back(gy), "gh")
    wg, wu = lr.glu_grad(*ff.refs, x, GH, "silu")
    GG, GU = half(gg, 520, T), half(gu, 520, T)
    lr.check(GG, wg, "grad_gate")
    lr.check(GU, wu, "grad_up")
    lr.check(half(gx, 264, T), ff.refs[0].back(GG, [(ff.refs[1], GU)]), "grad_x")


@pytest.mark.parametrize("T", [3, 48, 45])
def test_same_bits_every_time_and_in_a_graph(T):
    """Deterministic, captured and replayed on another stream, with inputs
    changed between replays; two graphs hold a workspace each."""
    c = Case(300, 1032, 2, 8, 60, layers=2)
    x, gy = acts(1032, T, 1), acts(300, T, 2, 0.1)
    first = c.glu_grad(x, gy, "silu")
    again = c.glu_grad(x, gy, "silu")
    assert all(np.array_equal(a.view(np.uint16), b.view(np.uint16)) for a, b in zip(first, again))
    xd, gyd = fenced(np.zeros_like(x)), fenced(gy)
    graphs = []
    for _ in range(2):
        ws = workspace(aq.aq_glu_grad_workspace_bytes(c.desc, T))
        outs = [torch.zeros(r * T, dtype=torch.int16, device="cuda") for r in (300, 300, 1032)]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            aq.aq_glu_grad(c.desc, *c.weights, xd, gyd, T, 4, *outs, ws)
        graphs.append((g, outs, ws))
    xd.copy_(torch.from_numpy(x.view(np.int16).ravel()).cuda())
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in graphs]
    for (g, _, _), s in zip(graphs, side):
        with torch.cuda.stream(s):
            g.replay()
            g.replay()
    torch.cuda.synchronize()
    for _, outs, _ in graphs:
        for got, want in zip(outs, first):
            assert np.array_equal(to_f16(got).view(np.uint16), want.view(np.uint16).ravel())


def test_two_streams_at_once_with_a_workspace_each():
    c = Case(1000, 1032, 1, 16, 61, layers=2)
    d = Case(1000, 1032, 2, 8, 62, layers=2)
    x = acts(1032, 16, 1)
    want = [k.glu(x, "silu") for k in (c, d)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    xd = fenced(x)
    outs = [torch.empty(1000 * 16, dtype=torch.int16, device="cuda") for _ in range(2)]
    wss = [workspace(aq.aq_glu_gemv_workspace_bytes(k.desc, 16)) for k in (c, d)]
    torch.cuda.synchronize()
    for _ in range(8):
        for k, s, o, ws in zip((c, d), streams, outs, wss):
            aq.aq_glu_gemv(k.desc, *k.weights, xd, 16, 4, o, ws, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert np.array_equal(to_f16(o).view(np.uint16), w.view(np.uint16).ravel())


@pytest.mark.parametrize("K,B,n", [(1, 16, 1), (2, 8, 1), (1, 16, 16), (2, 8, 8)])
def test_llama_rows_decode(K, B, n):
    """4096 features and 1024 rows: many splits per row range."""
    c = Case(1024, 4096, K, B, 70, layers=2, sigma=0.02)
    x, r = acts(4096, n, 1), acts(1024, n, 2)
    lr.check(c.glu(x, "silu"), lr.glu(*c.refs, x, "silu"), "glu")
    lr.check(c.fused(x, "none", None, r), lr.fused(c.refs[0], x, "none", None, r), "residual")


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8)])
@pytest.mark.parametrize("T", [512, 1001])
def test_llama_rows_prompt_and_backward(K, B, T):
    c = Case(1536, 2048, K, B, 71, layers=2, sigma=0.02)
    x, gy = acts(2048, T, 1), acts(1536, T, 2, 0.1)
    lr.check(c.glu(x, "silu"), lr.glu(*c.refs, x, "silu"), "glu")
    gg, gu, gx = c.glu_grad(x, gy, "silu")
    wg, wu = lr.glu_grad(*c.refs, x, gy, "silu")
    lr.check(gg, wg, "grad_gate")
    lr.check(gu, wu, "grad_up")
    lr.check(gx, c.refs[0].back(gg, [(c.refs[1], gu)]), "grad_x")


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8)])
def test_prompt_of_several_waves_of_tiles(K, B):
    """More tiles of 128 rows x 512 tokens than SMs, the last wave part full
    (11008 rows, 1024 tokens: 172 tiles): sampled rows."""
    c = Case(11008, 264, K, B, 72, layers=2, sigma=0.05)
    T = 1024
    x, b, r, gy = acts(264, T, 1), acts(11008, 1, 2).ravel(), acts(11008, T, 3), acts(11008, T, 4, 0.1)
    rows = np.r_[0:64, 5000:5064, 10880:11008]
    sub = []
    for R in c.refs:
        S = lr.Ref.__new__(lr.Ref)
        S.spec, S.W, S.C, S.s = R.spec, R.W[rows], R.C[rows], R.s[rows]
        sub.append(S)
    lr.check(c.fused(x, "silu", b, r)[rows], lr.fused(sub[0], x, "silu", b[rows], r[rows]), "fused")
    lr.check(c.glu(x, "silu")[rows], lr.glu(*sub, x, "silu"), "glu")
    gz, gb, _ = c.fused_grad(x, gy, "silu", b, want_x=False)
    want_z, want_b = lr.fused_grad(sub[0], x, gy[rows], "silu", b[rows])
    lr.check(gz[rows], want_z, "grad_z")
    lr.check(gb[rows], want_b, "grad_bias")


def _rows_of(ref, rows):
    R = lr.Ref.__new__(lr.Ref)
    R.spec, R.W, R.C, R.s = ref.spec, ref.W[rows], ref.C[rows], ref.s[rows]
    return R


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8), (8, 8)])
@pytest.mark.parametrize("out,inp,T", [(2312, 264, 2048), (2048, 1032, 2048), (11008, 1032, 1024), (2312, 520, 1999)])
def test_pairs_of_row_tiles(K, B, out, inp, T):
    """512-token tiles as CTA pairs: an odd number of row tiles (the last
    pair's second tile empty), features split in two, the last wave's tiles
    split over the features, ragged tokens; sampled rows."""
    if K == 8 and out > 4096:
        pytest.skip("one scheme less at the largest shape")
    c = Case(out, inp, K, B, 80, layers=2)
    x, r, gy = acts(inp, T, 1), acts(out, T, 3), acts(out, T, 4, 0.1)
    rows = np.unique(np.r_[0:40, out // 2:out // 2 + 40, out - 72:out])
    sub = [_rows_of(R, rows) for R in c.refs]
    lr.check(c.fused(x, "none", None, r)[rows], lr.fused(sub[0], x, "none", None, r[rows]), "fused")
    lr.check(c.glu(x, "silu")[rows], lr.glu(*sub, x, "silu"), "glu")
    gg, gu, gx = c.glu_grad(x, gy, "silu")
    wg, wu = lr.glu_grad(*sub, x, gy[rows], "silu")
    lr.check(gg[rows], wg, "grad_gate")
    lr.check(gu[rows], wu, "grad_up")
    toks = np.unique(np.r_[0:24, T // 2:T // 2 + 24, T - 24:T])
    lr.check(gx[:, toks], c.refs[0].back(gg[:, toks], [(c.refs[1], gu[:, toks])]), "grad_x")


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8)])
@pytest.mark.parametrize("inp,T", [(2312, 2048), (4104, 1024)])
def test_input_grad_pairs(K, B, inp, T):
    c = Case(1032, inp, K, B, 81)
    gy = acts(1032, T, 4, 0.1)
    toks = np.unique(np.r_[0:32, T // 2:T // 2 + 32, T - 32:T])
    lr.check(c.input_grad(gy)[:, toks], c.refs[0].back(gy[:, toks]), "input grad")


@pytest.mark.parametrize("K,B", SCHEMES)
@pytest.mark.parametrize("n", [1, 4, 40, 45, 520])
def test_padding_codes_select_nothing(K, B, n):
    """Rows and groups that only the padded storage holds have code 0: a
    codeword 0 of infinities, which no real code selects, reaches no result."""
    c = Case(20, 520, K, B, 90, layers=2)
    for i, L in enumerate(c.layers):
        L.codes[L.codes == 0] = 1
        L.codebooks.reshape(K, -1, 8)[:, 0] = np.inf
    c2 = Case.__new__(Case)
    c2.out, c2.inp, c2.layers = 20, 520, c.layers
    finite = []
    for L in c.layers:
        keep = L.codebooks.copy()
        L.codebooks.reshape(K, -1, 8)[:, 0] = 0
        finite.append(lr.Ref(L))
        L.codebooks[...] = keep
    c2.refs = finite
    c2.dls = [DevLayer(L) for L in c.layers]
    c2.desc = c2.dls[0].desc
    c2.books = [fenced(L.codebooks.view(np.float16)) for L in c.layers]
    c2.scales = [fenced(L.scales.view(np.float16)) for L in c.layers]
    c2.weights = [aq.Weights.make(d.packed, b, s) for d, b, s in zip(c2.dls, c2.books, c2.scales)]
    x, gy = acts(520, n, 1), acts(20, n, 2, 0.1)
    lr.check(c2.fused(x, "silu"), lr.fused(finite[0], x, "silu"), "fused")
    lr.check(c2.glu(x, "silu"), lr.glu(*finite, x, "silu"), "glu")
    lr.check(c2.input_grad(gy), finite[0].back(gy), "input grad")
    gg, gu, gx = c2.glu_grad(x, gy, "silu")
    lr.check(gx, finite[0].back(gg, [(finite[1], gu)]), "grad_x")


@pytest.mark.parametrize("n", [1, 8, 40])
def test_gate_and_up_may_be_the_same_layer(n):
    c = Case(136, 264, 2, 8, 91)
    x, gy = acts(264, n, 1), acts(136, n, 2, 0.1)
    c.weights, c.refs = c.weights * 2, c.refs * 2
    lr.check(c.glu(x, "silu"), lr.glu(*c.refs, x, "silu"), "glu")
    gg, gu, gx = c.glu_grad(x, gy, "silu")
    lr.check(gx, c.refs[0].back(gg, [(c.refs[1], gu)]), "grad_x")


@pytest.mark.parametrize("T", [16, 40, 45])
def test_one_layer_with_scales_and_one_without(T):
    c = Case(136, 264, 1, 16, 92, layers=2)
    d = Case(136, 264, 2, 8, 92, layers=2)
    for k in (c, d):
        k.weights[1] = aq.Weights.make(k.dls[1].packed, k.books[1], None)
        k.refs[1].s = np.ones(136)
        x, gy = acts(264, T, 1), acts(136, T, 2, 0.1)
        lr.check(k.glu(x, "silu", gemm=True), lr.glu(*k.refs, x, "silu"), "glu")
        gg, gu, gx = k.glu_grad(x, gy, "silu")
        lr.check(gx, k.refs[0].back(gg, [(k.refs[1], gu)]), "grad_x")


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8)])
def test_input_grad_of_several_waves_of_tiles(K, B):
    """11008 features, 1024 tokens: 172 tiles, the last 24 split over the rows."""
    c = Case(1544, 11008, K, B, 73, sigma=0.05)
    gy = acts(1544, 1024, 4, 0.1)
    lr.check(c.input_grad(gy), c.refs[0].back(gy), "input grad")
