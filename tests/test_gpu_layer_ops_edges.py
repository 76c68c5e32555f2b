"""Layer operators on the GPU at their edges: a workspace shared by any
sequence of calls, addresses of any alignment that the header allows, values
near the ends of binary16's range."""
import numpy as np
import pytest
import torch

import additive_quantized_matmul_b200 as aq
import layer_ref as lr
from aqtest import CANARY, guarded, guards_intact, to_f16, workspace
from test_gpu_layer_ops import Case, acts, fenced, half

pytestmark = pytest.mark.gpu

HEAD = slice(0, 16 + 4 * 1024)  # status word, largest scaled gradient, arrival counters


class Block:
    """Two layers of one shape with random codes, and a call of every entry
    point that takes a workspace: calls() gives (name, size, run(ws) -> outputs
    filled with a canary before the call)."""

    def __init__(self, out, inp, K, B, seed):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.out, self.inp = out, inp
        self.d = aq.LayerDesc.make(out, inp, K, B)
        self.w = []
        for _ in range(2):
            codes = torch.randint(0, 1 << B, (out, inp // 8, K), device="cuda", generator=gen, dtype=torch.int32)
            codes = codes.to(torch.uint8) if B == 8 else codes.to(torch.int16)
            packed = torch.empty(aq.aq_packed_codes_bytes(self.d), dtype=torch.uint8, device="cuda")
            aq.aq_pack_codes(self.d, codes, packed)
            books = (torch.randn((K, 1 << B, 8), device="cuda", generator=gen) * 0.02).half()
            scales = (torch.rand(out, device="cuda", generator=gen) + 0.5).half()
            self.w.append((packed, books, scales))
        self.weights = [aq.Weights.make(*w) for w in self.w]
        self.gen = gen

    def halves(self, rows, n, sigma=1.0):
        return (torch.randn((rows, n), device="cuda", generator=self.gen) * sigma).half()

    def calls(self, T, batch):
        d, w, (gate, up), out, inp = self.d, self.w[0], self.weights, self.out, self.inp
        x, gy, xb, res = self.halves(inp, T), self.halves(out, T, 0.1), self.halves(inp, batch), self.halves(out, T)

        def fresh(*shapes):
            return [torch.full(s, CANARY, dtype=torch.int16, device="cuda").view(torch.float16) for s in shapes]

        def run(fn, shapes, call):
            def go(ws):
                outs = fresh(*shapes)
                call(outs, ws)
                return outs
            return go

        def entry(name, size, shapes, call):
            return name, size, run(name, shapes, call)

        bias = torch.empty(out, dtype=torch.float32, device="cuda")

        def fused_grad(o, ws):
            bias.fill_(7.25)
            aq.aq_gemm_fused_grad(d, *w, x, gy, T, o[0], bias, o[1], ws, activation=4)
            o.append(bias.clone())

        return [
            entry("input_grad", aq.aq_input_grad_workspace_bytes(d, T), [(inp, T)],
                  lambda o, ws: aq.aq_input_grad(d, *w, gy, T, o[0], ws)),
            entry("gemm", aq.aq_gemm_workspace_bytes(d, T), [(out, T)],
                  lambda o, ws: aq.aq_gemm(d, *w, x, T, o[0], ws)),
            entry("glu_grad", aq.aq_glu_grad_workspace_bytes(d, T), [(out, T), (out, T), (inp, T)],
                  lambda o, ws: aq.aq_glu_grad(d, gate, up, x, gy, T, 4, *o, ws)),
            entry("gemv", aq.aq_gemv_workspace_bytes(d, batch), [(out, batch)],
                  lambda o, ws: aq.aq_gemv(d, *w, xb, batch, o[0], ws)),
            entry("fused_grad", aq.aq_gemm_fused_grad_workspace_bytes(d, T), [(out, T), (inp, T)], fused_grad),
            entry("gemm_fused", aq.aq_gemm_fused_workspace_bytes(d, T), [(out, T)],
                  lambda o, ws: aq.aq_gemm_fused(d, *w, x, T, o[0], ws, residual=res)),
            entry("gemv_fused", aq.aq_gemv_workspace_bytes(d, batch), [(out, batch)],
                  lambda o, ws: aq.aq_gemv_fused(d, *w, xb, batch, o[0], ws, activation=4)),
            entry("glu_gemm", aq.aq_glu_gemm_workspace_bytes(d, T), [(out, T)],
                  lambda o, ws: aq.aq_glu_gemm(d, gate, up, x, T, 4, o[0], ws)),
            entry("glu_gemv", aq.aq_glu_gemv_workspace_bytes(d, batch), [(out, batch)],
                  lambda o, ws: aq.aq_glu_gemv(d, gate, up, xb, batch, 4, o[0], ws)),
        ]


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8), (8, 8)])
@pytest.mark.parametrize("out,inp,T,batch", [(11008, 4096, 2048, 1), (4096, 11008, 2047, 1), (4096, 4096, 45, 4),
                                             (11008, 4096, 1, 16), (1000, 1032, 333, 2)])
def test_one_workspace_for_any_sequence_of_calls(K, B, out, inp, T, batch):
    """Every call, on a workspace that every other call used before it, gives
    the bits it gives on a workspace of its own, and leaves status word and
    counters at zero."""
    calls = Block(out, inp, K, B, 5).calls(T, batch)
    alone = {}
    for name, size, go in calls:
        ws = workspace(size)
        alone[name] = [o.view(torch.int16) if o.dtype == torch.float16 else o for o in go(ws)]
        torch.cuda.synchronize()
        assert aq.aq_workspace_status(ws) == 0
    shared = workspace(max(size for _, size, _ in calls))
    order = [*calls, *reversed(calls)]
    for name, _, go in order:
        got = go(shared)
        torch.cuda.synchronize()
        assert int(shared[HEAD].max()) == 0, f"{name} left something in the head"
        for i, (a, b) in enumerate(zip(got, alone[name])):
            a = a.view(torch.int16) if a.dtype == torch.float16 else a
            assert torch.equal(a, b), f"{name} output {i}"
    assert aq.aq_workspace_status(shared) == 0


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8)])
@pytest.mark.parametrize("T", [1, 5, 40, 77])
def test_training_step_twice_on_one_workspace(K, B, T):
    """A block's forward and backward, twice on one workspace, the outputs
    refilled with canaries between: each step of the second pass is held to its
    own error on the values it was given."""
    ff = Case(520, 264, K, B, 60 + T, layers=2)
    down = Case(264, 520, K, B, 61 + T)
    x, gy = acts(264, T, 1), acts(264, T, 2, 0.1)
    sizes = [aq.aq_glu_gemm_workspace_bytes(ff.desc, T), aq.aq_gemm_fused_workspace_bytes(down.desc, T),
             aq.aq_glu_grad_workspace_bytes(ff.desc, T), aq.aq_input_grad_workspace_bytes(down.desc, T),
             aq.aq_gemm_workspace_bytes(down.desc, T)]
    ws = workspace(max(sizes))
    xd, gyd = fenced(x), fenced(gy)
    for _ in range(2):
        (h, y, z, gh, gg, gu, gx) = (guarded(r * T) for r in (520, 264, 264, 520, 520, 520, 264))
        aq.aq_glu_gemm(ff.desc, *ff.weights, xd, T, 4, h[1], ws)
        aq.aq_gemm_fused(*down.w(), h[1], T, y[1], ws, residual=xd)
        aq.aq_input_grad(*down.w(), gyd, T, gh[1], ws)
        aq.aq_glu_grad(ff.desc, *ff.weights, xd, gh[1], T, 4, gg[1], gu[1], gx[1], ws)
        aq.aq_gemm(*down.w(), h[1], T, z[1], ws)
    torch.cuda.synchronize()
    assert aq.aq_workspace_status(ws) == 0 and int(ws[HEAD].max()) == 0
    assert all(guards_intact(b[0]) for b in (h, y, z, gh, gg, gu, gx))
    H, GH, GG, GU = (half(b[1], 520, T) for b in (h, gh, gg, gu))
    lr.check(H, lr.glu(*ff.refs, x, "silu"), "h")
    lr.check(half(y[1], 264, T), lr.fused(down.refs[0], H, "none", None, x), "y")
    lr.check(half(z[1], 264, T), lr.fused(down.refs[0], H, "none"), "plain product")
    lr.check(GH, down.refs[0].back(gy), "gh")
    wg, wu = lr.glu_grad(*ff.refs, x, GH, "silu")
    lr.check(GG, wg, "grad_gate")
    lr.check(GU, wu, "grad_up")
    lr.check(half(gx[1], 264, T), ff.refs[0].back(GG, [(ff.refs[1], GU)]), "grad_x")


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8), (1, 8), (2, 16), (8, 8)])
@pytest.mark.parametrize("inp", [264, 1032, 2056, 4096, 4616, 8200])
@pytest.mark.parametrize("offset", [1, 2, 3])
def test_plain_products_take_scales_at_any_even_address(K, B, inp, offset):
    """Scales that start 2, 4 or 6 bytes past an 8-byte boundary: the bits of
    aligned ones, whether the table kernel's splits (one per 512 features of 2x8
    layers, 1024 of 1x8) are summed from L2 (2 to 8) or staged."""
    b = Block(300, inp, K, B, 7)
    packed, books, scales = b.w[0]
    shifted = torch.full((300 + 8,), float("nan"), dtype=torch.float16, device="cuda")[offset:offset + 300]
    shifted.copy_(scales)
    assert shifted.data_ptr() % 8 == 2 * offset
    for n in (1, 2, 8, 40):
        x = b.halves(inp, n)
        fns = [(aq.aq_gemm, aq.aq_gemm_workspace_bytes)]
        if n <= 16:
            fns += [(aq.aq_gemv, aq.aq_gemv_workspace_bytes), (aq.aq_gemv_ordered, aq.aq_gemv_workspace_bytes),
                    (aq.aq_gemv_noalloc, None)]
        for fn, size in fns:
            got = []
            for s in (scales, shifted):
                full, y = guarded(300 * n)
                ws = [] if size is None else [workspace(size(b.d, n))]
                fn(b.d, packed, books, s, x, n, y, *ws)
                torch.cuda.synchronize()
                assert guards_intact(full)
                got.append(y.clone())
            assert torch.equal(*got), (fn.__name__, n)


def _same_kind(got, want):
    """NaN, +inf, -inf and finite values in the same places."""
    got = got.astype(np.float64)
    kinds = [(np.isnan(a), np.isposinf(a), np.isneginf(a)) for a in (got, want)]
    return all(np.array_equal(a, b) for a, b in zip(*kinds))


@pytest.mark.parametrize("n", [2, 6, 40])
@pytest.mark.parametrize("K,B", [(1, 16), (2, 8), (8, 8)])
@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_an_infinity_becomes_what_the_formula_makes_of_it(K, B, n, kind):
    """One token with an infinity, another with a NaN: the infinite token's
    rows are +inf, -inf or NaN as the formula has them in IEEE arithmetic (z is
    infinite of the sign of the weight that meets the infinity), the others
    keep their bits."""
    c = Case(72, 264, K, B, 31, layers=2)
    x = acts(264, n, 1)
    clean = (c.fused(x, kind), c.glu(x, kind))
    bad = x.copy()
    bad[70, 0] = np.float16(np.inf)
    bad[5, n - 1] = np.float16(np.nan)
    got = (c.fused(bad, kind), c.glu(bad, kind))
    with np.errstate(invalid="ignore", over="ignore"):
        z = [r.s * r.W[:, 70] * np.inf for r in c.refs]
        a = lr.act(kind, z[0])[0]
        want = (a, a * z[1])
    for g, w, k in zip(got, want, clean):
        assert _same_kind(g[:, 0], w)
        if kind != "relu":
            assert not np.isfinite(g[:, 0].astype(np.float64)).any()
        assert np.isnan(g[:, n - 1].astype(np.float64)).all()
        assert np.array_equal(g[:, 1:n - 1].view(np.uint16), k[:, 1:n - 1].view(np.uint16))


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8), (1, 8)])
@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_an_infinity_in_the_only_token(K, B, kind):
    c = Case(72, 264, K, B, 31, layers=2)
    x = acts(264, 1, 1)
    x[70, 0] = np.float16(np.inf)
    with np.errstate(invalid="ignore", over="ignore"):
        z = [r.s * r.W[:, 70] * np.inf for r in c.refs]
        a = lr.act(kind, z[0])[0]
        assert _same_kind(c.fused(x, kind)[:, 0], a)
        assert _same_kind(c.glu(x, kind)[:, 0], a * z[1])


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8)])
@pytest.mark.parametrize("T", [1, 5, 40, 520])
@pytest.mark.parametrize("kind", ["relu", "gelu", "gelu_tanh", "silu"])
def test_slopes_keep_a_nan(K, B, T, kind):
    """A NaN in one token's activations: that token's gradients are NaN, the
    others keep their bits."""
    c = Case(72, 264, K, B, 33, layers=2)
    x, gy = acts(264, T, 1), acts(72, T, 2, 0.1)
    bad = x.copy()
    bad[9, T - 1] = np.float16(np.nan)
    with_bias = acts(72, 1, 3).ravel()
    clean = c.fused_grad(x, gy, kind, with_bias, want_bias=False)[0], *c.glu_grad(x, gy, kind)[:2]
    got = c.fused_grad(bad, gy, kind, with_bias, want_bias=False)[0], *c.glu_grad(bad, gy, kind)[:2]
    for g, k in zip(got, clean):
        assert np.isnan(g[:, T - 1].astype(np.float64)).all()
        assert np.array_equal(g[:, :T - 1].view(np.uint16), k[:, :T - 1].view(np.uint16))


def _step2(v):
    """Mean square error of rounding v to binary16: a twelfth of the step's square."""
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -40))), -14)
    return np.where(v == 0, 0.0, 4.0 ** (e - 10) / 12)


def _table_sums(ref, layer, x):
    """s (sum of codewords) x, unrounded, and the mean square error that
    rounding each table entry <codeword, x_g> once to 11 bits makes of it."""
    K = layer.spec.num_codebooks
    cb = lr.f64(layer.codebooks).reshape(K, -1, 8)
    codes = layer.codes.reshape(layer.spec.out_features, -1, K).astype(np.int64)
    xg = x.astype(np.float64).reshape(-1, 8)
    total = var = 0.0
    for k in range(K):
        entries = np.take_along_axis(np.einsum("cj,gj->gc", cb[k], xg), codes[:, :, k].T, axis=1)  # [groups][rows]
        total = total + entries.sum(0)
        steps = np.where(entries == 0, 0.0, 4.0 ** (np.floor(np.log2(np.abs(entries) + (entries == 0))) - 10) / 12)
        var = var + steps.sum(0)
    return ref.s * total, ref.s ** 2 * var


@pytest.mark.parametrize("K,B", [(2, 8), (1, 8)])
@pytest.mark.parametrize("sigma", [1.0, 1e-2, 1e-3, 1e-4, 1e-6])
def test_table_entries_of_small_activations_keep_their_bits(K, B, sigma):
    """One token, 8-bit codebooks: the root mean square error over 2048 rows is
    that of one 11-bit rounding per table entry and one of the result, whatever
    the size of the activations.  It is estimated from 2048 rows (2 % spread);
    binary16 additions of four entries would make it 1.7 times as large."""
    out, inp = 2048, 4096
    c = Case(out, inp, K, B, 15, layers=2, scale=min(1 / sigma, 16000.0))
    x = acts(inp, 1, 1, sigma)
    (zg, vg), (zu, vu) = (_table_sums(r, L, x) for r, L in zip(c.refs, c.layers))
    for got, want, var in ((c.fused(x, "none"), zg, vg), (c.glu(x, "none"), zg * zu, zu ** 2 * vg + zg ** 2 * vu)):
        err = got[:, 0].astype(np.float64) - want
        assert np.sqrt((err ** 2).mean()) <= 1.2 * np.sqrt((var + _step2(want)).mean())


def _back(pairs):
    """sum of W^T (s g) over [(Ref, g)], and its mean square error when each
    product s g is rounded once to 11 bits and so is the result."""
    total = var = 0.0
    for r, g in pairs:
        z = r.s[:, None] * lr.f64(g)
        steps = np.where(z == 0, 0.0, 4.0 ** (np.floor(np.log2(np.abs(z) + (z == 0))) - 10) / 12)
        total = total + r.W.T @ z
        var = var + (r.W ** 2).T @ steps
    return total, var + _step2(total)


def _check_rms(got, pairs, what):
    """The root mean square error over all elements; 1.2 leaves room for the
    estimate's spread (thousands of rounding errors) and the fp32 sums."""
    want, var = _back(pairs)
    err = got.astype(np.float64) - want
    assert np.isfinite(err).all(), what
    ratio = np.sqrt((err ** 2).mean() / var.mean())
    assert ratio <= 1.2, f"{what}: {ratio:.3g} times the error of one rounding"


SCHEMES = [(1, 16), (2, 8), (1, 8), (2, 16), (8, 8)]


@pytest.mark.parametrize("K,B", SCHEMES)
@pytest.mark.parametrize("T", [3, 40, 45, 520])
@pytest.mark.parametrize("sigma,scale", [(0.1, 1.0), (1e-3, 16.0), (1e-5, 1000.0), (1e-6, 10000.0), (100.0, 1e-3)])
def test_gradients_of_any_size_keep_their_bits(K, B, T, sigma, scale):
    """Small gradients times ordinary or large scales (and the other way round)
    are rounded to 11 bits as the rest are."""
    c = Case(520, 264, K, B, 34, scale=scale)
    gy = acts(520, T, 4, sigma)
    _check_rms(c.input_grad(gy), [(c.refs[0], gy)], "input grad")


@pytest.mark.parametrize("K,B", SCHEMES)
@pytest.mark.parametrize("T", [40, 45])
def test_a_dominating_scale_costs_the_other_rows_no_bits(K, B, T):
    c = Case(520, 264, K, B, 35)
    s = (c.refs[0].s * 2.0 ** -11).astype(np.float16)
    s[17] = np.float16(1024.0)
    c.scales[0] = fenced(s)
    c.refs[0].s = s.astype(np.float64)
    gy = acts(520, T, 4, 64.0)
    gy[17] = 0
    _check_rms(c.input_grad(gy), [(c.refs[0], gy)], "input grad")


@pytest.mark.parametrize("K,B", SCHEMES)
@pytest.mark.parametrize("T", [8, 45, 520])
@pytest.mark.parametrize("small", [0, 1])
@pytest.mark.parametrize("power", [10, 12, 14])
def test_gated_backward_of_layers_with_scales_of_different_size(K, B, T, small, power):
    """One projection's scales 2^-power of the other's: the two terms of grad_x
    are of one size (each layer's gradient carries the other's scale), so both
    keep their bits."""
    c = Case(520, 264, K, B, 36, layers=2)
    s = (c.refs[small].s * 2.0 ** -power).astype(np.float16)
    c.refs[small].s = s.astype(np.float64)
    c.scales[small] = fenced(s)
    c.weights = [aq.Weights.make(d.packed, b, k) for d, b, k in zip(c.dls, c.books, c.scales)]
    x, gy = acts(264, T, 1), acts(520, T, 2, 30.0)
    gg, gu, gx = c.glu_grad(x, gy, "silu")
    want_g, want_u = lr.glu_grad(*c.refs, x, gy, "silu")
    lr.check(gg, want_g, "grad_gate")
    lr.check(gu, want_u, "grad_up")
    _check_rms(gx, [(c.refs[0], gg), (c.refs[1], gu)], "grad_x")


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8)])
@pytest.mark.parametrize("T", [24, 45])
def test_infinite_and_nan_gradients_stay_in_their_tokens(K, B, T):
    """E follows the finite products: the other tokens keep their values' bits
    but for the power of two."""
    c = Case(520, 264, K, B, 37)
    gy = acts(520, T, 4, 0.1)
    bad = gy.copy()
    bad[3, 2] = np.float16(np.inf)
    bad[400, T - 1] = np.float16(np.nan)
    clean, got = c.input_grad(gy), c.input_grad(bad)
    keep = np.setdiff1d(np.arange(T), [2, T - 1])
    lr.check(got[:, keep], tuple(a[:, keep] for a in c.refs[0].back(gy)), "other tokens")
    assert np.isfinite(clean.astype(np.float64)).all()
    assert _same_kind(got[:, 2], c.refs[0].W[3] * np.inf) and np.isnan(got[:, T - 1].astype(np.float64)).all()


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8)])
@pytest.mark.parametrize("T", [8, 13])
@pytest.mark.parametrize("zero", ["gradients", "scales"])
def test_zero_gradients_or_scales_give_zero(K, B, T, zero):
    c = Case(136, 264, K, B, 38)
    gy = acts(136, T, 4)
    if zero == "gradients":
        gy[...] = 0
    else:
        c.scales[0] = fenced(np.zeros(136, np.float16))
    assert (c.input_grad(gy) == 0).all()


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8)])
@pytest.mark.parametrize("T,batch", [(48, 1), (45, 2), (520, 8)])
def test_weights_rewritten_by_ordinary_work_between_calls(K, B, T, batch):
    """Every entry point right behind another call and a copy that rewrites the
    codebooks (as an optimiser step would), all queued at once: each call sees the
    codebooks that the last copy left."""
    b = Block(1000, 1032, K, B, 9)
    calls = b.calls(T, batch)
    sets = [[books.clone() for _, books, _ in b.w],
            [(torch.randn(books.shape, device="cuda", generator=b.gen) * 0.02).half() for _, books, _ in b.w]]

    def write(i):
        for (_, books, _), new in zip(b.w, sets[i]):
            books.copy_(new)

    ws = workspace(max(size for _, size, _ in calls))
    want = []
    for i in (0, 1):
        write(i)
        torch.cuda.synchronize()
        want.append([[o.clone() for o in go(ws)] for _, _, go in calls])
        torch.cuda.synchronize()
    got = []
    for j in range(len(calls)):
        for i in (0, 1, 0):
            write(i)
            got.append((j, i, calls[j][2](ws), calls[j - 1][2](ws)))
    torch.cuda.synchronize()
    assert aq.aq_workspace_status(ws) == 0
    for j, i, outs, before in got:
        for k, o in ((j, outs), (j - 1, before)):
            for x, y in zip(o, want[i][k]):
                x, y = (t.view(torch.int16) if t.dtype == torch.float16 else t for t in (x, y))
                assert torch.equal(x, y), (calls[k][0], i)


@pytest.mark.parametrize("K,B", [(1, 16), (2, 8)])
@pytest.mark.parametrize("out,T", [(8, 5001), (24, 2056), (520, 4099)])
def test_the_largest_gradient_is_found_wherever_it_stands(K, B, out, T):
    """Gradients of 1e-3 and one of 6e4, in the first or last rows and tokens,
    the ends of a warp's share of a row (2048 tokens) among them: a largest one
    that was missed would overflow once scaled."""
    c = Case(out, 136, K, B, 39, sigma=1e-3)
    base = acts(out, T, 4, 1e-3)
    for r, t in ((0, 0), (out - 1, T - 1), (out // 2, 2047), (out - 1, 2048), (0, T - 2)):
        gy = base.copy()
        gy[r, t] = np.float16(6e4)
        got = c.input_grad(gy)
        toks = np.unique([0, 7, 8, 2046, 2047, 2048, 2049, T - 9, T - 2, T - 1, t])
        lr.check(got[:, toks], c.refs[0].back(gy[:, toks]), f"row {r} token {t}")
        assert np.isfinite(got.astype(np.float64)).all()


@pytest.mark.parametrize("K,B", SCHEMES)
@pytest.mark.parametrize("sigma,scale,g", [(3000.0, 1e-3, 0.01), (3000.0, 50.0, 1e-5), (100.0, 2.0 ** -14, 1.0),
                                           (1e-4, 16000.0, 1.0), (1e-4, 1.0, 1000.0)])
def test_codebooks_of_any_size(K, B, sigma, scale, g):
    """Large and small codebook entries, scales and gradients together: nothing
    overflows, and the error is that of one rounding."""
    c = Case(520, 264, K, B, 40, layers=2, sigma=sigma, scale=scale)
    assert all(np.isfinite(r.W).all() for r in c.refs)
    gy = acts(520, 40, 4, g)
    _check_rms(c.input_grad(gy), [(c.refs[0], gy)], "input grad")
