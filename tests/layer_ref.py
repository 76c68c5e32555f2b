"""64-bit references of the layer operators and the error each may carry.

Rounding to binary16 is off by at most 2^-11 of the value (2^-25 where it is
subnormal), an fp32 addition by at most 2^-23 (rounded or truncated).  The
error of the sum z = s (W x) + b, with A = sum_i |s| |C_1 + ..| |x_i| taken
over the codewords' magnitudes:

* fp32 accumulation in any order: (in + 64) 2^-23 A;
* 8-bit codebooks, one or two, one token: lookup tables in binary16, each
  entry rounded once and four entries added in two binary16 additions, so
  three roundings, 4 * 2^-11 A with the second-order terms, and 2^-25 for
  each entry that may be subnormal;
* eight codebooks: the sum of the codewords may round the other way, one
  binary16 step, 2^-10 |W|.

The activations' slopes are at most 1.13 (GELU; SiLU 1.10) and their second
derivatives at most 1 in magnitude (GELU 0.80, SiLU 0.50).
"""
import math

import numpy as np

import oracle

H = 2.0 ** -11   # binary16 rounding, relative
SUB = 2.0 ** -25  # and absolute, subnormal
F = 2.0 ** -23   # one fp32 addition


def f64(a):
    a = np.asarray(a)
    return (a.view(np.float16) if a.dtype in (np.uint16, np.int16) else a).astype(np.float64)


class Ref:
    """A layer in 64 bits: W (decoded), |C| (the codewords' magnitudes added), s."""

    def __init__(self, layer, scaled=True):
        self.spec = layer.spec
        self.W = f64(oracle.decode(layer.codes, layer.codebooks)).reshape(layer.spec.out_features, -1)
        cb = np.abs(f64(layer.codebooks)).reshape(layer.spec.num_codebooks, -1, 8)
        codes = layer.codes.reshape(layer.spec.out_features, -1, layer.spec.num_codebooks)
        self.C = sum(cb[k][codes[:, :, k]] for k in range(codes.shape[2])).reshape(self.W.shape)
        self.s = f64(layer.scales) if scaled else np.ones(layer.spec.out_features)

    def z(self, x, bias=None):
        """z and its error."""
        x = f64(x)
        sp = self.spec
        s = self.s[:, None]
        A = np.abs(s) * (self.C @ np.abs(x))
        err = (sp.in_features + 64) * F * A
        if sp.nbits == 8 and sp.num_codebooks <= 2 and x.shape[1] == 1:
            err = err + 4 * H * A + np.abs(s) * (sp.in_features // 8 * sp.num_codebooks * SUB)
        if sp.num_codebooks == 8:
            err = err + 2 * H * np.abs(s) * (np.abs(self.W) @ np.abs(x))
        z = s * (self.W @ x)
        if bias is not None:
            z = z + f64(bias)[:, None]
            err = err + 2 * F * (np.abs(z) + np.abs(f64(bias))[:, None])
        return z, err

    def back(self, g, others=()):
        """W^T (s g), added over this layer and `others` [(Ref, g)], and its error."""
        total = err = 0.0
        pairs = [(self, g), *others]
        # the weights are rounded after scaling by s 2^-E, 2^E just above the largest |s|
        smax = max(np.abs(r.s).max() for r, _ in pairs)
        two_e = 2.0 ** (math.floor(math.log2(smax)) + 1) if smax > 0 else 1.0
        terms = sum(r.spec.out_features for r, _ in pairs)
        for r, gv in pairs:
            gv = f64(gv)
            sg = r.s[:, None] * gv
            A = np.abs(r.W).T @ np.abs(sg)
            total = total + r.W.T @ sg
            # a scale may be subnormal once divided by 2^E (2^-25 of it); so may
            # its product with the weight or (1x16) with the gradient
            small = np.abs(r.W).T @ np.ones_like(gv) if r.spec.nbits == 16 and r.spec.num_codebooks == 1 \
                else np.abs(gv).sum(0)[None, :]
            err = err + (1.01 * H + (terms + 64) * F) * A \
                + SUB * two_e * (small + np.abs(r.W).T @ np.abs(gv))
            if r.spec.num_codebooks == 8:
                err = err + 2 * H * A
        return total, err + rounded(total)


def rounded(v):
    return H * np.abs(v) + SUB


def _erf(v):
    return np.vectorize(math.erf, otypes=[np.float64])(v) if v.size else v


def _sigmoid(v):
    return 0.5 * (1 + np.tanh(0.5 * v))


def act(kind, z):
    """(act(z), act'(z)) in 64 bits."""
    if kind == "relu":
        return np.maximum(z, 0), (z > 0).astype(np.float64)
    if kind == "gelu":
        cdf = 0.5 * (1 + _erf(z / math.sqrt(2)))
        return z * cdf, cdf + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if kind == "silu":
        p = _sigmoid(z)
        return z * p, p + z * p * (1 - p)
    return z, np.ones_like(z)


def act_error(kind, z, ez):
    """Errors of act(z) and act'(z), z off by ez.

    The logistic function p(a) comes from an exponential that is off by
    (2 + 1.2 |a|) 2^-23 of its value, so p by p (1 - p) of that and two more
    roundings: at most 2^-20 as |a| p (1 - p) < 0.25.  act(z) = z p is then
    off by |z| 2^-20, and the slope p + z p (1 - p) k, k = d a / d z, by 2^-20
    (1 + |z| k); for the error function the same bounds hold with k = 1.
    """
    if kind == "none":
        return ez, np.zeros_like(z)
    if kind == "relu":
        return ez, np.where(np.abs(z) <= ez, 1.0, 0.0)  # the slope's step lies within the error
    k = 1.6 * (1 + 0.1342 * z * z) if kind == "gelu_tanh" else 1.0
    fast = 2.0 ** -20
    return 1.13 * ez + fast * np.abs(z), ez + fast * (1 + np.abs(z) * k)


def fused(ref, x, kind, bias=None, residual=None):
    """y and its error."""
    z, ez = ref.z(x, bias)
    a, _ = act(kind, z)
    ea, _ = act_error(kind, z, ez)
    y = a if residual is None else a + f64(residual)
    return y, ea * (1 + H) + 2 * F * np.abs(y) + rounded(y)


def fused_grad(ref, x, gy, kind, bias=None):
    """(grad_z, error), (grad_bias, error)."""
    z, ez = ref.z(x, bias)
    _, slope = act(kind, z)
    _, es = act_error(kind, z, ez)
    g = f64(gy)
    gz, err = g * slope, np.abs(g) * es * (1 + H)
    T = g.shape[1]
    return (gz, err + 2 * F * np.abs(gz) + rounded(gz)), \
        (gz.sum(1), err.sum(1) + (T + 8) * F * np.abs(gz).sum(1) + 1e-30)


def glu(gate, up, x, kind):
    g, eg = gate.z(x)
    u, eu = up.z(x)
    a, _ = act(kind, g)
    ea, _ = act_error(kind, g, eg)
    y = a * u
    return y, (np.abs(u) * ea + np.abs(a) * eu + ea * eu) * (1 + H) + 4 * F * np.abs(y) + rounded(y)


def glu_grad(gate, up, x, gy, kind):
    g, eg = gate.z(x)
    u, eu = up.z(x)
    a, slope = act(kind, g)
    ea, es = act_error(kind, g, eg)
    d = f64(gy)
    gg, gu = d * u * slope, d * a
    e_gg = np.abs(d) * (np.abs(u) * es + np.abs(slope) * eu + es * eu)
    e_gu = np.abs(d) * ea
    return (gg, e_gg * (1 + H) + 4 * F * np.abs(gg) + rounded(gg)), \
        (gu, e_gu * (1 + H) + 4 * F * np.abs(gu) + rounded(gu))


def check(got, want_err, what):
    want, err = want_err
    got = np.asarray(got, dtype=np.float64).reshape(want.shape)
    bad = ~(np.abs(got - want) <= err)
    if bad.any():
        at = np.argwhere(bad)[:4]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first " + ", ".join(
            f"{tuple(map(int, i))} got {got[tuple(i)]:.6g} want {want[tuple(i)]:.6g} +- {err[tuple(i)]:.2g}" for i in at))
