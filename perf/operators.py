"""What is measured of the layer operators around the additive-quantised product.

Three operators over layers whose weights are stored as codes (W[o][8g+j] =
RN16(sum_k C_k[codes[o][g][k]][j])), activations [features][tokens] binary16:

* the product with bias, activation and residual in its epilogue, for single
  tokens and prompts, and its backward pass;
* the gated feed-forward block, act(gate) * up with both projections
  quantised, for single tokens and prompts, and its backward pass;
* the input gradient of a layer, W^T (s * gy).

``run`` computes them in plain torch operations, or with ``own`` through the
package's entry points.
"""
import math

import torch

own = False

SIGMA = 0.02  # spread of the codebook entries, as in the Llama-2-shaped layers of aq_inputs


def listed():
    return [
        # attention output projection of one token, residual stream added
        {"name": "fused b1 1x16", "op": "fused", "out": 4096, "in": 4096, "K": 1, "B": 16, "n": 1,
         "act": "none", "bias": False, "residual": True},
        # MLP down projection of eight sequences decoded together
        {"name": "fused b8 2x8", "op": "fused", "out": 4096, "in": 11008, "K": 2, "B": 8, "n": 8,
         "act": "none", "bias": False, "residual": True},
        # MLP down projection of a 2048-token prompt
        {"name": "fused T2048 1x16", "op": "fused", "out": 4096, "in": 11008, "K": 1, "B": 16, "n": 2048,
         "act": "none", "bias": False, "residual": True},
        # a small layer with ragged rows, features and tokens: bias and GELU
        {"name": "fused T77 ragged 2x8", "op": "fused", "out": 1000, "in": 1032, "K": 2, "B": 8, "n": 77,
         "act": "gelu", "bias": True, "residual": False},
        # fine-tuning step of an MLP up projection with bias and GELU
        {"name": "fused grad T512 2x8", "op": "fused_grad", "out": 11008, "in": 4096, "K": 2, "B": 8, "n": 512,
         "act": "gelu_tanh", "bias": True, "residual": False},
        # gated MLP of one token
        {"name": "glu b1 2x8", "op": "glu", "out": 11008, "in": 4096, "K": 2, "B": 8, "n": 1, "act": "silu"},
        # gated MLP of sixteen sequences decoded together
        {"name": "glu b16 1x16", "op": "glu", "out": 11008, "in": 4096, "K": 1, "B": 16, "n": 16, "act": "silu"},
        # gated MLP of a 2048-token prompt
        {"name": "glu T2048 2x8", "op": "glu", "out": 11008, "in": 4096, "K": 2, "B": 8, "n": 2048, "act": "silu"},
        # backward pass of the gated MLP, 2048 tokens
        {"name": "glu grad T2048 1x16", "op": "glu_grad", "out": 11008, "in": 4096, "K": 1, "B": 16, "n": 2048,
         "act": "silu"},
        # backward pass of a small gated block, ragged tokens
        {"name": "glu grad T1001 2x8", "op": "glu_grad", "out": 2752, "in": 1032, "K": 2, "B": 8, "n": 1001,
         "act": "gelu_tanh"},
        # input gradient of an attention projection, a short sequence
        {"name": "input grad T512 1x16", "op": "input_grad", "out": 4096, "in": 4096, "K": 1, "B": 16, "n": 512},
        # input gradient of an MLP up projection, odd token count
        {"name": "input grad T2047 2x8", "op": "input_grad", "out": 11008, "in": 4096, "K": 2, "B": 8, "n": 2047},
    ]


def draw(rng):
    def log_size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["fused", "fused", "fused_grad", "glu", "glu", "glu_grad", "input_grad"])
    out = log_size(64, 11008)
    inp = max(8, log_size(64, 11008) // 8 * 8)
    K, B = rng.choice([(1, 16), (1, 16), (2, 8), (2, 8), (1, 8), (2, 16), (8, 8)])
    if op in ("fused", "glu") and rng.random() < 0.5:
        n = rng.randint(1, 16)  # decode
    else:
        n = log_size(1, 2048)
    if n > 1 and rng.random() < 0.4:
        n = max(8, n // 8 * 8) if n > 16 else n
    # no drawn case costs more than the largest listed one
    while out * inp * n > 11008 * 4096 * 2048:
        n = max(1, n // 2)
    case = {"op": op, "out": out, "in": inp, "K": K, "B": B, "n": n}
    if op == "input_grad":
        return case
    case["act"] = rng.choice(["relu", "gelu", "gelu_tanh", "silu"] + (["none"] if op == "fused" else []))
    if op in ("fused", "fused_grad"):
        case["bias"] = rng.random() < 0.5
        case["residual"] = op == "fused" and rng.random() < 0.5
    return case


# ---- inputs ------------------------------------------------------------------


def _layer(case, gen):
    out, inp, K, B = case["out"], case["in"], case["K"], case["B"]
    G = inp // 8
    codes = torch.randint(0, 1 << B, (out, G, K), device="cuda", generator=gen, dtype=torch.int32)
    books = (torch.randn((K, 1 << B, 8), device="cuda", generator=gen) * SIGMA).half()
    scales = (torch.rand(out, device="cuda", generator=gen) + 0.5).half()
    # the stored form: words of 8 rows x 32 groups interleaved, zero padding
    rt, gp = (out + 7) // 8, (G + 31) // 32 * 32
    words = torch.zeros((rt * 8, gp, K), device="cuda", dtype=torch.int32)
    words[:out, :G] = codes
    words = words.view(rt, 8, gp, K).permute(0, 2, 1, 3).contiguous()
    packed = words.to(torch.uint8) if B == 8 else words.to(torch.int16)
    return {"codes": codes.to(torch.uint8) if B == 8 else codes.to(torch.int16), "packed": packed, "books": books,
            "scales": scales}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    out, inp, n, op = case["out"], case["in"], case["n"], case["op"]

    def normal(*shape, sigma=1.0):
        return (torch.randn(shape, device="cuda", generator=gen) * sigma).half()

    s = {"case": dict(case), "layers": [_layer(case, gen) for _ in range(2 if op.startswith("glu") else 1)]}
    if op != "input_grad":
        s["x"] = normal(inp, n)
    if op.endswith("grad"):
        s["gy"] = normal(out, n, sigma=0.1)
    s["bias"] = normal(out, sigma=0.1) if case.get("bias") else None
    s["residual"] = normal(out, n) if case.get("residual") else None
    if own:  # what a program keeps per layer: descriptor, weights' handles, workspace
        import additive_quantized_matmul_b200 as aq
        d = s["desc"] = aq.LayerDesc.make(out, inp, case["K"], case["B"])
        s["weights"] = [aq.Weights.make(w["packed"], w["books"], w["scales"]) for w in s["layers"]]
        if op == "fused":
            nbytes = (aq.aq_gemv_workspace_bytes if n <= 16 else aq.aq_gemm_fused_workspace_bytes)(d, n)
        elif op == "glu":
            nbytes = (aq.aq_glu_gemv_workspace_bytes if n <= 16 else aq.aq_glu_gemm_workspace_bytes)(d, n)
        elif op == "fused_grad":
            nbytes = aq.aq_gemm_fused_grad_workspace_bytes(d, n)
        elif op == "glu_grad":
            nbytes = aq.aq_glu_grad_workspace_bytes(d, n)
        else:
            nbytes = aq.aq_input_grad_workspace_bytes(d, n)
        s["workspace"] = torch.zeros(nbytes, device="cuda", dtype=torch.uint8)
    return s


# ---- plain form --------------------------------------------------------------


def _decode(w):
    """The decoded matrix in fp32: codewords summed (in 64 bits when more than
    two, where fp32 could round), one rounding to binary16."""
    codes = w["codes"].long()
    if w["books"].shape[1] > 256:
        codes = codes & 0xffff
    K = codes.shape[2]
    books = w["books"].double() if K > 2 else w["books"].float()
    total = sum(books[k][codes[:, :, k]] for k in range(K))
    return total.half().float().reshape(codes.shape[0], -1)


def _act(z, kind):
    if kind == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if kind == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _project(w, x):
    return w["scales"].float()[:, None] * (_decode(w) @ x.float())


def _back(w, g):
    return _decode(w).t() @ (w["scales"].float()[:, None] * g.float())


def _plain(s):
    case = s["case"]
    op, act = case["op"], case.get("act", "none")
    if op == "input_grad":
        return {"grad_x": _back(s["layers"][0], s["gy"]).half()}
    if op == "fused" or op == "fused_grad":
        z = _project(s["layers"][0], s["x"])
        if s["bias"] is not None:
            z = z + s["bias"].float()[:, None]
        if op == "fused":
            y = _act(z, act)
            return {"y": (y if s["residual"] is None else y + s["residual"].float()).half()}
        gz = s["gy"].float() * _act_grad(z, act)
        # the input gradient is taken of grad_z as it is handed on, in binary16
        return {"grad_z": gz.half(), "grad_bias": gz.sum(1), "grad_x": _back(s["layers"][0], gz.half()).half()}
    g, u = _project(s["layers"][0], s["x"]), _project(s["layers"][1], s["x"])
    if op == "glu":
        return {"y": (_act(g, act) * u).half()}
    gy = s["gy"].float()
    gg, gu = (gy * u * _act_grad(g, act)).half(), (gy * _act(g, act)).half()
    return {"grad_gate": gg, "grad_up": gu, "grad_x": (_back(s["layers"][0], gg) + _back(s["layers"][1], gu)).half()}


# ---- the package's entry points ----------------------------------------------


def _own(s):
    import additive_quantized_matmul_b200 as aq
    case = s["case"]
    op, out, inp, n = case["op"], case["out"], case["in"], case["n"]
    d, ws = s["desc"], s["workspace"]

    def empty(rows):
        return torch.empty((rows, n), device="cuda", dtype=torch.float16)

    if op == "glu" or op == "glu_grad":
        gate, up = s["weights"]
        act = aq.ACTIVATIONS[case["act"]]
        if op == "glu":
            y = empty(out)
            (aq.aq_glu_gemv if n <= 16 else aq.aq_glu_gemm)(d, gate, up, s["x"], n, act, y, ws)
            return {"y": y}
        gg, gu, gx = empty(out), empty(out), empty(inp)
        aq.aq_glu_grad(d, gate, up, s["x"], s["gy"], n, act, gg, gu, gx, ws)
        return {"grad_gate": gg, "grad_up": gu, "grad_x": gx}
    w = s["layers"][0]
    if op == "input_grad":
        gx = empty(inp)
        aq.aq_input_grad(d, w["packed"], w["books"], w["scales"], s["gy"], n, gx, ws)
        return {"grad_x": gx}
    act = aq.ACTIVATIONS[case["act"]]
    if op == "fused":
        y = empty(out)
        (aq.aq_gemv_fused if n <= 16 else aq.aq_gemm_fused)(
            d, w["packed"], w["books"], w["scales"], s["x"], n, y, ws, activation=act, bias=s["bias"],
            residual=s["residual"])
        return {"y": y}
    gz, gx = empty(out), empty(inp)
    gb = torch.empty(out, device="cuda", dtype=torch.float32)
    aq.aq_gemm_fused_grad(d, w["packed"], w["books"], w["scales"], s["x"], s["gy"], n, gz, gb, gx, ws,
                          activation=act, bias=s["bias"])
    return {"grad_z": gz, "grad_bias": gb, "grad_x": gx}


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without -------------------------------------------


def work(case):
    out, inp, n, K, B, op = case["out"], case["in"], case["n"], case["K"], case["B"], case["op"]
    layers = 2 if op.startswith("glu") else 1
    product = 2.0 * out * inp * n
    nbytes = layers * (out * (inp // 8) * K * B / 8 + K * (1 << B) * 16 + 2 * out)
    if op != "input_grad":
        nbytes += 2 * inp * n  # x
    nbytes += 2 * out * n      # y, or gy
    if op.endswith("grad"):
        nbytes += 2 * inp * n  # grad_x
    if op == "glu_grad":
        nbytes += 4 * out * n  # grad_gate, grad_up
    if op == "fused_grad":
        nbytes += 2 * out * n + 4 * out  # grad_z, grad_bias
    if case.get("bias"):
        nbytes += 2 * out
    if case.get("residual"):
        nbytes += 2 * out * n
    # a backward pass computes the projections once more: nothing was kept of them
    flops = layers * product * (2 if op in ("fused_grad", "glu_grad") else 1)
    return {"bytes": nbytes, "flops": flops}


# ---- the definition in 64 bits -----------------------------------------------


def _matrix64(w):
    rows, groups, K = w["codes"].shape
    m = torch.zeros((rows * groups, 8), device="cuda", dtype=torch.float64)
    for k in range(K):
        idx = w["codes"][:, :, k].reshape(-1).to(torch.int64) % w["books"].shape[1]
        m += torch.index_select(w["books"][k].to(torch.float64), 0, idx)
    # the stored weight is the codeword sum rounded to binary16
    return m.to(torch.float16).to(torch.float64).view(rows, groups * 8)


def _phi64(v, kind):
    """(act(v), act'(v))"""
    if kind == "none":
        return v, torch.ones_like(v)
    if kind == "relu":
        return v.clamp_min(0), torch.heaviside(v, torch.zeros((), device=v.device, dtype=v.dtype))
    if kind == "silu":
        p = torch.sigmoid(v)
        return v * p, p + v * p * (1 - p)
    if kind == "gelu":
        cdf = torch.special.ndtr(v)
        return v * cdf, cdf + v * torch.exp(-v * v / 2) * 0.39894228040143267794
    c = 0.79788456080286535588
    p = torch.sigmoid(2 * c * (v + 0.044715 * v ** 3))  # (1 + tanh) / 2
    return v * p, p + v * 2 * p * (1 - p) * c * (1 + 0.134145 * v * v)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    mats = [_matrix64(w) * w["scales"].to(torch.float64).unsqueeze(1) for w in s["layers"]]
    gy = s["gy"].to(torch.float64) if "gy" in s else None
    if op == "input_grad":
        return {"grad_x": torch.matmul(mats[0].T, gy)}
    pre = [torch.matmul(m, s["x"].to(torch.float64)) for m in mats]
    if s["bias"] is not None:
        pre[0] += s["bias"].to(torch.float64).unsqueeze(1)
    a, da = _phi64(pre[0], case["act"])
    if op == "fused":
        return {"y": a if s["residual"] is None else a + s["residual"].to(torch.float64)}
    if op == "glu":
        return {"y": a * pre[1]}
    if op == "fused_grad":
        gz = gy * da
        handed = gz.to(torch.float16).to(torch.float64)
        return {"grad_z": gz, "grad_bias": gz.sum(dim=1), "grad_x": torch.matmul(mats[0].T, handed)}
    gg, gu = gy * pre[1] * da, gy * a
    gx = torch.matmul(mats[0].T, gg.to(torch.float16).to(torch.float64))
    gx += torch.matmul(mats[1].T, gu.to(torch.float16).to(torch.float64))
    return {"grad_gate": gg, "grad_up": gu, "grad_x": gx}
