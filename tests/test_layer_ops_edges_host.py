"""Layer operators at their edges, without a GPU: what the sizes and the header
promise."""
import os
import re

import pytest

import additive_quantized_matmul_b200 as aq

SCHEMES = [(1, 16), (2, 8), (1, 8), (2, 16), (8, 8)]
DATA = 16 + 4 * 1024  # status word and arrival counters come first


def _padded(rows, T):
    return 2 * rows * ((T + 7) // 8 * 8)


@pytest.mark.parametrize("K,B", SCHEMES)
@pytest.mark.parametrize("out,inp", [(64, 256), (4096, 4096), (11008, 4096), (4096, 11008), (300, 1032)])
@pytest.mark.parametrize("T", [1, 7, 8, 45, 512, 1001, 1999, 2047, 2048, 4096])
def test_arrays_lie_behind_the_counters(K, B, out, inp, T):
    """A workspace serves any sequence of calls, so no array of an operator may
    lie among the arrival counters: each size covers them and, behind them, the
    arrays that the call cannot do without."""
    d = aq.LayerDesc.make(out, inp, K, B)
    pad_in, pad_out = (_padded(inp, T), _padded(out, T)) if T % 8 else (0, 0)
    scaled = 0 if B == 8 and K <= 2 else _padded(out, T)  # gradients multiplied by the scales
    sums = 4 * ((T + 15) // 16) * out
    for fn, arrays in ((aq.aq_gemm_fused_workspace_bytes, pad_in + 2 * pad_out),
                       (aq.aq_glu_gemm_workspace_bytes, pad_in + pad_out),
                       (aq.aq_input_grad_workspace_bytes, pad_in + max(pad_out, scaled)),
                       (aq.aq_gemm_fused_grad_workspace_bytes, sums + 2 * pad_in + 2 * pad_out + scaled),
                       (aq.aq_glu_grad_workspace_bytes, 2 * pad_in + 3 * pad_out + 2 * scaled)):
        if arrays:
            assert fn(d, T) >= DATA + arrays, fn.__name__


# entry points whose first launch may read weights before earlier launches complete
EARLY = ["aq_gemv", "aq_gemv_noalloc", "aq_gemm", "aq_gemv_fused", "aq_gemm_fused", "aq_input_grad",
         "aq_gemm_fused_grad", "aq_glu_gemv", "aq_glu_gemm", "aq_glu_grad"]


def _header():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "aq.h")
    with open(path, encoding="utf-8") as f:
        return f.read()


@pytest.mark.parametrize("fn", EARLY)
def test_the_header_names_the_rule_where_weights_are_read_early(fn):
    text = _header()
    at = text.index(f"aq_status {fn}(")
    comment = text[text.rindex("/*", 0, at):at]
    assert "early weight reads" in " ".join(comment.replace("*", " ").split()).lower()


def test_every_function_that_the_header_speaks_of_exists():
    text = _header()
    declared = set(re.findall(r"\b(aq_\w+)\(", text)) | set(re.findall(r"}\s*(aq_\w+);", text)) | {"aq_b200", "aq_stream_t"}
    spoken = set(re.findall(r"\b(aq_[a-z0-9_]+)\b", text))
    assert spoken <= declared, spoken - declared
    assert set(aq.EXPORTED_SYMBOLS) <= declared
