"""A token's values have the same bits alone, in a batch and in a prompt: every activation, every part of the epilogue, given
and made 8-bit tokens, products with tiles of their own and with tiles that clusters share, the expert."""

from __future__ import annotations

import pytest
import torch

ses = pytest.importorskip("sparse_expert_swiglu_gb300")
from tests.test_int8 import BF16, F16, F32, _cuda, _expert_case, _linear_case, _linear_ref, _linear_run, _product64, _within  # noqa: E402

gpu = pytest.mark.gpu

TOKENS = (1, 2, 3, 4, 7, 8, 13, 16, 17, 32, 33, 64, 65, 90, 130, 257, 400)


@pytest.fixture(scope="module", autouse=True)
def _built():
    ses.build_library()
    ses.lib()


@gpu
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("N,K", [(1031, 1040), (136, 8192), (8200, 272)])
def test_products(act, gated, N, K):
    M = 600
    for x, residual, dtype, out in (("int8", False, F16, F32), ("16 bits", True, BF16, F32), ("int8", True, F16, None)):
        c = _linear_case(M, N, K, dtype, x, act, True, gated, residual, out)
        if x == "int8":  # products of about 2, where activations bend
            c["x_scale"] = c["x_scale"] * 8
        a = {k: _cuda(v) for k, v in c.items()}
        kw = {k: v for k, v in a.items() if k not in ("x", "x_scale", "w", "w_scale", "residual")}

        def run(n):
            return ses.linear_int8(a["x"][:n], a["w"], a["w_scale"], x_scale=None if x != "int8" else a["x_scale"][:n],
                                   residual=a["residual"][:n] if residual else None, **kw)
        full = run(M)
        for n in TOKENS:
            assert torch.equal(run(n), full[:n]), (n, x)


@gpu
@pytest.mark.parametrize("d,f", [(512, 1040), (256, 4096), (4096, 272)])
def test_experts(d, f):
    M = 600
    for x, dtype in (("int8", F16), ("16 bits", BF16)):
        c = _expert_case(M, d, f, dtype, x, True)
        if x == "int8":
            c["x_scale"] = c["x_scale"] * 8
        ex = ses.Int8Experts(*(t.cuda() for t in c["w"]))
        xd, xs, r = _cuda(c["x"]), _cuda(c["x_scale"]), _cuda(c["residual"])

        def run(n):
            return ses.expert_int8_swiglu(xd[:n], ex, 2, x_scale=None if xs is None else xs[:n], residual=r[:n], dtype=dtype)
        full = run(M)
        for n in TOKENS:
            assert torch.equal(run(n), full[:n]), (n, x)


@gpu
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("N,K", [(1031, 1040), (136, 8192)])
def test_scales_of_all_sizes(gated, N, K):
    """Tokens and outputs of ordinary scales beside such whose products leave fp32's range."""
    M = 600
    c = _linear_case(M, N, K, BF16, "int8", "none", gated=gated, out=F32)
    g = torch.Generator().manual_seed(K)
    for k in ("x_scale", "w_scale", "w_mul_scale"):
        if c[k] is not None:
            c[k] = torch.ldexp(c[k], torch.randint(-120, 60, c[k].shape, generator=g))
    few = {**c, "x": c["x"][:40], "x_scale": c["x_scale"][:40]}
    y, (ref, bound) = _linear_run(few).cpu(), _linear_ref(few)
    # both factors are fp32 numbers: only where their exact values are normal ones do the relative bounds hold
    normal = torch.ones_like(ref, dtype=torch.bool)
    for w, ws in (("w", "w_scale"), ("w_mul", "w_mul_scale")):
        if c[w] is not None:
            size = _product64(few["x"].double(), few["x_scale"], c[w], c[ws], None)[0].abs()
            normal &= (size >= 2.0 ** -126) & (size < 2.0 ** 127)
    normal &= ref.abs() < 2.0 ** 127
    assert normal.double().mean() > 0.3
    _within(y[normal], ref[normal], bound[normal], F32)
    a = {k: _cuda(v) for k, v in c.items()}
    kw = {k: v for k, v in a.items() if k not in ("x", "x_scale", "w", "w_scale")}

    def run(n):
        return ses.linear_int8(a["x"][:n], a["w"], a["w_scale"], x_scale=a["x_scale"][:n], **kw)
    full = run(M)
    assert torch.isfinite(full).any() and (full == 0).any()
    for n in TOKENS:
        assert torch.equal(run(n).view(torch.int32), full[:n].view(torch.int32)), n
