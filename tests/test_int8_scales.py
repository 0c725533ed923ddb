"""Scales at the ends of fp32's range: the product of a token's and an output's scale alone may leave the range although the
result lies in it.

The bound is that of the operators' other tests, three roundings of a product to fp32, and half a step of the smallest
fp32 number where a result is that small.
"""

from __future__ import annotations

import pytest
import torch

ses = pytest.importorskip("sparse_expert_swiglu_gb300")
from tests.test_int8 import BF16, F32, U, _expert_case, _expert_run, _gated64, _linear_case, _linear_check, _linear_run, _within  # noqa: E402

gpu = pytest.mark.gpu

# tokens for each of the kernels
TOKENS = [1, 2, 4, 7, 16, 40, 90, 150, 300]


@pytest.fixture(scope="module", autouse=True)
def _built():
    ses.build_library()
    ses.lib()


@gpu
@pytest.mark.parametrize("M", TOKENS)
@pytest.mark.parametrize("K", [528, 8192])
def test_scales_whose_product_is_small(M, K):
    """2^-100 times 2^-40 is no normal number, 2^-120 times 2^-60 is none at all; with sums up to 2^27 the results are
    numbers down to 2^-153."""
    for x_exp, w_exp in ((-100, -40), (-40, -100), (-120, -20), (-100, -60), (-75, -75), (-130, -10)):
        c = _linear_case(M, 200, K, BF16, out=F32)
        c["x_scale"] = torch.ldexp(1 + c["x_scale"] * 16, torch.tensor(x_exp))
        c["w_scale"] = torch.ldexp(1 + torch.rand(200), torch.tensor(w_exp))
        y = _linear_check(c)
        assert (y != 0).any()


@gpu
@pytest.mark.parametrize("M", TOKENS)
def test_tokens_of_small_numbers(M):
    """bf16 tokens around 1e-36, quantised on the way; sums of two matrices."""
    for gated in (False, True):
        c = _linear_case(M, 200, 1040, BF16, "16 bits", gated=gated, out=F32)
        c["x"] = (c["x"].double() * 1e-36).to(BF16)
        c["w_scale"] = torch.full((200,), 1.6e-4)
        if gated:
            c["w_mul_scale"] = torch.full((200,), 1e30)
        _linear_check(c)


@gpu
@pytest.mark.parametrize("M", TOKENS)
def test_scales_whose_product_is_large(M):
    """A sum of zero under scales whose product is infinite is zero; tokens of 1e35 and weights of 1e-10 have finite
    results although a sum times the token's scale has none."""
    c = _linear_case(M, 200, 528, BF16, bias=True, out=F32)
    c["x"][:] = 0
    c["x_scale"][:], c["w_scale"][:] = 2.0 ** 100, 2.0 ** 60
    assert torch.equal(_linear_run(c).cpu(), c["bias"].float().expand(M, 200))
    c = _linear_case(M, 200, 528, BF16, out=F32)
    c["x_scale"] = (1 + c["x_scale"]) * 1e35
    c["w_scale"] = (1 + torch.rand(200)) * 1e-10
    y = _linear_check(c)
    assert torch.isfinite(y).all()
    c["x_scale"], c["w_scale"] = (1 + torch.rand(M)) * 1e-10, (1 + torch.rand(200)) * 1e35
    assert torch.isfinite(_linear_check(c)).all()


@gpu
@pytest.mark.parametrize("M", TOKENS)
def test_scales_that_are_no_number(M):
    """NaN in a token's or an output's scale spoils its row or column alone, beside scales of any size."""
    for other in (2.0 ** -140, 1.0, 2.0 ** 120):
        c = _linear_case(M, 200, 528, BF16, out=F32)
        c["x_scale"][:], c["w_scale"][:] = other, 2.0 ** -30
        c["x_scale"][M // 2], c["w_scale"][7] = float("nan"), float("nan")
        y = _linear_run(c).cpu()
        bad = torch.zeros(M, 200, dtype=torch.bool)
        bad[M // 2], bad[:, 7] = True, True
        assert torch.equal(torch.isnan(y), bad)


@gpu
@pytest.mark.parametrize("n", TOKENS)
def test_expert_of_small_numbers(n):
    """An expert whose up products are about 1e-33 and whose h and down rows have one sign: h, its scale and y are normal
    numbers, h's scale times down's is about 3e-44."""
    c = _expert_case(n, 256, 528, BF16)
    g, gs, _, _, dn, ds = c["w"]
    us, dn, ds = gs * 1e-33, dn.abs(), ds * 1e-5
    c["w"] = [g, gs, g, us, dn, ds]
    q, xs = c["x"].double(), c["x_scale"]
    h, dh = _gated64(dict(w=g[1], w_scale=gs[1], w_mul=g[1], w_mul_scale=us[1], bias=None, bias_mul=None, act="silu"), q, xs)
    m = h.abs().amax(1, keepdim=True)
    s, steps, off = m / 127, h * 127 / m, dh.amax(1, keepdim=True) / m
    hq, rows, ds64 = torch.round(steps), dn[1].double(), ds[1].double()
    y = (hq * s) @ rows.t() * ds64
    # an integer within h's error of a half may be one off, a step of its weight; the scale errs as the largest h does
    close = ((steps - torch.floor(steps) - 0.5).abs() <= 127 * dh / m + steps.abs() * off + 1e-12).double()
    lim = ((close * s) @ rows.t() + (hq.abs() * s) @ rows.t() * off) * ds64 + 4 * U * y.abs()
    assert float((s * ds64).max()) < torch.finfo(F32).smallest_normal
    _within(_expert_run(c, 1), y, lim, BF16)
