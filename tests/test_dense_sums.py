"""How far fp32 sums of long products may drift.

The tensor core cuts off what its fp32 additions cannot hold, so that an accumulator's error grows with the number of
products it adds up, always towards zero.  An fp32 result's accumulators add at most 1024 values of k, 64 steps of 16, and
their sums are joined by rounded additions.  A step cuts off half a unit of the partial sum on average, at most
2^-24 of it; after s of 64 steps that is sqrt(s / 64) of the accumulator's sum: (2/3) 64 2^-24 in all, however long k is.
The joins, rounded to nearest and of both signs, stay below 2^-22.  A gated result is a product of two sums: twice that.
16-bit results: 16384 values of k, so 16 times as much, beside their own rounding, which has no sign.
"""

from __future__ import annotations

import pytest
import torch

ses = pytest.importorskip("sparse_expert_swiglu_gb300")

gpu = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
DRIFT = 2 / 3 * 64 * 2.0 ** -24
JOIN = 2.0 ** -22


@pytest.fixture(scope="module", autouse=True)
def _built():
    ses.build_library()
    ses.lib()


def _product(M, N, K, dtype, gated, layout, out):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    shape = (N, K) if layout == "nk" else (K, N)
    x = torch.randn(M, K, device="cuda", generator=g).to(dtype)
    w = [torch.randn(shape, device="cuda", generator=g).mul_(0.02).to(dtype) for _ in range(1 + gated)]
    y = ses.linear(x, w[0], w_mul=w[1] if gated else None, w_layout=layout, out_dtype=out).double()
    ref = None
    for t in w:
        p = torch.zeros(M, N, dtype=torch.float64, device="cuda")
        for k in range(0, K, 16384):
            a, b = x[:, k:k + 16384].double(), t[:, k:k + 16384] if layout == "nk" else t[k:k + 16384].t()
            p += a @ b.double().t()
        ref = p if ref is None else ref * p
    return y, ref


@gpu
@pytest.mark.parametrize("M,N,K,gated,layout", [
    (1, 4096, 4096, False, "nk"), (1, 256, 262144, False, "nk"), (16, 264, 131072, True, "kn"), (64, 256, 262144, False, "nk"),
    (64, 4096, 16384, True, "nk"), (128, 8192, 4096, False, "nk"), (128, 8192, 4096, False, "kn"), (333, 4096, 4096, False, "nk"),
    (333, 4096, 4096, True, "kn"), (300, 2048, 16384, True, "nk"), (1024, 4095, 4096, False, "nk"), (700, 1031, 16384, True, "nk"),
    (1024, 4096, 16384, False, "kn"), (2048, 2048, 16384, False, "nk"), (2048, 1024, 4096, True, "nk"),
    (2048, 2048, 1032, False, "nk"), (500, 520, 65536, False, "nk"), (2100, 136, 20000, False, "kn")])
def test_fp32_results_of_long_products(M, N, K, gated, layout):
    for dtype in (F16, BF16):
        y, ref = _product(M, N, K, dtype, gated, layout, F32)
        rel = float((y - ref).norm() / ref.norm())
        assert rel <= (1 + gated) * (DRIFT + JOIN), (dtype, rel)


@gpu
@pytest.mark.parametrize("M,N,K,gated,layout", [(1, 256, 262144, False, "nk"), (64, 2048, 131072, False, "kn"),
                                                (333, 1031, 131072, False, "nk"), (2048, 2048, 131072, False, "nk"),
                                                (300, 2048, 131072, True, "nk"), (1024, 512, 262144, True, "kn")])
def test_16_bit_results_of_long_products(M, N, K, gated, layout):
    y, ref = _product(M, N, K, F16, gated, layout, F16)
    drift = float(((y - ref) * ref.sign()).sum() / ref.abs().sum())
    # the mean of n independent roundings of at most 2^-11 each: six times its spread
    assert abs(drift) <= (1 + gated) * 16 * (DRIFT + JOIN) + 6 * 2.0 ** -11 / (M * N) ** 0.5, drift
    assert float((y - ref).norm() / ref.norm()) <= 2.0 ** -11
