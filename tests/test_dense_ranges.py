"""The ends of the ranges that the calls on uncompressed weights accept, against 64 bits (tolerances as in
test_dense_weights.py; of large results the first rows, the last ones and some where the offsets pass 2^31 or 2^32)."""

from __future__ import annotations

import pytest
import torch

ses = pytest.importorskip("sparse_expert_swiglu_gb300")

from tests.test_dense_weights import BF16, F16, F32, _act64, _expert_ref, _half_step, _linear_case, _linear_check, _tau, _within  # noqa: E402

gpu = pytest.mark.gpu

MAX_M, MAX_N, MAX_K = 1 << 20, 1 << 20, 1 << 18


@pytest.fixture(scope="module", autouse=True)
def _built():
    ses.build_library()
    ses.lib()


def _randn(shape, dtype, std=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, device="cuda", dtype=dtype, generator=g).mul_(std)


def _rows(M, N, width):
    """Row slices: the ends, and around the element and byte offsets 2^31 and 2^32."""
    at = {0, M - 3}
    for border in (1 << 31, 1 << 32):
        for size in (N, N * width):
            if border // size + 2 < M:
                at.add(border // size - 1)
    return [slice(a, a + 3) for a in sorted(at)]


@gpu
@pytest.mark.parametrize("N,K,gated,layout,dtype,out", [(8, 8, False, "nk", F16, F16), (136, 72, True, "kn", BF16, BF16),
                                                       (7, 264, False, "nk", F16, F32), (2056, 64, True, "nk", F16, F16),
                                                       (2056, 1096, False, "nk", BF16, F32), (2049, 64, False, "nk", F16, F16)])
def test_linear_most_tokens(N, K, gated, layout, dtype, out):
    M, act = MAX_M, "gelu" if gated else "none"
    shape = (N, K) if layout == "nk" else (K, N)
    x, w = _randn((M, K), dtype), _randn(shape, dtype, 0.05, 1)
    w2, b = _randn(shape, dtype, 0.05, 2) if gated else None, _randn((N,), dtype, seed=3)
    r = _randn((M, N), dtype, seed=4)
    y = ses.linear(x, w, bias=b, act=act, w_mul=w2, residual=r, w_layout=layout, out_dtype=out)
    for s in _rows(M, N, out.itemsize):
        xs = x[s].double().cpu()
        ws = [t.double().cpu().t() if layout == "nk" else t.double().cpu() for t in (w, w2) if t is not None]
        a = xs @ ws[0] + b.double().cpu()
        da = _tau(K) * (xs.abs() @ ws[0].abs() + b.double().cpu().abs())
        v = _act64(act, a)
        dv = da if act == "none" else 1.13 * da + 2.0 ** -20 * (v.abs() + a.abs())
        if gated:
            u, du = xs @ ws[1], _tau(K) * (xs.abs() @ ws[1].abs())
            dv = dv * u.abs() + v.abs() * du + dv * du
            v = v * u
        v = v + r[s].double().cpu()
        _within(y[s], v, dv + 2.0 ** -23 * v.abs(), out)


@gpu
@pytest.mark.parametrize("M,K,layout,dtype,out", [(1, 64, "nk", F16, F32), (3, 200, "kn", BF16, BF16), (100, 72, "nk", F16, F16),
                                                  (2100, 64, "kn", BF16, BF16)])
def test_linear_most_outputs(M, K, layout, dtype, out):
    N = MAX_N
    shape = (N, K) if layout == "nk" else (K, N)
    x, w = _randn((M, K), dtype), _randn(shape, dtype, 0.05, 1)
    y = ses.linear(x, w, w_layout=layout, out_dtype=out)
    xs, w64 = x[-3:].double(), (w if layout == "nk" else w.t()).double()
    ref, bound = xs @ w64.t(), _tau(K) * (xs.abs() @ w64.t().abs())
    _within(y[-3:], ref.cpu(), bound.cpu(), out)


@gpu
@pytest.mark.parametrize("M,N,gated,layout", [(1, 1, False, "nk"), (5, 8, True, "kn"), (65, 136, False, "nk"), (300, 264, False, "kn"),
                                              (64, 1000, True, "nk")])
def test_linear_longest_sums(M, N, gated, layout):
    for out in (BF16, F32):
        _linear_check(_linear_case(M, N, MAX_K, BF16, "relu", True, gated, True, layout, out))


@gpu
@pytest.mark.parametrize("d,f", [(8, 8), (72, 136), (2056, 64)])
def test_expert_most_tokens(d, f):
    n = MAX_M
    x, ws = _randn((n, d), BF16), [_randn((2, f, d), BF16, 0.05, 1 + i) for i in range(3)]
    r = _randn((n, d), BF16, seed=9)
    y = ses.expert_dense_swiglu(x, ses.DenseExperts(*ws), 1, residual=r)
    for s in _rows(n, d, 2):
        ref, bound = _expert_ref(x[s].double().cpu(), *(t[1].cpu() for t in ws), BF16, True)
        ref = ref + r[s].double().cpu()
        _within(y[s], ref, bound + 2.0 ** -22 * ref.abs(), BF16)
    with pytest.raises(ValueError):
        ses.expert_dense_swiglu(_randn((n + 1, d), BF16), ses.DenseExperts(*ws), 1)


@gpu
def test_expert_of_the_largest_sizes():
    """d = 16384, f = 65536 and more than 64 tokens: sums of 65536 terms."""
    d, f, n = 16384, 65536, 70
    x, ws = _randn((n, d), BF16), [_randn((1, f, d), BF16, 0.01, 1 + i) for i in range(3)]
    y = ses.expert_dense_swiglu(x, ses.DenseExperts(*ws), 0)
    xd = x[:3].double()
    h = torch.nn.functional.silu(xd @ ws[0][0].double().t()) * (xd @ ws[1][0].double().t())
    ref = h @ ws[2][0].double()
    # h is rounded: half a step of each term, in the root of their squares; then the result's own rounding
    lim = 8 * _half_step(BF16) * 0.01 * float(h.norm(dim=1).max()) + _half_step(BF16) * ref.abs() * 1.01
    assert ((y[:3].double() - ref).abs() <= lim).all()
