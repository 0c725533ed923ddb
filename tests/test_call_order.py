"""Calls behind one another on a stream see what the calls and copies before them wrote, although the kernels start
early: a layer's router weight that the call before it writes, or one further back, is the new one."""

from __future__ import annotations

import pytest
import torch

ses = pytest.importorskip("sparse_expert_swiglu_gb300")
from sparse_expert_swiglu_gb300 import synth  # noqa: E402

gpu = pytest.mark.gpu

F16 = torch.float16


def _layer(d, f, E, k):
    w = synth.experts(E, d, f, 3)
    experts = ses.Experts.from_dense(w.w_up.cuda(), w.gate_t.cuda(), w.down.cuda(), torch.zeros(E, device="cuda"))
    return ses.Layer(torch.zeros(d, E, dtype=F16, device="cuda"), experts, k)


def _routers(d, E, k, x):
    """Two router weights under which every token of x chooses other experts, and the choices."""
    g = torch.Generator().manual_seed(9)
    out = []
    for shift in (0, E // 2):
        wr = torch.randn((d, E), generator=g) * 0.01
        for j in range(k):  # experts shift ... shift + k - 1 win, in this order, for x of one sign
            wr[:, shift + j] += 0.5 - 0.1 * j
        out.append(wr.to(F16).cuda())
    return out, [list(range(s, s + k)) for s in (0, E // 2)]


@gpu
@pytest.mark.parametrize("B,d,path", [(1, 1024, "decode_fused"), (2, 1024, "decode"), (1, 4096, "decode_fused"),
                                      (3, 1024, "decode_pairs"), (8, 1024, "general")])
def test_router_weight_written_two_calls_back(B, d, path):
    """A copy into the router weight, a small product that leaves most SMs free, then the layer."""
    f, E, k = 256, 8, 2
    layer = _layer(d, f, E, k)
    assert ses.layer_path(layer, B) == path
    x = torch.rand(B, d, device="cuda").add_(0.1).to(F16)
    (wrs, choices) = _routers(d, E, k, x)
    small, w = torch.randn(1, 256, device="cuda").to(F16), torch.randn(64, 256, device="cuda").to(F16)
    big = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    got = []
    for i in range(40):
        big.fill_(i)                                # the copy starts late
        layer.w_router.copy_(wrs[i % 2])
        ses.linear(small, w)
        got.append(ses.layer_decode(x, layer, debug=True)[1]["topk_idx"])
    torch.cuda.synchronize()
    for i, idx in enumerate(got):
        assert idx.cpu().tolist() == [choices[i % 2]] * B, i


@gpu
@pytest.mark.parametrize("B,d", [(1, 1024), (2, 1024), (1, 4096), (8, 1024)])
@pytest.mark.parametrize("dense", [False, True])
def test_router_weight_written_by_the_product_before(B, d, dense):
    """The router weight is the result of a product (W R for a fixed [K][E] matrix): it is written by the kernel that the
    layer's starts under."""
    f, E, k, K = 256, 8, 2, 512
    layer = _layer(d, f, E, k)
    if dense:
        g = torch.Generator(device="cuda").manual_seed(2)
        ex = ses.DenseExperts(*(torch.randn(E, f, d, device="cuda", generator=g).to(F16) for _ in range(3)))
        layer = ses.DenseLayer(layer.w_router, ex, k)
    x = torch.rand(B, d, device="cuda").add_(0.1).to(F16)
    wrs, choices = _routers(d, E, k, x)
    a = torch.zeros(d, K, dtype=F16, device="cuda")
    a[:, 0] = 1.0
    # row n of b = expert n's value in every row of the router weight
    bs = []
    for c in choices:
        b = torch.zeros(E, K, dtype=F16, device="cuda")
        for j, e in enumerate(c):
            b[e, 0] = 0.5 - 0.1 * j
        bs.append(b)
    call = ses.layer_dense_decode if dense else ses.layer_decode
    got = []
    for i in range(40):
        ses.linear(a, bs[i % 2], out=layer.w_router)
        got.append(call(x, layer, debug=True)[1]["topk_idx"])
    torch.cuda.synchronize()
    for i, idx in enumerate(got):
        assert idx.cpu().tolist() == [choices[i % 2]] * B, i
