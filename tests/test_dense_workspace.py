"""Workspaces of a dense layer: their size on the device, and that only the counts at their start have to be zero."""

from __future__ import annotations

import pytest
import torch

ses = pytest.importorskip("sparse_expert_swiglu_gb300")

from tests.test_dense_weights import BF16, F16, _layer_case, _layer_check  # noqa: E402

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ses.build_library()
    ses.lib()


@gpu
@pytest.mark.parametrize("B,d,f,E,k,ns,dtype", [
    (64, 256, 264, 64, 6, 2, F16), (1, 512, 1024, 16, 4, 0, BF16), (8, 1032, 520, 8, 2, 1, F16), (9, 200, 136, 60, 8, 2, BF16),
    (17, 1024, 520, 8, 2, 1, F16), (61, 2272, 280, 19, 8, 2, BF16), (63, 1664, 3776, 6, 2, 0, F16), (64, 264, 1160, 5, 5, 8, BF16),
    (33, 4096, 328, 255, 8, 0, F16), (2, 4104, 2048, 12, 3, 2, BF16), (40, 520, 8, 3, 1, 1, F16)])
def test_workspace_of_exact_size_and_any_content(B, d, f, E, k, ns, dtype):
    """NaN in every byte behind the counts, and a guard behind the workspace's last byte."""
    c = _layer_case(B, d, f, E, k, ns, dtype, True, True, True)
    n, head = ses.layer_dense_workspace_bytes(c["layer"], B), ses.linear_workspace_bytes(1, 1, 8)
    assert head < n
    fresh = _layer_check(c)
    ws = ses.Workspace(n + 4096)
    ws.nbytes = n
    for fill in (0xFF, 0x7B):
        ws.buf[head:].fill_(fill)
        y = _layer_check(c, ws)
        assert torch.equal(y, fresh)
        assert (ws.buf[n:] == fill).all()
        assert (ws.buf[:head] == 0).all()
    assert ws.status() == 0


@gpu
def test_a_call_of_its_own_workspace_clears_the_counts_alone():
    c = _layer_case(64, 512, 264, 64, 6, 0, F16, True, False, False)
    x = c["x"].cuda()
    ses.layer_dense_decode(x, c["layer"])
    n = ses.layer_dense_workspace_bytes(c["layer"], 64)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    mark = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    at, end = mark.data_ptr(), n // 4096 * 4096
    del mark
    ws = ses.Workspace(n, clear=ses.linear_workspace_bytes(1, 1, 8))  # the block that was just given back
    assert ws.buf.data_ptr() == at
    assert (ws.buf[:ses.linear_workspace_bytes(1, 1, 8)] == 0).all() and (ws.buf[end - 4096:end] == 0xA5).all()
    assert torch.equal(ses.layer_dense_decode(x, c["layer"], ws=ws), ses.layer_dense_decode(x, c["layer"]))


@gpu
def test_workspace_of_many_experts():
    g = torch.Generator(device="cuda").manual_seed(3)
    E, d, f = 256, 1024, 512
    w = [torch.randn(E, f, d, device="cuda", dtype=BF16, generator=g) * 0.05 for _ in range(3)]
    layer = ses.DenseLayer(torch.randn(d, E, device="cuda", dtype=BF16, generator=g) * 0.05, ses.DenseExperts(*w), 8)
    assert ses.layer_dense_workspace_bytes(layer, 64) < 50e6
    x = torch.randn(64, d, device="cuda", dtype=BF16, generator=g)
    y, dbg = ses.layer_dense_decode(x, layer, debug=True)
    for b in (0, 31, 63):
        ref = torch.zeros(d, dtype=torch.float64, device="cuda")
        for e, p in zip(dbg["topk_idx"][b].tolist(), dbg["topk_w"][b].tolist()):
            gate, up, down = (t[e].double() for t in w)
            a = x[b].double()
            ref += p * ((torch.nn.functional.silu(gate @ a) * (up @ a)) @ down)
        assert float((y[b].double() - ref).norm() / ref.norm()) < 2.0 ** -8
