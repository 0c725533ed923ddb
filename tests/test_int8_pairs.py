"""CTA pairs of the 8-bit products (more than 96 tokens): each CTA of a pair holds half of a tile's tokens in its own shared
memory, and one thread of the first CTA starts the products that read both halves."""

from __future__ import annotations

import pytest
import torch

ses = pytest.importorskip("sparse_expert_swiglu_gb300")
from tests.test_int8 import BF16, F32, _ints, _linear_case, _linear_check  # noqa: E402

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ses.build_library()
    ses.lib()


@gpu
@pytest.mark.parametrize("M,N,K,gated", [
    (130, 8200, 528, False), (130, 4096, 4096, True), (520, 4096, 4096, False), (520, 2048, 4096, True),  # a tile for each pair
    (300, 1024, 14336, False), (130, 2048, 4096, True), (520, 2048, 14336, False), (130, 4096, 14336, True)])  # ... for each cluster
def test_tokens_that_change_from_call_to_call(M, N, K, gated):
    """Calls without a break whose tokens and scales differ from the call's before: half a tile of tokens that came late
    would show as the ones that lay in the same stages before."""
    c = _linear_case(M, N, K, BF16, "int8", "silu" if gated else "none", gated=gated, out=F32)
    g = torch.Generator().manual_seed(M)
    tokens = [(c["x"].cuda(), c["x_scale"].cuda())]
    want = [_linear_check(c)]
    for _ in range(2):
        new = {**c, "x": _ints(g, (M, K)), "x_scale": torch.rand(M, generator=g) / 32}
        tokens.append((new["x"].cuda(), new["x_scale"].cuda()))
        want.append(_linear_check(new))
    ws = ses.Workspace(ses.linear_int8_workspace_bytes(M, N, K, gated))
    a = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    kw = {k: v for k, v in a.items() if k not in ("x", "x_scale", "w", "w_scale")}
    out, wrong = torch.empty(M, N, device="cuda"), torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(1500):
        x, scale = tokens[i % 3]
        ses.linear_int8(x, a["w"], a["w_scale"], x_scale=scale, out=out, ws=ws, **kw)
        if i % 5 == 4:  # (the calls between have the next one start under them)
            wrong += (out != want[i % 3]).sum()
    assert int(wrong) == 0 and ws.status() == 0
