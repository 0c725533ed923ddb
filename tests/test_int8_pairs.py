"""CTA pairs of the 8-bit products (more than 96 tokens): each CTA of a pair holds half of a tile's tokens in its own shared
memory, and one thread of the first CTA starts the products that read both halves."""

from __future__ import annotations

import ctypes
import time

import pytest
import torch

ses = pytest.importorskip("sparse_expert_swiglu_gb300")
from tests.test_int8 import BF16, F32, _ints, _linear_case, _linear_check  # noqa: E402
from tests.test_int8_timeouts import _op  # noqa: E402

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


@gpu
@pytest.mark.parametrize("M,N,K,gated", [(1024, 4095, 4096, False), (520, 2048, 4096, True), (520, 2048, 14336, False)])
def test_pairs_that_give_up_end(M, N, K, gated):
    """A pair that gives up waits for what is in flight, not for copies that its other CTA never issued: it ends within the time of
    one wait (and no multiple of it by the number of stages), and the next call is right."""
    c = _linear_case(M, N, K, BF16, "int8", "silu" if gated else "none", gated=gated)
    t = [c[k].cuda() if c[k] is not None else None for k in ("x", "x_scale", "w", "w_scale", "w_mul", "w_mul_scale")]
    ws = ses.Workspace(ses.linear_int8_workspace_bytes(M, N, K, gated))
    y = torch.empty(M, N, dtype=BF16, device="cuda")
    op = _op(M, N, K, *(v.data_ptr() if v is not None else None for v in t), y.data_ptr(), 1, gated)
    tries = 1000  # of a millisecond at most: a wait of one thread takes a second
    torch.cuda.synchronize()
    start = time.monotonic()
    stream = torch.cuda.current_stream().cuda_stream
    assert ses.lib().moe_selftest_linear_int8_timeout(ctypes.byref(op), ws.buf.data_ptr(), ws.nbytes, tries, stream) == 0
    torch.cuda.synchronize()
    assert time.monotonic() - start < 2.0
    assert ws.status() == -6
    _linear_check(c, ws=ws)
    assert ws.status() == 0
