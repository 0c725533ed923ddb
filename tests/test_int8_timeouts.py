"""What the 8-bit products' tensor-core kernels do when a wait runs out: they end, the workspace's status says so, and the
next call on the same workspace is right.  The waits run out on the host's word (an arrival that is never made), after 20
rounds of a millisecond."""

from __future__ import annotations

import ctypes

import pytest
import torch

ses = pytest.importorskip("sparse_expert_swiglu_gb300")

from sparse_expert_swiglu_gb300 import _lib  # noqa: E402
from tests.test_int8 import BF16, F32, _linear_case, _linear_check  # noqa: E402

gpu = pytest.mark.gpu

TIMEOUT, INVALID = -6, -1
TRIES = 20


@pytest.fixture(scope="module", autouse=True)
def _built():
    ses.build_library()
    ses.lib()


def _op(M, N, K, x, xs, w, ws, w2, ws2, y, out, gated):
    return _lib._LinearInt8(M, N, K, 3, 1, out, 4 if gated else 0, x, xs, w, ws, w2, ws2, None, None, None, y)


def test_timeout_diagnostic_refuses():
    lib = ses.lib()
    op = _op(4, 64, 64, 0x10000, 0x20000, 0x30000, 0x40000, None, None, 0x50000, 1, False)
    ws = ctypes.c_void_p(0x100000)
    for tries in (0, 4001):
        assert lib.moe_selftest_linear_int8_timeout(ctypes.byref(op), ws, 0, tries, None) == INVALID
    assert lib.moe_selftest_linear_int8_timeout(None, ws, 0, 1, None) == INVALID
    assert lib.moe_selftest_linear_int8_timeout(ctypes.byref(op), ws, 0, 1, None) == -4


@gpu
@pytest.mark.parametrize("M,N,K,gated,out", [
    (1, 512, 128, False, None),             # one stage
    (4, 40000, 512, False, F32),            # more tiles than CTAs
    (20, 512, 8192, True, None),            # a cluster's shares
    (48, 256, 16400, False, F32), (100, 2048, 4096, False, None), (150, 1031, 1008, False, None), (300, 4096, 2064, True, None),
    (300, 512, 14336, False, F32), (1024, 4095, 4096, False, None), (2048, 2048, 512, True, None)])
def test_products_that_give_up(M, N, K, gated, out):
    c = _linear_case(M, N, K, BF16, "int8", "silu" if gated else "none", gated=gated, out=out)
    t = [c[k].cuda() if c[k] is not None else None for k in ("x", "x_scale", "w", "w_scale", "w_mul", "w_mul_scale")]
    ws = ses.Workspace(ses.linear_int8_workspace_bytes(M, N, K, gated))
    y = torch.empty(M, N, dtype=out or BF16, device="cuda")
    op = _op(M, N, K, *(v.data_ptr() if v is not None else None for v in t), y.data_ptr(), 2 if out else 1, gated)
    stream = torch.cuda.current_stream().cuda_stream
    for _ in range(2):
        assert ses.lib().moe_selftest_linear_int8_timeout(ctypes.byref(op), ws.buf.data_ptr(), ws.nbytes, TRIES, stream) == 0
        assert ws.status() == TIMEOUT
        _linear_check(c, ws=ws)
        assert ws.status() == 0
