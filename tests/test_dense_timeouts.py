"""What the kernels on uncompressed weights do when a wait runs out: they end, the workspace's status says so, and the next
call on the same workspace is right.  The waits run out on the host's word (an arrival that is never made), after
20 rounds of a millisecond."""

from __future__ import annotations

import ctypes

import pytest
import torch

ses = pytest.importorskip("sparse_expert_swiglu_gb300")

from sparse_expert_swiglu_gb300 import _lib  # noqa: E402
from tests.test_dense_weights import BF16, F16, _layer_case, _layer_check, _linear_case, _linear_check  # noqa: E402

gpu = pytest.mark.gpu

TIMEOUT, INVALID = -6, -1
TRIES = 20


@pytest.fixture(scope="module", autouse=True)
def _built():
    ses.build_library()
    ses.lib()


def test_timeout_diagnostics_refuse():
    lib = ses.lib()
    v = dict(M=4, N=64, K=64, dtype=0, out_dtype=0, w_layout=0, act=0, x=0x10000, w=0x20000, w_mul=None, bias=None,
             bias_mul=None, residual=None, y=0x30000)
    op = _lib._Linear(*(v[n] for n, _ in _lib._Linear._fields_))
    ws = ctypes.c_void_p(0x100000)
    for tries in (0, 4001):
        assert lib.moe_selftest_linear_timeout(ctypes.byref(op), ws, 0, tries, None) == INVALID
    assert lib.moe_selftest_linear_timeout(None, ws, 0, 1, None) == INVALID
    assert lib.moe_selftest_linear_timeout(ctypes.byref(op), ws, 0, 1, None) == -4
    ex = _lib._DenseExperts(8, 64, 64, 0, 0x1000000, 0x2000000, 0x3000000)
    layer = _lib._DenseLayer(2, 1, 0x4000000, ex, _lib._DenseExperts(0, 64, 64, 0, None, None, None))
    call = lib.moe_selftest_layer_dense_timeout
    for rms, barrier, tries in ((0, 3, 1), (1, 4, 1), (1, -1, 1), (0, 0, 0), (0, 0, 4001)):
        assert call(0x10000, 1, ctypes.byref(layer), 0x30000, rms, barrier, ws, 0, tries, None) == INVALID


@gpu
@pytest.mark.parametrize("M,N,K,gated,layout,out", [
    (1, 1024, 512, False, "nk", None),        # one tile for each CTA
    (4, 40000, 512, False, "nk", torch.float32),   # more tiles than CTAs
    (1, 512, 8192, False, "nk", None),        # a cluster's sums in memory of their own
    (48, 512, 8192, True, "kn", None),        # ... in the stages
    (100, 300, 16384, False, "nk", None), (300, 14336, 512, True, "nk", None),       # pairs
    (592, 744, 6104, False, "kn", None), (1024, 4095, 4096, False, "nk", torch.float32),
    (128, 4096, 16384, False, "nk", torch.float32),
    (2048, 2048, 512, False, "nk", None), (700, 1032, 2048, True, "kn", torch.float32)])
def test_products_that_give_up(M, N, K, gated, layout, out):
    c = _linear_case(M, N, K, BF16, "silu" if gated else "none", gated=gated, layout=layout, out=out)
    x, w = c["x"].cuda(), c["w"].cuda()
    w2 = c["w_mul"].cuda() if gated else None
    ws = ses.Workspace(ses.linear_workspace_bytes(M, N, K, gated))
    y = torch.empty(M, N, dtype=out or BF16, device="cuda")
    op = _lib._Linear(M, N, K, 1, 2 if out else 1, 0 if layout == "nk" else 1, 4 if gated else 0, x.data_ptr(), w.data_ptr(),
                      w2.data_ptr() if gated else None, None, None, None, y.data_ptr())
    stream = torch.cuda.current_stream().cuda_stream
    for _ in range(2):
        assert ses.lib().moe_selftest_linear_timeout(ctypes.byref(op), ws.buf.data_ptr(), ws.nbytes, TRIES, stream) == 0
        assert ws.status() == TIMEOUT
        _linear_check(c, ws=ws)
        assert ws.status() == 0


@gpu
@pytest.mark.parametrize("barrier", [0, 1, 2, 3])
@pytest.mark.parametrize("B,d,f,E,k,ns,dtype", [(1, 512, 1024, 16, 4, 0, BF16), (5, 1032, 520, 8, 2, 1, F16),
                                                (17, 1024, 520, 8, 2, 1, F16), (64, 256, 264, 64, 6, 2, BF16)])
def test_layers_that_give_up(B, d, f, E, k, ns, dtype, barrier):
    """The counts that a layer leaves are zero again, so that the next call's barriers hold."""
    c = _layer_case(B, d, f, E, k, ns, dtype, True, False, True)
    x = c["x"].cuda()
    head = ses.linear_workspace_bytes(1, 1, 8)
    ws = ses.Workspace(ses.layer_dense_workspace_bytes(c["layer"], B))
    y = torch.empty_like(x)
    layer = c["layer"].c_struct()
    want = _layer_check(c)
    stream = torch.cuda.current_stream().cuda_stream
    for _ in range(2):
        assert ses.lib().moe_selftest_layer_dense_timeout(x.data_ptr(), B, ctypes.byref(layer), y.data_ptr(), 1, barrier,
                                                          ws.buf.data_ptr(), ws.nbytes, TRIES, stream) == 0
        assert ws.status() == TIMEOUT
        assert (ws.buf[:head] == 0).all()
        assert torch.equal(_layer_check(c, ws), want)
        assert ws.status() == 0
