"""Outputs and workspaces of the calls on uncompressed weights that lie in the call's own tensors are refused, on the
host, before anything is enqueued."""

from __future__ import annotations

import ctypes

import pytest
import torch

ses = pytest.importorskip("sparse_expert_swiglu_gb300")
from sparse_expert_swiglu_gb300 import _lib  # noqa: E402

gpu = pytest.mark.gpu

D, F, E = 64, 128, 4
STACK = E * F * D * 2
GATE, UP, DOWN, ROUTER, X, RES, Y, WS, SHARED = (0x1000000 * (i + 1) for i in range(9))
INVALID = -1


@pytest.fixture(scope="module", autouse=True)
def _built():
    ses.build_library()


def _stack(gate=GATE, up=UP, down=DOWN):
    return _lib._DenseExperts(E, D, F, 0, gate, up, down)


def _expert(y=Y, ws=WS, ex=None, res=None, ws_bytes=0):  # (0 bytes: nothing is enqueued whatever the checks say)
    return ses.lib().moe_expert_dense_swiglu(X, 2, ctypes.byref(ex or _stack()), 1, res, y, ws, ws_bytes, None)


def _layer(y=Y, ws=WS, ex=None, shared=None):
    empty = _lib._DenseExperts(0, D, F, 0, None, None, None)
    layer = _lib._DenseLayer(2, 1, ROUTER, ex or _stack(), shared or empty)
    return ses.lib().moe_layer_dense_decode(X, 2, ctypes.byref(layer), None, y, 0, None, ws, 0, None)


def test_calls_without_overlaps_pass_these_checks():
    assert _expert() != INVALID and _layer() != INVALID
    assert _expert(y=GATE + STACK) != INVALID and _layer(y=DOWN + STACK) != INVALID  # right behind the rows


@pytest.mark.parametrize("y", [GATE, GATE + STACK - 16, GATE - 2 * D * 2 + 16, UP, UP + STACK - 16, DOWN + 1024, DOWN + STACK - 16])
def test_output_in_the_experts(y):
    assert _expert(y=y) == INVALID
    assert _layer(y=y) == INVALID


def test_output_in_interleaved_rows():
    both = _stack(down=GATE + 2 * D)
    for y in (GATE, GATE + 2 * STACK - 16, GATE + STACK + 2 * D):
        assert _expert(y=y, ex=both) == INVALID
        assert _layer(y=y, ex=both) == INVALID
    assert _expert(y=GATE + 2 * STACK, ex=both) != INVALID
    assert _layer(y=GATE + 2 * STACK, ex=both) != INVALID


def test_output_in_the_router_and_in_shared_experts():
    assert _layer(y=ROUTER) == INVALID
    assert _layer(y=ROUTER + D * E * 2 - 16) == INVALID
    assert _layer(y=ROUTER + D * E * 2) != INVALID
    shared = _stack(SHARED, SHARED + STACK, SHARED + 2 * STACK)
    for y in (SHARED, SHARED + STACK + 64, SHARED + 3 * STACK - 16):
        assert _layer(y=y, shared=shared) == INVALID
    assert _layer(y=SHARED + 3 * STACK, shared=shared) != INVALID


@pytest.mark.parametrize("ws", [X, Y, RES, GATE, UP + 256, DOWN + STACK - 256])
def test_workspace_in_the_tensors_of_an_expert(ws):
    assert _expert(ws=ws, res=RES, ws_bytes=1 << 20) == INVALID
    assert _expert(ws=Y - 256, res=RES, ws_bytes=1 << 20) == INVALID


@pytest.mark.parametrize("ws", ["x", "w", "w_mul", "bias", "bias_mul", "residual", "y"])
def test_workspace_in_the_tensors_of_a_product(ws):
    at = dict(x=X, w=GATE, w_mul=UP, bias=ROUTER, bias_mul=ROUTER + 256, residual=RES, y=Y)
    v = dict(M=4, N=64, K=64, dtype=0, out_dtype=0, w_layout=0, act=0, **at)
    op = _lib._Linear(*(v[n] for n, _ in _lib._Linear._fields_))
    assert ses.lib().moe_linear(ctypes.byref(op), at[ws], 1 << 20, None) == INVALID
    assert ses.lib().moe_linear(ctypes.byref(op), WS, 0, None) != INVALID


@gpu
def test_refusals_on_the_device():
    """A layer's workspace size depends on the device; the output in the last expert's down rows, through the binding."""
    dt = torch.float16
    buf = torch.zeros(3 * E * F * D + D * E, dtype=dt, device="cuda")
    gate, up, down = (buf[i * E * F * D:(i + 1) * E * F * D].view(E, F, D) for i in range(3))
    router = buf[3 * E * F * D:].view(D, E)
    ex = ses.DenseExperts(gate, up, down)
    layer = ses.DenseLayer(router, ex, 2)
    x = torch.zeros(2, D, dtype=dt, device="cuda")
    before = buf.clone()
    for out in (down[E - 1, F - 2:], gate[0, :2], up[2, 3:5]):
        for call in (lambda: ses.expert_dense_swiglu(x, ex, 0, out=out), lambda: ses.layer_dense_decode(x, layer, out=out)):
            with pytest.raises(_lib.MoeError) as err:
                call()
            assert err.value.status == INVALID
    ws = ses.Workspace(ses.layer_dense_workspace_bytes(layer, 2))
    inside = ws.buf[4096:4096 + x.numel() * 2].view(dt).view(2, D)
    with pytest.raises(_lib.MoeError) as err:
        ses.layer_dense_decode(x, layer, ws=ws, out=inside)
    assert err.value.status == INVALID
    assert torch.equal(before, buf) and ws.status() == 0
    assert ses.layer_dense_decode(x, layer, ws=ws).shape == (2, D)
