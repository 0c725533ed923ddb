"""residual_norm against a plain implementation in 64 bits, and a decode block of the 8-bit operators together.

Tolerances, elementwise and derived before the first run: every fp32 operation errs by at most U = 2^-24 of its result.  A
mean over d has partial sums of at most 32 values, ten pairwise steps and the division, fewer than 64 roundings in a row:
64 U of the mean magnitude.  _norm64 carries an error of its input through both norms by the product rule; the last rounding
costs half a step of the type.
"""

from __future__ import annotations

import ctypes

import pytest
import torch

ses = pytest.importorskip("sparse_expert_swiglu_gb300")
from sparse_expert_swiglu_gb300 import _lib  # noqa: E402
from sparse_expert_swiglu_gb300._lib import MoeError  # noqa: E402
from tests.test_int8 import _cuda, _ints, _rows64, _within  # noqa: E402

gpu = pytest.mark.gpu

F16, BF16, F32, I8 = torch.float16, torch.bfloat16, torch.float32, torch.int8
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    ses.build_library()
    ses.lib()


def _norm64(v, dv, kind, weight, bias, eps):
    """The norm of v, known to dv, and its error."""
    if kind == "none":
        return v, dv
    if kind == "layer":
        mean = v.mean(1, keepdim=True)
        dv = dv + dv.mean(1, keepdim=True) + 64 * U * v.abs().mean(1, keepdim=True)
        v = v - mean
        dv = dv + U * v.abs()
    ms = (v * v).mean(1, keepdim=True)
    dms = (2 * v.abs() * dv + dv * dv).mean(1, keepdim=True) + 64 * U * ms + 2 * U * (ms + eps)
    ms = ms + eps
    root = torch.sqrt(ms)
    off = dms / ms + 4 * U  # relative, of 1 / root, with room
    y = v / root
    dy = dv / root * (1 + off) + y.abs() * (off + U)
    if weight is not None:
        y, dy = y * weight.double(), dy * weight.double().abs()
        dy = dy + U * y.abs()
    if bias is not None:
        y = y + bias.double()
        dy = dy + U * y.abs()
    return y, dy


def _case(M, d, dtype, post="none", norm="rms", residual=True, wide=False, gate=0, affine=True, scales=(1.0, 1.0), int8=False,
          eps=1e-6, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed + M + 3 * d)

    def vec(on, one=0.0):
        return (one + 0.3 * torch.randn(d, generator=g)).to(dtype) if on and affine else None
    return dict(x=(torch.randn((M, d), generator=g) * std).to(dtype),
                residual=torch.randn((M, d), generator=g).to(F32 if wide else dtype) if residual else None,
                post=post, post_weight=vec(post != "none", 1.0), post_bias=vec(post != "none"),
                gate=(torch.randn((gate, d), generator=g)).to(dtype) if gate else None,
                residual_scale=scales[0], block_scale=scales[1], norm=norm, weight=vec(norm != "none", 1.0),
                bias=vec(norm != "none"), eps=eps, int8=int8)


def _ref(c):
    """(s, its error, y, its error)."""
    x = c["x"].double()
    u, du = _norm64(x, torch.zeros_like(x), c["post"], c["post_weight"], c["post_bias"], c["eps"])
    if c["gate"] is not None:
        g = c["gate"].double().repeat_interleave(len(x) // len(c["gate"]), dim=0)
        u, du = u * g, du * g.abs()
        du = du + U * u.abs()
    bs, rs = (torch.tensor(v, dtype=F32).double().item() for v in (c["block_scale"], c["residual_scale"]))
    s, ds = u * bs, du * abs(bs) + U * (u * bs).abs()
    if c["residual"] is not None:
        s = s + rs * c["residual"].double()
        ds = ds + U * s.abs()
    y, dy = _norm64(s, ds, c["norm"], c["weight"], c["bias"], c["eps"])
    return s, ds, y, dy


def _run(c, **more):
    return ses.residual_norm(**{k: _cuda(v) for k, v in c.items()}, **more)


def _check(c, **more):
    out = _run(c, **more)
    s, ds, y, dy = _ref(c)
    got = list(out) if isinstance(out, tuple) else [out]
    if c["residual"] is not None or c["norm"] == "none":
        kept = got.pop(0)
        assert kept.dtype == (c["residual"].dtype if c["residual"] is not None else c["x"].dtype)
        _within(kept, s, ds, kept.dtype)
    if c["norm"] == "none":
        assert not got
        return out
    if not c["int8"]:
        assert len(got) == 1 and got[0].dtype == c["x"].dtype
        _within(got[0], y, dy, got[0].dtype)
        return out
    q, scale = got[0].cpu().double(), got[1].cpu().double()
    assert got[0].dtype == I8 and got[1].dtype == F32 and got[1].shape == (len(y),)
    m = y.abs().amax(1)
    assert ((scale - m / 127).abs() <= (dy.amax(1) + 2 * U * m) / 127).all()
    # half a step, y's error, and the scale's
    lim = scale[:, None] * 0.5 * (1 + 1e-5) + dy + 2 * dy.amax(1, keepdim=True) + 8 * U * m[:, None]
    assert ((q * scale[:, None] - y).abs() <= lim).all()
    assert (q.abs().amax(1) == torch.where(m > 0, 127, 0)).all()
    return out


@gpu
@pytest.mark.parametrize("M,d", [(1, 8), (3, 16), (2, 72), (5, 264), (9, 1032), (33, 2048), (4, 4096), (3, 4104), (2, 6144),
                                 (3, 8192), (2, 8200), (2, 12288), (2, 16384)])
def test_sizes(M, d):
    for dtype, post, norm, wide in ((F16, "none", "rms", False), (BF16, "rms", "layer", True), (F16, "layer", "none", True),
                                    (BF16, "layer", "rms", False)):
        _check(_case(M, d, dtype, post, norm, wide=wide))
        if d % 16 == 0 and norm != "none":
            _check(_case(M, d, dtype, post, norm, wide=wide, int8=True))


@gpu
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("norm", ["none", "rms", "layer"])
@pytest.mark.parametrize("residual,wide", [(False, False), (True, False), (True, True)])
def test_parts(post, norm, residual, wide):
    for gate in (0, 1, 3, 12):
        for affine in (False, True):
            for scales in ((1.0, 1.0), (0.75, -0.3), (0.0, 2.0)):
                for int8 in (False, True) if norm != "none" else (False,):
                    _check(_case(12, 528, BF16, post, norm, residual, wide, gate, affine, scales, int8, eps=1e-5))


@gpu
def test_gate_of_one_row_and_weights_alone():
    c = _case(6, 256, F16, gate=1)
    a = _run(c)
    b = _run({**c, "gate": c["gate"][0]})
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    for drop in ("weight", "bias"):
        _check({**_case(6, 256, F16, "rms", "layer"), drop: None, "post_" + drop: None})


@gpu
def test_a_large_mean_and_small_values():
    """LayerNorm of values far from zero (the differences from the mean are formed first), rows of zeros and of subnormals."""
    c = _case(7, 1024, F16, norm="layer", affine=False, residual=False)
    c["x"] = (c["x"].double() + 500).to(F16)
    _check(c)
    for norm in ("rms", "layer"):
        c = _case(4, 512, F16, norm=norm, residual=False, eps=1e-5)
        c["x"][0] = 0
        c["x"][1] = (c["x"][1].double() * 2.0 ** -22).to(F16)
        _check(c)
        y = _run(c).cpu()
        assert torch.equal(y[0], c["bias"])
        c = _case(4, 512, F16, norm=norm, residual=False, affine=False, int8=True)
        c["x"][2] = 0
        q, scale = _run(c)
        assert (q[2] == 0).all() and scale[2] == 0
        _check(c)


@gpu
@pytest.mark.parametrize("int8", [False, True])
def test_tokens_without_a_number(int8):
    c = _case(6, 512, BF16, "rms", "rms", int8=int8)
    c["x"][1, 5], c["residual"][4, 100] = float("nan"), float("inf")
    out = [t.cpu() for t in _run(c)]
    keep = torch.tensor([0, 2, 3, 5])
    clean = {**c, "x": c["x"][keep], "residual": c["residual"][keep]}
    for a, b in zip(out, _run(clean)):
        assert torch.equal(a[keep], b.cpu())
    _check(clean)
    if int8:
        assert torch.isnan(out[2][[1, 4]]).all() and (out[1][[1, 4]] == 0).all()
    else:
        assert torch.isnan(out[1][1]).all() and torch.isnan(out[1][4, 100])


@gpu
@pytest.mark.parametrize("d", [264, 8192])
def test_in_place_streams_and_graphs(d):
    for wide in (False, True):
        c = _case(10, d, BF16, "rms", "rms", wide=wide, gate=2)
        want = _run(c)
        x, r = c["x"].cuda(), c["residual"].cuda()
        s, y = _run({**c, "x": x, "residual": r}, residual_out=r, out=x)
        assert s is r and y is x and torch.equal(r, want[0]) and torch.equal(x, want[1])
        a = {k: _cuda(v) for k, v in c.items()}
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            out = _run(a)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(p, q) for p, q in zip(out, want))
        graph, bufs = torch.cuda.CUDAGraph(), [torch.empty_like(t) for t in want]
        with torch.cuda.graph(graph):
            _run(a, residual_out=bufs[0], out=bufs[1])
        new = _case(10, d, BF16, "rms", "rms", wide=wide, gate=2, seed=7)
        for k, v in new.items():
            if isinstance(v, torch.Tensor):
                a[k].copy_(v)
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(bufs, _run(new)))
    x = c["x"].cuda()  # without a residual x itself may become the stream
    s = ses.residual_norm(x, post="rms", norm="none", residual_out=x)
    assert s is x and torch.equal(s, ses.residual_norm(c["x"].cuda(), post="rms", norm="none"))
    empty = ses.residual_norm(x[:0], x[:0])
    assert empty[0].shape == empty[1].shape == (0, d)


@gpu
@pytest.mark.parametrize("n", [1, 5, 70, 300])
def test_a_block_of_the_8_bit_operators(n):
    """A block as a model runs it: residual and norm to 8-bit tokens, a projection of 16-bit values, an expert on 8-bit
    tokens with the residual; the same with each step's input taken from the step before, in a graph too."""
    d, f = 512, 1040
    g = torch.Generator().manual_seed(n)

    def weight(*shape):
        return torch.randn(shape, generator=g) * shape[-1] ** -0.5
    proj = ses.quantize_int8(weight(d, d).cuda())
    ex = ses.Int8Experts(*ses.quantize_int8(weight(1, f, d).cuda()), *ses.quantize_int8(weight(1, f, d).cuda()),
                         *ses.quantize_int8(weight(1, d, f).cuda()))
    w1, w2 = ((1 + 0.1 * torch.randn(d, generator=g)).to(BF16).cuda() for _ in range(2))
    x, stream = (torch.randn((n, d), generator=g).to(BF16).cuda() for _ in range(2))
    ws = ses.Workspace(max(ses.expert_int8_workspace_bytes(n, d, f), ses.linear_int8_workspace_bytes(n, d, d)))

    def block(x, stream):
        a = ses.linear_int8(x, *proj, ws=ws)
        s, q, scale = ses.residual_norm(a, stream, post="rms", post_weight=w1, weight=w2, int8=True)
        return a, s, q, scale, ses.expert_int8_swiglu(q, ex, 0, x_scale=scale, residual=s, dtype=BF16, ws=ws)
    a, s, q, scale, y = block(x, stream)

    # every step against 64 bits on the step's own inputs, to half a bf16 step and fp32's roundings
    def near(got, want, room):
        got = got.cpu().double()
        assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + room).all()
    xq, xs = _rows64(x.cpu())
    # (the integers' sum first: with scaled operands a sum that is zero comes out as 64 bits' rounding errors)
    want = (xq @ proj[0].cpu().double().t()) * xs.double()[:, None] * proj[1].cpu().double()
    near(a, want, 8 * U * want.abs())
    v = a.cpu().double()
    u = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * w1.cpu().double()
    near(s, stream.cpu().double() + u, 256 * U * (u.abs() + stream.cpu().double().abs()))
    one = ses.expert_int8_swiglu(q, ex, 0, x_scale=scale, dtype=BF16)
    # one is off by half a step of the value that y adds, and y by half a step of its own sum, which that moves too
    near(y, s.cpu().double() + one.cpu().double(), 2.0 ** -8 * (1 + 2.0 ** -6) * one.cpu().double().abs())

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = block(x, stream)
    x.copy_(torch.randn((n, d), generator=g).to(BF16))
    graph.replay()
    assert all(torch.equal(p, r) for p, r in zip(out, block(x, stream)))
    assert ws.status() == 0


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

X, RES, GATE, PW, PB, W, B, S, Y, YS = (0x1000000 * (i + 1) for i in range(10))
INVALID, SHAPE, ALIGN = -1, -2, -3


def _c(**more):
    v = dict(M=4, d=64, dtype=0, s_dtype=0, y_dtype=0, post=0, norm=1, gate_rows=0, residual_scale=1, block_scale=1, eps=1e-6,
             x=X, residual=RES, gate=None, post_weight=None, post_bias=None, weight=None, bias=None, s=S, y=Y, y_scale=None)
    v.update(more)
    op = _lib._ResidualNorm(*(v[n] for n, _ in _lib._ResidualNorm._fields_))
    return ses.lib().moe_residual_norm(ctypes.byref(op), None)


def test_refuses_on_the_host():
    assert ses.lib().moe_residual_norm(None, None) == INVALID
    assert _c(M=0) == 0
    i8 = dict(y_dtype=3, y_scale=YS)
    for bad in (dict(M=-1), dict(d=0), dict(dtype=2), dict(s_dtype=1), dict(s_dtype=3), dict(y_dtype=2), dict(y_dtype=1),
                dict(post=3), dict(norm=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(gate_rows=1), dict(gate=GATE),
                dict(gate=GATE, gate_rows=3), dict(gate=GATE, gate_rows=-4), dict(x=None), dict(y=None), dict(norm=0),
                dict(s=None, y=None, norm=0), dict(y_dtype=3), dict(y_scale=YS), dict(post_weight=PW), dict(post_bias=PB),
                dict(norm=0, y=None, weight=W), dict(norm=0, y=None, bias=B)):
        assert _c(**bad) == INVALID, bad
    for bad in (dict(M=(1 << 20) + 1), dict(d=16392), dict(d=68), dict(i8, d=72)):
        assert _c(**bad) == SHAPE, bad
    for bad in (dict(x=X + 8), dict(residual=RES + 2), dict(s=S + 8), dict(y=Y + 8), dict(i8, y_scale=YS + 4),
                dict(gate=GATE + 2, gate_rows=1), dict(weight=W + 2), dict(post=1, post_bias=PB + 8)):
        assert _c(**bad) == ALIGN, bad
    n = 4 * 64 * 2
    for bad in (dict(s=X + 16), dict(s=RES + 16), dict(y=RES), dict(y=X + n - 16), dict(y=S), dict(y=S + n - 16), dict(s=X, s_dtype=2),
                dict(i8, y=X), dict(i8, y_scale=X + 16), dict(i8, y_scale=S), dict(i8, y_scale=Y + 32), dict(i8, y_scale=RES),
                dict(weight=S, s=S), dict(bias=Y), dict(gate=S + 64, gate_rows=1), dict(post=2, post_weight=Y + n - 16),
                dict(i8, weight=YS), dict(s=X, y=X), dict(s=X - 16), dict(s_dtype=2, residual=S + n)):
        assert _c(**bad) == INVALID, bad


@gpu
def test_binding_refusals():
    x = torch.zeros(4, 32, dtype=F16, device="cuda")
    v = x[0]
    for bad in (dict(post="l2"), dict(norm="batch"), dict(norm="none", int8=True), dict(post_weight=v), dict(norm="none", weight=v),
                dict(norm="none", out=x), dict(out_scale=v.float()), dict(residual_out=x), dict(residual=x.to(BF16)),
                dict(residual=x[:2]), dict(gate=x[:3].clone()), dict(gate=v.float()), dict(weight=v[:16]), dict(bias=v.float()),
                dict(out=x.float()), dict(residual=x.t()), dict(gate=x[:0])):
        with pytest.raises((TypeError, ValueError)):
            ses.residual_norm(x, **bad)
    for bad in (x.float(), x[0], x[:, ::2], x.cpu()):
        with pytest.raises((TypeError, ValueError)):
            ses.residual_norm(bad)
    for bad in (dict(out=x, residual_out=x, residual=x), dict(eps=-1.0)):
        with pytest.raises(MoeError) as err:
            ses.residual_norm(x, **bad)
        assert err.value.status == INVALID
    with pytest.raises(MoeError) as err:
        ses.residual_norm(torch.zeros(2, 24, dtype=F16, device="cuda"), int8=True)
    assert err.value.status == SHAPE
