"""Operators on 8-bit integers (quantize_int8, linear_int8, expert_int8_swiglu) against plain implementations in 64 bits.

Tolerances, elementwise and derived before the first run.  Quantised rows are exact: a quotient 127 x / m of two numbers of
at most 24 bits is no nearer to a half than 2^-26 of itself unless it is one, so that 64 bits decide it.  Sums over k are
exact integers.  A product then has three roundings to fp32 (the sum, the scales' product, their product): 3 * 2^-24 of it,
and the bias one more.  The activations have slopes up to 1.13 and a relative error of 2^-20 of their own; the last rounding
costs half a step.
"""

from __future__ import annotations

import ctypes

import pytest
import torch

ses = pytest.importorskip("sparse_expert_swiglu_gb300")
from sparse_expert_swiglu_gb300 import _lib  # noqa: E402
from sparse_expert_swiglu_gb300._lib import MoeError  # noqa: E402

gpu = pytest.mark.gpu

F16, BF16, F32, I8 = torch.float16, torch.bfloat16, torch.float32, torch.int8
U = 2.0 ** -24  # a rounding to fp32


@pytest.fixture(scope="module", autouse=True)
def _built():
    ses.build_library()
    ses.lib()


def _cuda(t):
    return t.cuda() if isinstance(t, torch.Tensor) else t


def _act64(name, a):
    f = torch.nn.functional
    return {"none": lambda v: v, "relu": f.relu, "gelu": f.gelu, "gelu_tanh": lambda v: f.gelu(v, approximate="tanh"),
            "silu": f.silu}[name](a)


def _within(y, ref, bound, dtype):
    y = y.cpu().double()
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    lim = bound + torch.finfo(dtype).eps / 2 * ref.abs() * (1 + 2.0 ** -10) + tiny
    bad = ~((y - ref).abs() <= lim)
    assert not bad.any(), (int(bad.sum()), float(((y - ref).abs() - lim)[bad].max()))


def _rows64(x):
    """q and scale (fp32) of finite rows."""
    m = x.double().abs().amax(-1, keepdim=True)
    q = torch.round(x.double() * 127 / torch.where(m == 0, 1.0, m))
    return q, (m[..., 0].float() / 127)


# ---------------------------------------------------------------------------
# quantize_int8
# ---------------------------------------------------------------------------

def _quantize_check(x):
    q, scale = ses.quantize_int8(x.cuda())
    want, want_scale = _rows64(x)
    assert q.dtype == I8 and scale.dtype == F32 and q.shape == x.shape and scale.shape == x.shape[:-1]
    assert torch.equal(q.cpu().double(), want)
    assert torch.equal(scale.cpu(), want_scale)


@gpu
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,K", [(1, 16), (7, 48), (9, 512), (33, 1008), (5, 4096), (3, 14336), (2, 16400), (2, 40976),
                                    (2, 65536)])
def test_quantize_sizes(rows, K, dtype):
    g = torch.Generator().manual_seed(rows + K)
    _quantize_check(torch.randn((rows, K), generator=g).to(dtype))


@gpu
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_quantize_halves(dtype):
    """Quotients that are halves exactly, and their neighbours in the type: every row's largest value is 127 * 2^e or twice
    that, so that odd multiples of 2^(e-1) are halves."""
    rows = []
    for e in (-3, 0, 4):
        for top in (127.0, 254.0):
            k = torch.arange(-126, 127, dtype=torch.float64)
            half = ((k + 0.5) * (top / 127) * 2.0 ** e).to(dtype)
            near = [half, torch.nextafter(half.float(), torch.tensor(1e9)).to(dtype),
                    torch.nextafter(half.float(), torch.tensor(-1e9)).to(dtype)]
            v = torch.cat([*near, torch.tensor([top * 2.0 ** e, 0.0, -top * 2.0 ** e]).to(dtype)])
            rows.append(torch.nn.functional.pad(v, (0, -len(v) % 16)))
    # ... and largest values without such a factor
    g = torch.Generator().manual_seed(5)
    for _ in range(40):
        m = (torch.rand((), generator=g).double() + 0.5).to(dtype)
        v = ((torch.arange(-127, 127).double() + 0.5) * m.double() / 127).to(dtype)
        v = torch.cat([v, m[None], -m[None]])
        rows.append(torch.nn.functional.pad(v, (0, len(rows[0]) - len(v))))
    _quantize_check(torch.stack(rows))


@gpu
def test_quantize_ends_of_the_types():
    for dtype in (F16, BF16, F32):
        fi = torch.finfo(dtype)
        sub = fi.smallest_normal * fi.eps
        for m in (fi.max, fi.smallest_normal, sub, sub * 5, fi.smallest_normal * 3, 1.0):
            v = torch.linspace(-1, 1, 64).double() * m
            v[0] = m
            _quantize_check(v.to(dtype)[None])
    _quantize_check(torch.zeros(3, 32, dtype=BF16))
    x = torch.randn(6, 32).to(F16)
    x[1, 3], x[3, 0], x[4, 31] = float("inf"), float("nan"), -float("inf")
    q, scale = ses.quantize_int8(x.cuda())
    bad = torch.tensor([1, 3, 4])
    assert torch.isnan(scale.cpu()[bad]).all() and (q.cpu()[bad] == 0).all()
    good = torch.tensor([0, 2, 5])
    want, ws = _rows64(x[good])
    assert torch.equal(q.cpu()[good].double(), want) and torch.equal(scale.cpu()[good], ws)


@gpu
def test_quantize_outputs_and_leading_dimensions():
    x = torch.randn(2, 5, 48).to(BF16)
    _quantize_check(x)
    q, s = torch.empty(2, 5, 48, dtype=I8, device="cuda"), torch.empty(2, 5, device="cuda")
    a, b = ses.quantize_int8(x.cuda(), out=q, out_scale=s)
    assert a is q and b is s and torch.equal(q.cpu().double(), _rows64(x)[0])
    a, b = ses.quantize_int8(torch.empty(0, 48, dtype=F16, device="cuda"))
    assert a.shape == (0, 48) and b.shape == (0,)


# ---------------------------------------------------------------------------
# linear_int8
# ---------------------------------------------------------------------------

def _ints(g, shape):
    return torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)


def _linear_case(M, N, K, dtype, x="int8", act="none", bias=False, gated=False, residual=False, out=None, seed=0):
    g = torch.Generator().manual_seed(seed + M + 3 * N + 7 * K)
    c = dict(w=_ints(g, (N, K)), w_scale=torch.rand(N, generator=g) / (127 * K ** 0.5), act=act, dtype=dtype, out_dtype=out)
    if x == "int8":
        c.update(x=_ints(g, (M, K)), x_scale=torch.rand(M, generator=g) / 32)
    else:
        c.update(x=torch.randn((M, K), generator=g).to(dtype), x_scale=None)
    c["w_mul"] = _ints(g, (N, K)) if gated else None
    c["w_mul_scale"] = torch.rand(N, generator=g) / (127 * K ** 0.5) if gated else None
    c["bias"] = torch.randn(N, generator=g).to(dtype) if bias else None
    c["bias_mul"] = torch.randn(N, generator=g).to(dtype) if bias and gated else None
    c["residual"] = torch.randn((M, N), generator=g).to(dtype) if residual else None
    return c


def _product64(q, xs, w, ws, b):
    a = (q @ w.double().t()) * xs.double()[:, None] * ws.double()
    if b is None:
        return a, 3 * U * a.abs()
    y = a + b.double()
    return y, 3 * U * a.abs() + U * y.abs()


def _gated64(c, q, xs):
    a, da = _product64(q, xs, c["w"], c["w_scale"], c["bias"])
    y = _act64(c["act"], a)
    dy = da if c["act"] in ("none", "relu") else 1.13 * da + 2.0 ** -20 * (y.abs() + a.abs())
    if c["w_mul"] is not None:
        u, du = _product64(q, xs, c["w_mul"], c["w_mul_scale"], c["bias_mul"])
        dy = dy * u.abs() + y.abs() * du + dy * du
        y = y * u
        dy = dy + U * y.abs()
    return y, dy * (1 + 1e-6)


def _linear_ref(c):
    q, xs = (c["x"].double(), c["x_scale"]) if c["x_scale"] is not None else _rows64(c["x"])
    y, dy = _gated64(c, q, xs)
    if c["residual"] is not None:
        y = y + c["residual"].double()
        dy = dy + U * y.abs()
    return y, dy


def _linear_run(c, **more):
    kw = {k: _cuda(v) for k, v in c.items() if k not in ("x", "w", "w_scale")}
    return ses.linear_int8(_cuda(c["x"]), _cuda(c["w"]), _cuda(c["w_scale"]), **kw, **more)


def _linear_check(c, **more):
    y = _linear_run(c, **more)
    ref, bound = _linear_ref(c)
    assert y.dtype == (c["out_dtype"] or c["dtype"]) and y.shape == ref.shape
    _within(y, ref, bound, y.dtype)
    return y


SIZES = [(1, 128, 64), (1, 1, 16), (2, 7, 48), (3, 40, 112), (4, 257, 1008), (5, 1031, 528), (8, 333, 2064), (9, 64, 4096),
         (16, 256, 128), (17, 264, 1008), (31, 129, 160), (33, 1000, 8192), (64, 2048, 272), (130, 1032, 528), (257, 136, 64),
         (333, 648, 2064)]


@gpu
@pytest.mark.parametrize("x", ["int8", "16 bits"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_sizes(M, N, K, x):
    _linear_check(_linear_case(M, N, K, F16, x, out=F32))
    _linear_check(_linear_case(M, N, K, BF16, x, "silu", gated=True))


@gpu
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M", [1, 3, 21, 140])
def test_linear_epilogues(act, gated, M):
    for dtype, out in ((F16, None), (BF16, None), (F16, F32), (BF16, F32)):
        for bias, residual in ((False, False), (True, False), (True, True)):
            _linear_check(_linear_case(M, 200, 272, dtype, "int8", act, bias, gated, residual, out))


@gpu
@pytest.mark.parametrize("M", [1, 4, 7, 12, 48, 100, 300])
@pytest.mark.parametrize("N", [64, 1000, 4096])
def test_linear_long_rows(M, N):
    """A long k over few outputs, which several warps or CTAs share; the largest K."""
    for K in (14336, 16400) if N > 64 else (14336, 65536):
        for x in ("int8", "16 bits"):
            c = _linear_case(M, N, K, BF16, x, residual=True, out=F32)
            y = _linear_check(c)
            assert torch.equal(y, _linear_run(c))


@gpu
@pytest.mark.parametrize("M", [1, 2, 6, 16, 40, 200, 600])
def test_linear_sums_are_exact(M):
    """Sums far above 2^24, and such as cancel to a small number at the end."""
    for K in (1024, 4096, 65536):
        x, w = torch.full((M, K), 127, dtype=I8), torch.full((130, K), 127, dtype=I8)
        w[1], w[2, K // 2:], w[3, K // 2:] = -127, -127, -127
        w[3, K - 5] = -126
        w[4], x[M - 1] = -128, -128
        w[5, 1::2] = -127
        w[6] = torch.arange(K).remainder(255).sub(127).to(I8)
        one, ones = torch.ones(M), torch.ones(130)
        y = ses.linear_int8(x.cuda(), w.cuda(), ones.cuda(), one.cuda(), dtype=F16, out_dtype=F32).cpu()
        want = (x.double() @ w.double().t()).float()  # the sum, rounded once
        assert torch.equal(y, want)


@gpu
def test_linear_results_do_not_depend_on_the_batch():
    """A token's values have the same bits alone, in a batch and in a prompt, whatever plan the sizes take."""
    g = torch.Generator().manual_seed(3)
    M, N, K = 700, 1031, 2064
    x, w, ws = _ints(g, (M, K)).cuda(), _ints(g, (N, K)).cuda(), torch.rand(N, generator=g).cuda()
    xs, bias = torch.rand(M, generator=g).cuda(), torch.randn(N, generator=g).half().cuda()
    full = ses.linear_int8(x, w, ws, xs, bias=bias, act="gelu", dtype=F16, out_dtype=F32)
    for n in (1, 2, 4, 8, 15, 33, 90, 257):
        some = ses.linear_int8(x[:n], w, ws, xs[:n], bias=bias, act="gelu", dtype=F16, out_dtype=F32)
        assert torch.equal(some, full[:n])


@gpu
@pytest.mark.parametrize("M", [2, 20, 150])
def test_linear_values_without_a_number(M):
    """A token with NaN or infinity spoils its own row alone; a row of zeros gives the bias; large values round to
    infinity."""
    c = _linear_case(M, 130, 256, F16, "16 bits", bias=True)
    c["x"][1, 100] = float("nan")
    c["x"][0] = 0
    y = _linear_run(c).cpu()
    assert torch.isnan(y[1]).all() and torch.equal(y[0], c["bias"])
    keep = [i for i in range(M) if i != 1]
    ref, bound = _linear_ref({**c, "x": c["x"][keep]})
    _within(y[keep], ref, bound, F16)
    c = _linear_case(M, 130, 256, F16)
    c["x_scale"][:] = 1e4
    ref = _linear_ref(c)[0]
    y = _linear_run(c).cpu()
    big = ref.abs() > 70000
    assert big.any() and torch.isinf(y[big]).all()


@gpu
@pytest.mark.parametrize("M", [1, 3, 30, 300])
def test_linear_in_place_streams_and_graphs(M):
    """The residual's tensor as output; another stream; a captured call, replayed with new inputs; two calls on one
    workspace."""
    c = _linear_case(M, 520, 1040, BF16, "16 bits", "silu", True, True, True)
    want = _linear_run(c)
    res = _cuda(c["residual"])
    got = _linear_run({**c, "residual": res}, out=res)
    assert got is res and torch.equal(got, want)
    ws = ses.Workspace(ses.linear_int8_workspace_bytes(M, 520, 1040, True))
    a = {k: _cuda(v) for k, v in c.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first, second = _linear_run(a, ws=ws), _linear_run(a, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, want) and torch.equal(second, want)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    with torch.cuda.graph(graph):
        _linear_run(a, ws=ws, out=out)
    for seed in (1, 2):
        new = _linear_case(M, 520, 1040, BF16, "16 bits", "silu", True, True, True, seed=seed)
        for k, v in new.items():
            if isinstance(v, torch.Tensor):
                a[k].copy_(v)
        graph.replay()
        assert torch.equal(out, _linear_run(new))
    assert ws.status() == 0


@gpu
@pytest.mark.parametrize("M,N,K,gated,calls", [(4, 32000, 4096, False, 20000), (40, 2048, 2048, True, 20000),
                                               (300, 1024, 14336, False, 10000), (100, 4096, 4096, False, 10000)])
def test_linear_many_calls_in_a_row(M, N, K, gated, calls):
    """Thousands of calls without a break: every one ends by itself, and the last one's result is the first one's."""
    c = _linear_case(M, N, K, F16, "int8", "silu" if gated else "none", gated=gated, out=F32)
    a = {k: _cuda(v) for k, v in c.items()}
    ws = ses.Workspace(ses.linear_int8_workspace_bytes(M, N, K, gated))
    first, out = _linear_check(c, ws=ws), torch.empty(M, N, device="cuda")
    kw = {k: v for k, v in a.items() if k not in ("x", "w", "w_scale")}
    for i in range(calls):
        ses.linear_int8(a["x"], a["w"], a["w_scale"], out=out, ws=ws, **kw)
    assert ws.status() == 0 and torch.equal(out, first)


@gpu
def test_linear_output_behind_2_to_the_31():
    M, N, K = 65537, 40000, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randint(-127, 128, (M, K), device="cuda", dtype=I8, generator=g)
    w = torch.randint(-127, 128, (N, K), device="cuda", dtype=I8, generator=g)
    xs, ws = torch.rand(M, device="cuda") / 100, torch.rand(N, device="cuda") / 100
    y = ses.linear_int8(x, w, ws, xs, dtype=F16)
    for rows in (slice(0, 3), slice(53685, 53690), slice(M - 3, M)):  # 53687 * 40000 crosses 2^31
        ref, bound = _product64(x[rows].cpu().double(), xs[rows].cpu(), w.cpu(), ws.cpu(), None)
        _within(y[rows], ref, bound, F16)


# ---------------------------------------------------------------------------
# expert_int8_swiglu
# ---------------------------------------------------------------------------

def _expert_case(n, d, f, dtype, x="int8", residual=False, E=3, seed=0):
    g = torch.Generator().manual_seed(seed + n + 3 * d + 7 * f)
    w = [_ints(g, (E, f, d)), torch.rand((E, f), generator=g) / (64 * d ** 0.5), _ints(g, (E, f, d)),
         torch.rand((E, f), generator=g) / (64 * d ** 0.5), _ints(g, (E, d, f)), torch.rand((E, d), generator=g) / (64 * f ** 0.5)]
    c = dict(w=w, dtype=dtype, residual=torch.randn((n, d), generator=g).to(dtype) if residual else None)
    if x == "int8":
        c.update(x=_ints(g, (n, d)), x_scale=torch.rand(n, generator=g) / 32)
    else:
        c.update(x=torch.randn((n, d), generator=g).to(dtype), x_scale=None)
    return c


def _expert_ref(c, e):
    """y and its bound: h's integers may be one off where the quotient lies within h's error of a half, and their scale
    errs as the largest h does."""
    q, xs = (c["x"].double(), c["x_scale"]) if c["x_scale"] is not None else _rows64(c["x"])
    g, gs, u, us, dn, ds = (t[e] for t in c["w"])
    h, dh = _gated64(dict(w=g, w_scale=gs, w_mul=u, w_mul_scale=us, bias=None, bias_mul=None, act="silu"), q, xs)
    m = h.abs().amax(1, keepdim=True)
    off = (dh.amax(1, keepdim=True) / m)  # of the scale, relative
    step = torch.where(m == 0, 0.0, h * 127 / torch.where(m == 0, 1.0, m))
    hq = torch.round(step)
    close = ((step - torch.floor(step) - 0.5).abs() <= 127 * dh / m + step.abs() * off + 1e-12).double()
    s = m / 127
    a, mag = (hq * s) @ dn.double().t(), (hq.abs() * s) @ dn.double().abs().t()
    y = a * ds.double()
    # a changed integer moves the sum by one step of its weight; a change of the scale moves all of it
    dy = ((close * s) @ dn.double().abs().t() + mag * off) * ds.double() + 4 * U * y.abs()
    if c["residual"] is not None:
        y = y + c["residual"].double()
        dy = dy + U * y.abs()
    return y, dy


def _expert_run(c, e, **more):
    ex = ses.Int8Experts(*(t.cuda() for t in c["w"]))
    return ses.expert_int8_swiglu(_cuda(c["x"]), ex, e, x_scale=_cuda(c["x_scale"]), residual=_cuda(c["residual"]),
                                  dtype=c["dtype"], **more)


@gpu
@pytest.mark.parametrize("n,d,f", [(1, 64, 48), (1, 2048, 1408), (2, 256, 528), (4, 1040, 272), (7, 512, 1024), (20, 528, 80),
                                   (64, 256, 2064), (130, 400, 1008), (300, 1024, 512)])
def test_expert(n, d, f):
    for dtype, x, residual in ((F16, "int8", False), (BF16, "16 bits", True), (F16, "16 bits", True), (BF16, "int8", False)):
        c = _expert_case(n, d, f, dtype, x, residual)
        for e in (0, 2):
            y = _expert_run(c, e)
            ref, bound = _expert_ref(c, e)
            assert y.dtype == dtype and y.shape == (n, d)
            _within(y, ref, bound, dtype)


@gpu
@pytest.mark.parametrize("n", [1, 3, 40, 200])
def test_expert_buffers_and_graphs(n):
    d, f = 512, 784
    c = _expert_case(n, d, f, BF16, "16 bits", True)
    want = _expert_run(c, 1)
    x = c["x"].cuda()
    assert torch.equal(_expert_run({**c, "x": x}, 1, out=x), want)
    r = c["residual"].cuda()
    assert torch.equal(_expert_run({**c, "residual": r}, 1, out=r), want)
    ws = ses.Workspace(ses.expert_int8_workspace_bytes(n, d, f))
    a = {**c, "w": [t.cuda() for t in c["w"]], "x": c["x"].cuda(), "residual": c["residual"].cuda()}
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _expert_run(a, 1, ws=ws, out=out)
    new = _expert_case(n, d, f, BF16, "16 bits", True, seed=9)
    for to, v in zip([*a["w"], a["x"], a["residual"]], [*new["w"], new["x"], new["residual"]]):
        to.copy_(v)
    graph.replay()
    assert torch.equal(out, _expert_run(new, 1)) and ws.status() == 0


@gpu
def test_expert_tokens_without_a_number():
    """A token with NaN spoils its own row alone; a token of zeros gives the residual."""
    for n in (3, 40):
        c = _expert_case(n, 256, 528, F16, "16 bits", True)
        c["x"][1, 7] = float("nan")
        c["x"][2] = 0
        y = _expert_run(c, 0).cpu()
        assert torch.isnan(y[1]).all() and torch.equal(y[2], c["residual"][2])
        keep = [i for i in range(n) if i not in (1, 2)]
        ref, bound = _expert_ref({**c, "x": c["x"][keep], "residual": c["residual"][keep]}, 0)
        _within(y[keep], ref, bound, F16)


@gpu
def test_expert_from_uncompressed_experts():
    """from_dense keeps the expert's function up to the steps of its integers."""
    g = torch.Generator().manual_seed(1)
    w = [(torch.randn((2, f, 256), generator=g) * 0.05).to(BF16) for f in (528, 528, 528)]
    dense = ses.DenseExperts(*(t.cuda() for t in w))
    ex = ses.Int8Experts.from_dense(dense)
    for t, want in zip((ex.gate_t, ex.up_t, ex.down_t), (w[0], w[1], w[2].transpose(1, 2))):
        assert torch.equal(t.cpu().double(), _rows64(want)[0])
    x = torch.randn((5, 256), generator=g).to(BF16).cuda()
    a, b = ses.expert_int8_swiglu(x, ex, 1).double(), ses.expert_dense_swiglu(x, dense, 1).double()
    # each of the five quantised operands errs by at most half a step, m / 254, uniformly: with m below 4.5 standard
    # deviations 4.5 / 254 / sqrt(3) = 1.02 % of their norm each; x's and h's reach y through both factors of h
    assert float((a - b).norm() / b.norm()) <= 0.0102 * (2 + 1 + 1 + 1 + 1)


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

X, XS, W, WS_, W2, WS2, BIAS, BIAS2, RES, Y, WORK = (0x1000000 * (i + 1) for i in range(11))
INVALID, SHAPE, ALIGN, SMALL = -1, -2, -3, -4


def _c_linear(ws=WORK, ws_bytes=0, **more):
    v = dict(M=4, N=64, K=64, x_dtype=3, dtype=0, out_dtype=0, act=0, x=X, x_scale=XS, w=W, w_scale=WS_, w_mul=None,
             w_mul_scale=None, bias=None, bias_mul=None, residual=None, y=Y)
    v.update(more)
    op = _lib._LinearInt8(*(v[n] for n, _ in _lib._LinearInt8._fields_))
    return ses.lib().moe_linear_int8(ctypes.byref(op), ws, ws_bytes, None)


def test_linear_refuses_on_the_host():
    assert ses.lib().moe_linear_int8(None, WORK, 1 << 20, None) == INVALID
    assert _c_linear() == SMALL  # the checks pass
    assert _c_linear(M=0) == 0
    gated = dict(w_mul=W2, w_mul_scale=WS2)
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(x_dtype=2), dict(x_dtype=1, x_scale=None), dict(dtype=2), dict(dtype=3),
                dict(out_dtype=1), dict(out_dtype=3), dict(act=5), dict(act=-1), dict(x=None), dict(w=None), dict(w_scale=None),
                dict(y=None), dict(ws=None), dict(x_scale=None), dict(x_dtype=0), dict(w_mul=W2), dict(w_mul_scale=WS2),
                dict(bias_mul=BIAS2)):
        assert _c_linear(**bad) == INVALID, bad
    for bad in (dict(M=(1 << 20) + 1), dict(N=(1 << 20) + 1), dict(K=65552), dict(K=72)):
        assert _c_linear(**bad) == SHAPE, bad
    for bad in (dict(x=X + 8), dict(x_scale=XS + 4), dict(w=W + 8), dict(w_scale=WS_ + 4), dict(y=Y + 2), dict(ws=WORK + 16),
                dict(bias=BIAS + 2), dict(residual=RES + 8), dict(gated, w_mul=W2 + 1), dict(gated, w_mul_scale=WS2 + 4),
                dict(gated, bias_mul=BIAS2 + 2)):
        assert _c_linear(**bad) == ALIGN, bad
    for bad in (dict(y=X), dict(y=X + 240), dict(y=X - 496), dict(y=XS), dict(y=W + 64 * 64 - 16), dict(y=WS_ + 240),
                dict(gated, y=W2), dict(gated, y=WS2), dict(y=BIAS, bias=BIAS), dict(residual=Y + 16),
                dict(residual=Y, out_dtype=2), dict(gated, y=BIAS2, bias_mul=BIAS2)):
        assert _c_linear(**bad) == INVALID, bad
    assert _c_linear(residual=Y) == SMALL and _c_linear(y=X + 256) == SMALL
    for at in (X, XS, W, WS_, W2, WS2, BIAS, BIAS2, RES, Y):
        assert _c_linear(ws=at, ws_bytes=1 << 23, w_mul=W2, w_mul_scale=WS2, bias=BIAS, bias_mul=BIAS2, residual=RES) == INVALID


def _c_expert(ws=WORK, ws_bytes=0, x=X, xs=XS, x_dtype=3, dtype=0, n=2, expert=1, residual=None, y=Y, **more):
    v = dict(E=4, d=64, f=128, gate_t=W, gate_scale=WS_, up_t=W2, up_scale=WS2, down_t=BIAS, down_scale=BIAS2)
    v.update(more)
    ex = _lib._Int8Experts(*(v[k] for k, _ in _lib._Int8Experts._fields_))
    return ses.lib().moe_expert_int8_swiglu(x, xs, x_dtype, dtype, n, ctypes.byref(ex), expert, residual, y, ws, ws_bytes, None)


def test_expert_refuses_on_the_host():
    assert _c_expert() == SMALL and _c_expert(n=0) == 0
    for bad in (dict(n=-1), dict(dtype=2), dict(x_dtype=1), dict(expert=-1), dict(expert=4), dict(E=-1), dict(d=0), dict(f=-16),
                dict(x=None), dict(y=None), dict(xs=None), dict(x_dtype=0), dict(ws=None), dict(gate_t=None), dict(up_scale=None),
                dict(down_scale=None), dict(y=W + 4 * 64 * 128 - 16), dict(y=WS2), dict(y=BIAS2), dict(y=X), dict(y=XS),
                dict(residual=Y + 32)):
        assert _c_expert(**bad) == INVALID, bad
    for bad in (dict(d=72), dict(f=136), dict(d=16400), dict(f=65552), dict(n=(1 << 20) + 1), dict(E=257), dict(E=0)):
        assert _c_expert(**bad) == SHAPE, bad
    for bad in (dict(x=X + 8), dict(y=Y + 8), dict(up_t=W2 + 8), dict(down_scale=BIAS2 + 4), dict(ws=WORK + 16), dict(xs=XS + 4)):
        assert _c_expert(**bad) == ALIGN, bad
    assert _c_expert(x_dtype=0, xs=None, y=X) == SMALL and _c_expert(residual=Y) == SMALL
    for at in (X, XS, W, WS_, W2, WS2, BIAS, BIAS2, RES, Y):
        assert _c_expert(ws=at, ws_bytes=1 << 23, residual=RES) == INVALID
    lib = ses.lib()
    assert lib.moe_expert_int8_workspace_bytes(1, 72, 64) == 0 and lib.moe_linear_int8_workspace_bytes(1, 8, 24, 0) == 0
    assert lib.moe_expert_int8_workspace_bytes(1, 64, 64) > 0 and lib.moe_linear_int8_workspace_bytes(0, 1, 16, 0) > 0


def test_quantize_refuses_on_the_host():
    q = ses.lib().moe_quantize_int8
    assert q(X, 0, 0, 64, Y, RES, None) == 0
    for bad in ((X, 3, 2, 64, Y, RES), (X, -1, 2, 64, Y, RES), (X, 0, -1, 64, Y, RES), (X, 0, 2, 0, Y, RES), (None, 0, 2, 64, Y, RES),
                (X, 0, 2, 64, None, RES), (X, 0, 2, 64, Y, None), (X, 0, 2, 64, X + 128, RES), (X, 2, 2, 64, Y, X + 496),
                (X, 0, 2, 64, Y, Y + 112)):
        assert q(*bad, None) == INVALID, bad
    for K in (8, 72, 65552):
        assert q(X, 0, 2, K, Y, RES, None) == SHAPE
    for bad in ((X + 8, 0, 2, 64, Y, RES), (X, 0, 2, 64, Y + 8, RES), (X, 0, 2, 64, Y, RES + 4)):
        assert q(*bad, None) == ALIGN, bad


def test_binding_refuses_host_tensors():
    t = torch.zeros(2, 16)
    for call in (lambda: ses.quantize_int8(t), lambda: ses.linear_int8(t.half(), t.to(I8), t[:, 0]), lambda: ses.quantize_int8(None),
                 lambda: ses.Int8Experts(*[t.to(I8)[None], t] * 3).c_struct()):
        with pytest.raises(TypeError):
            call()


@gpu
def test_binding_refusals():
    x, xs = torch.zeros(4, 32, dtype=I8, device="cuda"), torch.ones(4, device="cuda")
    w, ws = torch.zeros(8, 32, dtype=I8, device="cuda"), torch.ones(8, device="cuda")
    ok = dict(x_scale=xs, dtype=F16)
    for bad, kind in ((dict(ok, x_scale=None), ValueError), (dict(ok, dtype=None), TypeError), (dict(ok, dtype=F32), TypeError),
                      (dict(ok, act="tanh"), ValueError), (dict(ok, out_dtype=BF16), TypeError), (dict(ok, w_mul=w), ValueError),
                      (dict(ok, w_mul_scale=ws), ValueError), (dict(ok, bias_mul=ws.half()), ValueError),
                      (dict(ok, bias=ws), TypeError), (dict(ok, x_scale=xs[:3]), ValueError),
                      (dict(ok, residual=torch.zeros(4, 9, dtype=F16, device="cuda")), ValueError),
                      (dict(ok, out=torch.zeros(4, 8, device="cuda")), TypeError)):
        with pytest.raises(kind):
            ses.linear_int8(x, w, ws, **bad)
    for args in ((x.float(), w, ws), (x.half(), w.half(), ws), (x.half(), w, ws.half()), (x.t(), w, ws), (x[:, ::2], w, ws),
                 (x.half(), w[:, :16], ws), (x.half(), w, ws[:4]), (x[0], w, ws)):
        with pytest.raises((TypeError, ValueError)):
            ses.linear_int8(*args)
    with pytest.raises(TypeError):
        ses.linear_int8(x.half(), w, ws, dtype=BF16)
    with pytest.raises(ValueError):
        ses.linear_int8(x.half(), w, ws, x_scale=xs)
    with pytest.raises(MoeError) as err:  # an inner size that is no multiple of 16
        ses.linear_int8(torch.zeros(2, 24, dtype=F16, device="cuda"), torch.zeros(8, 24, dtype=I8, device="cuda"), ws,
                        ws=ses.Workspace(1 << 20))
    assert err.value.status == SHAPE
    with pytest.raises(MoeError) as err:
        ses.linear_int8(x, w, ws, **ok, ws=ses.Workspace(16))
    assert err.value.status == SMALL
    assert ses.linear_int8(x[:0], w, ws, x_scale=xs[:0], dtype=BF16).shape == (0, 8)
    ex = ses.Int8Experts(torch.zeros(2, 48, 32, dtype=I8, device="cuda"), torch.ones(2, 48, device="cuda"),
                         torch.zeros(2, 48, 32, dtype=I8, device="cuda"), torch.ones(2, 48, device="cuda"),
                         torch.zeros(2, 32, 48, dtype=I8, device="cuda"), torch.ones(2, 32, device="cuda"))
    assert (ex.E, ex.d, ex.f) == (2, 32, 48)
    for bad in (dict(x=x[:, :16].contiguous()), dict(expert=2), dict(dtype=None), dict(residual=x)):
        with pytest.raises((TypeError, ValueError, MoeError)):
            kw = dict(dict(x=x, experts=ex, expert=0, x_scale=xs, dtype=F16), **bad)
            ses.expert_int8_swiglu(**kw)
    ex.up_scale = ex.up_scale[:, :40]
    with pytest.raises(ValueError):
        ses.expert_int8_swiglu(x, ex, 0, x_scale=xs, dtype=F16)
