"""Operators on uncompressed 16-bit weights (linear, expert_dense_swiglu, layer_dense_decode) against plain
implementations in 64 bits.

Tolerances, elementwise and derived before the first run.  The last rounding costs half a step,
eps/2 * |y|.  A product of K terms with fp32 sums costs at most tau(K) * S, where S is the sum of the
terms' magnitudes: K/16 tensor-core steps that may each cut off (2^-23 of the partial sum) and as much
again for the alignment within a step, and up to 20 more additions when the shares of a split sum are
joined: tau(K) = (K/16 + 20) * 2^-22.  The activations have slopes up to 1.13, a relative error of
2^-20 of their own (exp and erf of fp32), and their derived bounds follow the product rule.
"""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from oracle import moe_oracle as orc
from tests import parity

ses = pytest.importorskip("sparse_expert_swiglu_gb300")
from sparse_expert_swiglu_gb300._lib import MoeError  # noqa: E402

gpu = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    ses.build_library()
    ses.lib()


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _tau(K):
    return (K / 16 + 20) * 2.0 ** -22


def _rand(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype)


def _cuda(t):
    return None if t is None else t.cuda()


def _act64(name, a):
    f = torch.nn.functional
    return {"none": lambda v: v, "relu": f.relu, "gelu": f.gelu, "gelu_tanh": lambda v: f.gelu(v, approximate="tanh"),
            "silu": f.silu}[name](a)


def _within(y, ref, bound, dtype):
    """Every element within its bound; the type's largest value and subnormal steps are allowed for."""
    y = y.cpu().double()
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    lim = bound + _half_step(dtype) * ref.abs() * (1 + 2.0 ** -10) + tiny
    bad = ~((y - ref).abs() <= lim)
    assert not bad.any(), (int(bad.sum()), float(((y - ref).abs() - lim)[bad].max()))


# ---------------------------------------------------------------------------
# linear
# ---------------------------------------------------------------------------

def _linear_case(M, N, K, dtype, act="none", bias=False, gated=False, residual=False, layout="nk", out=None, seed=0):
    g = torch.Generator().manual_seed(seed + M + 3 * N + 7 * K)
    shape = (N, K) if layout == "nk" else (K, N)
    x, w = _rand(g, (M, K), dtype), _rand(g, shape, dtype, 0.05)
    w2 = _rand(g, shape, dtype, 0.05) if gated else None
    b = _rand(g, (N,), dtype) if bias else None
    b2 = _rand(g, (N,), dtype) if bias and gated else None
    r = _rand(g, (M, N), dtype) if residual else None
    return dict(x=x, w=w, w_mul=w2, bias=b, bias_mul=b2, residual=r, act=act, w_layout=layout, out_dtype=out)


def _linear_ref(c):
    """(y, bound without the last rounding) in 64 bits."""
    x = c["x"].double()
    K = x.shape[1]

    def product(w, b):
        w = w.double().t() if c["w_layout"] == "nk" else w.double()
        s = x.abs() @ w.abs()
        a = x @ w
        if b is not None:
            a, s = a + b.double(), s + b.double().abs()
        return a, _tau(K) * s
    a, da = product(c["w"], c["bias"])
    y = _act64(c["act"], a)
    dy = da if c["act"] in ("none", "relu") else 1.13 * da + 2.0 ** -20 * (y.abs() + a.abs())
    if c["w_mul"] is not None:
        u, du = product(c["w_mul"], c["bias_mul"])
        dy = dy * u.abs() + y.abs() * du + dy * du
        y = y * u
    if c["residual"] is not None:
        y = y + c["residual"].double()
    return y, dy + 2.0 ** -23 * y.abs()


def _linear_run(c, **more):
    kw = {k: _cuda(v) if isinstance(v, torch.Tensor) else v for k, v in c.items() if k not in ("x", "w")}
    return ses.linear(_cuda(c["x"]), _cuda(c["w"]), **kw, **more)


def _linear_check(c, **more):
    y = _linear_run(c, **more)
    ref, bound = _linear_ref(c)
    assert y.dtype == (c["out_dtype"] or c["x"].dtype) and y.shape == ref.shape
    _within(y, ref, bound, y.dtype)
    return y


@gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("M,N,K", [(1, 128, 64), (16, 256, 128), (1, 8, 8), (3, 40, 72), (17, 264, 1000),
                                   (130, 1032, 520), (257, 136, 64), (333, 648, 2056)])
def test_linear_sizes(M, N, K, layout, dtype):
    _linear_check(_linear_case(M, N, K, dtype, layout=layout))


@gpu
@pytest.mark.parametrize("N", [1, 7, 127, 129, 255, 257, 1031])
def test_linear_odd_outputs(N):
    for M in (1, 5, 48):
        _linear_check(_linear_case(M, N, 200, BF16, bias=True, residual=True))


@gpu
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_epilogues(act, gated):
    for dtype, out in ((F16, None), (BF16, None), (F16, F32), (BF16, F32)):
        for bias, residual in ((False, False), (True, False), (True, True)):
            _linear_check(_linear_case(21, 200, 264, dtype, act, bias, gated, residual, out=out))


@gpu
def test_linear_split_sum_and_full_waves():
    """One tile cut into many shares, more tiles than SMs, and both at once; equal calls give equal bits."""
    for M, N, K, gated, layout in ((1, 256, 16384, False, "nk"), (1, 256, 16384, True, "kn"), (64, 40960, 128, False, "nk"),
                                   (700, 12288, 136, False, "kn"), (300, 5000, 1032, True, "nk")):
        c = _linear_case(M, N, K, F16, "silu" if gated else "none", gated=gated, layout=layout)
        ws = ses.Workspace(ses.linear_workspace_bytes(M, N, K, gated))
        y = _linear_check(c, ws=ws)
        for _ in range(3):
            assert torch.equal(y, _linear_run(c, ws=ws))
        assert ws.status() == 0


@gpu
@pytest.mark.parametrize("M,N,K,gated,layout", [
    (1, 4096, 4096, False, "nk"), (1, 1024, 8192, False, "kn"), (4, 512, 16384, True, "nk"), (5, 520, 8200, True, "kn"),
    (16, 2048, 2048, False, "nk"), (33, 768, 8192, False, "nk"), (64, 1000, 4096, True, "kn"), (100, 300, 16384, False, "nk"),
    (128, 2048, 2048, False, "kn"), (300, 264, 8192, False, "nk")])
def test_linear_sums_shared_by_a_cluster(M, N, K, gated, layout):
    """Few tiles and a long k: two to eight CTAs share a tile."""
    for bias, residual, out in ((False, False, None), (True, True, F32)):
        c = _linear_case(M, N, K, BF16, "gelu_tanh", bias, gated, residual, layout, out)
        y = _linear_check(c)
        assert torch.equal(y, _linear_run(c))


@gpu
@pytest.mark.parametrize("M,N,K", [(256, 256, 64), (512, 520, 1000), (700, 1032, 520), (1500, 1040, 136), (1025, 4096, 72),
                                   (2048, 2048, 264)])
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_linear_many_tokens(M, N, K, layout):
    for dtype, gated, bias, residual, out in ((BF16, False, False, True, None), (F16, True, True, False, None),
                                              (F16, False, True, True, F32), (BF16, True, False, True, F32)):
        _linear_check(_linear_case(M, N, K, dtype, "silu", bias, gated, residual, layout, out))


@gpu
def test_linear_output_behind_2_to_the_31():
    M, N, K = 65537, 40000, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(M, K, device="cuda", dtype=F16, generator=g)
    w = torch.randn(N, K, device="cuda", dtype=F16, generator=g)
    y = ses.linear(x, w)
    for rows in (slice(0, 3), slice(53685, 53690), slice(M - 3, M)):  # 53687 * 40000 crosses 2^31
        a, b = x[rows].double().cpu(), w.double().cpu()
        _within(y[rows], a @ b.t(), _tau(K) * (a.abs() @ b.abs().t()), F16)
    odd = ses.linear(x, w[:39999])
    assert torch.equal(odd[-3:], y[-3:, :39999]) and torch.equal(odd[53687], y[53687, :39999])


@gpu
def test_linear_large_values_and_nan():
    """A token with NaN or inf spoils its own row alone; sums beyond fp16 round to inf."""
    c = _linear_case(20, 130, 256, F16, "relu")
    c["x"][3, 100] = float("nan")
    c["x"][17, 0] = float("inf")
    y = _linear_run(c).cpu()
    ref, bound = _linear_ref(c)
    assert torch.isnan(y[3]).all()
    assert torch.equal(torch.isfinite(y), torch.isfinite(ref))
    keep = [i for i in range(20) if i not in (3, 17)]
    _within(y[keep], ref[keep], bound[keep], F16)
    big = dict(c, x=torch.full((1, 256), 1000.0, dtype=F16), w=torch.full((130, 256), 1.0, dtype=F16), act="none")
    assert torch.isinf(_linear_run(big)).all()
    assert torch.equal(_linear_run(dict(big, out_dtype=F32)).cpu(), torch.full((1, 130), 256000.0))


@gpu
def test_linear_output_tensor_in_place_and_empty():
    c = _linear_case(9, 72, 96, BF16, "gelu", bias=True, residual=True)
    y = _linear_run(c)
    r = c["residual"].cuda()
    kw = {k: _cuda(v) if isinstance(v, torch.Tensor) else v for k, v in c.items() if k not in ("x", "w", "residual")}
    got = ses.linear(c["x"].cuda(), c["w"].cuda(), residual=r, out=r, **kw)
    assert got is r and torch.equal(r, y)
    assert ses.linear(c["x"].cuda()[:0], c["w"].cuda()).shape == (0, 72)


@gpu
@pytest.mark.parametrize("M,N,K,gated,layout,out", [
    (128, 4096, 4096, False, "nk", None), (86, 4420, 2176, True, "nk", None), (592, 744, 6104, False, "kn", None),
    (384, 7808, 120, True, "kn", None), (1421, 6484, 1000, False, "nk", None), (300, 14336, 512, True, "nk", None),
    (128, 4096, 4096, False, "nk", F32), (592, 744, 6104, True, "kn", F32), (97, 2056, 1304, False, "kn", None)])
def test_linear_of_cta_pairs_with_halved_tokens(M, N, K, gated, layout, out):
    _linear_check(_linear_case(M, N, K, BF16, "silu" if gated else "none", bias=True, gated=gated, residual=True,
                               layout=layout, out=out))


@gpu
@pytest.mark.parametrize("out", [F16, F32])
@pytest.mark.parametrize("M,N,K,gated", [(2048, 4096, 256, False), (2048, 2048, 256, True), (300, 2048, 128, False),
                                         (5, 512, 128, True)])
def test_linear_output_on_any_16_bytes(M, N, K, gated, out):
    c = _linear_case(M, N, K, F16, "silu", bias=True, gated=gated, residual=True, out=out)
    y = _linear_run(c)
    step = 128 // torch.finfo(out).bits
    for at in range(1, 4):
        buf = torch.full((M * N + 4 * step,), 7.0, dtype=out, device="cuda")
        z = buf[at * step:at * step + M * N].view(M, N)
        assert _linear_run(c, out=z) is z and torch.equal(z, y)
        assert (buf[:at * step] == 7.0).all() and (buf[at * step + M * N:] == 7.0).all()


# ---------------------------------------------------------------------------
# experts and layers
# ---------------------------------------------------------------------------

def _experts(g, E, d, f, dtype, interleave=False, std=0.05):
    gate, up, down = (_rand(g, (E, f, d), dtype, std) for _ in range(3))
    if interleave:
        both = torch.stack((gate, down), dim=2).cuda()
        return (gate, up, down), ses.DenseExperts(both[:, :, 0, :], up.cuda(), both[:, :, 1, :])
    return (gate, up, down), ses.DenseExperts(gate.cuda(), up.cuda(), down.cuda())


def _expert_ref(x, gate, up, down, dtype, rounded_h):
    """(y, bound) of one expert on x (64 bits)."""
    d, f = x.shape[1], gate.shape[0]
    gate, up, down = gate.double(), up.double(), down.double()
    a, u = x @ gate.t(), x @ up.t()
    da, du = _tau(d) * (x.abs() @ gate.abs().t()), _tau(d) * (x.abs() @ up.abs().t())
    s = torch.nn.functional.silu(a)
    h = s * u
    ds = 1.13 * da + 2.0 ** -20 * (s.abs() + a.abs())
    dh = ds * u.abs() + s.abs() * du + ds * du + 2.0 ** -22 * h.abs()
    # h in the operand: one value of the type, or two (the second one's half step; fp16's smallest step)
    half = _half_step(dtype)
    dh = dh + (half if rounded_h else half * half) * 1.01 * (h.abs() + dh) + 2.0 ** -25
    return h @ down, dh @ down.abs() + _tau(f) * (h.abs() @ down.abs())


def _expert_check(n, d, f, dtype, residual=False, interleave=False, E=2, e=1, ws=None):
    g = torch.Generator().manual_seed(n + 3 * d + 5 * f)
    (gate, up, down), ex = _experts(g, E, d, f, dtype, interleave)
    x = _rand(g, (n, d), dtype)
    r = _rand(g, (n, d), dtype) if residual else None
    y = ses.expert_dense_swiglu(x.cuda(), ex, e, residual=_cuda(r), ws=ws)
    ref, bound = _expert_ref(x.double(), gate[e], up[e], down[e], dtype, n > 64)
    if residual:
        ref = ref + r.double()
    _within(y, ref, bound + 2.0 ** -22 * ref.abs(), dtype)


@gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n,d,f", [(1, 64, 128), (1, 8, 8), (2, 256, 136), (7, 200, 264), (8, 512, 1000), (9, 72, 520),
                                   (33, 520, 72), (64, 256, 1408), (65, 256, 264), (200, 136, 520), (300, 1024, 256)])
def test_expert_sizes(n, d, f, dtype):
    _expert_check(n, d, f, dtype)


@gpu
@pytest.mark.parametrize("n", [1, 64, 65, 150])
def test_expert_residual_and_interleaved_rows(n):
    for interleave in (False, True):
        for residual in (False, True):
            _expert_check(n, 264, 200, BF16, residual, interleave, E=3, e=2)


def _layer_case(B, d, f, E, k, ns, dtype, renorm, residual, rmsnorm, interleave=False, seed=0):
    g = torch.Generator().manual_seed(seed + B + 3 * d + 5 * f + 7 * E)
    routed, ex = _experts(g, E, d, f, dtype, interleave)
    shared, sh = _experts(g, ns, d, f, dtype, interleave) if ns else (None, None)
    wr = _rand(g, (d, E), dtype, 0.05)
    x = _rand(g, (B, d), dtype)
    r = _rand(g, (B, d), dtype) if residual else None
    return dict(x=x, wr=wr, routed=routed, shared=shared, residual=r, k=k, renorm=renorm, rmsnorm=rmsnorm,
                layer=ses.DenseLayer(wr.cuda(), ex, k, renorm, sh))


def _layer_check(c, ws=None, idx_as_oracle=True):
    x, dtype, k = c["x"], c["x"].dtype, c["k"]
    B, d = x.shape
    y, dbg = ses.layer_dense_decode(x.cuda(), c["layer"], residual=_cuda(c["residual"]), rmsnorm=c["rmsnorm"], ws=ws,
                                    debug=True)
    idx, w = dbg["topk_idx"].cpu(), dbg["topk_w"].cpu().double()
    xd, wr = x.double(), c["wr"].double()
    idx_ref, _, logits = orc.route_topk(xd.numpy(), wr.numpy(), k, c["renorm"])
    ok, n_band = parity.route_band(logits, (xd.abs() @ wr.abs()).numpy(), idx.numpy(), k)
    assert ok and (n_band == 0 or not idx_as_oracle)
    lo = torch.from_numpy(logits)
    sel = torch.gather(lo, 1, idx.long())
    p = torch.exp(sel - sel[:, :1]) / torch.exp((sel if c["renorm"] else lo) - sel[:, :1]).sum(1, keepdim=True)
    # logits off by tau(d) S; a softmax weight by twice that
    dw = 2 * _tau(d) * float((xd.abs() @ wr.abs()).max()) + 2.0 ** -20
    assert float((w - p).abs().max()) <= dw
    ref, bound = torch.zeros(B, d, dtype=torch.float64), torch.zeros(B, d, dtype=torch.float64)
    for e in range(wr.shape[1]):
        b, j = torch.nonzero(idx == e, as_tuple=True)
        if len(b):
            v, dv = _expert_ref(xd[b], *(t[e] for t in c["routed"]), dtype, False)
            ref[b] += p[b, j][:, None] * v
            bound[b] += p[b, j][:, None] * dv + dw * (v.abs() + dv)
    if c["shared"] is not None:
        for e in range(c["shared"][0].shape[0]):
            v, dv = _expert_ref(xd, *(t[e] for t in c["shared"]), dtype, False)
            ref, bound = ref + v, bound + dv
    if c["residual"] is not None:
        ref = ref + c["residual"].double()
    bound = bound + 2.0 ** -20 * ref.abs()
    if c["rmsnorm"]:
        rms = torch.sqrt((ref * ref).mean(1, keepdim=True) + 1e-6)
        drms = torch.sqrt((bound * bound).mean(1, keepdim=True)) + 2.0 ** -20 * rms
        bound = bound / rms + (ref.abs() + bound) / rms * (drms / (rms - drms))
        ref = ref / rms
    _within(y, ref, bound, dtype)
    return y


@gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("B,d,f,E,k,ns", [(1, 256, 512, 8, 2, 0), (1, 256, 264, 64, 6, 2), (2, 520, 200, 7, 3, 1),
                                          (8, 256, 512, 8, 2, 0), (9, 200, 136, 60, 8, 2), (17, 1024, 520, 8, 2, 1),
                                          (64, 256, 264, 64, 6, 2), (64, 136, 72, 1, 1, 0), (33, 72, 1000, 256, 8, 0),
                                          (5, 8, 8, 3, 3, 8)])
def test_layer_sizes(B, d, f, E, k, ns, dtype):
    for renorm, residual, rmsnorm in ((True, False, False), (False, True, True), (True, True, False)):
        _layer_check(_layer_case(B, d, f, E, k, ns, dtype, renorm, residual, rmsnorm))


@gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("B,d,f,E,k,ns", [(50, 1464, 840, 22, 4, 1), (13, 1344, 1680, 4, 3, 2), (61, 2272, 280, 19, 8, 2),
                                          (2, 2720, 496, 9, 3, 2), (40, 1512, 600, 60, 4, 0), (20, 512, 256, 250, 8, 1),
                                          (33, 1032, 264, 1, 1, 1), (9, 776, 328, 255, 8, 0), (64, 264, 1160, 5, 5, 8)])
def test_layer_tiles_and_routers(B, d, f, E, k, ns, dtype):
    _layer_check(_layer_case(B, d, f, E, k, ns, dtype, True, True, True))


@gpu
def test_layer_of_the_largest_experts():
    """d = 16384, f = 65536: an expert's rows lie behind 2^31 elements."""
    d, f, E = 16384, 65536, 3
    g = torch.Generator(device="cuda").manual_seed(4)
    gate, up, down = (torch.empty(E, f, d, device="cuda", dtype=BF16).normal_(0, 0.01, generator=g) for _ in range(3))
    wr = torch.randn(d, E, device="cuda", dtype=BF16, generator=g) * 0.05
    x = torch.randn(3, d, device="cuda", dtype=BF16, generator=g)
    y, dbg = ses.layer_dense_decode(x, ses.DenseLayer(wr, ses.DenseExperts(gate, up, down), 1), debug=True)
    idx = dbg["topk_idx"][:, 0].cpu()
    assert torch.equal(idx, (x.double() @ wr.double()).argmax(1).int().cpu())
    for e in sorted(set(idx.tolist())):
        one = ses.expert_dense_swiglu(x, ses.DenseExperts(gate, up, down), e)
        b = [i for i in range(3) if idx[i] == e]
        xd = x[b].double()
        h = torch.nn.functional.silu(xd @ gate[e].double().t()) * (xd @ up[e].double().t())
        ref = (h @ down[e].double()).cpu()
        for got in (y[b], one[b]):
            # h and its sums: at most a part in 2^14 of the terms' root sum of squares; then the rounding
            lim = 2.0 ** -14 * float(h.norm(dim=1).max()) * 0.01 * 8 + _half_step(BF16) * ref.abs() * 1.01
            assert ((got.double().cpu() - ref).abs() <= lim).all()


@gpu
def test_layers_on_two_streams_at_once():
    """Each call's kernel takes every SM and waits for its own CTAs: two streams, two workspaces."""
    a = _layer_case(17, 1024, 520, 8, 2, 1, BF16, True, False, False)
    b = _layer_case(1, 512, 1024, 16, 4, 0, F16, False, False, True)
    want = [ses.layer_dense_decode(c["x"].cuda(), c["layer"], rmsnorm=c["rmsnorm"]) for c in (a, b)]
    ws = [ses.Workspace(ses.layer_dense_workspace_bytes(c["layer"], len(c["x"]))) for c in (a, b)]
    xs = [c["x"].cuda() for c in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, c in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(ses.layer_dense_decode(xs[i], c["layer"], rmsnorm=c["rmsnorm"], ws=ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert ws[i].status() == 0
        assert all(torch.equal(y, want[i]) for y in got[i])


@gpu
def test_calls_of_two_threads():
    import threading

    cases = [[_linear_case(*s, F16, bias=True) for s in ((1, 264, 1000), (40, 520, 264), (200, 264, 136), (3, 72, 2048))],
             [_linear_case(*s, BF16, "silu", gated=True) for s in ((300, 520, 264), (2, 264, 520), (70, 72, 1000))]]
    serial = [[_linear_run(c) for c in cs] for cs in cases]
    torch.cuda.synchronize()
    wrong = []

    def calls(cs, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    for c, y in zip(cs, want):
                        if not torch.equal(_linear_run(c), y):
                            wrong.append(tuple(y.shape))
        except Exception as e:  # an exception of a thread fails the test
            wrong.append(e)

    threads = [threading.Thread(target=calls, args=a) for a in zip(cases, serial)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@gpu
def test_outputs_in_the_residual():
    c = _layer_case(5, 264, 200, 8, 2, 1, F16, True, True, False)
    x, r = c["x"].cuda(), c["residual"].cuda()
    for rmsnorm in (False, True):
        y = ses.layer_dense_decode(x, c["layer"], residual=r, rmsnorm=rmsnorm)
        z = r.clone()
        assert ses.layer_dense_decode(x, c["layer"], residual=z, rmsnorm=rmsnorm, out=z) is z and torch.equal(z, y)
    for n in (5, 70):
        xn, rn = x.repeat(14, 1)[:n].contiguous(), r.repeat(14, 1)[:n].contiguous()
        y = ses.expert_dense_swiglu(xn, c["layer"].routed, 2, residual=rn)
        z = rn.clone()
        assert ses.expert_dense_swiglu(xn, c["layer"].routed, 2, residual=z, out=z) is z and torch.equal(z, y)
        y, z = ses.expert_dense_swiglu(xn, c["layer"].routed, 2, residual=xn), xn.clone()
        assert ses.expert_dense_swiglu(z, c["layer"].routed, 2, residual=z, out=z) is z and torch.equal(z, y)


@gpu
def test_layer_interleaved_rows():
    _layer_check(_layer_case(3, 264, 200, 8, 2, 1, F16, True, True, False, interleave=True))


@gpu
def test_layer_calls_share_a_workspace():
    """Calls of all three operators with different sizes, in turn, on one workspace; equal calls, equal bits."""
    big = _layer_case(64, 256, 264, 64, 6, 2, F16, True, True, True)
    small = _layer_case(1, 512, 1024, 8, 2, 0, BF16, True, False, False)
    lin = _linear_case(33, 264, 2056, F16, "silu", gated=True)
    need = max(ses.layer_dense_workspace_bytes(big["layer"], 64), ses.layer_dense_workspace_bytes(small["layer"], 1),
               ses.linear_workspace_bytes(33, 264, 2056, True))
    ws = ses.Workspace(need)
    first = None
    for _ in range(3):
        got = (_layer_check(big, ws), _layer_check(small, ws), _linear_run(lin, ws=ws))
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    assert ws.status() == 0


@gpu
def test_layer_exact_ties_go_to_the_lower_expert():
    d, E, k = 64, 12, 3
    g = torch.Generator().manual_seed(1)
    c = _layer_case(20, d, 64, E, k, 0, F16, True, False, False)
    c["x"] = torch.randint(-2, 3, (20, d), generator=g).to(F16)
    c["wr"] = torch.randint(-1, 2, (d, E), generator=g).to(F16)
    c["layer"].w_router = c["wr"].cuda()
    _layer_check(c)


@gpu
def test_layer_token_without_finite_values():
    """A NaN token gets valid experts and a NaN row; the other tokens are untouched by it."""
    c = _layer_case(10, 256, 264, 16, 2, 1, BF16, True, False, False)
    clean = _layer_check(c)
    x = c["x"].clone()
    x[4, 7] = float("nan")
    y, dbg = ses.layer_dense_decode(x.cuda(), c["layer"], debug=True)
    assert torch.isnan(y[4]).all()
    keep = [i for i in range(10) if i != 4]
    assert torch.equal(y[keep], clean[keep])
    idx = dbg["topk_idx"].cpu()
    assert (idx >= 0).all() and (idx < 16).all() and idx[4, 0] != idx[4, 1]


@gpu
def test_layer_matches_the_sparse_layer_at_threshold_zero():
    """The sparse layer's up projection is INT2; with the dequantised values as the dense layer's up rows and
    threshold 0 both compute the same layer (the fp16 rounding of the dequantised weights apart)."""
    d, f, E, k = 256, 512, 8, 2
    g = torch.Generator().manual_seed(3)
    wu = _rand(g, (E, d, f), F16, 0.02)
    gate, down = _rand(g, (E, f, d), F16, 0.02), _rand(g, (E, f, d), F16, 0.02)
    wr, x = _rand(g, (d, E), F16, 0.05), _rand(g, (8, d), F16)
    deq = np.stack([orc.dequantize_int2(*orc.quantize_int2(wu[e].numpy())) for e in range(E)])
    up = torch.from_numpy(deq).to(F16).transpose(1, 2).contiguous()
    sparse = ses.Experts.from_dense(wu.cuda(), gate.cuda(), down.cuda(), torch.zeros(E, device="cuda"), interleave=True)
    y0 = ses.layer_decode(x.cuda(), ses.Layer(wr.cuda(), sparse, k))
    dense = ses.DenseExperts(sparse.gate_t, up.cuda(), sparse.down)  # the same gate and down buffer
    y1 = ses.layer_dense_decode(x.cuda(), ses.DenseLayer(wr.cuda(), dense, k))
    a, b = y0.double().cpu(), y1.double().cpu()
    assert float((a - b).norm() / a.norm()) < 2e-3


@gpu
def test_decode_step_of_a_small_stack():
    """The operators as a model runs them: output projection with residual, MoE layer with residual, a dense
    gated block by two products, fp32 logits; against 64 bits of the same chain with rounding in between."""
    d, f, V = 256, 520, 1000
    g = torch.Generator().manual_seed(5)
    c = _layer_case(6, d, f, 8, 2, 1, BF16, True, False, False)
    wo, wh = _rand(g, (d, d), BF16, 0.05), _rand(g, (V, d), BF16, 0.05)
    wg, wu, wd = _rand(g, (f, d), BF16, 0.05), _rand(g, (f, d), BF16, 0.05), _rand(g, (f, d), BF16, 0.05)
    att, h0 = _rand(g, (6, d), BF16), _rand(g, (6, d), BF16)

    def step():
        h = ses.linear(att.cuda(), wo.cuda(), residual=h0.cuda())
        h = ses.layer_dense_decode(h, c["layer"], residual=h)
        t = ses.linear(h, wg.cuda(), act="silu", w_mul=wu.cuda())
        h2 = ses.linear(t, wd.cuda(), residual=h, w_layout="kn")
        return h, h2, ses.linear(h2, wh.cuda(), out_dtype=F32)
    h, h2, logits = step()
    hd = h.double().cpu()
    t = torch.nn.functional.silu(hd @ wg.double().t()) * (hd @ wu.double().t())
    ref = t @ wd.double() + hd
    assert float((h2.double().cpu() - ref).norm() / ref.norm()) < 2.0 ** -8
    ref = h2.double().cpu() @ wh.double().t()
    assert float((logits.double().cpu() - ref).norm() / ref.norm()) < 2.0 ** -16
    assert all(torch.equal(a, b) for a, b in zip((h, h2, logits), step()))


@gpu
def test_captured_calls_and_other_streams():
    """Each operator captured into a graph and replayed on new inputs, on a stream of its own, while the
    default stream works on other workspaces."""
    c = _layer_case(4, 256, 264, 8, 2, 1, F16, True, True, False)
    lin = _linear_case(4, 264, 256, F16, "gelu", bias=True)
    x, r = c["x"].cuda(), c["residual"].cuda()
    w, b = lin["w"].cuda(), lin["bias"].cuda()
    ex = c["layer"].routed
    ws = ses.Workspace(max(ses.layer_dense_workspace_bytes(c["layer"], 4), ses.linear_workspace_bytes(4, 264, 256),
                           ses.expert_dense_workspace_bytes(4, 256, 264)))
    out = [torch.empty(4, 256, dtype=F16, device="cuda"), torch.empty(4, 264, dtype=F16, device="cuda"),
           torch.empty(4, 256, dtype=F16, device="cuda")]

    def calls():
        ses.layer_dense_decode(x, c["layer"], residual=r, ws=ws, out=out[0])
        ses.linear(out[0], w, bias=b, act="gelu", ws=ws, out=out[1])
        ses.expert_dense_swiglu(out[0], ex, 3, ws=ws, out=out[2])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        calls()
    for seed in range(3):
        g = torch.Generator().manual_seed(seed)
        x.copy_(_rand(g, (4, 256), F16))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        other = ses.linear(x, w, bias=b, act="gelu")  # the default stream, its own workspace
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        with torch.cuda.stream(s):
            calls()
        torch.cuda.synchronize()
        assert all(torch.equal(a, t) for a, t in zip(got, out))
        assert torch.equal(other, ses.linear(x, w, bias=b, act="gelu"))
    assert ws.status() == 0


# ---------------------------------------------------------------------------
# refusals (no GPU needed: found on the host before anything is enqueued)
# ---------------------------------------------------------------------------

def _lin_op(**kw):
    from sparse_expert_swiglu_gb300 import _lib
    v = dict(M=4, N=64, K=64, dtype=0, out_dtype=0, w_layout=0, act=0, x=0x10000, w=0x20000, w_mul=None, bias=None,
             bias_mul=None, residual=None, y=0x30000)
    v.update(kw)
    return _lib._Linear(*(v[n] for n, _ in _lib._Linear._fields_))


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), -1), (dict(N=0), -1), (dict(K=0), -1), (dict(K=60), -2), (dict(K=1 << 19), -2), (dict(M=(1 << 20) + 1), -2),
    (dict(N=(1 << 20) + 1), -2), (dict(w_layout=1, N=60), -2), (dict(w_layout=2), -1), (dict(act=5), -1), (dict(act=-1), -1),
    (dict(dtype=2), -1), (dict(out_dtype=1), -1), (dict(x=None), -1), (dict(w=None), -1), (dict(y=None), -1),
    (dict(bias_mul=0x40000), -1), (dict(x=0x10008), -3), (dict(w=0x20002), -3), (dict(y=0x30004), -3),
    (dict(bias=0x40002), -3), (dict(residual=0x40008), -3), (dict(w_mul=0x40008), -3), (dict(M=0), 0),
    (dict(y=0x10000), -1), (dict(y=0x0FE10), -1), (dict(y=0x101F0), -1), (dict(y=0x21FF0), -1),
    (dict(w_mul=0x40000, y=0x40000), -1), (dict(bias=0x30010), -1), (dict(w_mul=0x40000, bias_mul=0x301F0), -1),
    (dict(residual=0x30010), -1), (dict(residual=0x30000, out_dtype=2), -1)])
def test_linear_refusals(change, status):
    lib = ses.lib()
    ws = ctypes.c_void_p(0x100000)
    assert lib.moe_linear(ctypes.byref(_lin_op(**change)), ws, 0, None) == status


def test_linear_refuses_null_and_workspace():
    lib = ses.lib()
    assert lib.moe_linear(None, ctypes.c_void_p(0x100000), 1 << 30, None) == -1
    assert lib.moe_linear(ctypes.byref(_lin_op()), None, 1 << 30, None) == -1
    assert lib.moe_linear(ctypes.byref(_lin_op()), ctypes.c_void_p(0x100080), 1 << 30, None) == -3
    assert lib.moe_linear_workspace_bytes(4, 64, 60, 0) == 0
    assert lib.moe_linear_workspace_bytes(-1, 64, 64, 0) == 0


def _dense_structs(**kw):
    from sparse_expert_swiglu_gb300 import _lib
    v = dict(E=8, d=256, f=512, dtype=0, gate_t=0x10000, up_t=0x20000, down=0x30000)
    layer = dict(k=2, renorm=1, w_router=0x50000)
    sh = dict(E=0, d=256, f=512, dtype=0, gate_t=None, up_t=None, down=None)
    for key, val in kw.items():
        if key in layer:
            layer[key] = val
        elif key.startswith("s_"):
            sh[key[2:]] = val
        else:
            v[key] = val
            if key in ("d", "f", "dtype") and sh["E"] == 0:
                sh[key] = val
    ex = _lib._DenseExperts(*(v[n] for n, _ in _lib._DenseExperts._fields_))
    s = _lib._DenseExperts(*(sh[n] for n, _ in _lib._DenseExperts._fields_))
    return ex, _lib._DenseLayer(layer["k"], layer["renorm"], layer["w_router"], ex, s)


@pytest.mark.parametrize("change,status", [
    (dict(d=250), -2), (dict(f=250), -2), (dict(d=0), -1), (dict(d=16392), -2), (dict(f=65544), -2), (dict(E=0), -2),
    (dict(E=257), -2), (dict(E=-1), -1), (dict(dtype=2), -1), (dict(gate_t=None), -1), (dict(up_t=None), -1),
    (dict(down=None), -1), (dict(gate_t=0x10008), -3), (dict(up_t=0x20002), -3), (dict(down=0x30008), -3)])
def test_expert_and_layer_refusals(change, status):
    lib = ses.lib()
    ex, layer = _dense_structs(**change)
    p, ws = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x200000)
    assert lib.moe_expert_dense_swiglu(p, 1, ctypes.byref(ex), 0, None, p, ws, 0, None) == status
    assert lib.moe_layer_dense_decode(p, 1, ctypes.byref(layer), None, p, 0, None, ws, 0, None) == status
    assert lib.moe_layer_dense_workspace_bytes(ctypes.byref(layer), 1) == 0


def test_expert_refusals():
    lib = ses.lib()
    ex, _ = _dense_structs()
    p, odd, ws = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100008), ctypes.c_void_p(0x200000)
    call = lib.moe_expert_dense_swiglu
    assert call(p, 0, ctypes.byref(ex), 0, None, p, ws, 0, None) == 0
    assert call(p, -1, ctypes.byref(ex), 0, None, p, ws, 0, None) == -1
    assert call(p, (1 << 20) + 1, ctypes.byref(ex), 0, None, p, ws, 0, None) == -2
    assert call(p, 1, None, 0, None, p, ws, 0, None) == -1
    assert call(p, 1, ctypes.byref(ex), 8, None, p, ws, 0, None) == -1
    assert call(p, 1, ctypes.byref(ex), -1, None, p, ws, 0, None) == -1
    assert call(None, 1, ctypes.byref(ex), 0, None, p, ws, 0, None) == -1
    assert call(p, 1, ctypes.byref(ex), 0, None, None, ws, 0, None) == -1
    assert call(p, 1, ctypes.byref(ex), 0, None, p, None, 0, None) == -1
    assert call(odd, 1, ctypes.byref(ex), 0, None, p, ws, 0, None) == -3
    assert call(p, 1, ctypes.byref(ex), 0, odd, p, ws, 0, None) == -3
    assert call(p, 4, ctypes.byref(ex), 0, ctypes.c_void_p(0x100010), p, ws, 0, None) == -1
    assert lib.moe_expert_dense_workspace_bytes(-1, 256, 512) == 0
    assert lib.moe_expert_dense_workspace_bytes(1, 250, 512) == 0


@pytest.mark.parametrize("change,B,status", [
    (dict(k=0), 1, -1), (dict(k=9), 1, -1), (dict(E=16, k=9), 1, -2), (dict(w_router=None), 1, -1),
    (dict(w_router=0x50008), 1, -3), (dict(), 65, -2), (dict(), -1, -1), (dict(), 0, 0),
    (dict(s_E=9, s_gate_t=0x10000, s_up_t=0x10000, s_down=0x30000), 1, -2), (dict(s_E=-1), 1, -1),
    (dict(s_E=1, s_gate_t=0x10000, s_up_t=0x10000, s_down=None), 1, -1),
    (dict(s_E=1, s_d=264, s_gate_t=0x10000, s_up_t=0x10000, s_down=0x30000), 1, -1),
    (dict(s_E=1, s_dtype=1, s_gate_t=0x10000, s_up_t=0x10000, s_down=0x30000), 1, -1)])
def test_layer_refusals(change, B, status):
    _, layer = _dense_structs(**change)
    p, ws = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x200000)
    assert ses.lib().moe_layer_dense_decode(p, B, ctypes.byref(layer), None, p, 0, None, ws, 0, None) == status


def test_layer_refuses_outputs_in_its_inputs():
    _, layer = _dense_structs()
    ws = ctypes.c_void_p(0x200000)
    for x, r, y in ((0x100000, None, 0x100000), (0x100000, None, 0x1001F0), (0x100000, 0x100000, 0x100000),
                    (0x100000, 0x300010, 0x300000)):
        assert ses.lib().moe_layer_dense_decode(ctypes.c_void_p(x), 1, ctypes.byref(layer), r, ctypes.c_void_p(y), 0, None,
                                                ws, 0, None) == -1


def test_binding_refuses_host_tensors_and_types():
    t = torch.zeros(4, 8, dtype=F16)
    with pytest.raises(TypeError, match="CUDA tensor"):
        ses.linear(t, t)
    with pytest.raises(TypeError, match="must be a tensor"):
        ses.linear([1.0], t)
    ex = ses.DenseExperts(t[None], t[None], t[None])
    with pytest.raises(TypeError, match="CUDA tensor"):
        ex.c_struct()
    with pytest.raises(TypeError, match="CUDA tensor"):
        ses.expert_dense_swiglu(t, ex, 0)
    with pytest.raises(ValueError, match="shape"):
        ses.DenseExperts(t, t, t).c_struct()


@gpu
def test_binding_refusals_on_the_device():
    x, w = torch.zeros(4, 64, dtype=F16, device="cuda"), torch.zeros(32, 64, dtype=F16, device="cuda")
    for bad, exc in ((dict(bias=torch.zeros(31, dtype=F16, device="cuda")), ValueError),
                     (dict(bias=torch.zeros(32, dtype=F32, device="cuda")), TypeError),
                     (dict(residual=torch.zeros(4, 31, dtype=F16, device="cuda")), ValueError),
                     (dict(w_layout="kn"), ValueError), (dict(w_layout="x"), ValueError), (dict(act="tanh"), ValueError),
                     (dict(bias_mul=torch.zeros(32, dtype=F16, device="cuda")), ValueError),
                     (dict(out_dtype=BF16), TypeError), (dict(out=torch.zeros(4, 32, device="cuda")), TypeError),
                     (dict(w_mul=w.t().contiguous().t()), ValueError)):
        with pytest.raises(exc):
            ses.linear(x, w, **bad)
    with pytest.raises(TypeError):
        ses.linear(x.float(), w)
    with pytest.raises(TypeError):
        ses.linear(x, w.bfloat16())
    with pytest.raises(ValueError):
        ses.linear(x.t().contiguous().t(), w)
    with pytest.raises(MoeError) as err:
        ses.linear(torch.zeros(4, 60, dtype=F16, device="cuda"), torch.zeros(32, 60, dtype=F16, device="cuda"),
                   ws=ses.Workspace(1 << 20))
    assert err.value.status == -2
    with pytest.raises(MoeError) as err:
        ses.linear(x, w, ws=ses.Workspace(256))
    assert err.value.status == -4
    c = _layer_case(2, 64, 72, 4, 2, 0, F16, True, False, False)
    for call in (lambda ws: ses.layer_dense_decode(c["x"].cuda(), c["layer"], ws=ws),
                 lambda ws: ses.expert_dense_swiglu(c["x"].cuda(), c["layer"].routed, 0, ws=ws)):
        with pytest.raises(MoeError) as err:
            call(ses.Workspace(256))
        assert err.value.status == -4
    with pytest.raises(ValueError):  # 65 tokens: more than the layer takes
        ses.layer_dense_decode(torch.zeros(65, 64, dtype=F16, device="cuda"), c["layer"])
    with pytest.raises(ValueError):
        ses.layer_dense_decode(torch.zeros(2, 72, dtype=F16, device="cuda"), c["layer"])
    with pytest.raises(ValueError):
        ses.layer_dense_decode(c["x"].cuda().bfloat16(), c["layer"])
