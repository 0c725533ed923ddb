"""Cases, inputs, plain forms and exact values of three operators on uncompressed 16-bit weights:

  linear         y = act(x w^T + bias) [* (x w_mul^T + bias_mul)] [+ residual]
  expert_dense   one SwiGLU expert on n tokens: y = (SiLU(x gate^T) * (x up^T)) down [+ residual]
  layer_dense    a whole mixture-of-experts layer on up to 64 tokens: routing, the chosen experts,
                 the always-on shared experts, their weighted sum [+ residual] [RMSNorm]

With `own` false, `run` computes them in elementary torch operations in 32 bits (the router's logits,
whose order decides the experts, in 64); with `own` true it calls the package.
"""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS = 1e-6


def _linear(name, M, N, K, dtype, act="none", bias=False, gated=False, residual=False, layout="nk", out=None):
    return dict(name=name, op="linear", M=M, N=N, K=K, dtype=dtype, act=act, bias=bias, gated=gated,
                residual=residual, layout=layout, out=out or dtype)


def _expert(name, n, d, f, dtype, residual=False):
    return dict(name=name, op="expert_dense", n=n, d=d, f=f, dtype=dtype, residual=residual)


def _layer(name, B, d, f, E, k, shared, dtype, renorm=True, residual=False, rmsnorm=False):
    return dict(name=name, op="layer_dense", B=B, d=d, f=f, E=E, k=k, shared=shared, dtype=dtype, renorm=renorm,
                residual=residual, rmsnorm=rmsnorm)


def listed():
    return [
        # one decode token through the attention's output projection of a d = 4096 model, with its residual
        _linear("linear 1 token bf16", 1, 4096, 4096, "bf16", residual=True),
        # four drafted tokens through the output head: fp32 logits for the sampler
        _linear("linear head 4 tokens fp16", 4, 32000, 4096, "fp16", out="fp32"),
        # an odd batch, odd output size and a ragged inner size, every part of the epilogue on
        _linear("linear ragged fp16", 333, 1031, 1000, "fp16", act="gelu", bias=True, residual=True),
        # a prompt of 2048 tokens through the gated up projection of a d = 4096, f = 14336 block
        _linear("linear gated prompt bf16", 2048, 14336, 4096, "bf16", act="silu", gated=True),
        # a prompt through the down projection, stored [f][d] as the experts' down rows are
        _linear("linear down prompt fp16", 2048, 4096, 14336, "fp16", residual=True, layout="kn"),
        # one token through one small expert (d = 2048, f = 1408): the shortest call of the expert operator
        _expert("expert 1 token fp16", 1, 2048, 1408, "fp16"),
        # the tokens of one expert in a prompt's chunk
        _expert("expert 300 tokens bf16", 300, 4096, 14336, "bf16", residual=True),
        # one decode token, 8 large experts, 2 per token
        _layer("layer 8x14336 1 token fp16", 1, 4096, 14336, 8, 2, 0, "fp16"),
        # a few drafted tokens of a d = 6144 stack: RMSNorm on the way out
        _layer("layer 8x16384 5 tokens bf16", 5, 6144, 16384, 8, 2, 0, "bf16", rmsnorm=True),
        # one decode token, 64 small experts, 6 per token, 2 shared: launch latency counts
        _layer("layer 64x1408 1 token bf16", 1, 2048, 1408, 64, 6, 2, "bf16", renorm=False, residual=True),
        # a full decode batch over the same layer: every expert has a few tokens
        _layer("layer 64x1408 64 tokens fp16", 64, 2048, 1408, 64, 6, 2, "fp16", renorm=False),
        # a small decode batch of the large experts, next layer's input
        _layer("layer 8x14336 17 tokens bf16", 17, 4096, 14336, 8, 2, 0, "bf16", residual=True, rmsnorm=True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("linear", "expert_dense", "layer_dense"))
    dtype = rng.choice(("fp16", "bf16"))
    if op == "linear":
        layout = rng.choice(("nk", "nk", "kn"))
        gated = rng.random() < 0.3
        c = _linear("", _log_int(rng, 1, 2048), _log_int(rng, 16, 14336, 8 if layout == "kn" else 1),
                    _log_int(rng, 64, 8192, 8), dtype, act=rng.choice(ACTS), bias=rng.random() < 0.5, gated=gated,
                    residual=rng.random() < 0.5, layout=layout, out=rng.choice((dtype, dtype, "fp32")))
    elif op == "expert_dense":
        c = _expert("", _log_int(rng, 1, 1024), _log_int(rng, 256, 6144, 8), _log_int(rng, 256, 14336, 8), dtype,
                    residual=rng.random() < 0.5)
    else:
        E = _log_int(rng, 4, 64)
        c = _layer("", _log_int(rng, 1, 64), _log_int(rng, 512, 4096, 8), _log_int(rng, 256, 4096, 8), E,
                   rng.randint(1, min(8, E)), rng.randint(0, 2), dtype, renorm=rng.random() < 0.5,
                   residual=rng.random() < 0.5, rmsnorm=rng.random() < 0.5)
    del c["name"]
    return c


def _normal(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        wshape = (N, K) if case["layout"] == "nk" else (K, N)
        s["x"] = _normal(g, (M, K), dt)
        s["w"] = _normal(g, wshape, dt, 0.02)
        s["w_mul"] = _normal(g, wshape, dt, 0.02) if case["gated"] else None
        s["bias"] = _normal(g, (N,), dt, 0.1) if case["bias"] else None
        s["bias_mul"] = _normal(g, (N,), dt, 0.1) if case["bias"] and case["gated"] else None
        s["residual"] = _normal(g, (M, N), dt) if case["residual"] else None
        if own:
            import sparse_expert_swiglu_gb300 as ses
            # the workspace that a program keeps for its calls of these sizes
            s["ws"] = ses.Workspace(ses.linear_workspace_bytes(M, N, K, case["gated"]))
        return s
    d, f = case["d"], case["f"]
    if case["op"] == "expert_dense":
        n, E, shared = case["n"], 1, 0
    else:
        n, E, shared = case["B"], case["E"], case["shared"]
        s["w_router"] = _normal(g, (d, E), dt, 0.02)
    s["x"] = _normal(g, (n, d), dt)
    s["residual"] = _normal(g, (n, d), dt) if case["residual"] else None
    for which, count in (("routed", E), ("shared", shared)):
        s[which] = [_normal(g, (count, f, d), dt, 0.02) for _ in range(3)] if count else None
    if own:
        import sparse_expert_swiglu_gb300 as ses
        experts = ses.DenseExperts(*s["routed"])
        if case["op"] == "expert_dense":
            s["experts"] = experts
            s["ws"] = ses.Workspace(ses.expert_dense_workspace_bytes(n, d, f))
        else:
            more = ses.DenseExperts(*s["shared"]) if shared else None
            s["layer"] = ses.DenseLayer(s["w_router"], experts, case["k"], case["renorm"], more)
            s["ws"] = ses.Workspace(ses.layer_dense_workspace_bytes(s["layer"], n))
    return s


def _act(name, a):
    if name == "relu":
        return torch.where(a > 0, a, torch.zeros_like(a))
    if name == "gelu":
        return 0.5 * a * (1 + torch.erf(a * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a * a * a)))
    if name == "silu":
        return a / (1 + torch.exp(-a))
    return a


def _plain_linear(s):
    c = s["case"]
    x = s["x"].float()
    turn = (lambda w: w.float().t()) if c["layout"] == "nk" else (lambda w: w.float())
    a = x @ turn(s["w"])
    if s["bias"] is not None:
        a = a + s["bias"].float()
    a = _act(c["act"], a)
    if s["w_mul"] is not None:
        b = x @ turn(s["w_mul"])
        if s["bias_mul"] is not None:
            b = b + s["bias_mul"].float()
        a = a * b
    if s["residual"] is not None:
        a = a + s["residual"].float()
    return a.to(DTYPES[c["out"]])


def _plain_experts(x, gate_t, up_t, down):
    """x [E or 1, n, d] through experts [E, f, d] -> [E, n, d], all in fp32."""
    h = _act("silu", x @ gate_t.float().transpose(-1, -2)) * (x @ up_t.float().transpose(-1, -2))
    return h @ down.float()


def _plain_layer(s):
    c = s["case"]
    B, E, k = c["B"], c["E"], c["k"]
    x = s["x"].float()
    logits = s["x"].double() @ s["w_router"].double()
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    over = top if c["renorm"] else logits
    w = (torch.exp(top - top[:, :1]) / torch.exp(over - top[:, :1]).sum(1, keepdim=True)).float()
    if B * k <= E:  # few pairs: the chosen experts' weights by index
        pick = idx.reshape(-1)
        xs = x.repeat_interleave(k, dim=0)[:, None, :]
        out = _plain_experts(xs, *(t[pick] for t in s["routed"]))[:, 0].reshape(B, k, -1)
        y = (out * w[:, :, None]).sum(1)
    else:           # every expert on every token, weighted by what the router gave it
        table = torch.zeros((B, E), device=x.device).scatter_(1, idx, w)
        y = (_plain_experts(x[None], *s["routed"]) * table.t()[:, :, None]).sum(0)
    if s["shared"] is not None:
        y = y + _plain_experts(x[None], *s["shared"]).sum(0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    if c["rmsnorm"]:
        y = y / torch.sqrt((y * y).mean(1, keepdim=True) + EPS)
    return y.to(DTYPES[c["dtype"]])


def run(state):
    s = state
    c = s["case"]
    if own:
        import sparse_expert_swiglu_gb300 as ses
        if c["op"] == "linear":
            return ses.linear(s["x"], s["w"], bias=s["bias"], act=c["act"], w_mul=s["w_mul"], bias_mul=s["bias_mul"],
                              residual=s["residual"], w_layout=c["layout"], out_dtype=DTYPES[c["out"]], ws=s["ws"])
        if c["op"] == "expert_dense":
            return ses.expert_dense_swiglu(s["x"], s["experts"], 0, residual=s["residual"], ws=s["ws"])
        return ses.layer_dense_decode(s["x"], s["layer"], residual=s["residual"], rmsnorm=c["rmsnorm"], ws=s["ws"])
    if c["op"] == "linear":
        return _plain_linear(s)
    if c["op"] == "expert_dense":
        y = _plain_experts(s["x"].float()[None], *s["routed"])[0]
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(DTYPES[c["dtype"]])
    return _plain_layer(s)


def work(case):
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        mats = 2 if case["gated"] else 1
        wide = 4 if case["out"] == "fp32" else 2
        nbytes = 2 * mats * N * K + 2 * M * K + wide * M * N
        nbytes += 2 * M * N * case["residual"] + 2 * mats * N * case["bias"]
        return {"bytes": nbytes, "flops": 2 * mats * M * N * K}
    d, f = case["d"], case["f"]
    if case["op"] == "expert_dense":
        n, active, pairs, router = case["n"], 1, case["n"], 0
    else:
        n, E, k = case["B"], case["E"], case["k"]
        # experts that n tokens of independent choice reach, on average
        active = E * (1 - (1 - k / E) ** n) + case["shared"]
        pairs, router = n * (k + case["shared"]), d * E
    nbytes = 2 * (3 * active * f * d + router + n * d * (3 if case["residual"] else 2))
    return {"bytes": nbytes, "flops": 6 * pairs * f * d + 2 * n * router}


def _exact_expert(x, gate_t, up_t, down):
    a, u = x @ gate_t.double().t(), x @ up_t.double().t()
    return (a * torch.sigmoid(a) * u) @ down.double()


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    x = s["x"].double()
    res = s["residual"].double() if s["residual"] is not None else 0.0
    if case["op"] == "linear":
        def product(w, b):
            a = torch.matmul(x, w.double().t() if case["layout"] == "nk" else w.double())
            return a if b is None else a + b.double()
        a = product(s["w"], s["bias"])
        f = torch.nn.functional
        a = {"none": lambda v: v, "relu": f.relu, "gelu": f.gelu, "gelu_tanh": lambda v: f.gelu(v, approximate="tanh"),
             "silu": f.silu}[case["act"]](a)
        if case["gated"]:
            a = a * product(s["w_mul"], s["bias_mul"])
        return a + res
    if case["op"] == "expert_dense":
        return _exact_expert(x, *(t[0] for t in s["routed"])) + res
    logits = x @ s["w_router"].double()
    y = torch.zeros_like(x)
    order = torch.argsort(-logits, dim=1, stable=True)[:, :case["k"]]
    prob = torch.softmax(torch.gather(logits, 1, order) if case["renorm"] else logits, dim=1)
    weight = prob if case["renorm"] else torch.gather(prob, 1, order)
    for e in range(case["E"]):
        b, j = torch.nonzero(order == e, as_tuple=True)
        if len(b):
            y[b] += weight[b, j][:, None] * _exact_expert(x[b], *(t[e] for t in s["routed"]))
    for e in range(case["shared"]):
        y += _exact_expert(x, *(t[e] for t in s["shared"]))
    y = y + res
    return y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) if case["rmsnorm"] else y
