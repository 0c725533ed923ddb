"""Cases, inputs, plain forms and exact values of the operators on 8-bit integer weights and tokens, and of the norms
around a block:

  quantize_int8  rows of 8-bit integers with a scale each: scale = max |x| / 127, q = x * 127 / max |x| rounded to the
                 nearest, halves to even
  linear_int8    y = act(s_x s_w (q_x q_w^T) + bias) [* (s_x s_mul (q_x q_mul^T) + bias_mul)] [+ residual]; x in 16 bits is
                 quantised by token on the way
  expert_int8    one SwiGLU expert: h = SiLU(x gate^T) * (x up^T), quantised by token, y = h down^T [+ residual]
  residual_norm  s = residual_scale * residual + block_scale * gate * post_norm(x), y = norm(s), in 16 bits or quantised

With `own` false, `run` computes them in elementary torch operations in 32 bits; with `own` true it calls the package.
"""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS = 1e-6


def _quantize(name, R, K, dtype):
    return dict(name=name, op="quantize_int8", R=R, K=K, dtype=dtype)


def _linear(name, M, N, K, dtype, x="16 bits", act="none", bias=False, gated=False, residual=False, out=None):
    return dict(name=name, op="linear_int8", M=M, N=N, K=K, dtype=dtype, x=x, act=act, bias=bias, gated=gated,
                residual=residual, out=out or dtype)


def _expert(name, n, d, f, dtype, x="16 bits", residual=False):
    return dict(name=name, op="expert_int8", n=n, d=d, f=f, dtype=dtype, x=x, residual=residual)


def _norm(name, M, d, dtype, post="none", norm="rms", gate_rows=0, residual_scale=1.0, block_scale=1.0, affine=False,
          wide=False, int8=False):
    return dict(name=name, op="residual_norm", M=M, d=d, dtype=dtype, post=post, norm=norm, gate_rows=gate_rows,
                residual_scale=residual_scale, block_scale=block_scale, affine=affine, wide=wide, int8=int8)


def listed():
    return [
        # a decode batch's hidden values before a down projection
        _quantize("quantize 48 tokens fp16", 48, 14336, "fp16"),
        # one projection's weights of a d = 4096, f = 14336 block, on loading a model
        _quantize("quantize weights bf16", 14336, 4096, "bf16"),
        # one decode token through the attention's output projection of a d = 4096 model, with its residual
        _linear("linear 1 token bf16", 1, 4096, 4096, "bf16", residual=True),
        # four drafted tokens, quantised by the norm before, through the output head: fp32 logits for the sampler
        _linear("linear head 4 tokens fp16", 4, 32000, 4096, "fp16", x="int8", out="fp32"),
        # an odd batch, odd output size and a ragged inner size, every part of the epilogue on
        _linear("linear ragged fp16", 333, 1031, 1008, "fp16", act="gelu", bias=True, residual=True),
        # a decode batch of 48 through the gated up projection of a d = 6144, f = 16384 block
        _linear("linear gated 48 tokens bf16", 48, 16384, 6144, "bf16", x="int8", act="silu", gated=True),
        # a prompt of 2048 tokens through the gated up projection of a d = 4096, f = 14336 block
        _linear("linear gated prompt bf16", 2048, 14336, 4096, "bf16", act="silu", gated=True),
        # one token through one small expert (d = 2048, f = 1408): the shortest call of the expert operator
        _expert("expert 1 token fp16", 1, 2048, 1408, "fp16"),
        # the tokens of one expert in a prompt's chunk, quantised by the norm before the layer
        _expert("expert 300 tokens bf16", 300, 4096, 14336, "bf16", x="int8", residual=True),
        # one decode token between two blocks: residual and RMSNorm, launch latency alone
        _norm("norm 1 token bf16", 1, 4096, "bf16", affine=True),
        # a decode batch of a d = 6144 stack with a norm behind the block as well, the next block's input in 8 bits
        _norm("norm 64 tokens int8 fp16", 64, 6144, "fp16", post="rms", affine=True, int8=True),
        # a prompt's tokens: two LayerNorms, a gate for each of 4 sequences, the residual stream in fp32
        _norm("norm 8192 tokens bf16", 8192, 4096, "bf16", post="layer", norm="layer", gate_rows=4, residual_scale=0.9,
              block_scale=0.5, affine=True, wide=True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("quantize_int8", "linear_int8", "expert_int8", "residual_norm"))
    dtype = rng.choice(("fp16", "bf16"))
    if op == "quantize_int8":
        c = _quantize("", _log_int(rng, 1, 8192), _log_int(rng, 64, 6144, 16), rng.choice((dtype, "fp32")))
    elif op == "linear_int8":
        gated = rng.random() < 0.3
        c = _linear("", _log_int(rng, 1, 2048), _log_int(rng, 16, 14336), _log_int(rng, 64, 8192, 16) // (2 if gated else 1) // 16 * 16,
                    dtype, x=rng.choice(("16 bits", "int8")), act=rng.choice(ACTS), bias=rng.random() < 0.5, gated=gated,
                    residual=rng.random() < 0.5, out=rng.choice((dtype, dtype, "fp32")))
    elif op == "expert_int8":
        c = _expert("", _log_int(rng, 1, 1024), _log_int(rng, 256, 6144, 16), _log_int(rng, 256, 8192, 16), dtype,
                    x=rng.choice(("16 bits", "int8")), residual=rng.random() < 0.5)
    else:
        M = _log_int(rng, 1, 4096)
        c = _norm("", M, _log_int(rng, 64, 16384, 8), dtype, post=rng.choice(("none", "rms", "layer")),
                  norm=rng.choice(("rms", "layer", "none")), gate_rows=rng.choice((0, 1, M)),
                  residual_scale=rng.choice((1.0, 0.75)), block_scale=rng.choice((1.0, 0.5)), affine=rng.random() < 0.7,
                  wide=rng.random() < 0.3)
        c["int8"] = c["norm"] != "none" and c["d"] % 16 == 0 and rng.random() < 0.4
    del c["name"]
    return c


def _normal(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _tokens(g, M, K, dtype):
    """Hidden states: most channels near one, one in 128 about ten times as large."""
    big = torch.rand((K,), generator=g, device="cuda") < 1 / 128
    x = torch.randn((M, K), generator=g, device="cuda", dtype=torch.float32)
    return x.mul_(torch.where(big, 10.0, 1.0)).to(dtype)


def _plain_quantize(x):
    """(q as fp32 integers, scale [rows, 1]).  64 bits where 32 could miss on which side of a half a quotient lies."""
    v = x.double() if x.dtype == torch.float32 else x.float()
    most = v.abs().amax(-1, keepdim=True)
    q = torch.round(v * 127 / torch.where(most == 0, torch.ones_like(most), most))
    return q.float(), most.float() / 127


def _weights(g, shape, std=0.02):
    q, scale = _plain_quantize(_normal(g, shape, torch.float32, std))
    return q.to(torch.int8), scale[..., 0].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "quantize_int8":
        s["x"] = _tokens(g, case["R"], case["K"], dt)
        return s
    if case["op"] == "residual_norm":
        M, d = case["M"], case["d"]
        s["x"] = _tokens(g, M, d, dt)
        s["residual"] = _normal(g, (M, d), torch.float32 if case["wide"] else dt, 2.0)
        s["gate"] = _normal(g, (case["gate_rows"], d), dt, 0.5) if case["gate_rows"] else None
        for which in ("post", "norm"):
            with_it = case["affine"] and case[which] != "none"
            s[which + "_weight"] = (1 + _normal(g, (d,), torch.float32, 0.1)).to(dt) if with_it else None
            s[which + "_bias"] = _normal(g, (d,), dt, 0.1) if with_it and case[which] == "layer" else None
        return s
    if case["op"] == "linear_int8":
        M, N, K = case["M"], case["N"], case["K"]
        s["w"], s["w_scale"] = _weights(g, (N, K))
        s["w_mul"], s["w_mul_scale"] = _weights(g, (N, K)) if case["gated"] else (None, None)
        s["bias"] = _normal(g, (N,), dt, 0.1) if case["bias"] else None
        s["bias_mul"] = _normal(g, (N,), dt, 0.1) if case["bias"] and case["gated"] else None
        s["residual"] = _normal(g, (M, N), dt) if case["residual"] else None
    else:
        M, d, f = case["n"], case["d"], case["f"]
        K = d
        for name, shape in (("gate", (1, f, d)), ("up", (1, f, d)), ("down", (1, d, f))):
            s[name], s[name + "_scale"] = _weights(g, shape)
        s["residual"] = _normal(g, (M, d), dt) if case["residual"] else None
    s["x"], s["x_scale"] = _tokens(g, M, K, dt), None
    if case["x"] == "int8":
        q, scale = _plain_quantize(s["x"])
        s["x"], s["x_scale"] = q.to(torch.int8), scale[:, 0].contiguous()
    if own:
        import sparse_expert_swiglu_gb300 as ses
        # the workspace that a program keeps for its calls of these sizes
        if case["op"] == "linear_int8":
            s["ws"] = ses.Workspace(ses.linear_int8_workspace_bytes(M, N, K, case["gated"]))
        else:
            s["experts"] = ses.Int8Experts(s["gate"], s["gate_scale"], s["up"], s["up_scale"], s["down"], s["down_scale"])
            s["ws"] = ses.Workspace(ses.expert_int8_workspace_bytes(M, d, f))
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


def _plain_x(s):
    if s["x_scale"] is None:
        return _plain_quantize(s["x"])
    return s["x"].float(), s["x_scale"][:, None]


def _plain_product(q, scale, w, w_scale, bias=None):
    a = (q @ w.float().t()) * scale * w_scale
    return a if bias is None else a + bias.float()


def _plain_linear(s):
    c = s["case"]
    q, scale = _plain_x(s)
    y = _act(c["act"], _plain_product(q, scale, s["w"], s["w_scale"], s["bias"]))
    if c["gated"]:
        y = y * _plain_product(q, scale, s["w_mul"], s["w_mul_scale"], s["bias_mul"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DTYPES[c["out"]])


def _plain_expert(s):
    q, scale = _plain_x(s)
    h = _act("silu", _plain_product(q, scale, s["gate"][0], s["gate_scale"][0]))
    h = h * _plain_product(q, scale, s["up"][0], s["up_scale"][0])
    y = _plain_product(*_plain_quantize(h), s["down"][0], s["down_scale"][0])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DTYPES[s["case"]["dtype"]])


def _plain_norm_of(v, kind, weight, bias):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    if weight is not None:
        v = v * weight.float()
    return v if bias is None else v + bias.float()


def _plain_residual_norm(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    u = _plain_norm_of(s["x"].float(), c["post"], s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        g = s["gate"].float()
        u = (u.view(len(g), -1, c["d"]) * g[:, None]).view(c["M"], c["d"])
    v = c["residual_scale"] * s["residual"].float() + c["block_scale"] * u
    kept = v.to(s["residual"].dtype)
    if c["norm"] == "none":
        return kept
    y = _plain_norm_of(v, c["norm"], s["norm_weight"], s["norm_bias"])
    if c["int8"]:
        q, scale = _plain_quantize(y)
        return kept, (q * scale).to(dt), scale[:, 0]
    return kept, y.to(dt)


def _values(q, scale, dtype):
    """What 8-bit integers stand for, rounded to the type."""
    return torch.mul(q, scale[:, None], out=torch.empty(q.shape, dtype=dtype, device=q.device))


def run(state):
    s = state
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if own:
        import sparse_expert_swiglu_gb300 as ses
        if c["op"] == "quantize_int8":
            q, scale = ses.quantize_int8(s["x"])
            return q * scale[:, None], scale
        if c["op"] == "linear_int8":
            return ses.linear_int8(s["x"], s["w"], s["w_scale"], x_scale=s["x_scale"], bias=s["bias"], act=c["act"],
                                   w_mul=s["w_mul"], w_mul_scale=s["w_mul_scale"], bias_mul=s["bias_mul"],
                                   residual=s["residual"], dtype=dt, out_dtype=DTYPES[c["out"]], ws=s["ws"])
        if c["op"] == "expert_int8":
            return ses.expert_int8_swiglu(s["x"], s["experts"], 0, x_scale=s["x_scale"], residual=s["residual"], dtype=dt,
                                          ws=s["ws"])
        out = ses.residual_norm(s["x"], s["residual"], post=c["post"], post_weight=s["post_weight"], post_bias=s["post_bias"],
                                gate=s["gate"], residual_scale=c["residual_scale"], block_scale=c["block_scale"],
                                norm=c["norm"], weight=s["norm_weight"], bias=s["norm_bias"], eps=EPS, int8=c["int8"])
        return (out[0], _values(out[1], out[2], dt), out[2]) if c["int8"] else out
    if c["op"] == "quantize_int8":
        q, scale = _plain_quantize(s["x"])
        return q * scale, scale[:, 0]
    if c["op"] == "linear_int8":
        return _plain_linear(s)
    return _plain_expert(s) if c["op"] == "expert_int8" else _plain_residual_norm(s)


def work(case):
    two = {"fp16": 2, "bf16": 2, "fp32": 4}
    if case["op"] == "quantize_int8":
        n = case["R"] * case["K"]
        return {"bytes": n * (two[case["dtype"]] + 1) + 4 * case["R"], "flops": 4 * n}
    if case["op"] == "residual_norm":
        M, d = case["M"], case["d"]
        wide = 4 if case["wide"] else 2
        last = 0 if case["norm"] == "none" else 1 if case["int8"] else 2
        vectors = 2 * d * (case["gate_rows"] + sum((case[k] != "none") + (case[k] == "layer") for k in ("post", "norm")) * case["affine"])
        return {"bytes": M * d * (2 + 2 * wide + last) + vectors + 4 * M * case["int8"], "flops": 16 * M * d}
    if case["op"] == "linear_int8":
        M, N, K, mats = case["M"], case["N"], case["K"], 2 if case["gated"] else 1
        nbytes = mats * (N * K + 4 * N + 2 * N * case["bias"]) + M * N * (two[case["out"]] + 2 * case["residual"])
        products = mats * N * K
    else:
        M, d, f = case["n"], case["d"], case["f"]
        N, K = d, d
        nbytes = 3 * d * f + 4 * (2 * f + d) + M * d * (2 + 2 * case["residual"])
        products = 3 * d * f
    nbytes += M * K + 4 * M if case["x"] == "int8" else 2 * M * K
    return {"bytes": nbytes, "flops": 2 * M * products}


def _exact_rows(x):
    """Integers and scale of rows in 64 bits."""
    most = x.abs().max(dim=-1, keepdim=True).values
    steps = x / torch.clamp(most, min=1e-300) * 127
    # a quotient that is a half to 12 digits is one (16-bit inputs): to the even neighbour
    half = torch.floor(steps) + 0.5
    steps = torch.where((steps - half).abs() < 1e-12 * 127, half, steps)
    return torch.round(steps), most / 127


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "quantize_int8":
        q, scale = _exact_rows(s["x"].double())
        return q * scale, scale[:, 0]
    res = s["residual"].double() if s["residual"] is not None else 0.0
    if case["op"] == "residual_norm":
        f = torch.nn.functional
        d = case["d"]

        def normed(v, kind, weight, bias):
            w = None if weight is None else weight.double()
            if kind == "layer":
                return f.layer_norm(v, (d,), w, None if bias is None else bias.double(), EPS)
            if kind == "rms":
                v = v * torch.rsqrt(v.pow(2).mean(dim=1, keepdim=True) + EPS)
                return v if w is None else v * w
            return v
        u = normed(s["x"].double(), case["post"], s["post_weight"], s["post_bias"])
        if case["gate_rows"]:
            u = u * s["gate"].double().repeat_interleave(case["M"] // case["gate_rows"], dim=0)
        v = res * case["residual_scale"] + u * case["block_scale"]
        if case["norm"] == "none":
            return v
        y = normed(v, case["norm"], s["norm_weight"], s["norm_bias"])
        if case["int8"]:
            q, scale = _exact_rows(y)
            return v, q * scale, scale[:, 0]
        return v, y
    if s["x_scale"] is None:
        q, scale = _exact_rows(s["x"].double())
    else:
        q, scale = s["x"].double(), s["x_scale"].double()[:, None]
    x = q * scale

    def product(a, w, w_scale, b):
        y = torch.matmul(a, (w.double() * w_scale.double()[:, None]).t())
        return y if b is None else y + b.double()
    if case["op"] == "linear_int8":
        f = torch.nn.functional
        a = {"none": lambda v: v, "relu": f.relu, "gelu": f.gelu, "gelu_tanh": lambda v: f.gelu(v, approximate="tanh"),
             "silu": f.silu}[case["act"]](product(x, s["w"], s["w_scale"], s["bias"]))
        if case["gated"]:
            a = a * product(x, s["w_mul"], s["w_mul_scale"], s["bias_mul"])
        return a + res
    g = product(x, s["gate"][0], s["gate_scale"][0], None)
    q, scale = _exact_rows(g * torch.sigmoid(g) * product(x, s["up"][0], s["up_scale"][0], None))
    return product(q * scale, s["down"][0], s["down_scale"][0], None) + res
