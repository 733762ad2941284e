"""The operators on either side of the framework's projections, in plain torch and
as a user calls them: the residual's addition with the RMS norm in front of a
projection (rows out, or straight into an INT8 or FP8 linear; forward and backward),
and a whole mixture-of-experts layer for a few tokens.

`run(prepare(case, seed))` is one pass.  With `own` false it is elementary torch
arithmetic in 32 bits (routing in 64); with `own` true it is the calls of
`w8a8_int8_rotated_amd.convrot`.  Cases are plain dicts; `exact` evaluates the
definitions in 64 bits.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}
EPS = 1e-6


def listed():
    return [
        # one token's hidden state in front of a layer: latency
        norm("norm_step", M=1, K=5376),
        # a text prompt's fp32 rows of a width that is no multiple of 128
        norm("norm_text", M=1093, K=4104, x="f32", res="f32", out="f32"),
        # a 768p packed sequence, its residual stream kept in fp32
        norm("norm_768p", M=38656, K=5376, res="f32"),
        # straight into the INT8 QKV projection: drafted tokens, and the packed sequence
        norm_linear("norm_int8_drafts", M=5, K=5376, N=16128),
        norm_linear("norm_int8_768p", M=38656, K=5376, N=16128, res="f32"),
        # into an FP8 output projection with power-of-two scales: an odd prompt
        norm_linear("norm_fp8_prompt", M=333, K=5376, N=5376, kind="fp8_pow2", bias=True),
        # backward: a small fp32 batch, and fine-tuning on the packed sequence with
        # bf16 branches beside the fp32 stream
        norm_bwd("norm_bwd_batch", M=1527, K=2304, g="f32", h="f32", x="f32"),
        norm_bwd("norm_bwd_768p", M=38656, K=5376, g="bf16", h="f32", x="bf16"),
        # one token through many small experts: latency
        moe("moe_token", T=1, K=2048, F=768, E=128, k=8),
        # drafted tokens through wide experts, sigmoid scores with a balancing bias and
        # a shared expert
        moe("moe_drafts", T=5, K=5376, F=1408, E=32, k=4, S=1, score="sigmoid", bias=True,
            scale=2.5, scales="pow2", router="f32"),
        # an odd batch, weights not renormalised, fp32 out
        moe("moe_batch", T=23, K=2560, F=640, E=40, k=6, renorm=False, out="f32"),
        # a serving batch that touches every expert
        moe("moe_serving", T=64, K=5376, F=1408, E=64, k=6),
    ]


def norm(name, M, K, x="bf16", res="bf16", out="bf16"):
    return {"name": name, "op": "norm", "M": M, "K": K, "x": x, "res": res, "out": out}


def norm_linear(name, M, K, N, res="bf16", kind="int8", block=128, rotation="sylvester",
                bias=False):
    return {"name": name, "op": "norm_linear", "M": M, "K": K, "N": N, "x": "bf16", "res": res,
            "kind": kind, "block": block, "rotation": rotation, "bias": bias}


def norm_bwd(name, M, K, g, h, x):
    return {"name": name, "op": "norm_bwd", "M": M, "K": K, "g": g, "h": h, "x": x}


def moe(name, T, K, F, E, k, S=0, score="softmax", bias=False, renorm=True, scale=1.0,
        scales="f32", router="bf16", out="bf16"):
    return {"name": name, "op": "moe", "T": T, "K": K, "F": F, "E": E, "k": k, "S": S,
            "score": score, "bias": bias, "renorm": renorm, "scale": scale, "scales": scales,
            "router": router, "out": out}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_linear", "norm_bwd", "moe", "moe"])
    top = 38656 * 5376
    if op == "moe":
        E = _log_int(rng, 4, 160)
        K, F = 128 * _log_int(rng, 2, 42), 128 * _log_int(rng, 1, 16)
        S = rng.choice([0, 0, 1, 2])
        E = max(4, min(E, 64 * 5376 * 1408 // (K * F) - S))
        c = moe("", _log_int(rng, 1, 96), K, F, E, rng.randint(1, min(E, 10)), S,
                rng.choice(["softmax", "sigmoid"]), rng.random() < 0.4, rng.random() < 0.6,
                rng.choice([1.0, 2.5]), rng.choice(["f32", "pow2"]), rng.choice(["bf16", "f32"]),
                rng.choice(["bf16", "bf16", "f32"]))
    elif op == "norm_linear":
        K, N = 128 * _log_int(rng, 1, 96), 16 * _log_int(rng, 8, 1008)
        M = _log_int(rng, 1, min(38656, 38656 * 5376 * 16128 // (K * N), top // K))
        block, rotation = rng.choice([(64, "sylvester"), (128, "sylvester"), (64, "regular")] +
                                     ([(256, "sylvester"), (256, "regular")] if K % 256 == 0
                                      else []))
        c = norm_linear("", M, K, N, rng.choice(["none", "bf16", "f32"]),
                        rng.choice(["int8", "fp8_f32", "fp8_pow2"]), block, rotation,
                        rng.random() < 0.5)
    else:
        K = 8 * _log_int(rng, 4, 2048)
        M = _log_int(rng, 1, min(top // K, 1 << 17))
        if op == "norm":
            x = rng.choice(["bf16", "bf16", "f32"])
            c = norm("", M, K, x, rng.choice(["none", "bf16", "f32"] if x == "bf16"
                                             else ["none", "f32"]), rng.choice(["bf16", "f32"]))
        else:
            h = rng.choice(["bf16", "f32"])
            c = norm_bwd("", M, K, rng.choice(["bf16", "f32"]), h,
                         rng.choice(["bf16", "f32"]) if h == "f32" else "bf16")
    del c["name"]
    return c


_SIZE = {"bf16": 2, "f32": 4, "none": 0}


def work(case):
    if case["op"] == "moe":
        T, K, F, E, k, S = (case[n] for n in "TKFEkS")
        used = E * (1 - (1 - k / E) ** T) + S        # experts that T tokens choose, expected
        nbytes = used * 3 * F * K * (1 + 4 / 128 ** 2) + E * K * _SIZE[case["router"]] \
            + T * K * (2 + _SIZE[case["out"]])
        return {"bytes": nbytes, "flops": 2 * T * ((k + S) * 3 * F * K + E * K)}
    M, K = case["M"], case["K"]
    if case["op"] == "norm_bwd":
        per = _SIZE[case["g"]] + 3 * _SIZE[case["h"]] + (2 if case["x"] != case["h"] else 0)
        return {"bytes": M * K * per + 8 * K, "flops": 12 * M * K}
    nbytes = M * K * (_SIZE[case["x"]] + 2 * _SIZE[case["res"]]) + 4 * K
    if case["op"] == "norm":
        return {"bytes": nbytes + M * K * _SIZE[case["out"]], "flops": 6 * M * K}
    N = case["N"]
    return {"bytes": nbytes + N * K + 2 * M * N, "flops": 2 * M * N * K}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=F32)


def prepare(case, seed):
    if case["op"] == "moe":
        return _prepare_moe(case, seed)
    g = _gen(seed)
    M, K = case["M"], case["K"]
    state = {"case": case, "w": 1 + 0.2 * _randn(g, K)}
    # a few channels of a residual stream carry outliers
    hot = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 30.0, 1.0)
    if case["op"] == "norm_bwd":
        state["g"] = (_randn(g, M, K) * 0.01).to(DTYPES[case["g"]])
        state["h"] = (_randn(g, M, K) * hot).to(DTYPES[case["h"]])
        state["g_h"] = (_randn(g, M, K) * 0.01).to(DTYPES[case["h"]])
        return state
    state["x"] = _randn(g, M, K).to(DTYPES[case["x"]])
    state["res"] = None
    if case["res"] != "none":
        state["res"] = (_randn(g, M, K) * hot * 3).to(DTYPES[case["res"]])
    if case["op"] == "norm_linear":
        _prepare_linear(case, g, state)
    return state


def run(state):
    return {"norm": _run_norm, "norm_linear": _run_norm_linear, "norm_bwd": _run_norm_bwd,
            "moe": _run_moe}[state["case"]["op"]](state)


def exact(case, seed):
    was = own
    globals()["own"] = False
    try:
        state = prepare(case, seed)
    finally:
        globals()["own"] = was
    return {"norm": _exact_norm, "norm_linear": _exact_norm_linear, "norm_bwd": _exact_norm_bwd,
            "moe": _exact_moe}[case["op"]](state)


# ------------------------------------ the residual's addition and the norm ----
# h = x + residual, rounded to the residual's type; y = h rsqrt(mean h^2 + eps) w.

def _add_norm(state):
    """(h or None, y in 32 bits)"""
    h = None
    v = state["x"].to(F32)
    if state["res"] is not None:
        h = (v + state["res"].to(F32)).to(state["res"].dtype)
        v = h.to(F32)
    return h, v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * state["w"]


def _run_norm(state):
    case = state["case"]
    if own:
        from w8a8_int8_rotated_amd import convrot
        return convrot.convrot_add_rms_norm_forward(state["x"], state["w"], state["res"], eps=EPS,
                                                    out_dtype=DTYPES[case["out"]])
    h, y = _add_norm(state)
    return y.to(DTYPES[case["out"]]), h


def _exact_add_norm(state):
    h, v = None, state["x"].double()
    if state["res"] is not None:
        h = (v + state["res"].double()).to(state["res"].dtype).double()
        v = h
    norm = ((v * v).sum(-1, keepdim=True) / v.shape[-1] + EPS).sqrt()
    return h, v / norm * state["w"].double()


def _exact_norm(state):
    h, y = _exact_add_norm(state)
    return y, h


# ------------------------------------------- the norm in front of a linear ----
# INT8: v = H_b y over blocks of b channels; codes rint(v 127 / amax) and one scale
# amax / 127 / sqrt(b) a row; weights are codes of rotated rows with a scale each.
# FP8: e4m3 codes with a scale per 128 inputs of a row and per 128 x 128 weight block.

def _hadamard(block, rotation, dtype):
    h4 = torch.ones(4, 4, dtype=dtype, device="cuda")
    h4 = h4 - 2 * torch.eye(4, dtype=dtype, device="cuda")
    h2 = torch.tensor([[1, 1], [1, -1]], dtype=dtype, device="cuda")
    part = h4 if rotation == "regular" else h2
    times = int(round(math.log(block, part.shape[0])))
    h = torch.ones(1, 1, dtype=dtype, device="cuda")
    for _ in range(times):
        h = torch.kron(h, part)
    return h


def _prepare_linear(case, g, state):
    K, N = case["K"], case["N"]
    w = _randn(g, N, K) * 0.02
    state["bias"] = _randn(g, N) * 0.01 if case["bias"] else None
    if case["kind"] == "int8":
        H = _hadamard(case["block"], case["rotation"], F32)
        v = (w.view(N, -1, case["block"]) @ H).view(N, K)
        amax = v.abs().amax(-1, keepdim=True)
        state["codes"] = (v * (127 / amax)).round().to(torch.int8)
        state["scale"] = (amax / 127 / math.sqrt(case["block"])).view(N)
    else:
        state["codes"], state["scale"] = _quantize_weight(w, case["kind"][4:])
    if own:
        from w8a8_int8_rotated_amd import convrot
        if case["kind"] == "int8":
            state["weights"] = convrot.convrot_linear_prepare_weights(
                state["codes"], case["block"], src_scale=state["scale"],
                rotation=case["rotation"])
        else:
            state["weights"] = convrot.convrot_fp8_prepare_weights(
                state["codes"], src_scale=state["scale"], scales=case["kind"][4:])


def _pow2_up(s):
    m, e = torch.frexp(s)                            # s = m 2^e, 0.5 <= m < 1
    e = torch.where(m == 0.5, e - 1, e)
    return torch.where(s > 0, torch.ldexp(torch.ones_like(s), e), s)


def _scale(amax, kind):
    # the quotients in 64 bits, rounded once: correctly rounded 32-bit division
    s = (amax.double() / 448).to(F32).clamp_min(2.0 ** -126)
    return torch.where(amax > 0, _pow2_up(s) if kind == "pow2" else s, amax)


def _quantize_weight(w, kind):
    N, K = w.shape
    pad = -N % 128
    wb = torch.nn.functional.pad(w, (0, 0, 0, pad)).view((N + pad) // 128, 128, K // 128, 128)
    s = _scale(wb.abs().amax((1, 3)), kind)
    q = (wb / s.clamp_min(1e-38)[:, None, :, None]).view(N + pad, K)[:N]
    return q.clamp(-448, 448).to(torch.float8_e4m3fn), s


def _run_norm_linear(state):
    case = state["case"]
    if own:
        from w8a8_int8_rotated_amd import convrot
        return convrot.convrot_norm_linear_forward(state["x"], state["w"], state["weights"],
                                                   state["res"], bias=state["bias"], eps=EPS)
    M, K, N = case["M"], case["K"], case["N"]
    h, y = _add_norm(state)
    if case["kind"] == "int8":
        b = case["block"]
        v = (y.view(M, -1, b) @ _hadamard(b, case["rotation"], F32)).view(M, K)
        amax = v.abs().amax(-1, keepdim=True)
        q = (v * (127 / amax)).round()
        out = (q @ state["codes"].to(F32).t()) * (amax / 127 / math.sqrt(b)) * state["scale"]
    else:
        x = y.view(M, K // 128, 128)
        s = _scale(x.abs().amax(-1, keepdim=True), case["kind"][4:])
        inv = torch.where(s > 0, (1 / s.double()).to(F32), s)
        xq = ((x * inv).clamp(-448, 448).to(torch.float8_e4m3fn).to(F32) * s).view(M, K)
        sw = state["scale"].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
        out = xq @ (state["codes"].to(F32) * sw).t()
    if state["bias"] is not None:
        out = out + state["bias"]
    return out.to(BF16), h


def _exact_norm_linear(state):
    case = state["case"]
    M, K, N = case["M"], case["K"], case["N"]
    h, y = _exact_add_norm(state)
    if case["kind"] == "int8":
        b = case["block"]
        v = torch.matmul(y.reshape(-1, b), _hadamard(b, case["rotation"], torch.float64))
        v = v.reshape(M, K)
        top = v.abs().max(-1, keepdim=True).values
        q = torch.round(v * 127.0 / top)
        sx = top / 127.0 / b ** 0.5
        w = state["codes"].double() * state["scale"].double()[:, None]
        out = torch.matmul(q * sx, w.t())
    else:
        x = y.reshape(M, K // 128, 128)
        s = torch.clamp(x.abs().max(-1, keepdim=True).values / 448.0, min=2.0 ** -126)
        if case["kind"] == "fp8_pow2":
            s = torch.exp2(torch.ceil(torch.log2(s)).clamp_min(-126))
        v = x / s
        # e4m3: steps of 2^(e - 3) from 2^e up, 2^-9 below 2^-6; ties to even
        e = torch.frexp(v)[1].double().sub(1).clamp_min(-6)
        step = torch.exp2(e - 3)
        q = (torch.round(v / step) * step).clamp(-448, 448)
        xq = (q * s).reshape(M, K)
        del x, v, e, step, q
        w = state["codes"].float().double()
        idx = torch.arange(N, device="cuda") // 128
        for kb in range(K // 128):
            w[:, 128 * kb:128 * kb + 128] *= state["scale"].double()[idx, kb][:, None]
        out = torch.matmul(xq, w.t())
    if state["bias"] is not None:
        out = out + state["bias"].double()
    return out, h


# ------------------------------------------------------ the norm's backward ----
# From g, the gradient of y, and g_h, the one that reaches h along the residual
# stream: the gradient of h (which is the residual's, and x's in x's type) and of w.

def _run_norm_bwd(state):
    case = state["case"]
    if own:
        from w8a8_int8_rotated_amd import convrot
        dh, dx, dw = convrot.convrot_add_rms_norm_backward(
            state["g"], state["h"], state["w"], g_h=state["g_h"], eps=EPS,
            x_dtype=DTYPES[case["x"]])
        return (dh, dw) if case["x"] == case["h"] else (dh, dw, dx)
    h, g = state["h"].to(F32), state["g"].to(F32)
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    hh = h * r
    t = g * state["w"]
    d = state["g_h"].to(F32) + r * (t - hh * (t * hh).mean(-1, keepdim=True))
    # sums over all rows: 64 bits where 32 would lose them
    dw = (g * hh).sum(0, dtype=torch.float64).to(F32)
    out = (d.to(state["h"].dtype), dw)
    return out if case["x"] == case["h"] else (*out, d.to(DTYPES[case["x"]]))


def _exact_norm_bwd(state):
    """By differentiation of the definition, in 64 bits."""
    case = state["case"]
    h = state["h"].double().requires_grad_()
    w = state["w"].double().requires_grad_()
    y = h / ((h * h).sum(-1, keepdim=True) / h.shape[-1] + EPS).sqrt() * w
    dh, dw = torch.autograd.grad(y, (h, w), state["g"].double())
    dh = dh + state["g_h"].double()
    return (dh, dw) if case["x"] == case["h"] else (dh, dw, dh)


# ------------------------------------------------ a mixture-of-experts layer ----
# logits = x router^T; the k experts of the largest logits (with a bias: of the
# largest score + bias), ties to the lowest index; weights: their scores, divided by
# their sum or not, times a factor.  Expert e: D_e (silu(G_e x) * (U_e x)), [G_e; U_e]
# and D_e of e4m3 codes with a scale per 128 x 128 block.  The last S experts serve
# every token with weight 1.

def _prepare_moe(case, seed):
    g = _gen(seed)
    T, K, F, E, S = (case[n] for n in ("T", "K", "F", "E", "S"))
    hot = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 10.0, 1.0)
    state = {"case": case, "x": (_randn(g, T, K) * hot).to(BF16)}
    state["router"] = (_randn(g, E, K) / math.sqrt(K)).to(DTYPES[case["router"]])
    state["bias"] = _randn(g, E) * 0.05 if case["bias"] else None
    gu = torch.empty(E + S, 2 * F, K, dtype=torch.float8_e4m3fn, device="cuda")
    dn = torch.empty(E + S, K, F, dtype=torch.float8_e4m3fn, device="cuda")
    sgu = torch.empty(E + S, 2 * F // 128, K // 128, device="cuda")
    sdn = torch.empty(E + S, K // 128, F // 128, device="cuda")
    for e in range(E + S):
        gu[e], sgu[e] = _quantize_weight(_randn(g, 2 * F, K) / math.sqrt(K), case["scales"])
        dn[e], sdn[e] = _quantize_weight(_randn(g, K, F) / math.sqrt(F), case["scales"])
    state.update(gate_up=gu, down=dn, gate_up_scale=sgu, down_scale=sdn)
    if own:
        from w8a8_int8_rotated_amd import convrot
        state["weights"] = convrot.convrot_moe_prepare_weights(
            gu, dn, shared=S, src_scale_gate_up=sgu, src_scale_down=sdn)
    return state


def _route(state):
    """ids [T, k] and weights [T, k], in 64 bits: the choice next to a border does not
    hang on the order of a sum."""
    case = state["case"]
    logits = state["x"].double() @ state["router"].double().t()
    p = torch.sigmoid(logits) if case["score"] == "sigmoid" else torch.softmax(logits, -1)
    order = logits if state["bias"] is None else p + state["bias"].double()
    ids = torch.sort(order, dim=-1, descending=True, stable=True).indices[:, :case["k"]]
    w = p.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return ids, w * case["scale"]


def _widen(codes, scale, ids=None):
    """fp32 weights of the experts `ids` (all when None)."""
    if ids is not None:
        codes, scale = codes.view(torch.uint8)[ids].view(torch.float8_e4m3fn), scale[ids]
    n, a, b = codes.shape
    w = codes.to(F32).view(n, a // 128, 128, b // 128, 128)
    return (w * scale[:, :, None, :, None]).view(n, a, b)


def _run_moe(state):
    case = state["case"]
    if own:
        from w8a8_int8_rotated_amd import convrot
        return convrot.convrot_moe_forward(
            state["x"], state["router"], state["weights"], case["k"], router_bias=state["bias"],
            score=case["score"], renormalize=case["renorm"], scale=case["scale"],
            out_dtype=DTYPES[case["out"]])
    T, F, E, k, S = (case[n] for n in ("T", "F", "E", "k", "S"))
    ids, w = _route(state)
    x = state["x"].to(F32)
    # the shared experts as further choices of every token, of weight 1
    every = torch.cat([ids, torch.arange(E, E + S, device="cuda").expand(T, S)], 1)
    part = torch.cat([w.to(F32), torch.ones(T, S, device="cuda")], 1)
    if T * (k + S) <= E + S:                         # few tokens: the chosen experts' weights
        at = every.reshape(-1)
        a = _widen(state["gate_up"], state["gate_up_scale"], at) \
            @ x.repeat_interleave(k + S, 0)[:, :, None]
        g = torch.nn.functional.sigmoid(a[:, :F]) * a[:, :F] * a[:, F:]
        o = (_widen(state["down"], state["down_scale"], at) @ g).view(T, k + S, -1)
        y = (o * part[:, :, None]).sum(1)
    else:                                            # every expert on every token
        a = torch.matmul(x, _widen(state["gate_up"], state["gate_up_scale"]).transpose(1, 2))
        g = torch.sigmoid(a[..., :F]) * a[..., :F] * a[..., F:]
        o = torch.matmul(g, _widen(state["down"], state["down_scale"]).transpose(1, 2))
        share = torch.zeros(T, E + S, device="cuda").scatter(1, every, part)
        y = (o * share.t()[:, :, None]).sum(0)
    return y.to(DTYPES[case["out"]]), ids.to(torch.int32), w.to(F32)


def _exact_moe(state):
    case = state["case"]
    T, K, F, E, k, S = (case[n] for n in ("T", "K", "F", "E", "k", "S"))
    x = state["x"].double()
    logits = (x[:, None, :] * state["router"].double()).sum(-1) if T * E * K < 1 << 28 \
        else torch.nn.functional.linear(x, state["router"].double())
    e = (logits - logits.max(-1, keepdim=True).values).exp()
    p = 1 / (1 + (-logits).exp()) if case["score"] == "sigmoid" else e / e.sum(-1, keepdim=True)
    order = logits.clone() if state["bias"] is None else p + state["bias"].double()
    ids = torch.empty(T, k, dtype=torch.int64, device="cuda")
    for j in range(k):
        top = order.max(-1, keepdim=True).values
        ids[:, j] = torch.where(order == top, torch.arange(E, device="cuda"), E).min(-1).values
        order.scatter_(1, ids[:, j:j + 1], -math.inf)
    w = torch.gather(p, 1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    w = w * case["scale"]

    def wide(codes, scale):
        s = scale.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        return codes.float().double() * s

    y = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    for i in range(E + S):
        if i < E:
            hit = ids == i
            share = torch.where(hit, w, torch.zeros_like(w)).sum(1)
            rows = hit.any(1).nonzero()[:, 0]
        else:
            share, rows = torch.ones(T, dtype=torch.float64, device="cuda"), \
                torch.arange(T, device="cuda")
        if rows.numel() == 0:
            continue
        a = torch.matmul(wide(state["gate_up"][i], state["gate_up_scale"][i]), x[rows].t())
        act = a[:F] / (1 + (-a[:F]).exp()) * a[F:]
        out = torch.matmul(wide(state["down"][i], state["down_scale"][i]), act)
        y[rows] += (out * share[rows]).t()
    return y, ids.to(torch.int32), w
