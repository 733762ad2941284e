"""The framework's operators beside the INT8 projections, in plain torch and as
a user calls them: the FP8 block-scaled linear, the rotary positions with
several axes, and the per-head norm of queries and keys with the rotation in
the same pass (forward and backward).

`run(prepare(case, seed))` is one pass.  With `own` false it is elementary
torch arithmetic in 32 bits (angles in 64); with `own` true it is the calls of
`w8a8_int8_rotated_amd.convrot`.  Cases are plain dicts; `exact` evaluates the
definitions in 64 bits.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}


def listed():
    return [
        # one conditioning vector through a QKV-sized layer: latency
        fp8("fp8_vector", M=1, K=5376, N=16128),
        # the modulation projection (six hidden widths) of 8 timestep embeddings
        fp8("fp8_modulation", M=8, K=5376, N=32256, bias=True, out="f32"),
        # a text prompt's tokens through an output projection, odd count
        fp8("fp8_prompt", M=333, K=5376, N=5376, bias=True),
        # a square projection over an image's tokens, power-of-two scales
        fp8("fp8_image", M=4096, K=5376, N=5376, scales="pow2", bias=True),
        # the fused QKV projection of a 768p packed sequence, both scale kinds
        fp8("fp8_qkv", M=38656, K=5376, N=16128),
        fp8("fp8_qkv_pow2", M=38656, K=5376, N=16128, scales="pow2"),
        # rotary positions alone: image patches (height, width) in fp32 ...
        rope("rope", "rope_patches", B=2, T=1021, Hq=16, Hk=16, D=64, dims="32,32",
             pairing="half", dtype="f32", layout="bhtd"),
        # ... and the last token of 8 sequences at far positions, shared K heads
        rope("rope", "rope_step", B=8, T=1, Hq=32, Hk=8, D=128, dims="128", far=True),
        # Q/K norm and rotation on the Q and K columns of the QKV rows: a short
        # clip with an odd token count, and the 768p packed sequence
        rope("norm", "norm_rope_clip", B=1, T=2381, Hq=42, Hk=42, D=128, dims="16,56,56",
             layout="qkv", pos="f32"),
        rope("norm", "norm_rope_768p", B=1, T=38656, Hq=42, Hk=42, D=128, dims="16,56,56",
             layout="qkv", pos="f32"),
        # its backward pass: fine-tuning on a small batch with shared K heads,
        # and on the whole packed sequence
        rope("norm_bwd", "norm_rope_bwd_batch", B=3, T=509, Hq=24, Hk=8, D=96, dims="32,32,32",
             pairing="half", spectrum="whole", dtype="f32"),
        rope("norm_bwd", "norm_rope_bwd_768p", B=1, T=38656, Hq=42, Hk=42, D=128,
             dims="16,56,56", layout="qkv", pos="f32"),
    ]


def fp8(name, M, K, N, scales="f32", bias=False, out="bf16"):
    return {"name": name, "op": "fp8", "M": M, "K": K, "N": N, "scales": scales, "bias": bias,
            "out": out}


def rope(op, name, B, T, Hq, Hk, D, dims, pairing="interleaved", spectrum="axis", dtype="bf16",
         layout="bthd", pos="i32", far=False):
    return {"name": name, "op": op, "B": B, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "dims": dims,
            "pairing": pairing, "spectrum": spectrum, "dtype": dtype, "layout": layout,
            "pos": pos, "far": far}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        K = 128 * _log_int(rng, 1, 168)
        N = 16 * _log_int(rng, 1, 2016)
        top = min(38656, 38656 * 5376 * 16128 // (K * N), (1 << 31) // K - 16)
        c = fp8("", _log_int(rng, 1, top), K, N, rng.choice(["f32", "pow2"]),
                rng.random() < 0.5, rng.choice(["bf16", "f32"]))
    else:
        pairing = rng.choice(["interleaved", "half"])
        axes = rng.choice([1, 2, 3])
        D = rng.choice([32, 64, 80, 96, 128, 192, 256])
        R = D if rng.random() < 0.7 else D // 2
        unit = 2                                      # an axis holds whole pairs
        cuts = sorted(rng.sample(range(1, R // unit), axes - 1))
        ends = [0] + [c * unit for c in cuts] + [R]
        dims = ",".join(str(b - a) for a, b in zip(ends, ends[1:]))
        Hk = rng.choice([1, 2, 4, 8, 21, 42])
        Hq = Hk * rng.choice([1, 2, 4]) if Hk < 21 else Hk
        dtype = rng.choice(["bf16", "bf16", "f32"])
        op = rng.choice(["rope", "norm", "norm_bwd"])
        per_token = (Hq + Hk) * D * (2 if dtype == "f32" else 1)
        tokens = _log_int(rng, 1, 38656 * 84 * 128 // max(per_token, 84 * 128))
        B = rng.choice([1, 1, 2, 3]) if tokens >= 3 else 1
        c = rope(op, "", B, max(1, tokens // B), Hq, Hk, D, dims, pairing,
                 rng.choice(["axis", "whole"]), dtype, rng.choice(["qkv", "bthd", "bhtd"]),
                 rng.choice(["i32", "f32"]), rng.random() < 0.25)
    del c["name"]
    return c


def work(case):
    if case["op"] == "fp8":
        M, K, N = case["M"], case["K"], case["N"]
        out = 2 if case["out"] == "bf16" else 4
        nbytes = 2 * M * K + N * K + 4 * -(-N // 128) * (K // 128) + out * M * N
        return {"bytes": nbytes + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    tokens = case["B"] * case["T"]
    n = tokens * (case["Hq"] + case["Hk"]) * case["D"]
    es = 2 if case["dtype"] == "bf16" else 4
    axes = len(_dims(case))
    passes = {"rope": 2, "norm": 2, "norm_bwd": 3}[case["op"]]
    flops = {"rope": 3, "norm": 7, "norm_bwd": 14}[case["op"]] * n
    return {"bytes": passes * n * es + 4 * axes * tokens, "flops": flops}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=F32)


def prepare(case, seed):
    return _prepare_fp8(case, seed) if case["op"] == "fp8" else _prepare_rope(case, seed)


def run(state):
    return {"fp8": _run_fp8, "rope": _run_rope, "norm": _run_norm,
            "norm_bwd": _run_norm_bwd}[state["case"]["op"]](state)


def exact(case, seed):
    was = own
    globals()["own"] = False
    try:
        state = prepare(case, seed)
    finally:
        globals()["own"] = was
    if case["op"] == "fp8":
        return _exact_fp8(state)
    return _exact_rope(state)


# ------------------------------------------------- FP8 block-scaled linear ----
# x bf16 [M, K]; w e4m3 codes [N, K] with one fp32 scale per 128 x 128 block.
# Activation scales: amax / 448 of each token's 128 inputs, or the smallest
# power of two not below it; at least 2^-126, 0 for a block of zeros.

def _prepare_fp8(case, seed):
    g = _gen(seed)
    M, K, N = case["M"], case["K"], case["N"]
    x = _randn(g, M, K)
    # a few channels carry outliers, as a residual stream's do
    hot = torch.rand(K, generator=g, device="cuda") < 0.01
    x = torch.where(hot, x * 30, x).to(BF16)
    w = _randn(g, N, K) * 0.02
    codes, scale = _quantize_weight(w, case["scales"])
    state = {"case": case, "x": x, "codes": codes, "scale": scale, "bias": None}
    if case["bias"]:
        state["bias"] = _randn(g, N) * 0.01
    if own:
        from w8a8_int8_rotated_amd import convrot
        state["weights"] = convrot.convrot_fp8_prepare_weights(codes, src_scale=scale,
                                                               scales=case["scales"])
    return state


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


def _run_fp8(state):
    case = state["case"]
    if own:
        from w8a8_int8_rotated_amd import convrot
        return convrot.convrot_fp8_linear_forward(state["x"], state["weights"], state["bias"],
                                                  out_dtype=DTYPES[case["out"]])
    x = state["x"].to(F32).view(case["M"], case["K"] // 128, 128)
    amax = x.abs().amax(-1, keepdim=True)
    s = _scale(amax, case["scales"])
    inv = torch.where(s > 0, (1 / s.double()).to(F32), s)
    xq = ((x * inv).to(torch.float8_e4m3fn).to(F32) * s).view(case["M"], case["K"])
    sw = state["scale"].repeat_interleave(128, 0)[:case["N"]].repeat_interleave(128, 1)
    y = xq @ (state["codes"].to(F32) * sw).t()
    if state["bias"] is not None:
        y = y + state["bias"]
    return y.to(DTYPES[case["out"]])


def _exact_fp8(state):
    case = state["case"]
    M, K, N = case["M"], case["K"], case["N"]
    x = state["x"].double().reshape(M, K // 128, 128)
    amax = x.abs().max(-1, keepdim=True).values
    s = torch.clamp((amax / 448.0).float().double(), min=2.0 ** -126)
    if case["scales"] == "pow2":
        s = torch.exp2(torch.ceil(torch.log2(s)).clamp_min(-126))
    zero = amax == 0
    inv = (1.0 / s).float().double()
    v = (x * inv).float().double()
    # e4m3: steps of 2^(e - 3) from 2^e up, 2^-9 below 2^-6; ties to even
    e = torch.frexp(v)[1].double().sub(1).clamp_min(-6)
    step = torch.exp2(e - 3)
    q = (torch.round(v / step) * step).clamp(-448, 448)
    xq = torch.where(zero, torch.zeros_like(q), q * s).reshape(M, K)
    del x, v, e, step, q
    ws = state["scale"].double()
    w = state["codes"].float().double()
    idx = torch.arange(N, device="cuda") // 128
    for kb in range(K // 128):
        w[:, 128 * kb:128 * kb + 128] *= ws[idx, kb][:, None]
    y = torch.matmul(xq, w.t())
    return y if state["bias"] is None else y + state["bias"].double()


# ------------------------------- rotary positions, with and without norms ----
# q [B, T, Hq, D], k [B, T, Hk, D]; positions [B, T, axes].  Pair p of the
# R = sum(dims) rotated channels turns by positions[axis(p)] * freq(p):
# channels (2p, 2p + 1), or (p, p + R/2) for "half".

def _dims(case):
    return [int(d) for d in case["dims"].split(",")]


def _prepare_rope(case, seed):
    g = _gen(seed)
    B, T, Hq, Hk, D = (case[k] for k in ("B", "T", "Hq", "Hk", "D"))
    dtype, dims = DTYPES[case["dtype"]], _dims(case)

    def heads(gain):
        if case["layout"] == "qkv":                  # columns of the fused projection
            row = (_randn(g, B, T, (Hq + 2 * Hk) * D) * gain).to(dtype)
            return (row[..., :Hq * D].unflatten(-1, (Hq, D)),
                    row[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D)))
        if case["layout"] == "bhtd":
            return tuple((_randn(g, B, H, T, D) * gain).to(dtype).transpose(1, 2)
                         for H in (Hq, Hk))
        return tuple((_randn(g, B, T, H, D) * gain).to(dtype) for H in (Hq, Hk))

    state = {"case": case}
    state["q"], state["k"] = heads(3.0)
    state["wq"] = 1 + 0.2 * _randn(g, D)
    state["wk"] = 1 + 0.2 * _randn(g, D)
    if case["op"] == "norm_bwd":
        state["gq"], state["gk"] = heads(0.01)
    # a raster of frames x height x width, from a random start
    t = torch.arange(T, device="cuda").expand(B, T)
    start = torch.randint(0, (1 << 20) if case["far"] else 64, (B, 1, len(dims)), generator=g,
                          device="cuda")
    raster = [t] if len(dims) == 1 else \
        [t // 1536 if len(dims) == 3 else t // 48, t // 48 % 32, t % 48][-len(dims):]
    if len(dims) == 2:
        raster = [t // 48, t % 48]
    pos = torch.stack(raster, -1) + start
    # frames at a fractional rate where the positions are fp32
    state["pos"] = (pos * torch.tensor([0.24, 1, 1][:len(dims)], device="cuda")).to(F32) \
        if case["pos"] == "f32" else pos.to(torch.int32)
    if own:
        from w8a8_int8_rotated_amd import convrot
        state["plan"] = convrot.convrot_rope_prepare(dims, D, theta=10000.0,
                                                     pairing=case["pairing"],
                                                     spectrum=case["spectrum"])
    return state


def _rates(case):
    """Frequency and axis of every pair."""
    dims = _dims(case)
    R = sum(dims)
    axis = [a for a, d in enumerate(dims) for _ in range(d // 2)]
    if case["spectrum"] == "whole":
        f = [10000.0 ** (-2.0 * p / R) for p in range(R // 2)]
    else:
        f = [10000.0 ** (-2.0 * j / d) for d in dims for j in range(d // 2)]
    return (torch.tensor(f, dtype=torch.float64, device="cuda"),
            torch.tensor(axis, dtype=torch.int64, device="cuda"))


def _cos_sin(state):
    f, axis = _rates(state["case"])
    angle = state["pos"].double()[..., axis] * f
    return angle.cos()[:, :, None], angle.sin()[:, :, None]      # [B, T, 1, R/2]


def _rotate(x, c, s, pairing):
    R = 2 * c.shape[-1]
    if pairing == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        out = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        out = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([out, x[..., R:]], -1)


EPS = 1e-6


def _run_rope(state):
    case = state["case"]
    if own:
        from w8a8_int8_rotated_amd import convrot
        return convrot.convrot_rope_forward(state["q"], state["k"], state["plan"], state["pos"])
    c, s = (v.to(F32) for v in _cos_sin(state))
    return tuple(_rotate(x.to(F32), c, s, case["pairing"]).to(x.dtype)
                 for x in (state["q"], state["k"]))


def _run_norm(state):
    case = state["case"]
    if own:
        from w8a8_int8_rotated_amd import convrot
        return convrot.convrot_qk_norm_rope_forward(state["q"], state["k"], state["wq"],
                                                    state["wk"], state["plan"], state["pos"],
                                                    eps=EPS)
    c, s = (v.to(F32) for v in _cos_sin(state))
    out = []
    for x, w in ((state["q"], state["wq"]), (state["k"], state["wk"])):
        x32 = x.to(F32)
        n = x32 * torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS) * w
        out.append(_rotate(n, c, s, case["pairing"]).to(x.dtype))
    return tuple(out)


def _run_norm_bwd(state):
    case = state["case"]
    if own:
        from w8a8_int8_rotated_amd import convrot
        return convrot.convrot_qk_norm_rope_backward(state["gq"], state["gk"], state["q"],
                                                     state["k"], state["wq"], state["wk"],
                                                     state["plan"], state["pos"], eps=EPS)
    c, s = (v.to(F32) for v in _cos_sin(state))
    dx, dw = [], []
    for g, x, w in ((state["gq"], state["q"], state["wq"]),
                    (state["gk"], state["k"], state["wk"])):
        x32 = x.to(F32)
        r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS)
        xh = x32 * r
        gn = _rotate(g.to(F32), c, -s, case["pairing"])
        t = gn * w
        dx.append((r * (t - xh * (t * xh).mean(-1, keepdim=True))).to(x.dtype))
        # sums over all tokens and heads: 64 bits where 32 would lose them
        dw.append((gn * xh).sum((0, 1, 2), dtype=torch.float64).to(F32))
    return (*dx, *dw)


def _exact_rope(state):
    """The definitions with every pair as a complex number times e^(i angle)."""
    case = state["case"]
    f, axis = _rates(case)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.index_select(state["pos"].double(), 2, axis) * f)[:, :, None]
    R = 2 * f.numel()

    def rotate(x, z):
        y = x.clone()
        if case["pairing"] == "half":
            p = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * z
            y[..., :R // 2], y[..., R // 2:R] = p.real, p.imag
        else:
            p = torch.complex(x[..., 0:R:2].contiguous(), x[..., 1:R:2].contiguous()) * z
            y[..., 0:R:2], y[..., 1:R:2] = p.real, p.imag
        return y

    out, dws = [], []
    for n in "qk":
        x, w = state[n].double(), state["w" + n].double()
        if case["op"] == "rope":
            out.append(rotate(x, turn))
            continue
        norm = ((x * x).sum(-1, keepdim=True) / case["D"] + EPS).sqrt()
        if case["op"] == "norm":
            out.append(rotate(x / norm * w, turn))
            continue
        gn = rotate(state["g" + n].double(), turn.conj())
        u = gn * w
        out.append(u / norm - x * ((u * x).sum(-1, keepdim=True) / case["D"]) / norm ** 3)
        dws.append((gn * x / norm).sum((0, 1, 2)))
    return (*out, *dws)
