"""The mixture-of-experts layer against its definition in 64 bits.

Bounds.  Products of bf16 values and e4m3 codes are exact in fp32; a sum over n inputs adds
at most 128 products and joins n / 128 blocks and 16 waves, each addition off by at most a
unit: (n / 128 + 144) 2^-23 of the sum of magnitudes.  |silu'| <= 1.1 and silu is off by a
few units (8 * 2^-24 of itself), so the errors of gate and up reach g as written in `layer`;
bf16 outputs round g once (2^-8 of it, F32 outputs not).  The down projection sums them with
|weight D|, adds its own sum's error, the experts' additions (within the same count) and the
output's half step.  Choices are equal; weights are one rounding of a value that is off by
1e-12."""
import pytest
import torch

from gpu_util import announce

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
FP8 = torch.float8_e4m3fn
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module")
def cr():
    from w8a8_int8_rotated_amd import convrot
    convrot.library()
    return convrot


def randn(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def experts(seed, n, K, F):
    """Random codes (no NaN) and scales of n experts."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def codes(*shape):
        c = torch.randn(*shape, generator=g, device="cuda") * 60
        return c.clamp(-448, 448).to(FP8)

    def scale(*shape):
        return 0.5 + torch.rand(*shape, generator=g, device="cuda")

    return {"gu": codes(n, 2 * F, K), "gus": scale(n, 2 * F // 128, K // 128) / (60 * K ** 0.5),
            "dn": codes(n, K, F), "dns": scale(n, K // 128, F // 128) / (60 * F ** 0.5)}


def prepare(cr, ex, shared=0):
    return cr.convrot_moe_prepare_weights(ex["gu"], ex["dn"], shared, ex["gus"], ex["dns"])


def wide(codes, scale):
    s = scale.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    return codes.float().double() * s


def route(x, router, k, bias=None, score="softmax", renormalize=True, scale=1.0):
    logits = x.double() @ router.double().t()
    p = torch.sigmoid(logits) if score == "sigmoid" else torch.softmax(logits, -1)
    order = logits if bias is None else p + bias.double()
    order = torch.where(order.isnan(), torch.full_like(order, -float("inf")), order)
    ids = torch.sort(order, dim=-1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if renormalize:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total == 0, torch.zeros_like(w), w / total)
    return ids, w * scale


def layer(x, ex, ids, w, shared, out_t):
    """(y, bound) in 64 bits for given choices and weights."""
    T, K = x.shape
    F, n = ex["dn"].shape[2], ex["dn"].shape[0]
    y, off = (torch.zeros(T, K, dtype=F64, device="cuda") for _ in range(2))
    eps = lambda m: (m / 128 + 144) * 2.0 ** -23                     # noqa: E731
    for e in range(n):
        share = torch.where(ids == e, w, torch.zeros_like(w)).sum(1)
        hit = (ids == e).any(1)
        if e >= n - shared:
            share, hit = torch.ones_like(share), torch.ones_like(hit)
        if not bool(hit.any()):
            continue
        xe, s = x[hit].double(), share[hit][:, None]
        W, D = wide(ex["gu"][e], ex["gus"][e]), wide(ex["dn"][e], ex["dns"][e])
        a = xe @ W.t()
        da = (xe.abs() @ W.abs().t()) * eps(K)
        gate, up = a[:, :F], a[:, F:]
        silu = gate * torch.sigmoid(gate)
        g = silu * up
        dg = 1.1 * da[:, :F] * (up.abs() + da[:, F:]) + silu.abs() * da[:, F:] \
            + g.abs() * (8 * 2.0 ** -24 + (HALF[BF16] if out_t == BF16 else 0.0))
        y[hit] += s * (g @ D.t())
        off[hit] += s.abs() * (dg @ D.abs().t() + ((g.abs() + dg) @ D.abs().t())
                               * (eps(F) + (n + 16) * 2.0 ** -23))
    return y, off + (y.abs() + off) * HALF[out_t]


CASES = [
    dict(T=1, K=2048, F=768, E=128, k=8),
    dict(T=1, K=128, F=128, E=1, k=1),
    dict(T=2, K=256, F=128, E=3, k=3, S=1, score="sigmoid"),
    dict(T=5, K=1280, F=1408, E=32, k=4, S=1, score="sigmoid", bias=True, scale=2.5,
         router="f32"),
    dict(T=15, K=640, F=384, E=40, k=6, renormalize=False, out="f32"),
    dict(T=16, K=5376, F=256, E=8, k=2, bias=True),
    dict(T=17, K=896, F=640, E=20, k=5, S=2, out="f32", router="f32"),
    dict(T=23, K=2560, F=640, E=40, k=6, renormalize=False, out="f32"),
    dict(T=31, K=512, F=256, E=130, k=10, score="sigmoid", renormalize=False),
    dict(T=33, K=384, F=512, E=257, k=7, bias=True, out="f32"),
    dict(T=48, K=256, F=128, E=512, k=32, S=3),
    dict(T=64, K=1024, F=384, E=16, k=4, S=1, bias=True, score="sigmoid"),
    dict(T=64, K=640, F=256, E=64, k=1, out="f32"),
    dict(T=65, K=512, F=256, E=12, k=3, S=1),
    dict(T=64, K=256, F=384, E=40, k=32, S=16),
    dict(T=64, K=384, F=256, E=40, k=32, S=16, out="f32"),
    dict(T=3, K=384, F=128, E=300, k=12, S=2, score="sigmoid", bias=True),
    dict(T=4, K=512, F=640, E=6, k=5, S=1, out="f32"),
    dict(T=8, K=2048, F=1024, E=70, k=8, bias=True),
    dict(T=9, K=640, F=384, E=143, k=3),
    dict(T=26, K=384, F=512, E=59, k=9, S=1, score="sigmoid", out="f32"),
    dict(T=60, K=2560, F=128, E=20, k=4, S=1, router="f32"),
    dict(T=200, K=384, F=128, E=9, k=2, out="f32", router="f32"),
    dict(T=3, K=256, F=128, E=300, k=32),
    dict(T=4, K=384, F=128, E=40, k=32, S=2, bias=True),
    dict(T=37, K=640, F=384, E=12, k=3, S=1, out="f32"),
    dict(T=64, K=512, F=640, E=8, k=3),
]


def make(case, seed=1):
    T, K, F, E, S = case["T"], case["K"], case["F"], case["E"], case.get("S", 0)
    hot = torch.where(torch.arange(K, device="cuda") % 97 == 5, 10.0, 1.0)
    x = (randn(seed, T, K) * hot).to(BF16)
    router = (randn(seed + 1, E, K) / K ** 0.5).to(F32 if case.get("router") == "f32" else BF16)
    bias = randn(seed + 2, E) * 0.05 if case.get("bias") else None
    kw = dict(score=case.get("score", "softmax"), renormalize=case.get("renormalize", True),
              scale=case.get("scale", 1.0))
    return x, router, bias, experts(seed + 3, E + S, K, F), kw


@pytest.mark.parametrize("case", CASES, ids=str)
def test_layer(cr, case):
    announce(f"moe {case}")
    x, router, bias, ex, kw = make(case)
    T, K, k, S = case["T"], case["K"], case["k"], case.get("S", 0)
    out_t = F32 if case.get("out") == "f32" else BF16
    W = prepare(cr, ex, S)
    whole = torch.full((T + 2, K), 7.0, dtype=out_t, device="cuda")
    y, ids, w = cr.convrot_moe_forward(x, router, W, k, router_bias=bias, out=whole[:T], **kw)
    assert bool((whole[T:] == 7).all())
    ids64, w64 = route(x, router, k, bias, **kw)
    assert torch.equal(ids.long(), ids64)
    assert bool(((w.double() - w64).abs() <= w64.abs() * (2.0 ** -24 + 1e-11)).all())
    ref, bound = layer(x, ex, ids64, w64, S, out_t)
    over = (y.double() - ref).abs() / bound
    print(f"[moe] worst share of the bound {float(over.max()):.3f}, rel "
          f"{float((y.double() - ref).norm() / ref.norm()):.2e}", flush=True)
    assert bool((over <= 1).all())
    again = cr.convrot_moe_forward(x, router, W, k, router_bias=bias, out_dtype=out_t, **kw)
    assert all(torch.equal(a, b) for a, b in zip(again, (y, ids, w)))


def test_choice_is_the_tokens_own(cr):
    """Choices and weights do not depend on the batch; outputs agree to their rounding."""
    case = dict(T=64, K=1024, F=256, E=32, k=4, S=1)
    x, router, _, ex, kw = make(case)
    W = prepare(cr, ex, 1)
    y, ids, w = cr.convrot_moe_forward(x, router, W, 4, **kw)
    for part in (slice(0, 1), slice(3, 20), slice(17, 50)):
        y1, ids1, w1 = cr.convrot_moe_forward(x[part].clone(), router, W, 4, **kw)
        assert torch.equal(ids1, ids[part]) and torch.equal(w1, w[part])
        ref, bound = layer(x[part], ex, ids1.long(), w1.double(), 1, BF16)
        assert bool(((y1.double() - ref).abs() <= bound).all())


def test_ties_go_to_the_lowest_index(cr):
    K, F, E = 256, 128, 70
    ex = experts(1, E, K, F)
    W = prepare(cr, ex)
    router = randn(2, E, K)
    router[5:] = router[5 - torch.arange(5, E, device="cuda") % 5]   # many equal experts
    x = randn(3, 9, K).to(BF16)
    x[0] = 0                                                         # every logit equal
    for bias in (None, torch.zeros(E, device="cuda")):
        for score in ("softmax", "sigmoid"):
            _, ids, w = cr.convrot_moe_forward(x, router, W, 12, router_bias=bias, score=score)
            assert ids[0].tolist() == list(range(12))
            logits = (x.double()[:, None] * router.double()).sum(-1)
            for t in range(1, 9):
                # equal rows of the router have equal logits, whatever the order of the sums
                got, p = ids[t].tolist(), w[t].tolist()
                for a, b, pa, pb in zip(got, got[1:], p, p[1:]):
                    assert pa >= pb
                    if torch.equal(router[a], router[b]):
                        assert a < b and pa == pb
                rest = [e for e in range(E) if e not in got]
                least = min(float(logits[t, e]) for e in got)
                assert all(float(logits[t, e]) <= least + 1e-12 for e in rest)


def test_masked_experts(cr):
    """A bias of -infinity, or of the type's lowest value, keeps an expert from being chosen
    while others are left; the weights are the scores without the bias."""
    K, F, E = 256, 128, 12
    ex = experts(1, E, K, F)
    W = prepare(cr, ex)
    router, x = randn(2, E, K) / K ** 0.5, randn(3, 20, K).to(BF16)
    for low in (-float("inf"), torch.finfo(F32).min, float("nan")):
        for score in ("softmax", "sigmoid"):
            bias = torch.zeros(E, device="cuda")
            bias[[0, 3, 4, 11]] = low
            y, ids, w = cr.convrot_moe_forward(x, router, W, 4, router_bias=bias, score=score)
            ids64, w64 = route(x, router, 4, bias, score)
            assert torch.equal(ids.long(), ids64)
            assert not bool((ids[..., None] == torch.tensor([0, 3, 4, 11], device="cuda")).any())
            ref, bound = layer(x, ex, ids64, w64, 0, BF16)
            assert bool(((y.double() - ref).abs() <= bound).all())
            bias[:] = low                                            # nothing left: the first ones
            _, ids, w = cr.convrot_moe_forward(x, router, W, 4, router_bias=bias, score=score)
            if low != torch.finfo(F32).min:
                assert bool((ids == torch.arange(4, device="cuda", dtype=torch.int32)).all())
            assert bool(w.isfinite().all())


def test_scores_that_vanish(cr):
    """Sigmoid scores of 0: weights 0, not NaN; and far logits, whose scores tie while the
    logits do not."""
    K, F, E = 128, 128, 6
    ex = experts(1, E, K, F)
    W = prepare(cr, ex)
    router = torch.zeros(E, K, device="cuda")
    router[:, 0] = -1000.0 - torch.arange(E, device="cuda").flip(0)
    x = torch.zeros(1, K, dtype=BF16, device="cuda")
    x[0, 0] = 1
    y, ids, w = cr.convrot_moe_forward(x, router, W, 2, score="sigmoid")
    assert ids.tolist() == [[5, 4]] and w.tolist() == [[0, 0]] and bool((y == 0).all())
    router[:, 0] = 1000.0 + torch.arange(E, device="cuda")
    y, ids, w = cr.convrot_moe_forward(x, router, W, 2, score="sigmoid")
    assert ids.tolist() == [[5, 4]] and w.tolist() == [[0.5, 0.5]]


@pytest.mark.parametrize("out_t", [BF16, F32], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T", [1, 5, 40])
def test_non_finite_tokens_stay_alone(cr, bad, T, out_t):
    case = dict(T=T, K=384, F=256, E=10, k=3, S=1)
    x, router, _, ex, kw = make(case)
    W = prepare(cr, ex, 1)
    xb = x.clone()
    xb[T // 2, 7] = bad
    others = [t for t in range(T) if t != T // 2]
    a = cr.convrot_moe_forward(x, router, W, 3, out_dtype=out_t, **kw)
    b = cr.convrot_moe_forward(xb, router, W, 3, out_dtype=out_t, **kw)
    assert bool(b[0][T // 2].isnan().all())
    ids = b[1][T // 2].tolist()
    assert len(set(ids)) == 3 and min(ids) >= 0 and max(ids) < 10
    assert torch.equal(a[1][others], b[1][others]) and torch.equal(a[2][others], b[2][others])
    if others:
        ref, bound = layer(x[others], ex, a[1][others].long(), a[2][others].double(), 1, out_t)
        assert bool(((b[0][others].double() - ref).abs() <= bound).all())


def test_broken_expert_stays_alone(cr):
    """Codes of NaN reach the tokens that chose the expert and no other."""
    case = dict(T=40, K=384, F=256, E=10, k=3)
    x, router, _, ex, kw = make(case)
    for name in ("gu", "dn"):
        broken = dict(ex)
        c = ex[name].view(torch.uint8).clone()
        c[4, 5, 9] = 0x7F
        broken[name] = c.view(FP8)
        y0, ids, _ = cr.convrot_moe_forward(x, router, prepare(cr, ex), 3, **kw)
        y1, _, _ = cr.convrot_moe_forward(x, router, prepare(cr, broken), 3, **kw)
        hit = (ids == 4).any(1)
        assert bool(hit.any()) and not bool(hit.all())
        assert bool(y1[hit].isnan().any(1).all()) and torch.equal(y0[~hit], y1[~hit])


@pytest.mark.parametrize("scales", ["f32", "pow2"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_prepare_from_floats(cr, dtype, scales):
    """Each expert as convrot_fp8_prepare_weights quantises it."""
    n, K, F = 3, 384, 256
    gu, dn = (randn(1, n, 2 * F, K) * 0.02).to(dtype), (randn(2, n, K, F) * 0.02).to(dtype)
    W = cr.convrot_moe_prepare_weights(gu, dn, shared=1, scales=scales)
    assert (W.experts, W.shared, W.K, W.F) == (2, 1, K, F)
    for e in range(n):
        for w, codes, sc in ((gu, W.gate_up, W.gate_up_scale), (dn, W.down, W.down_scale)):
            one = cr.convrot_fp8_prepare_weights(w[e], scales=scales)
            size = one.codes.numel()
            assert torch.equal(codes[e * size:(e + 1) * size], one.codes)
            assert torch.equal(sc[e], one.scale)


def test_no_tokens(cr):
    ex = experts(1, 4, 128, 128)
    W = prepare(cr, ex)
    x, router = torch.empty(0, 128, dtype=BF16, device="cuda"), randn(2, 4, 128)
    y, ids, w = cr.convrot_moe_forward(x, router, W, 2)
    assert y.shape == (0, 128) and ids.shape == (0, 2) and w.shape == (0, 2)


def test_offsets_past_32_bits(cr):
    """Stacks of more than 2^32 bytes of codes: the last experts against a stack of their
    own."""
    n, K, F = 90, 5376, 5120
    gu = torch.zeros(n, 2 * F, K, dtype=torch.uint8, device="cuda")
    dn = torch.zeros(n, K, F, dtype=torch.uint8, device="cuda")
    last = experts(1, 2, K, F)
    gu[-2:], dn[-2:] = last["gu"].view(torch.uint8), last["dn"].view(torch.uint8)
    gus, dns = torch.ones(n, 2 * F // 128, K // 128, device="cuda"), \
        torch.ones(n, K // 128, F // 128, device="cuda")
    gus[-2:], dns[-2:] = last["gus"], last["dns"]
    W = cr.convrot_moe_prepare_weights(gu.view(FP8), dn.view(FP8), 0, gus, dns)
    del gu, dn
    x = randn(2, 3, K).to(BF16)
    router = randn(3, n, K) / K ** 0.5
    bias = torch.zeros(n, device="cuda")
    bias[-2:] = 10.0
    y, ids, w = cr.convrot_moe_forward(x, router, W, 2, router_bias=bias, score="sigmoid")
    assert bool((ids >= n - 2).all())
    y2, ids2, w2 = cr.convrot_moe_forward(x, router[-2:].contiguous(), prepare(cr, last), 2,
                                          router_bias=bias[-2:].contiguous(), score="sigmoid")
    assert torch.equal(y, y2) and torch.equal(ids, ids2 + n - 2) and torch.equal(w, w2)
    assert float(y.abs().max()) > 0


def test_graphs_and_streams(cr):
    """Two graphs that share a workspace, replayed several times with eager work in between,
    choices changing from replay to replay; then two streams at once."""
    case = dict(T=21, K=640, F=256, E=24, k=4, S=1)
    x, router, _, ex, kw = make(case)
    W = prepare(cr, ex, 1)
    ws = torch.empty(cr.convrot_moe_workspace_bytes(21, W, 4), dtype=torch.uint8, device="cuda")
    xs = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cr.convrot_moe_forward(xs, router, W, 4, workspace=ws, **kw)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for dt in (BF16, F32):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = cr.convrot_moe_forward(xs, router, W, 4, workspace=ws, out_dtype=dt, **kw)
        graphs.append((gr, out, dt))
    for i in range(5):
        xs.copy_(randn(50 + i, 21, 640).to(BF16))
        ws.fill_(0xA5)                               # nothing of the workspace is kept
        for gr, out, dt in graphs:
            want = cr.convrot_moe_forward(xs, router, W, 4, out_dtype=dt, **kw)
            for t in out:
                t.fill_(3)
            gr.replay()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), i
        torch.cuda.synchronize()
    want = cr.convrot_moe_forward(x, router, W, 4, **kw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [cr.convrot_moe_forward(x, router, W, 4, stream=streams[i % 2], **kw) for i in range(6)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))


@pytest.mark.parametrize("T", [1, 7])
def test_pre_norm_layers(cr, T):
    """As a model uses them: norm -> experts -> the residual's addition and the next norm, over
    two layers, against the definitions on the same rounded intermediates."""
    K, F, E, k = 640, 256, 16, 3
    x = randn(1, T, K).to(BF16)
    h = randn(2, T, K) * 3
    wn = 1 + 0.1 * randn(3, K)
    for i in range(2):
        ex = experts(10 + i, E, K, F)
        W, router = prepare(cr, ex), randn(20 + i, E, K) / K ** 0.5
        n, h2 = cr.convrot_add_rms_norm_forward(x, wn, h)
        assert torch.equal(h2, x.float() + h)
        v = h2.double()
        ref = v / ((v * v).mean(-1, keepdim=True) + 1e-6).sqrt() * wn.double()
        assert bool(((n.double() - ref).abs() <= ref.abs() * (2.0 ** -18 + 2.0 ** -8)).all())
        y, ids, w = cr.convrot_moe_forward(n, router, W, k)
        ids64, w64 = route(n, router, k)
        assert torch.equal(ids.long(), ids64)
        ref, bound = layer(n, ex, ids64, w64, 0, BF16)
        assert bool(((y.double() - ref).abs() <= bound).all())
        x, h = y, h2


@pytest.mark.parametrize("T", [1, 5, 12, 20, 40])
def test_values_past_bf16(cr, T):
    """F32 outputs carry g up to the largest fp32 value, which is beyond bf16's: even tokens have
    a g of that value at every channel, odd ones a quarter of it, the last (of several) an
    infinite one, whose outputs are not finite.  Only channel 0 of g is summed, so outputs are
    off by the additions of its three parts: 2^-22."""
    K = F = 128
    gu, dn = torch.zeros(1, 2 * F, K, device="cuda"), torch.zeros(1, K, F, device="cuda")
    gu[:, :, 0], dn[:, :, 0] = 1, 1
    gus, dns = torch.empty(1, 2, 1, device="cuda"), torch.full((1, 1, 1), 2.0 ** -120, device="cuda")
    gus[0, 0], gus[0, 1] = 2.0 ** 63, (2 - 2.0 ** -23) * 2.0 ** 64
    W = cr.convrot_moe_prepare_weights(gu.to(FP8), dn.to(FP8), 0, gus, dns)
    x = torch.zeros(T, K, dtype=BF16, device="cuda")
    x[0::2, 0], x[1::2, 0] = 1, 0.5
    if T > 1:
        x[-1, 0] = 2
    n = max(T - 1, 1)
    y, _, _ = cr.convrot_moe_forward(x, torch.zeros(1, K, device="cuda"), W, 1, out_dtype=F32)
    ref = x.double()[:, :1] ** 2 * ((2 - 2.0 ** -23) * 2.0 ** 7)
    assert bool(((y[:n].double() - ref[:n]).abs() <= ref[:n] * 2.0 ** -22).all())
    assert not bool(y[n:].isfinite().any())


# one token, and three: the experts' own workgroups choose, with two, four and eight experts a
# lane; or in more than a round of them (F / 16 (k + S) > 768) the kernel of its own
FEW_TOKENS = [
    dict(T=1, K=256, F=128, E=256, k=32, S=1, bias=True, score="sigmoid"),
    dict(T=1, K=384, F=256, E=129, k=8, out="f32"),
    dict(T=3, K=256, F=128, E=200, k=10, S=2, bias=True, router="f32"),
    dict(T=1, K=256, F=128, E=512, k=32, S=2, score="sigmoid", renormalize=False),
    dict(T=1, K=128, F=384, E=257, k=5, bias=True, out="f32", scale=2.5),
    dict(T=1, K=128, F=512, E=128, k=32, S=16, out="f32"),
    dict(T=1, K=256, F=512, E=200, k=32, bias=True, score="sigmoid"),
    dict(T=1, K=128, F=512, E=300, k=31, S=1, renormalize=False),
    dict(T=1, K=128, F=1024, E=14, k=14, S=1),
]


@pytest.mark.parametrize("case", FEW_TOKENS, ids=str)
def test_few_tokens_of_many_experts(cr, case):
    test_layer(cr, case)
