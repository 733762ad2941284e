"""The residual's addition with the RMS norm, forward (rows, INT8 and FP8 codes, in front
of a linear) and backward, against the definitions in 64 bits.

Bounds.  h = x + r is one fp32 addition and one rounding: equal bits.  A lane adds at most
64 squares in turn (8 steps of 8), 5 additions join a half-wave and at most 16 the waves,
so the sum of squares is off by less than 96 * 2^-24 of itself; its reciprocal root by half
of that, 3 roundings and the root's own unit: under 60 * 2^-24, and n by 2 roundings more.
2^-18 (64 * 2^-24) bounds it, plus half a step of the output's type.  Backward, q^3 carries
three times that and the mean of t h another 96 * 2^-24 of the mean of |t h|: 2^-15 of the
sum of the terms' magnitudes bounds dh.  dw adds at most M terms in fp32, each off by
2^-18 of itself, before the sums are joined in fp64."""
import numpy as np
import pytest
import torch

from gpu_util import announce, padded_rows, untile

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module")
def cr():
    from w8a8_int8_rotated_amd import convrot
    convrot.library()
    return convrot


def rows(seed, M, K, dtype, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda")
    hot = torch.where(torch.rand(K, generator=g, device="cuda") < 0.02, 30.0, 1.0)
    return (x * hot * gain).to(dtype)


def weight(K, seed=9):
    return 1 + 0.2 * rows(seed, 1, K, F32)[0]


def guarded(M, K, dtype, fill=7.0):
    """[M, K] with two rows of canaries behind it."""
    whole = torch.full((M + 2, K), fill, dtype=dtype, device="cuda")
    return whole, whole[:M]


def unharmed(whole, M, fill=7.0):
    assert bool((whole[M:] == fill).all())


def reference(x, w, r):
    """(h as stored, n in 64 bits)"""
    h = x if r is None else (x.float() + r.float()).to(r.dtype)
    v = h.double()
    n = v / ((v * v).mean(-1, keepdim=True) + EPS).sqrt()
    return h, n if w is None else n * w.double()


SHAPES = [(1, 8), (3, 24), (2, 128), (5, 264), (17, 1000), (1, 2056), (40, 2304), (33, 4104),
          (1, 5376), (9, 5376), (7, 8192), (3, 8200), (2, 16384), (5, 16392), (1, 32768),
          (3, 32760)]
TYPES = [("bf16", None), ("bf16", "bf16"), ("bf16", "f32"), ("f32", None), ("f32", "f32")]
DT = {"bf16": BF16, "f32": F32, None: None}


@pytest.mark.parametrize("x_t,r_t", TYPES, ids=str)
@pytest.mark.parametrize("M,K", SHAPES, ids=str)
def test_forward(cr, M, K, x_t, r_t):
    announce(f"norm M={M} K={K} x={x_t} r={r_t}")
    x = rows(1, M, K, DT[x_t])
    r = None if r_t is None else rows(2, M, K, DT[r_t], 3.0)
    for w in (weight(K), None):
        h_ref, n = reference(x, w, r)
        for out_t in (BF16, F32):
            whole, out = guarded(M, K, out_t)
            hw, h = guarded(M, K, r.dtype) if r is not None else (None, None)
            y, h2 = cr.convrot_add_rms_norm_forward(x, w, r, eps=EPS, out=out, residual_out=h)
            assert y is out and h2 is h
            unharmed(whole, M)
            if r is not None:
                unharmed(hw, M)
                assert torch.equal(h, h_ref)
            assert bool(((y.double() - n).abs() <= n.abs() * (2.0 ** -18 + HALF[out_t])).all())


def test_leading_dimensions_and_defaults(cr):
    x, r = rows(1, 6, 256, BF16).view(2, 3, 256), rows(2, 6, 256, F32).view(2, 3, 256)
    w = weight(256)
    y, h = cr.convrot_add_rms_norm_forward(x, w, r)
    assert y.shape == x.shape and y.dtype == BF16 and h.shape == x.shape and h.dtype == F32
    y2, h2 = cr.convrot_add_rms_norm_forward(x.view(6, 256), w, r.view(6, 256))
    assert torch.equal(y.view(6, 256), y2) and torch.equal(h.view(6, 256), h2)
    y3, none = cr.convrot_add_rms_norm_forward(h, w)             # the norm of the stored h
    assert none is None and torch.equal(y3, y)


def test_extreme_rows(cr):
    """Zeros, tiny and large values: eps carries a zero row, 2.4e5 is far from overflow."""
    K = 512
    x = torch.zeros(6, K, device="cuda")
    x[1, 5] = 2.4e5
    x[2] = 1e-30
    x[3] = 1e15
    x[4] = torch.linspace(-3, 3, K, device="cuda")
    x[5, 0] = 1e-4
    w = weight(K)
    y, _ = cr.convrot_add_rms_norm_forward(x, w, out_dtype=F32)
    n = reference(x, w, None)[1]
    assert bool(((y.double() - n).abs() <= n.abs() * 2.0 ** -18 + 2.0 ** -149).all())
    assert bool((y[0] == 0).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_rows_stay_alone(cr, bad):
    M, K = 37, 1024
    x, r, w = rows(1, M, K, BF16), rows(2, M, K, F32), weight(K)
    xb = x.clone()
    xb[4, 100] = bad
    xb[5, 1023] = bad
    others = [i for i in range(M) if i not in (4, 5)]
    y0, h0 = cr.convrot_add_rms_norm_forward(x, w, r)
    y1, h1 = cr.convrot_add_rms_norm_forward(xb, w, r)
    assert torch.equal(y0[others], y1[others]) and torch.equal(h0[others], h1[others])
    assert bool(y1[4].isnan().any()) and bool(y1[5].isnan().any())
    W = cr.convrot_linear_prepare_weights(rows(3, 256, K, F32) * 0.02, 128)
    F, P = (cr.convrot_fp8_prepare_weights(rows(3, 256, K, F32) * 0.02, scales=s)
            for s in ("f32", "pow2"))
    for weights in (W, F, P):
        for n in (M, 9):                             # tiles, and the kernels for few rows
            for out in (BF16, F32):
                a, _ = cr.convrot_norm_linear_forward(x[:n], w, weights, r[:n], out_dtype=out)
                b, _ = cr.convrot_norm_linear_forward(xb[:n], w, weights, r[:n], out_dtype=out)
                assert torch.equal(a[others[:n - 2]], b[others[:n - 2]])
                assert bool(b[4].isnan().all()) and bool(b[5].isnan().all())


@pytest.mark.parametrize("eps", [1e-30, 1e-38, 2e-45])
def test_tiny_eps(cr, eps):
    """A zero row is 0 times a large number, forward and backward, not 0 times infinity."""
    K = 256
    x, w, g = torch.zeros(3, K, device="cuda"), weight(K), rows(1, 3, K, F32) * 1e-9
    x[1] = 1e-25
    x[2, 3] = -2.0
    y, _ = cr.convrot_add_rms_norm_forward(x, w, eps=eps, out_dtype=F32)
    assert bool((y[0] == 0).all()) and bool(y.isfinite().all())
    dh, _, dw = cr.convrot_add_rms_norm_backward(g, x, w, eps=eps)
    assert not bool(dh.isnan().any()) and bool(dw.isfinite().all())
    v = x[2].double()
    q = 1 / ((v * v).mean() + eps).sqrt()
    t = g[2].double() * w.double()
    d = q * (t - v * q * (t * v * q).mean())
    size = q * (t.abs() + (v * q).abs() * (t * v * q).abs().mean())
    assert bool(((dh[2].double() - d).abs() <= size * 2.0 ** -15 + 2.0 ** -130).all())


BLOCKS = [(64, "sylvester"), (128, "sylvester"), (256, "sylvester"), (64, "regular"),
          (256, "regular")]


@pytest.mark.parametrize("x_t,r_t", TYPES, ids=str)
@pytest.mark.parametrize("block,rotation", BLOCKS, ids=str)
def test_int8_codes(cr, block, rotation, x_t, r_t):
    """Equal bits: rotate_quantize of the fp32 rows of the norm."""
    for M, K in ((1, 256), (3, 768), (18, 1280), (35, 5376), (2, 8192 + 256), (5, 16384 + 256),
                 (1, 32768)):
        announce(f"norm int8 M={M} K={K} b={block} {rotation} x={x_t} r={r_t}")
        x = rows(1, M, K, DT[x_t])
        r = None if r_t is None else rows(2, M, K, DT[r_t], 3.0)
        w = weight(K)
        n, h0 = cr.convrot_add_rms_norm_forward(x, w, r, out_dtype=F32)
        q0, s0 = cr.convrot_rotate_quantize(n, block, rotation=rotation)
        q1 = torch.full((padded_rows(M), K), 99, dtype=torch.int8, device="cuda")
        s1 = torch.full((M + 4,), 7.0, device="cuda")
        _, _, h1 = cr.convrot_add_rms_norm_rotate_quantize(x, w, block, r, rotation=rotation,
                                                           q=q1, s=s1[:M])
        assert torch.equal(s1[:M], s0) and bool((s1[M:] == 7).all())
        assert np.array_equal(untile(q1, M, K), untile(q0, M, K))
        assert (h1 is None and h0 is None) or torch.equal(h1, h0)
        if M % 16:                                   # the padding rows are left as they were
            assert np.all(untile(q1, padded_rows(M), K)[M:] == 99)


@pytest.mark.parametrize("scales", ["f32", "pow2"])
@pytest.mark.parametrize("x_t,r_t", TYPES, ids=str)
def test_fp8_codes(cr, scales, x_t, r_t):
    """Equal bits: the fp32 rows of the norm quantised by the definition."""
    for M, K in ((1, 128), (3, 640), (18, 1280), (35, 5376), (2, 8320), (5, 16512), (1, 32768)):
        announce(f"norm fp8 M={M} K={K} {scales} x={x_t} r={r_t}")
        x = rows(1, M, K, DT[x_t])
        x[:, :128] = 0                               # with the residual's zeros: a zero block
        r = None if r_t is None else rows(2, M, K, DT[r_t], 3.0)
        if r is not None:
            r[:, :128] = 0
        w = weight(K)
        n, _ = cr.convrot_add_rms_norm_forward(x, w, r, out_dtype=F32)
        b = n.view(M, K // 128, 128)
        amax = b.abs().amax(-1)
        s = (amax.double() / 448).float().clamp_min(2.0 ** -126)
        if scales == "pow2":
            m, e = torch.frexp(s)
            s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
        s = torch.where(amax > 0, s, amax)
        inv = torch.where(s > 0, (1 / s.double()).float(), s)
        codes = (b * inv[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        Mp = padded_rows(M)
        q = torch.full((Mp, K), 99, dtype=torch.uint8, device="cuda")
        s1 = torch.full((K // 128, Mp), 7.0, device="cuda")
        cr.convrot_add_rms_norm_fp8_quantize(x, w, scales, r, q=q, s=s1)
        assert torch.equal(s1[:, :M].t(), s) and bool((s1[:, M:] == 7).all())
        assert np.array_equal(untile(q, M, K), codes.view(M, K).cpu().numpy())
        if M % 16:
            assert np.all(untile(q, Mp, K)[M:] == 99)


@pytest.mark.parametrize("kind", ["int8", "int8_regular", "fp8_f32", "fp8_pow2"])
@pytest.mark.parametrize("M", [0, 1, 16, 17, 300])
def test_norm_linear(cr, kind, M):
    """Equal bits: the codes, then the linear's own product."""
    K, N = 1280, 528
    x, r, w = rows(1, M, K, BF16), rows(2, M, K, F32, 3.0), weight(K)
    W32, bias = rows(3, N, K, F32) * 0.02, rows(4, 1, N, F32)[0]
    for out_t in (BF16, F32):
        if kind.startswith("int8"):
            rot = "regular" if kind.endswith("regular") else "sylvester"
            W = cr.convrot_linear_prepare_weights(W32, 64, rotation=rot)
            q, s, h0 = cr.convrot_add_rms_norm_rotate_quantize(x, w, 64, r, rotation=rot)
            ref = cr.convrot_gemm_dequant(q, s, W, bias, out_dtype=out_t)
        else:
            sc = kind[4:]
            W = cr.convrot_fp8_prepare_weights(W32, scales=sc)
            q, s, h0 = cr.convrot_add_rms_norm_fp8_quantize(x, w, sc, r)
            ref = cr.convrot_fp8_gemm_dequant(q, s, M, W, bias, out_dtype=out_t, scales=sc)
        whole, out = guarded(M, N, out_t)
        y, h = cr.convrot_norm_linear_forward(x, w, W, r, bias=bias, out=out)
        assert torch.equal(y, ref) and torch.equal(h, h0)
        unharmed(whole, M)
    if M > 1:
        # and near the product with the exact norm: the codes' steps, at random over K
        n = reference(x, w, r)[1]
        exact = n @ W32.double().t() + bias.double()
        assert float((y.double() - exact).norm() / exact.norm()) < 0.06


def test_pre_norm_block(cr):
    """As a layer uses them: norm -> QKV -> Q/K norms and positions in place, and the residual
    stream carried in fp32, against the unfused calls."""
    B, T, K, H, D = 2, 75, 512, 4, 64
    x, r, w = rows(1, B * T, K, BF16), rows(2, B * T, K, F32, 3.0), weight(K)
    W = cr.convrot_linear_prepare_weights(rows(3, 3 * H * D, K, F32) * 0.02, 128)
    rope = cr.convrot_rope_prepare([D], D)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    y, h = cr.convrot_norm_linear_forward(x.view(B, T, K), w, W, r.view(B, T, K))
    q, k, v = y.view(B, T, 3, H, D).unbind(2)
    cr.convrot_qk_norm_rope_forward(q, k, None, None, rope, pos, out_q=q, out_k=k)
    n, h2 = cr.convrot_add_rms_norm_forward(x, w, r)
    ref = cr.convrot_qkv_forward(n.view(B, T, K), W, H, H, None, None, rope, pos)
    assert torch.equal(h.view(-1, K), h2)
    # the unfused path rounds n to bf16 before it is quantised: a code step here and there
    assert float((y.float() - ref.float()).norm() / ref.float().norm()) < 0.02


def test_in_place(cr):
    M, K = 19, 1288
    for x_t, r_t in TYPES[1:3] + TYPES[4:]:
        x, r, w = rows(1, M, K, DT[x_t]), rows(2, M, K, DT[r_t]), weight(K)
        y, h = cr.convrot_add_rms_norm_forward(x, w, r, out_dtype=x.dtype)
        xi, ri = x.clone(), r.clone()
        cr.convrot_add_rms_norm_forward(xi, w, ri, out=xi, residual_out=ri)
        assert torch.equal(xi, y) and torch.equal(ri, h)
        if x.dtype == r.dtype:
            xi = x.clone()
            cr.convrot_add_rms_norm_forward(xi, w, r, out=(o := torch.empty_like(x)),
                                            residual_out=xi)
            assert torch.equal(xi, h) and torch.equal(o, y)
    g, h, gh, w = rows(5, M, K, F32), rows(6, M, K, F32), rows(7, M, K, F32), weight(K)
    dh, dx, dw = cr.convrot_add_rms_norm_backward(g, h, w, g_h=gh, x_dtype=BF16)
    for which in range(3):
        t = [g.clone(), h.clone(), gh.clone()]
        d2, dx2, dw2 = cr.convrot_add_rms_norm_backward(t[0], t[1], w, g_h=t[2], x_dtype=BF16,
                                                        dh=t[which])
        assert torch.equal(d2, dh) and torch.equal(dx2, dx) and torch.equal(dw2, dw)
    gb = g.to(BF16)
    dh, dx, dw = cr.convrot_add_rms_norm_backward(gb, h, w, g_h=gh, x_dtype=BF16)
    gi = gb.clone()
    d2, _, dw2 = cr.convrot_add_rms_norm_backward(gi, h, w, g_h=gh, x_dtype=BF16, dx=gi)
    assert torch.equal(d2, dh) and torch.equal(gi, dx) and torch.equal(dw2, dw)


GRAD_SHAPES = [(1, 8), (3, 24), (2, 504), (130, 512), (67, 520), (17, 1000), (301, 2304),
               (5, 5376), (1100, 5376), (6, 8192), (5, 8200), (3, 16384), (4, 16392), (2, 32768)]


def reference_backward(g, h, w, gh):
    v, t = h.double(), g.double()
    if w is not None:
        t = t * w.double()
    K = v.shape[-1]
    q = 1 / ((v * v).mean(-1, keepdim=True) + EPS).sqrt()
    a, b = q * t, v * q ** 3 * ((t * v).sum(-1, keepdim=True) / K)
    size = a.abs() + v.abs() * q ** 3 * ((t * v).abs().sum(-1, keepdim=True) / K)
    d = a - b
    if gh is not None:
        d, size = d + gh.double(), size + gh.double().abs()
    terms = g.double() * v * q
    return d, size, terms.sum(0), terms.abs().sum(0)


@pytest.mark.parametrize("g_t,h_t", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"),
                                     ("f32", "f32")])
@pytest.mark.parametrize("M,K", GRAD_SHAPES, ids=str)
def test_backward(cr, M, K, g_t, h_t):
    announce(f"norm backward M={M} K={K} g={g_t} h={h_t}")
    g, h = rows(1, M, K, DT[g_t], 0.01), rows(2, M, K, DT[h_t])
    for w in (weight(K), None):
        for gh in (rows(3, M, K, DT[h_t], 0.01), None):
            whole, out = guarded(M, K, h.dtype)
            want_dx = h_t == "f32"
            dh, dx, dw = cr.convrot_add_rms_norm_backward(
                g, h, w, g_h=gh, eps=EPS, dh=out, x_dtype=BF16 if want_dx else None)
            unharmed(whole, M)
            d, size, ref_dw, dw_size = reference_backward(g, h, w, gh)
            bound = size * 2.0 ** -15
            assert bool(((dh.double() - d).abs() <= bound + d.abs() * HALF[h.dtype]
                         + 2.0 ** -130).all())
            if want_dx:
                assert torch.equal(dx, dh.to(BF16))
            else:
                assert dx is dh
            if w is None:
                assert dw is None
            else:
                off = (dw.double() - ref_dw).abs()
                assert bool((off <= dw_size * ((M + 64) * 2.0 ** -24) + 2.0 ** -130).all())
    again = cr.convrot_add_rms_norm_backward(g, h, weight(K), g_h=None)
    first = cr.convrot_add_rms_norm_backward(g, h, weight(K), g_h=None)
    assert torch.equal(again[0], first[0]) and torch.equal(again[2], first[2])


def test_backward_against_differences(cr):
    """<g, dn> along a direction of x, r and w, from central differences of the definition in
    64 bits (their own error: under 1e-7 of the derivative at this step)."""
    M, K, e = 5, 136, 1e-5
    g, h, w = rows(1, M, K, F32), rows(2, M, K, F32), weight(K)
    dh, _, dw = cr.convrot_add_rms_norm_backward(g, h, w, g_h=None)
    dv, dwv = rows(3, M, K, F32).double(), rows(4, 1, K, F32)[0].double()
    f = lambda a, b: (g.double() * a / ((a * a).mean(-1, keepdim=True) + EPS).sqrt() * b).sum()  # noqa: E731
    want = (f(h.double() + e * dv, w.double()) - f(h.double() - e * dv, w.double())) / (2 * e)
    _, size, _, dw_size = reference_backward(g, h, w, None)
    assert abs(float((dh.double() * dv).sum() - want)) <= \
        float((size * dv.abs()).sum()) * (2.0 ** -15 + 2.0 ** -24 + 1e-7)
    want = (f(h.double(), w.double() + e * dwv) - f(h.double(), w.double() - e * dwv)) / (2 * e)
    assert abs(float((dw.double() * dwv).sum() - want)) <= \
        float((dw_size * dwv.abs()).sum()) * (80 * 2.0 ** -24 + 1e-7)


def test_no_rows(cr):
    x = torch.empty(0, 512, dtype=BF16, device="cuda")
    w = weight(512)
    y, h = cr.convrot_add_rms_norm_forward(x, w, x)
    assert y.shape == (0, 512) and h.shape == (0, 512)
    dh, dx, dw = cr.convrot_add_rms_norm_backward(x, x, w)
    assert dh.shape == (0, 512) and bool((dw == 0).all())
    q, s, _ = cr.convrot_add_rms_norm_rotate_quantize(x, w, 128)
    assert s.shape == (0,)


def test_graphs(cr):
    """Forward, quantised forward and backward in two graphs that share a workspace, replayed
    several times with eager work in between; an eager autograd graph of the same leaves lives
    meanwhile."""
    M, K = 70, 2304
    x, r, g, gh = (torch.empty(M, K, dtype=t, device="cuda") for t in (BF16, F32, BF16, F32))
    w = weight(K)
    W = cr.convrot_linear_prepare_weights(rows(3, 256, K, F32) * 0.02, 128)
    ws = torch.empty(max(cr.convrot_add_rms_norm_workspace_bytes(M, K),
                         cr.convrot_linear_workspace_bytes(M, K, 256, 128)), dtype=torch.uint8,
                     device="cuda")
    leaf = w.detach().clone().requires_grad_()
    kept = (leaf * leaf).sum()

    def step():
        y, h = cr.convrot_add_rms_norm_forward(x, w, r)
        z, _ = cr.convrot_norm_linear_forward(x, w, W, r, workspace=ws)
        dh, dx, dw = cr.convrot_add_rms_norm_backward(g, h, w, g_h=gh, x_dtype=BF16, workspace=ws)
        return y, h, z, dh, dx, dw

    def fill(i):
        for j, t in enumerate((x, r, g, gh)):
            t.copy_(rows(10 * i + j, M, K, t.dtype))

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = step()
        graphs.append((gr, out))
    for i in range(1, 5):
        fill(i)
        want = [t.clone() for t in step()]
        for gr, out in graphs:
            for t in out:
                t.fill_(3)
            gr.replay()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), i
        torch.cuda.synchronize()
    kept.backward()


def test_callers_stream(cr):
    M, K = 333, 2304
    x, r, w = rows(1, M, K, BF16), rows(2, M, K, F32), weight(K)
    W = cr.convrot_fp8_prepare_weights(rows(3, 256, K, F32) * 0.02)
    want = (*cr.convrot_add_rms_norm_forward(x, w, r), *cr.convrot_norm_linear_forward(x, w, W, r),
            *cr.convrot_add_rms_norm_backward(x, r, w, g_h=r))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(6):                               # two streams at once
        s = streams[i % 2]
        outs.append((*cr.convrot_add_rms_norm_forward(x, w, r, stream=s),
                     *cr.convrot_norm_linear_forward(x, w, W, r, stream=s),
                     *cr.convrot_add_rms_norm_backward(x, r, w, g_h=r, stream=s)))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_offsets_past_32_bits(cr):
    """More than 2^31 elements (2^33 bytes of fp32): the last rows against their own call."""
    M, K = 66000, 32768
    w = weight(K)
    x = torch.empty(M, K, dtype=BF16, device="cuda").fill_(0.25)
    r = torch.empty(M, K, dtype=F32, device="cuda").fill_(0.5)
    x[-3:], r[-3:] = rows(1, 3, K, BF16), rows(2, 3, K, F32)
    y, h = cr.convrot_add_rms_norm_forward(x, w, r)
    a, b = cr.convrot_add_rms_norm_forward(x[-4:].clone(), w, r[-4:].clone())
    assert torch.equal(y[-4:], a) and torch.equal(h[-4:], b)
    del r
    dh, _, dw = cr.convrot_add_rms_norm_backward(y, h, None, g_h=h, dh=h)
    d2, _, _ = cr.convrot_add_rms_norm_backward(a, b, None, g_h=b)
    assert torch.equal(dh[-4:], d2) and dw is None


def test_more_rows_than_a_grid_dimension_holds(cr):
    """A grid of more than 2^32 threads in a row: every row against a second call in parts."""
    M, K = 2 ** 27 + 37, 8
    x = torch.empty(M, K, dtype=BF16, device="cuda")
    x.view(torch.int16).copy_(torch.arange(K, device="cuda", dtype=torch.int16) + 0x3f80)
    x[:, 3] = (torch.arange(M, device="cuda") % 251).to(BF16)
    y, _ = cr.convrot_add_rms_norm_forward(x, None)
    for at in range(0, M, 2 ** 25 + 8):
        part, _ = cr.convrot_add_rms_norm_forward(x[at:at + 2 ** 25 + 8], None)
        assert torch.equal(y[at:at + 2 ** 25 + 8], part)


@pytest.mark.parametrize("K", [256, 1280, 5376, 8448, 16640])
@pytest.mark.parametrize("block,rotation", BLOCKS, ids=str)
def test_non_finite_weights_reach_every_row(cr, block, rotation, K):
    """A NaN in the norm's weight, or infinities that meet as NaN in a block's rotation (an odd
    number of minus signs over four of its channels), show in the outputs of the INT8 form as
    in those of the others: no row looks finite."""
    x, w = rows(1, 18, K, BF16), weight(K)
    x[:, :4] = 1
    bad = []
    for at in (0, K // 2 + 3, K - 1):
        wb = w.clone()
        wb[at] = float("nan")
        bad.append(wb)
    wb = w.clone()
    wb[:4] = torch.tensor([1.0, 1, 1, -1], device="cuda") * float("inf")
    bad.append(wb)
    W8 = cr.convrot_linear_prepare_weights(rows(3, 64, K, F32) * 0.02, block, rotation=rotation)
    F = cr.convrot_fp8_prepare_weights(rows(3, 64, K, F32) * 0.02)
    for wb in bad:
        y, _ = cr.convrot_add_rms_norm_forward(x, wb)
        assert not bool(y.isfinite().all(1).any())
        _, s, _ = cr.convrot_add_rms_norm_rotate_quantize(x, wb, block, rotation=rotation)
        assert bool(s.isnan().all())
        for W in (W8, F):
            y, _ = cr.convrot_norm_linear_forward(x, wb, W)
            assert bool(y.isnan().all())


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("M", [3, 40, 300])
def test_norm_linear_in_place(cr, kind, M):
    """Y in the place of x, or of the residual, which the first launch has read by then."""
    K = N = 640
    x, r, w = rows(1, M, K, BF16), rows(2, M, K, F32, 3.0), weight(K)
    W32 = rows(3, N, K, F32) * 0.02
    W = cr.convrot_linear_prepare_weights(W32, 128) if kind == "int8" else \
        cr.convrot_fp8_prepare_weights(W32)
    for out_t in (BF16, F32):
        y, h = cr.convrot_norm_linear_forward(x, w, W, r, out_dtype=out_t)
        t = (x.clone(), r.clone())
        at = t[0] if out_t == BF16 else t[1]
        y1, h1 = cr.convrot_norm_linear_forward(t[0], w, W, t[1], out=at)
        assert y1 is at and torch.equal(y1, y) and torch.equal(h1, h)


def rows_past_caches(K, bytes_a_channel):
    """The least odd number of rows whose call moves more than 2^28 bytes (such calls read and
    write past the caches)."""
    return (2 ** 28 // (K * bytes_a_channel) + 1) | 1


@pytest.mark.parametrize("out_t", [BF16, F32], ids=str)
@pytest.mark.parametrize("x_t,r_t", TYPES, ids=str)
@pytest.mark.parametrize("K", [40, 520, 4104, 8192])
def test_forward_past_the_caches(cr, K, x_t, r_t, out_t):
    """Against the definition, and bit for bit against parts of the rows, whose calls go through
    the caches; in place too."""
    size = {"bf16": 2, "f32": 4, None: 0}
    M = rows_past_caches(K, size[x_t] + 2 * size[r_t] + (4 if out_t == F32 else 2))
    announce(f"norm past the caches M={M} K={K} x={x_t} r={r_t} {out_t}")
    x = rows(1, M, K, DT[x_t])
    r = None if r_t is None else rows(2, M, K, DT[r_t], 3.0)
    w = weight(K)
    whole, out = guarded(M, K, out_t)
    hw, h = guarded(M, K, r.dtype) if r is not None else (None, None)
    y, _ = cr.convrot_add_rms_norm_forward(x, w, r, eps=EPS, out=out, residual_out=h)
    unharmed(whole, M)
    if r is not None:
        unharmed(hw, M)
    step = M // 3 + 1
    for at in range(0, M, step):
        part = slice(at, min(at + step, M))
        rp = None if r is None else r[part]
        y1, h1 = cr.convrot_add_rms_norm_forward(x[part], w, rp, eps=EPS, out_dtype=out_t)
        h_ref, n = reference(x[part], w, rp)
        assert torch.equal(y[part], y1)
        assert r is None or (torch.equal(h[part], h1) and torch.equal(h1, h_ref))
        assert bool(((y[part].double() - n).abs()
                     <= n.abs() * (2.0 ** -18 + HALF[out_t])).all())
        del n, h_ref
    if r is not None:
        xi, ri = x.clone(), r.clone()
        y2, h2 = cr.convrot_add_rms_norm_forward(xi, w, ri, eps=EPS, out_dtype=out_t,
                                                 out=xi if x.dtype == out_t else None,
                                                 residual_out=ri)
        assert h2 is ri and torch.equal(y2, y) and torch.equal(h2, h)


@pytest.mark.parametrize("g_t,h_t", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"),
                                     ("f32", "f32")])
@pytest.mark.parametrize("K", [40, 520, 4104, 8192, 16384, 16392])
def test_backward_past_the_caches(cr, K, g_t, h_t):
    """Against the definition, the rows of dh bit for bit against parts of them, whose calls go
    through the caches; in place too."""
    size = {"bf16": 2, "f32": 4}
    want_dx = h_t == "f32"
    M = rows_past_caches(K, size[g_t] + 3 * size[h_t] + (2 if want_dx else 0))
    announce(f"norm backward past the caches M={M} K={K} g={g_t} h={h_t}")
    g, h, gh = rows(1, M, K, DT[g_t], 0.01), rows(2, M, K, DT[h_t]), rows(3, M, K, DT[h_t], 0.01)
    w = weight(K)
    whole, out = guarded(M, K, h.dtype)
    dh, dx, dw = cr.convrot_add_rms_norm_backward(g, h, w, g_h=gh, eps=EPS, dh=out,
                                                  x_dtype=BF16 if want_dx else None)
    unharmed(whole, M)
    dx_ok = torch.equal(dx, dh.to(BF16)) if want_dx else dx is dh
    assert dx_ok
    ref_dw, dw_size = (torch.zeros(K, dtype=torch.float64, device="cuda") for _ in range(2))
    step = M // 3 + 1
    for at in range(0, M, step):
        part = slice(at, min(at + step, M))
        d1, _, _ = cr.convrot_add_rms_norm_backward(g[part], h[part], w, g_h=gh[part], eps=EPS)
        assert torch.equal(dh[part], d1)
        d, size_d, a, b = reference_backward(g[part], h[part], w, gh[part])
        assert bool(((dh[part].double() - d).abs() <= size_d * 2.0 ** -15
                     + d.abs() * HALF[h.dtype] + 2.0 ** -130).all())
        ref_dw += a
        dw_size += b
        del d, size_d
    assert bool(((dw.double() - ref_dw).abs()
                 <= dw_size * ((M + 64) * 2.0 ** -24) + 2.0 ** -130).all())
    t = gh.clone()
    d2, _, dw2 = cr.convrot_add_rms_norm_backward(g, h, w, g_h=t, eps=EPS, dh=t)
    assert d2 is t and torch.equal(d2, dh) and torch.equal(dw2, dw)


def test_more_rows_than_a_grid_dimension_holds_in_small_parts(cr):
    """The same rows against calls below the border of the caches, at the ends and in the middle."""
    M, K = 2 ** 27 + 37, 8
    x = torch.empty(M, K, dtype=BF16, device="cuda")
    x.view(torch.int16).copy_(torch.arange(K, device="cuda", dtype=torch.int16) + 0x3f80)
    x[:, 3] = (torch.arange(M, device="cuda") % 251).to(BF16)
    y, _ = cr.convrot_add_rms_norm_forward(x, None)
    n = 2 ** 22 + 8                                  # 2^27 bytes
    for at in (0, 5 * n + 3, M // 2 - n // 2, 2 ** 26 - n + 5, M - n):
        part, _ = cr.convrot_add_rms_norm_forward(x[at:at + n], None)
        ref = reference(x[at:at + n], None, None)[1]
        assert torch.equal(y[at:at + n], part)
        assert bool(((part.double() - ref).abs() <= ref.abs() * (2.0 ** -18 + HALF[BF16])).all())
