"""GPU tests of the FP8 block-scaled linear against its definition in 64 bits.

Codes and scales are compared bit for bit.  Outputs: the reference sums the
exact products of the codes and scales in fp64; a kernel may round each of its
fp32 additions and the product of the two scales, so an output is within
(K + K/128 + 4) 2^-24 of the sum of the terms' magnitudes, plus the rounding to
the output type (2^-8 of the value for bf16, 2^-24 for fp32).  Where s_x s_w
falls below 2^-126, fp32 holds it in steps of 2^-149: it is then off by up to
2^-150 whatever its size, and the block's term by that times |sum qx qw|, at
most 2^-150 sum |qx qw|.  bf16 outputs use the FP8 matrix instructions, which cut
each of 8 neighbouring products to a multiple of 2^-13 of the power of two of the
largest (the public header says so): less than 2^-13 of the largest for 7 of
them, and the largest product is at most the product of the largest codes."""
import numpy as np
import pytest
import torch

from gpu_util import announce, padded_rows, tile, untile

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def cr():
    from w8a8_int8_rotated_amd import convrot
    convrot.library()
    return convrot


def block_scale(amax, kind):
    """fp32 scales of fp64 block maxima."""
    s = np.maximum((amax / 448).astype(np.float32), np.float32(2.0 ** -126))
    if kind == "pow2":
        m, e = np.frexp(s.astype(np.float64))
        s = np.ldexp(1.0, np.where(m == 0.5, e - 1, e)).astype(np.float32)
    return np.where(amax > 0, s, np.float32(0)).astype(np.float32)


def to_codes(v):
    """e4m3 bits of fp32 values (torch's conversion: round to nearest even)."""
    return torch.from_numpy(v.astype(np.float32)).to(F8).view(torch.uint8).numpy()


def from_codes(q):
    return torch.from_numpy(np.ascontiguousarray(q)).view(F8).to(torch.float64).numpy()


def quantize_rows(x, kind):
    M, K = x.shape
    xb = x.astype(np.float64).reshape(M, K // 128, 128)
    s = block_scale(np.abs(xb).max(-1), kind)
    inv = np.zeros_like(s)
    inv[s > 0] = (1.0 / s[s > 0].astype(np.float64)).astype(np.float32)
    v = (xb * inv.astype(np.float64)[..., None]).astype(np.float32)
    return to_codes(v.reshape(M, K)), s


def quantize_blocks(w, kind):
    N, K = w.shape
    nb = -(-N // 128)
    full = np.zeros((nb * 128, K), np.float64)
    full[:N] = w
    fb = full.reshape(nb, 128, K // 128, 128)
    s = block_scale(np.abs(fb).max((1, 3)), kind)
    inv = np.zeros_like(s)
    inv[s > 0] = (1.0 / s[s > 0].astype(np.float64)).astype(np.float32)
    v = (fb * inv.astype(np.float64)[:, None, :, None]).astype(np.float32)
    return to_codes(v.reshape(nb * 128, K)[:N]), s


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def rows(rng, M, K):
    """Activations with outliers, a block of zeros and a tiny block."""
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, rng.random(K) < 0.02] *= 30
    x = bf16(x).float().numpy()
    x[M // 2, :128] = 0
    x[-1, -128:] = np.float32(2.0 ** -130) * np.arange(128)
    return bf16(x).float().numpy()


def check(y, xq, sx, wq, sw, bias=None, what=""):
    """y against the fp64 sum, with the bound of the module's docstring."""
    M, K = xq.shape
    N = wq.shape[0]
    xd = from_codes(xq) * np.repeat(sx.astype(np.float64), 128, 1)
    wd = from_codes(wq) * np.repeat(np.repeat(sw.astype(np.float64), 128, 0)[:N], 128, 1)
    ref, mag = xd @ wd.T, np.abs(xd) @ np.abs(wd).T
    codes = np.abs(from_codes(xq)) @ np.abs(from_codes(wq)).T
    if bias is not None:
        ref, mag = ref + bias, mag + np.abs(bias)
    half = 2.0 ** (-8 if y.dtype == torch.bfloat16 else -24)
    got = y.double().cpu().numpy()
    bound = (K + K // 128 + 4) * 2.0 ** -24 * mag + 2.0 ** -150 * codes
    if y.dtype == torch.bfloat16:
        g = lambda a: np.abs(a).reshape(a.shape[0], K // 8, 8).max(-1)
        bound += 7 * 2.0 ** -13 * (g(xd) @ g(wd).T)
    bound = bound + half * (np.abs(ref) + bound) + 2.0 ** -140
    worst = np.max(np.abs(got - ref) / bound) if got.size else 0.0
    print(f"[parity] {what}: worst error {worst:.3f} of its bound", flush=True)
    assert worst <= 1.0


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("M,K", [(1, 128), (5, 384), (17, 1024), (130, 5376), (33, 2176)])
def test_quantize_rows(cr, kind, M, K):
    announce(f"fp8 quantize {M}x{K} {kind}")
    x = rows(np.random.default_rng(M + K), M, K)
    Mp = padded_rows(M)
    q = torch.full((Mp, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((K // 128, Mp), -7.0, device="cuda")
    cr.convrot_fp8_quantize(bf16(x).cuda(), kind, q=q, s=s)
    qr, sr = quantize_rows(x, kind)
    got = untile(q.view(torch.int8), M, K).view(np.uint8)
    assert np.array_equal(got, qr)
    assert np.array_equal(s[:, :M].t().cpu().numpy(), sr)
    # the padding rows and columns are left as they were
    assert bool((s[:, M:] == -7.0).all())
    pad = untile(q.view(torch.int8), Mp, K)[M:]
    assert np.all(pad == 0x55)


def test_quantize_every_e4m3_neighbourhood(cr):
    """A block holding 448 (factor 1): every bf16 value in the code range, ties
    and subnormals among them, is rounded as the definition rounds it."""
    announce("fp8 quantize: every bf16 up to 448")
    bits = np.arange(0x0000, 0x43E1, dtype=np.uint32)               # 0 .. 448
    vals = (bits << 16).astype(np.uint32).view(np.float32)
    vals = np.concatenate([vals, -vals])
    vals = np.pad(vals, (0, -len(vals) % 127))
    x = np.concatenate([vals.reshape(-1, 127), np.full((len(vals) // 127, 1), 448.0)], 1)
    x = x.astype(np.float32)
    M = x.shape[0]
    q, s = cr.convrot_fp8_quantize(bf16(x).cuda())
    assert bool((s[0, :M] == 1).all())
    assert np.array_equal(untile(q.view(torch.int8), M, 128).view(np.uint8), to_codes(x))


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("N,K", [(16, 128), (48, 256), (272, 640)])
def test_prepare_weights(cr, kind, N, K):
    rng = np.random.default_rng(N)
    w = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    w[:16, :128] = 0
    for dt in (torch.float32, torch.bfloat16):
        wt = torch.from_numpy(w).to(dt)
        qr, sr = quantize_blocks(wt.float().numpy(), kind)
        for layout in (cr.OUT_MAJOR, cr.IN_MAJOR):
            announce(f"fp8 prepare {N}x{K} {kind} {dt} layout {layout}")
            src = wt.cuda() if layout == cr.OUT_MAJOR else wt.t().contiguous().cuda()
            pw = cr.convrot_fp8_prepare_weights(src, layout, scales=kind)
            assert np.array_equal(untile(pw.codes.view(torch.int8), N, K).view(np.uint8), qr)
            assert np.array_equal(pw.scale.cpu().numpy(), sr)
    codes, scale = torch.from_numpy(qr).view(F8).cuda(), torch.from_numpy(sr).cuda()
    for layout in (cr.OUT_MAJOR, cr.IN_MAJOR):
        src = codes if layout == cr.OUT_MAJOR else codes.view(torch.uint8).t().contiguous().view(F8)
        pw = cr.convrot_fp8_prepare_weights(src, layout, src_scale=scale, scales=kind)
        assert np.array_equal(untile(pw.codes.view(torch.int8), N, K).view(np.uint8), qr)
        assert np.array_equal(pw.scale.cpu().numpy(), sr)


SHAPES = [(1, 128, 16), (1, 5376, 272), (3, 640, 48), (16, 1024, 144), (17, 128, 16),
          (37, 384, 400), (64, 256, 1040), (129, 896, 272), (255, 1152, 528), (256, 512, 512),
          (333, 5376, 256), (700, 768, 784), (1025, 640, 1296)]


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_forward(cr, kind, M, K, N):
    rng = np.random.default_rng(M * 7 + N)
    x, w = rows(rng, M, K), (rng.standard_normal((N, K)) * 0.05).astype(np.float32)
    bias = rng.standard_normal(N).astype(np.float32)
    pw = cr.convrot_fp8_prepare_weights(torch.from_numpy(w).cuda(), scales=kind)
    (xq, sx), (wq, sw) = quantize_rows(x, kind), quantize_blocks(w, kind)
    X = bf16(x).cuda()
    ws = torch.full((max(1, cr.convrot_fp8_linear_workspace_bytes(M, K, N)),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    for dt, b in ((torch.float32, None), (torch.bfloat16, bias)):
        announce(f"fp8 forward {M}x{K}x{N} {kind} {dt} bias={b is not None}")
        bt = None if b is None else torch.from_numpy(b).cuda()
        # rows behind the output stay as they were
        buf = torch.full((M + 2, N), 3.0, dtype=dt, device="cuda")
        cr.convrot_fp8_linear_forward(X, pw, bias=bt, out=buf[:M], workspace=ws)
        check(buf[:M], xq, sx, wq, sw, b, f"fp8 {M}x{K}x{N} {kind} {dt}")
        assert bool((buf[M:] == 3.0).all())
        # the same call repeats bit for bit
        again = cr.convrot_fp8_linear_forward(X, pw, bias=bt, out_dtype=dt)
        assert torch.equal(again, buf[:M])


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_hooks_equal_forward(cr, kind, M):
    K, N = 640, 272
    rng = np.random.default_rng(M)
    X = bf16(rows(rng, M, K)).cuda()
    pw = cr.convrot_fp8_prepare_weights(
        torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32)).cuda(), scales=kind)
    announce(f"fp8 hooks {M}x{K}x{N} {kind}")
    q, s = cr.convrot_fp8_quantize(X, kind)
    y = cr.convrot_fp8_gemm_dequant(q, s, M, pw, out_dtype=torch.float32)
    want = cr.convrot_fp8_linear_forward(X, pw, out_dtype=torch.float32)
    if M > 16:
        assert torch.equal(y, want)
    wq, sw = untile(pw.codes.view(torch.int8), N, K).view(np.uint8), pw.scale.cpu().numpy()
    xq, sx = quantize_rows(X.float().cpu().numpy(), kind)
    check(y, xq, sx, wq, sw, what=f"hooks M={M}")


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("M,N", [(4, 272), (50, 272), (300, 272), (520, 5392)])
def test_non_finite_rows_stay_alone(cr, kind, M, N):
    """NaN and infinities make their own token's outputs NaN, no other's."""
    K = 512
    rng = np.random.default_rng(5)
    x = rng.standard_normal((M, K)).astype(np.float32)
    pw = cr.convrot_fp8_prepare_weights(
        torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32)).cuda(), scales=kind)
    clean = cr.convrot_fp8_linear_forward(bf16(x).cuda(), pw)
    bad = {0: np.nan, 1: np.inf, M - 1: -np.inf}
    for m, v in bad.items():
        x[m, (130 + m) % K] = v
    announce(f"fp8 non-finite M={M} {kind}")
    y = cr.convrot_fp8_linear_forward(bf16(x).cuda(), pw)
    keep = [m for m in range(M) if m not in bad]
    assert bool(torch.isnan(y[list(bad)]).all())
    assert torch.equal(y[keep], clean[keep])


def test_zero_and_empty(cr):
    K, N = 256, 144
    pw = cr.convrot_fp8_prepare_weights(torch.randn(N, K, device="cuda"))
    bias = torch.randn(N, device="cuda")
    for M in (0, 1, 20):
        announce(f"fp8 zero rows M={M}")
        y = cr.convrot_fp8_linear_forward(torch.zeros(M, K, dtype=torch.bfloat16, device="cuda"),
                                          pw, bias=bias, out_dtype=torch.float32)
        assert y.shape == (M, N) and torch.equal(y, bias.expand(M, N))


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("M,N", [(2, 528), (40, 528), (520, 528), (1025, 5392)])
def test_graph_and_streams(cr, kind, M, N):
    """Captured calls replay to the eager result, with eager work between the
    replays; a call on another stream gives it too."""
    K = 640
    X = torch.randn(M, K, device="cuda").to(torch.bfloat16)
    pw = cr.convrot_fp8_prepare_weights(torch.randn(N, K, device="cuda"), scales=kind)
    want = cr.convrot_fp8_linear_forward(X, pw)
    ws = torch.empty(max(1, cr.convrot_fp8_linear_workspace_bytes(M, K, N)), dtype=torch.uint8,
                     device="cuda")
    out = torch.zeros_like(want)
    announce(f"fp8 graph M={M} {kind}")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cr.convrot_fp8_linear_forward(X, pw, out=out, workspace=ws)
    for i in range(3):
        X2 = torch.randn(M, K, device="cuda").to(torch.bfloat16)
        X.copy_(X2)
        want = cr.convrot_fp8_linear_forward(X2, pw)
        ws.fill_(0xFF)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {i}"
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = cr.convrot_fp8_linear_forward(X, pw, stream=s)
    s.synchronize()
    assert torch.equal(y, want)


def test_pow2_import_refuses_other_scales(cr):
    codes = torch.zeros(128, 128, device="cuda").to(F8)
    for scale in (3.0, -2.0, float("inf"), float("nan")):
        with pytest.raises(ValueError, match="powers of two"):
            cr.convrot_fp8_prepare_weights(codes, scales="pow2",
                                           src_scale=torch.full((1, 1), scale, device="cuda"))


# every tile shape, the two-launch plan, ragged edges, odd and even counts of k-blocks
PLANS = [(100, 384, 528), (192, 256, 21504), (520, 128, 5376), (768, 384, 10880),
         (1000, 256, 5376), (2041, 256, 5392), (4133, 640, 5392), (2500, 128, 16128)]
# few rows or few outputs: the shapes of the kernel whose waves split the k-blocks
# (fewer k-blocks than waves, counts that 8 does not divide), and a long axis
PLANS += [(43, 4224, 32), (37, 640, 272), (333, 1280, 272), (93, 1664, 1776), (64, 1152, 5392),
          (70, 2176, 16144), (300, 896, 2064), (65, 21504, 48), (333, 1920, 5376)]


@pytest.mark.parametrize("M,K,N", PLANS)
def test_tile_plans(cr, M, K, N):
    """Every output of the tiled kernels against the fp64 product of the library's
    own codes and scales (checked against the definition above), on the GPU, with
    the bound of the module's docstring; scales of a row differ by factors of up to
    2^12 from block to block."""
    g = torch.Generator(device="cuda").manual_seed(M + N)
    X = torch.randn(M, K, generator=g, device="cuda")
    X = (X * torch.exp2(torch.randint(-6, 7, (M, K // 128, 1), generator=g, device="cuda"))
         .expand(-1, -1, 128).reshape(M, K)).to(torch.bfloat16)
    W = torch.randn(N, K, generator=g, device="cuda")
    bias = torch.randn(N, generator=g, device="cuda")
    for kind in ("f32", "pow2"):
        pw = cr.convrot_fp8_prepare_weights(W, scales=kind)
        q, s = cr.convrot_fp8_quantize(X, kind)
        dec = lambda c, n: torch.from_numpy(untile(c.view(torch.int8), n, K).copy()).cuda() \
            .view(F8).double()
        xc, wc = dec(q, M), dec(pw.codes, N)
        xd = xc * s[:, :M].t().double().repeat_interleave(128, 1)
        wd = wc * pw.scale.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
        ref, mag = xd @ wd.t() + bias.double(), xd.abs() @ wd.abs().t() + bias.double().abs()
        top = lambda a: a.abs().view(a.shape[0], K // 8, 8).amax(-1)
        cut = 7 * 2.0 ** -13 * (top(xd) @ top(wd).t())
        for dt in (torch.bfloat16, torch.float32):
            announce(f"fp8 plan {M}x{K}x{N} {kind} {dt}")
            y = cr.convrot_fp8_linear_forward(X, pw, bias=bias, out_dtype=dt)
            bound = (K + K // 128 + 4) * 2.0 ** -24 * mag
            if dt == torch.bfloat16:
                bound = bound + cut
            bound = bound + (2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24) * (ref.abs() + bound)
            worst = float(((y.double() - ref).abs() / bound).max())
            print(f"[parity] plan {M}x{K}x{N} {kind} {dt}: worst error {worst:.3f} of its bound",
                  flush=True)
            assert worst <= 1.0


@pytest.mark.parametrize("M,N", [(8, 272), (200, 272), (300, 272), (520, 5392)])
def test_non_finite_rows_fp32(cr, M, N):
    """As above for the kernels behind fp32 outputs, where a NaN must not cross
    from one k-block's scales or one tile into another token either."""
    K = 384
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M))
    pw = cr.convrot_fp8_prepare_weights(torch.randn(N, K, device="cuda"))
    clean = cr.convrot_fp8_linear_forward(x.bfloat16().cuda(), pw, out_dtype=torch.float32)
    x[M - 1, 200] = float("nan")
    x[2, 7] = float("inf")
    announce(f"fp8 non-finite fp32 M={M}")
    y = cr.convrot_fp8_linear_forward(x.bfloat16().cuda(), pw, out_dtype=torch.float32)
    assert bool(torch.isnan(y[[2, M - 1]]).all())
    keep = [m for m in range(M) if m not in (2, M - 1)]
    assert torch.equal(y[keep], clean[keep])


def test_pow2_import_zero_scales(cr):
    """A zero scale stands only for a block of zeros."""
    codes = torch.zeros(128, 256, device="cuda")
    codes[:, 128:] = 2.0
    scale = torch.tensor([[0.0, 0.5]], device="cuda")
    pw = cr.convrot_fp8_prepare_weights(codes.to(F8), src_scale=scale, scales="pow2")
    for M in (1, 300):
        announce(f"fp8 zero scale M={M}")
        y = cr.convrot_fp8_linear_forward(torch.ones(M, 256, device="cuda").bfloat16(), pw)
        assert bool((y == 128.0).all())
    codes[5, 5] = 1.0
    with pytest.raises(ValueError, match="scale is 0"):
        cr.convrot_fp8_prepare_weights(codes.to(F8), src_scale=scale, scales="pow2")


def test_largest_extents(cr):
    """The most rows, inputs and outputs that the shape limits allow (byte offsets
    up to 2^31 in both code matrices, past it in the inputs and the output): rows and
    columns at the corners against the same rows and weight blocks in a call of their
    own.  Both calls form the same sum of each k-block; the K / 128 sums are then
    added in two orders, and both outputs are rounded to bf16."""
    M = N = 32752
    K = 65536
    announce(f"fp8 largest {M}x{K}x{N}")
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    W = torch.randn(N, K, generator=g, device="cuda", dtype=torch.bfloat16)
    rows = torch.tensor([0, 1, 255, 16384, 32512, M - 1], device="cuda")
    blocks = ((0, 128), (16384, 16512), (32640, N))
    assert cr.convrot_fp8_packed_bytes(N + 16, K) == 0       # one row block more is refused
    for kind in ("f32", "pow2"):
        y = cr.convrot_fp8_linear_forward(X, cr.convrot_fp8_prepare_weights(W, scales=kind))
        for a, b in blocks:
            part = cr.convrot_fp8_prepare_weights(W[a:b].contiguous(), scales=kind)
            want = cr.convrot_fp8_linear_forward(X[rows].contiguous(), part).double()
            mag = X[rows].double().abs() @ W[a:b].double().abs().t()
            # codes are within 1/16 of the values they stand for, products within 1/7
            bound = 2 * (K // 128 + 8) * 2.0 ** -24 * (8 / 7) * mag
            bound = bound + 2 * 2.0 ** -8 * (want.abs() + bound)
            worst = float(((y[rows][:, a:b].double() - want).abs() / bound).max())
            print(f"[parity] largest {kind} {a}: worst error {worst:.3f} of its bound", flush=True)
            assert worst <= 1.0
        del y


@pytest.mark.parametrize("rows_kind,kind", [("f32", "pow2"), ("pow2", "f32"), ("f32", "f32"),
                                            ("pow2", "pow2")])
@pytest.mark.parametrize("M,K,N", [(9, 640, 272), (40, 640, 272), (520, 256, 5392),
                                   (1000, 384, 5392)])
def test_gemm_dequant_takes_any_row_scales(cr, rows_kind, kind, M, K, N):
    """Rows of either kind of scales by weights of either kind, in the few-rows
    kernel and in tiles: the same product of codes and scales (the docstring's
    bound)."""
    rng = np.random.default_rng(M + N)
    x, w = rows(rng, M, K), rng.standard_normal((N, K)).astype(np.float32)
    bias = rng.standard_normal(N).astype(np.float32)
    pw = cr.convrot_fp8_prepare_weights(torch.from_numpy(w).cuda(), scales=kind)
    (xq, sx), (wq, sw) = quantize_rows(x, rows_kind), quantize_blocks(w, kind)
    q, s = cr.convrot_fp8_quantize(bf16(x).cuda(), rows_kind)
    for dt in (torch.bfloat16, torch.float32):
        announce(f"fp8 gemm {M}x{K}x{N}: {rows_kind} rows, {kind} weight, {dt}")
        y = cr.convrot_fp8_gemm_dequant(q, s, M, pw, bias=torch.from_numpy(bias).cuda(),
                                        out_dtype=dt)
        check(y, xq, sx, wq, sw, bias, f"gemm {M}x{K}x{N} {rows_kind}/{kind} {dt}")


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("M,K,N", [(40, 640, 272), (520, 256, 5392), (1000, 384, 5392)])
def test_stages_equal_forward(cr, kind, M, K, N):
    """The two stages, told the rows' kind, are the forward bit for bit."""
    rng = np.random.default_rng(M)
    X = bf16(rows(rng, M, K)).cuda()
    pw = cr.convrot_fp8_prepare_weights(torch.randn(N, K, device="cuda"), scales=kind)
    q, s = cr.convrot_fp8_quantize(X, kind)
    for dt in (torch.bfloat16, torch.float32):
        announce(f"fp8 stages {M}x{K}x{N} {kind} {dt}")
        y = cr.convrot_fp8_gemm_dequant(q, s, M, pw, out_dtype=dt, scales=kind)
        assert torch.equal(y, cr.convrot_fp8_linear_forward(X, pw, out_dtype=dt))


def product_bound(q, s, M, pw, bias, K, N):
    """fp64 product of the library's codes and scales, its bound for fp32 outputs and
    what bf16 outputs add to it (the module's docstring), on the GPU."""
    dec = lambda c, n: torch.from_numpy(untile(c.view(torch.int8), n, K).copy()).cuda() \
        .view(F8).double()
    xd = dec(q, M) * s[:, :M].t().double().repeat_interleave(128, 1)
    wd = dec(pw.codes, N) * pw.scale.double().repeat_interleave(128, 0)[:N] \
        .repeat_interleave(128, 1)
    ref, mag = xd @ wd.t(), xd.abs() @ wd.abs().t()
    if bias is not None:
        ref, mag = ref + bias.double(), mag + bias.double().abs()
    top = lambda a: a.abs().view(a.shape[0], K // 8, 8).amax(-1)
    return ref, (K + K // 128 + 4) * 2.0 ** -24 * mag, 7 * 2.0 ** -13 * (top(xd) @ top(wd).t())


def check_product(y, ref, bound, cut, what):
    bf = y.dtype == torch.bfloat16
    bound = bound + cut if bf else bound
    bound = bound + (2.0 ** -8 if bf else 2.0 ** -24) * (ref.abs() + bound)
    worst = float(((y.double() - ref).abs() / bound).max())
    print(f"[parity] {what}: worst error {worst:.3f} of its bound", flush=True)
    assert worst <= 1.0


# rows quantised by the product's kernel: 1, 2 and 4 row tiles a workgroup, counts of
# 16-row blocks that these do not divide, fewer and more k-blocks than waves
FEW_ROWS = [(1152, 2064), (384, 5392), (1152, 5392), (384, 10256), (384, 16144), (1152, 16144),
            (640, 17424), (384, 32272)]


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("M", [1, 8, 16])
@pytest.mark.parametrize("K,N", FEW_ROWS)
def test_few_rows(cr, kind, M, K, N):
    g = torch.Generator(device="cuda").manual_seed(M + N)
    X = torch.randn(M, K, generator=g, device="cuda")
    X = (X * torch.exp2(torch.randint(-6, 7, (M, K // 128, 1), generator=g, device="cuda"))
         .expand(-1, -1, 128).reshape(M, K)).to(torch.bfloat16)
    # blocks of 128 outputs differ in scale by factors up to 2^8
    W = torch.randn(N, K, generator=g, device="cuda") * torch.exp2(
        torch.randint(-4, 5, (-(-N // 128), 1), generator=g, device="cuda")
        .repeat_interleave(128, 0)[:N].float())
    bias = torch.randn(N, generator=g, device="cuda")
    pw = cr.convrot_fp8_prepare_weights(W, scales=kind)
    q, s = cr.convrot_fp8_quantize(X, kind)
    for dt, b in ((torch.bfloat16, bias), (torch.bfloat16, None), (torch.float32, bias),
                  (torch.float32, None)):
        announce(f"fp8 few rows {M}x{K}x{N} {kind} {dt} bias={b is not None}")
        buf = torch.full((M + 2, N), 3.0, dtype=dt, device="cuda")
        cr.convrot_fp8_linear_forward(X, pw, bias=b, out=buf[:M])
        assert bool((buf[M:] == 3.0).all())
        check_product(buf[:M], *product_bound(q, s, M, pw, b, K, N),
                      f"few rows {M}x{K}x{N} {kind} {dt}")


# whole rounds of the largest tiles, then the last rows in each of the other shapes, for
# bf16 and F32 outputs (tests/test_fp8_plans.py asks the chooser which)
TAILS = [(1185, 640, 15232), (574, 640, 14960), (1844, 384, 16704), (7390, 640, 3152),
         (8965, 384, 2064), (5676, 640, 6672), (1400, 640, 1680), (8588, 384, 32), (90, 256, 1120),
         (380, 640, 480)]


@pytest.mark.parametrize("kind", ["f32", "pow2"])
@pytest.mark.parametrize("M,K,N", TAILS)
def test_tails(cr, kind, M, K, N):
    g = torch.Generator(device="cuda").manual_seed(M + N)
    X = torch.randn(M, K, generator=g, device="cuda")
    X = (X * torch.exp2(torch.randint(-6, 7, (M, K // 128, 1), generator=g, device="cuda"))
         .expand(-1, -1, 128).reshape(M, K)).to(torch.bfloat16)
    W = torch.randn(N, K, generator=g, device="cuda")
    bias = torch.randn(N, generator=g, device="cuda")
    pw = cr.convrot_fp8_prepare_weights(W, scales=kind)
    q, s = cr.convrot_fp8_quantize(X, kind)
    ref, bound, cut = product_bound(q, s, M, pw, bias, K, N)
    for dt in (torch.bfloat16, torch.float32):
        announce(f"fp8 tails {M}x{K}x{N} {kind} {dt}")
        buf = torch.full((M + 2, N), 3.0, dtype=dt, device="cuda")
        cr.convrot_fp8_linear_forward(X, pw, bias=bias, out=buf[:M])
        assert bool((buf[M:] == 3.0).all())
        check_product(buf[:M], ref, bound, cut, f"tails {M}x{K}x{N} {kind} {dt}")
