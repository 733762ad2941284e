"""Host-side refusals of the residual's addition with the RMS norm: the C ABI with fake
pointers (never dereferenced) and the Python binding with host tensors.  Nothing is
launched."""
import ctypes
import os

import pytest
import torch

A = 0x7f0000000000                  # fake device addresses, far apart
B, C, D, E, G = (A + (i << 40) for i in range(1, 6))
ODD = A + 8


@pytest.fixture(scope="module")
def cr():
    from w8a8_int8_rotated_amd import convrot
    if not os.path.exists(convrot.LIB_PATH):
        pytest.fail("libconvrot.so not built (run __graft_entry__.build())")
    convrot.library()
    return convrot


def forward(cr, x=A, xt=1, r=B, rt=0, w=C, eps=1e-6, M=4, K=512, h=D, y=E, yt=1):
    return cr.library().convrot_add_rms_norm_forward(x, xt, r, rt, w, eps, M, K, h, y, yt, None)


def test_forward_refusals(cr):
    f = lambda **kw: forward(cr, **kw)                              # noqa: E731
    assert f(M=0, x=None, y=None) == cr.OK
    assert f(M=-1) == cr.EINVAL and f(K=0) == cr.EINVAL and f(K=-8) == cr.EINVAL
    for K in (4, 12, 1001, 32776, 1 << 40):
        assert f(K=K) == cr.EUNSUPPORTED
    assert f(M=1 << 31) == cr.EUNSUPPORTED and f(M=(1 << 63) - 1) == cr.EUNSUPPORTED
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert f(eps=eps) == cr.EINVAL
    assert f(x=None) == cr.EINVAL and f(y=None) == cr.EINVAL
    assert f(r=None) == cr.EINVAL and f(h=None) == cr.EINVAL        # both or neither
    assert f(xt=cr.I8) == cr.EUNSUPPORTED and f(rt=cr.I32) == cr.EUNSUPPORTED
    assert f(yt=cr.F8E4M3) == cr.EUNSUPPORTED
    assert f(xt=cr.F32, rt=cr.BF16) == cr.EUNSUPPORTED
    for name in "xrwhy":
        assert f(**{name: ODD + (ord(name) << 33)}) == cr.EALIGN


def test_forward_overlaps(cr):
    f = lambda **kw: forward(cr, **kw)                              # noqa: E731
    n = 4 * 512
    assert f(h=A) == cr.EINVAL                     # fp32 h on a bf16 x
    assert f(h=B + 16) == cr.EINVAL and f(h=A + 2 * n - 16) == cr.EINVAL
    assert f(y=A + 16) == cr.EINVAL and f(y=B) == cr.EINVAL         # bf16 y on the fp32 residual
    assert f(y=D) == cr.EINVAL and f(y=D + 4 * n - 16) == cr.EINVAL
    assert f(y=A, yt=cr.F32) == cr.EINVAL
    assert f(y=C) == cr.EINVAL and f(h=C) == cr.EINVAL


def test_quantize_refusals(cr):
    lib = cr.library()
    q8 = lambda M=4, K=512, b=128, flags=0, q=E, s=G, x=A, r=B, h=D: \
        lib.convrot_add_rms_norm_rotate_quantize(x, 1, r, 0, C, 1e-6, M, K, b, flags, h, q, s,
                                                 None)               # noqa: E731
    assert q8(M=0, x=None, q=None, s=None) == cr.OK
    assert q8(b=32) == cr.EINVAL and q8(b=256, K=384) == cr.EINVAL
    assert q8(flags=cr.ROT_REGULAR) == cr.EINVAL and q8(flags=1) == cr.EUNSUPPORTED
    assert q8(b=64, K=192) == cr.EUNSUPPORTED and q8(K=512 + 8) == cr.EINVAL
    assert q8(M=70000, K=32768) == cr.EUNSUPPORTED                  # 32-bit code offsets
    assert q8(K=65536) == cr.EUNSUPPORTED
    assert q8(q=None) == cr.EINVAL and q8(s=None) == cr.EINVAL
    assert q8(q=ODD) == cr.EALIGN and q8(s=ODD) == cr.EALIGN
    assert q8(q=A) == cr.EINVAL and q8(q=D) == cr.EINVAL and q8(s=C) == cr.EINVAL
    assert q8(s=E + 64) == cr.EINVAL
    f8 = lambda M=4, K=512, kind=0, q=E, s=G: lib.convrot_add_rms_norm_fp8_quantize(
        A, 1, B, 0, C, 1e-6, M, K, kind, D, q, s, None)              # noqa: E731
    assert f8(M=0, q=None) == cr.OK and f8(kind=2) == cr.EINVAL and f8(K=136) == cr.EINVAL
    assert f8(M=70000, K=32768) == cr.EUNSUPPORTED
    assert f8(q=None) == cr.EINVAL and f8(s=ODD) == cr.EALIGN and f8(q=B) == cr.EINVAL


def test_norm_linear_refusals(cr):
    lib = cr.library()
    d = cr.convrot_weights()
    d.magic, d.version, d.N, d.K, d.block = cr.WEIGHTS_MAGIC, cr.WEIGHTS_VERSION, 256, 512, 128
    d.codes, d.scale = G, G + (1 << 30)
    p = cr.convrot_fp8_weights()
    p.magic, p.version, p.N, p.K = cr.FP8_MAGIC, cr.FP8_VERSION, 256, 512
    p.codes, p.scale = G, G + (1 << 30)
    WS = G + (2 << 30)
    for fn, W in (("convrot_norm_linear_forward", d), ("convrot_fp8_norm_linear_forward", p)):
        f = lambda M=4, W=W, x=A, h=D, bias=None, Y=E, yt=1, ws=WS, wsb=1 << 30, eps=1e-6: \
            getattr(lib, fn)(x, 1, B, 0, C, eps, M, ctypes.byref(W), bias, h, Y, yt, ws, wsb,
                             None)                                   # noqa: E731
        assert getattr(lib, fn)(A, 1, B, 0, C, 1e-6, 4, None, None, D, E, 1, WS, 1 << 30,
                                None) == cr.EINVAL
        assert f(M=0, x=None, Y=None, ws=None, wsb=0) == cr.OK
        assert f(M=-1) == cr.EINVAL and f(x=None) == cr.EINVAL and f(Y=None) == cr.EINVAL
        assert f(h=None) == cr.EINVAL and f(eps=0.0) == cr.EINVAL
        assert f(yt=cr.I8) == cr.EUNSUPPORTED
        assert f(ws=None) == cr.EWORKSPACE and f(wsb=64) == cr.EWORKSPACE
        assert f(Y=ODD) == cr.EALIGN and f(bias=ODD) == cr.EALIGN and f(ws=ODD) == cr.EALIGN
        assert f(Y=D) == cr.EINVAL
        W.magic += 1
        assert f() == cr.ELAYOUT
        W.magic -= 1
        W.K = 65536                                                  # a wider row than the norm's
        assert f() == cr.EUNSUPPORTED
        W.K = 512
    d.flags, d.N = cr.SWIGLU_PAIRS, 512
    assert lib.convrot_norm_linear_forward(A, 1, B, 0, C, 1e-6, 4, ctypes.byref(d), None, D, E, 1,
                                           WS, 1 << 30, None) == cr.ELAYOUT
    ws = lib.convrot_fp8_norm_linear_workspace_bytes
    assert ws(1, 512, 256) >= 16 * 512 + 16 * 4 * 4 and ws(-1, 512, 256) == 0
    assert ws(5, 192, 256) == 0 and ws(5, 512, 24) == 0


def test_backward_refusals(cr):
    lib = cr.library()
    WS = G + (1 << 30)
    f = lambda g=A, gt=0, h=B, ht=0, gh=C, w=D, eps=1e-6, M=4, K=512, dh=E, dx=None, dw=G, ws=WS, \
        wsb=1 << 30: lib.convrot_add_rms_norm_backward(g, gt, h, ht, gh, w, eps, M, K, dh, dx, dw,
                                                       ws, wsb, None)  # noqa: E731
    assert f(M=0, dw=None, g=None, h=None, dh=None) == cr.OK
    assert f(M=-1) == cr.EINVAL and f(K=12) == cr.EUNSUPPORTED and f(eps=0.0) == cr.EINVAL
    assert f(K=32776) == cr.EUNSUPPORTED and f(M=1 << 31) == cr.EUNSUPPORTED
    assert f(gt=2) == cr.EUNSUPPORTED and f(ht=3) == cr.EUNSUPPORTED
    assert f(g=None) == cr.EINVAL and f(h=None) == cr.EINVAL and f(dh=None) == cr.EINVAL
    assert f(ht=1, dx=A + (1 << 30)) == cr.EINVAL                    # dx beside a bf16 h
    assert f(ws=None) == cr.EWORKSPACE and f(wsb=16) == cr.EWORKSPACE
    for name in ("g", "h", "gh", "w", "dh", "dx", "dw", "ws"):
        assert f(**{name: ODD}) == cr.EALIGN
    assert f(dh=A + 16) == cr.EINVAL and f(dh=A, gt=1) == cr.EINVAL
    assert f(dh=C + 4 * 4 * 512 - 16) == cr.EINVAL and f(dx=A) == cr.EINVAL
    assert f(dx=E + 16) == cr.EINVAL and f(dw=E) == cr.EINVAL and f(dw=D) == cr.EINVAL
    assert f(dw=B + 64) == cr.EINVAL and f(dh=D) == cr.EINVAL
    ws = lib.convrot_add_rms_norm_workspace_bytes
    assert ws(0, 512) == 0 and ws(-1, 512) == 0 and ws(4, 12) == 0
    assert ws(38656, 5376) >= 5376 * 4 and ws((1 << 31) - 1, 32768) > 0


def test_binding_refusals(cr):
    x, r, w = torch.zeros(4, 512, dtype=torch.bfloat16), torch.zeros(4, 512), torch.ones(512)
    bad = pytest.raises(ValueError)
    for call in (
            lambda: cr.convrot_add_rms_norm_forward(x.half(), w, r),
            lambda: cr.convrot_add_rms_norm_forward(x, w.double(), r),
            lambda: cr.convrot_add_rms_norm_forward(x, w[:256], r),
            lambda: cr.convrot_add_rms_norm_forward(x, w, r[:3]),
            lambda: cr.convrot_add_rms_norm_forward(x, w, r.t().contiguous().t()),
            lambda: cr.convrot_add_rms_norm_forward(x.float(), w, x),
            lambda: cr.convrot_add_rms_norm_forward(x, w, None, residual_out=r),
            lambda: cr.convrot_add_rms_norm_forward(x, w, r, residual_out=x),
            lambda: cr.convrot_add_rms_norm_forward(x, w, r),                      # on the host
            lambda: cr.convrot_add_rms_norm_forward(3.0, w, r),
            lambda: cr.convrot_add_rms_norm_rotate_quantize(x, w, 128, r, rotation="other"),
            lambda: cr.convrot_add_rms_norm_rotate_quantize(x, w, 128, r,
                                                            q=torch.zeros(4, 512)),
            lambda: cr.convrot_add_rms_norm_fp8_quantize(x, w, "f16", r),
            lambda: cr.convrot_add_rms_norm_fp8_quantize(x, w, "f32", r, s=torch.zeros(4, 4)),
            lambda: cr.convrot_norm_linear_forward(x, w, w),
            lambda: cr.convrot_add_rms_norm_backward(x, r[:3], w),
            lambda: cr.convrot_add_rms_norm_backward(x, x, w, g_h=r),
            lambda: cr.convrot_add_rms_norm_backward(x, x, w, x_dtype=torch.float32),
            lambda: cr.convrot_add_rms_norm_backward(x, r, w, dx=x),
            lambda: cr.convrot_add_rms_norm_backward(x, r, None, dw=w),
            lambda: cr.convrot_add_rms_norm_backward(x, r, w)):
        with bad:
            call()


SPREAD = [A + (i << 40) for i in range(12)]


def inside(base, size):
    """The first and the last 16 bytes of an extent."""
    return base, base + (size + 15) // 16 * 16 - 16


@pytest.mark.parametrize("fp8", [False, True], ids=["int8", "fp8"])
def test_norm_linear_overlaps(cr, fp8):
    """Y, residual_out and the workspace against every input, the bias and the prepared weights
    among them, and against each other."""
    lib, M, K, N = cr.library(), 4, 512, 256
    need = lib.convrot_fp8_norm_linear_workspace_bytes(M, K, N) if fp8 else \
        lib.convrot_linear_workspace_bytes(M, K, N, 128)
    ins = {"w": K * 4, "bias": N * 4, "codes": N * K, "scale": N // 128 * K // 128 * 4 if fp8 else N * 4}
    size = {"x": M * K * 2, "r": M * K * 4, "h": M * K * 4, "Y": M * N * 2, "ws": need, **ins}
    base = dict(zip(size, SPREAD))

    def f(**kw):
        a = {**base, **kw}
        d = cr.convrot_fp8_weights() if fp8 else cr.convrot_weights()
        if fp8:
            d.magic, d.version = cr.FP8_MAGIC, cr.FP8_VERSION
        else:
            d.magic, d.version, d.block = cr.WEIGHTS_MAGIC, cr.WEIGHTS_VERSION, 128
        d.N, d.K, d.codes, d.scale = N, K, a["codes"], a["scale"]
        fn = lib.convrot_fp8_norm_linear_forward if fp8 else lib.convrot_norm_linear_forward
        return fn(a["x"], 1, a["r"], 0, a["w"], 1e-6, M, ctypes.byref(d), a["bias"], a["h"], a["Y"],
                  1, a["ws"], need, None)

    for o, others in (("Y", ("x", "r", "h", "ws", *ins)), ("h", ("ws", *ins)),
                      ("ws", ("x", "r", *ins))):
        for n in others:
            for at in inside(base[n], size[n]):
                assert f(**{o: at}) == cr.EINVAL, (o, n)


def test_backward_workspace_overlaps(cr):
    lib, M, K = cr.library(), 4, 512
    need = lib.convrot_add_rms_norm_workspace_bytes(M, K)
    size = {"g": M * K * 4, "h": M * K * 4, "gh": M * K * 4, "w": K * 4, "dh": M * K * 4,
            "dx": M * K * 2, "dw": K * 4}
    base = dict(zip(size, SPREAD))
    for n in size:
        for at in inside(base[n], size[n]):
            b = base
            assert lib.convrot_add_rms_norm_backward(
                b["g"], 0, b["h"], 0, b["gh"], b["w"], 1e-6, M, K, b["dh"], b["dx"], b["dw"], at,
                need, None) == cr.EINVAL, n
