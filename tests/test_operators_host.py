"""Host-side refusals of the FP8 linear, the rotary positions and the Q/K norms:
the C ABI with fake pointers (never dereferenced) and the Python binding with
host tensors.  Nothing is launched."""
import ctypes
import os

import pytest
import torch

FAKE = 0x7f0000000000
ODD = FAKE + 8


@pytest.fixture(scope="module")
def cr():
    from w8a8_int8_rotated_amd import convrot
    if not os.path.exists(convrot.LIB_PATH):
        pytest.fail("libconvrot.so not built (run __graft_entry__.build())")
    convrot.library()
    return convrot


# ---------------------------------------------------------------- C ABI ----

def fp8_desc(cr, N=512, K=512, **kw):
    d = cr.convrot_fp8_weights()
    d.magic, d.version, d.N, d.K, d.scales = cr.FP8_MAGIC, cr.FP8_VERSION, N, K, 0
    d.codes, d.scale = FAKE, FAKE + 4096
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_fp8_sizes(cr):
    lib = cr.library()
    assert lib.convrot_fp8_packed_bytes(16128, 5376) == 16128 * 5376
    assert lib.convrot_fp8_scale_bytes(16128, 5376) == 126 * 42 * 4
    assert lib.convrot_fp8_scale_bytes(16, 128) == 4
    for N, K in ((24, 512), (16, 192), (0, 128), (16, 65536 + 128), (1 << 20, 4096)):
        assert lib.convrot_fp8_packed_bytes(N, K) == 0
        assert lib.convrot_fp8_scale_bytes(N, K) == 0
    ws = lib.convrot_fp8_linear_workspace_bytes
    assert ws(1, 5376, 16128) == 0 and ws(16, 5376, 16128) == 0
    assert ws(17, 5376, 16128) >= 32 * 5376 + 32 * 42 * 4
    assert ws(-1, 512, 512) == 0 and ws(40000, 65536, 16) == 0
    assert lib.convrot_fp8_prepare_workspace_bytes(256, 512, cr.F32, cr.IN_MAJOR) >= 256 * 512 * 4
    assert lib.convrot_fp8_prepare_workspace_bytes(256, 512, cr.F8E4M3, cr.IN_MAJOR) == 0


def test_fp8_forward_refusals(cr):
    lib = cr.library()
    f = lambda d, M=40, X=FAKE, Y=FAKE, y=cr.BF16, bias=None, ws=FAKE, wsb=1 << 30: \
        lib.convrot_fp8_linear_forward(X, M, ctypes.byref(d), bias, Y, y, ws, wsb, None)
    d = fp8_desc(cr)
    assert lib.convrot_fp8_linear_forward(FAKE, 4, None, None, FAKE, 1, FAKE, 1, None) == cr.EINVAL
    assert f(d, M=0, X=None, Y=None, ws=None, wsb=0) == cr.OK
    assert f(d, M=-1) == cr.EINVAL
    assert f(d, X=None) == cr.EINVAL and f(d, Y=None) == cr.EINVAL
    assert f(d, X=ODD) == cr.EALIGN and f(d, Y=ODD) == cr.EALIGN
    assert f(d, bias=ODD) == cr.EALIGN and f(d, ws=ODD) == cr.EALIGN
    assert f(d, ws=None) == cr.EWORKSPACE and f(d, wsb=100) == cr.EWORKSPACE
    assert f(d, y=cr.I8) == cr.EUNSUPPORTED
    for bad in (dict(magic=0), dict(version=9), dict(scales=2), dict(reserved=1), dict(N=24, K=0)):
        assert f(fp8_desc(cr, **bad)) == cr.ELAYOUT
    assert f(fp8_desc(cr, K=192)) == cr.ELAYOUT            # K % 128
    assert f(fp8_desc(cr, N=24)) == cr.EUNSUPPORTED        # N % 16
    assert f(fp8_desc(cr, N=16, K=65536), M=40000) == cr.EUNSUPPORTED
    assert f(fp8_desc(cr, codes=None)) == cr.EINVAL
    assert f(fp8_desc(cr, scale=ODD)) == cr.EALIGN


def test_fp8_prepare_and_hook_refusals(cr):
    lib = cr.library()
    d = cr.convrot_fp8_weights()
    d.codes, d.scale = FAKE, FAKE + 4096
    p = lambda W=FAKE, dt=cr.F32, layout=0, sc=None, N=512, K=512, d=d, ws=None, wsb=0: \
        lib.convrot_fp8_prepare_weights(W, dt, layout, sc, N, K, ctypes.byref(d), ws, wsb, None)
    assert p(W=None) == cr.EINVAL and p(layout=3) == cr.EINVAL
    assert p(K=192) == cr.EINVAL and p(N=24) == cr.EUNSUPPORTED
    assert p(dt=cr.I8) == cr.EUNSUPPORTED
    assert p(dt=cr.F8E4M3) == cr.EINVAL and p(sc=FAKE) == cr.EINVAL
    assert p(W=ODD) == cr.EALIGN
    assert p(layout=1) == cr.EWORKSPACE
    bad = cr.convrot_fp8_weights()
    assert p(d=bad) == cr.EINVAL
    bad.codes, bad.scale, bad.scales = FAKE, FAKE, 5
    assert p(d=bad) == cr.EINVAL
    assert d.magic == 0                                    # nothing written on error
    q = lambda M=4, K=512, kind=0, X=FAKE: lib.convrot_fp8_quantize(X, M, K, kind, FAKE, FAKE, None)
    assert q(M=0, X=None) == cr.OK and q(M=-1) == cr.EINVAL and q(K=500) == cr.EINVAL
    assert q(kind=2) == cr.EINVAL and q(X=None) == cr.EINVAL and q(X=ODD) == cr.EALIGN
    assert q(K=65536 + 128) == cr.EUNSUPPORTED
    g = lambda d, M=4, qx=FAKE, y=0: lib.convrot_fp8_gemm_dequant(
        qx, FAKE, M, ctypes.byref(d), None, FAKE, y, None)
    assert g(fp8_desc(cr), M=0, qx=None) == cr.OK
    assert g(fp8_desc(cr), qx=None) == cr.EINVAL and g(fp8_desc(cr), qx=ODD) == cr.EALIGN
    assert g(fp8_desc(cr, magic=1)) == cr.ELAYOUT and g(fp8_desc(cr), y=3) == cr.EUNSUPPORTED


def rope_desc(cr, **kw):
    r = cr.convrot_rope()
    r.magic, r.version, r.axes, r.head_dim, r.rotary_dim = cr.ROPE_MAGIC, cr.ROPE_VERSION, 3, 128, 128
    r.freq, r.axis = FAKE, FAKE
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def heads(cr, H=8, T=10, D=128, **kw):
    h = cr.convrot_heads(FAKE, H, 0, T * H * D, H * D, D)
    for k, v in kw.items():
        setattr(h, k, v)
    return ctypes.byref(h)


def test_rope_prepare_refusals(cr):
    lib = cr.library()

    def p(dims, D=128, theta=1e4, pairing=0, spectrum=0, freq=FAKE, axis=FAKE, n=None):
        r = cr.convrot_rope()
        r.freq, r.axis = freq, axis
        arr = (ctypes.c_int32 * max(1, len(dims)))(*dims)
        rc = lib.convrot_rope_prepare(arr, len(dims) if n is None else n, D, theta, pairing,
                                      spectrum, ctypes.byref(r), None)
        assert r.magic == 0
        return rc

    assert p([], n=0) == cr.EINVAL and p([64, 63]) == cr.EINVAL and p([64, 0]) == cr.EINVAL
    assert p([64, 66]) == cr.EINVAL                        # beyond the head
    assert p([8] * 5) == cr.EUNSUPPORTED                   # five axes
    assert p([64], theta=0.0) == cr.EINVAL and p([64], theta=float("nan")) == cr.EINVAL
    assert p([64], theta=float("inf")) == cr.EINVAL
    assert p([64], pairing=2) == cr.EINVAL and p([64], spectrum=2) == cr.EINVAL
    assert p([12], pairing=1) == cr.EUNSUPPORTED           # half: a multiple of 8
    assert p([64], D=100) == cr.EUNSUPPORTED and p([64], D=520) == cr.EUNSUPPORTED
    assert p([64], freq=None) == cr.EINVAL and p([64], axis=ODD) == cr.EALIGN
    assert p([2 ** 31 - 2] * 2) == cr.EINVAL               # no overflow in the sum


def test_rope_and_norm_refusals(cr):
    lib = cr.library()

    def both(expect, B=1, T=10, dt=cr.BF16, q=None, qo=None, k=None, ko=None, r=None, pos=FAKE,
             pdt=cr.I32, psb=0):
        q = heads(cr) if q is None else q
        qo = heads(cr) if qo is None else qo
        r = rope_desc(cr) if r is None else r
        assert lib.convrot_rope_forward(B, T, dt, q, qo, k, ko, ctypes.byref(r), pos, pdt, psb, 0,
                                        None) == expect
        assert lib.convrot_qk_norm_rope_forward(B, T, dt, q, qo, None, k, ko, None, 1e-6,
                                                ctypes.byref(r), pos, pdt, psb, None) == expect
        assert lib.convrot_qk_norm_rope_backward(
            B, T, dt, q, q, qo, None, FAKE, k, k, ko, None, FAKE if k is not None else None, 1e-6,
            ctypes.byref(r), pos, pdt, psb, FAKE, 1 << 30, None) == expect

    both(cr.EINVAL, B=-1)
    both(cr.EINVAL, T=-1)
    both(cr.EUNSUPPORTED, B=1 << 16, T=1 << 16)
    both(cr.EUNSUPPORTED, B=1 << 62, T=4)
    both(cr.EUNSUPPORTED, dt=cr.I8)
    both(cr.EUNSUPPORTED, pdt=cr.BF16)
    both(cr.EINVAL, pos=None)
    both(cr.EALIGN, pos=FAKE + 2)
    both(cr.EINVAL, psb=-1)
    both(cr.EINVAL, q=heads(cr, heads=0))
    both(cr.EUNSUPPORTED, q=heads(cr, heads=65537), qo=heads(cr, heads=65537))
    both(cr.EINVAL, qo=heads(cr, heads=7))
    both(cr.EINVAL, q=heads(cr, data=None))
    both(cr.EINVAL, q=heads(cr, reserved=1))
    both(cr.EALIGN, q=heads(cr, data=ODD))
    both(cr.EALIGN, qo=heads(cr, token_stride=8 * 128 + 4))
    both(cr.EALIGN, q=heads(cr, head_stride=129))
    both(cr.EINVAL, qo=heads(cr, token_stride=-1024))
    both(cr.EINVAL, qo=heads(cr, head_stride=0))           # rows on top of each other
    both(cr.EINVAL, qo=heads(cr, token_stride=0))
    both(cr.EINVAL, B=2, qo=heads(cr, batch_stride=0))
    both(cr.EINVAL, k=heads(cr, H=2))                      # no output for k
    for bad in (dict(magic=0), dict(version=2), dict(axes=0), dict(axes=5), dict(head_dim=100),
                dict(rotary_dim=130), dict(rotary_dim=63), dict(pairing=3),
                dict(pairing=1, rotary_dim=20)):
        both(cr.ELAYOUT, r=rope_desc(cr, **bad))
    both(cr.EINVAL, r=rope_desc(cr, freq=None))
    both(cr.EALIGN, r=rope_desc(cr, axis=ODD))
    h, r = heads(cr), ctypes.byref(rope_desc(cr))
    assert lib.convrot_rope_forward(1, 10, cr.BF16, h, h, None, None, r, FAKE, cr.I32, 0, 2, None) \
        == cr.EUNSUPPORTED                                 # unknown flag
    assert lib.convrot_rope_forward(1, 10, cr.BF16, h, h, None, None, None, FAKE, cr.I32, 0, 0,
                                    None) == cr.EINVAL
    assert lib.convrot_rope_forward(1, 0, cr.BF16, h, h, None, None, r, None, cr.I32, 0, 0, None) \
        == cr.OK                                           # no tokens
    n = lambda eps, wq=None: lib.convrot_qk_norm_rope_forward(
        1, 10, cr.BF16, h, h, wq, None, None, None, eps, r, FAKE, cr.I32, 0, None)
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert n(eps) == cr.EINVAL
    assert n(1e-6, ODD) == cr.EALIGN
    b = lambda g=h, dw=FAKE, ws=FAKE, wsb=1 << 30, gk=None, dwk=None: \
        lib.convrot_qk_norm_rope_backward(1, 10, cr.BF16, g, h, h, None, dw, gk, None, None, None,
                                          dwk, 1e-6, r, FAKE, cr.I32, 0, ws, wsb, None)
    assert b(g=None) == cr.EINVAL and b(dw=None) == cr.EINVAL
    assert b(gk=h) == cr.EINVAL and b(dwk=FAKE) == cr.EINVAL
    assert b(dw=ODD) == cr.EALIGN and b(ws=ODD) == cr.EALIGN
    assert b(ws=None) == cr.EWORKSPACE and b(wsb=64) == cr.EWORKSPACE


def test_norm_rope_workspace(cr):
    ws = cr.library().convrot_qk_norm_rope_workspace_bytes
    assert ws(1, 1, 1, 0, 64) >= 2 * 64 * 4
    assert ws(1, 38656, 42, 42, 128) % 256 == 0 and ws(1, 38656, 42, 42, 128) > 0
    assert ws(1, 0, 4, 4, 64) == 0
    for bad in ((-1, 1, 1, 1, 64), (1, -1, 1, 1, 64), (1, 1, 0, 1, 64), (1, 1, 1, -1, 64),
                (1, 1, 1, 1, 60), (1, 1, 1, 1, 520), (1 << 16, 1 << 16, 1, 1, 64)):
        assert ws(*bad) == 0


def test_qkv_refusals(cr):
    lib = cr.library()
    w = cr.convrot_weights()
    w.magic, w.version, w.N, w.K, w.block = cr.WEIGHTS_MAGIC, cr.WEIGHTS_VERSION, 1536, 512, 128
    w.codes, w.scale = FAKE, FAKE
    f8 = fp8_desc(cr, N=1536)
    r = rope_desc(cr)
    for fn, d in ((lib.convrot_qkv_forward, w), (lib.convrot_fp8_qkv_forward, f8)):
        f = lambda B=1, T=40, hq=8, hk=2, X=FAKE, Y=FAKE, y=cr.BF16, eps=1e-6, r=r, pos=FAKE, \
            ws=FAKE, wsb=1 << 30: fn(X, B, T, ctypes.byref(d), None, hq, hk, None, None, eps,
                                     ctypes.byref(r), pos, cr.I32, 0, Y, y, ws, wsb, None)
        assert f(T=0, X=None, Y=None, pos=None) == cr.OK
        assert f(hq=9) == cr.ELAYOUT and f(hq=0) == cr.EINVAL and f(hk=0) == cr.EINVAL
        assert f(r=rope_desc(cr, head_dim=64, rotary_dim=64)) == cr.ELAYOUT
        assert f(B=-1) == cr.EINVAL and f(B=1 << 40, T=1 << 40) == cr.EUNSUPPORTED
        assert f(T=1 << 30) == cr.EUNSUPPORTED and f(T=1 << 62) == cr.EUNSUPPORTED
        assert f(pos=FAKE + 2) == cr.EALIGN
        assert f(X=None) == cr.EINVAL and f(Y=None) == cr.EINVAL and f(pos=None) == cr.EINVAL
        assert f(Y=ODD) == cr.EALIGN and f(X=ODD) == cr.EALIGN
        assert f(y=cr.I32) == cr.EUNSUPPORTED and f(eps=0.0) == cr.EINVAL
        assert f(ws=None) == cr.EWORKSPACE and f(wsb=8) == cr.EWORKSPACE
        assert fn(FAKE, 1, 4, None, None, 8, 2, None, None, 1e-6, ctypes.byref(r), FAKE, cr.I32, 0,
                  FAKE, cr.BF16, FAKE, 1 << 30, None) == cr.EINVAL


# -------------------------------------------------------------- binding ----

bf, f32 = torch.bfloat16, torch.float32


def fake_fp8(cr, N=64, K=256):
    d = fp8_desc(cr, N, K)
    return cr.FP8Weights(d, torch.zeros(N * K, dtype=torch.uint8), torch.ones(1, K // 128))


def fake_plan(cr, D=64, axes=2):
    d = rope_desc(cr, head_dim=D, rotary_dim=D, axes=axes)
    return cr.RopePlan(d, torch.zeros(D // 2, dtype=torch.float64),
                       torch.zeros(D // 2, dtype=torch.int32))


@pytest.mark.parametrize("kw,msg", [
    (dict(X=torch.zeros(32, 256)), "X must be torch.bfloat16"),
    (dict(X=torch.zeros(32, 128, dtype=bf)), "X must have shape"),
    (dict(X=torch.zeros(256, 32, dtype=bf).t()), "X must be contiguous"),
    (dict(bias=torch.zeros(63)), "bias must have shape"),
    (dict(out=torch.zeros(31, 64, dtype=bf)), "out must have shape"),
    (dict(workspace=torch.zeros(64, dtype=torch.uint8)), "workspace holds"),
    (dict(W=3), "must be FP8Weights"),
    (dict(), "must be a GPU tensor"),
])
def test_fp8_binding_refuses(cr, kw, msg):
    args = dict(X=torch.zeros(32, 256, dtype=bf), W=fake_fp8(cr))
    args.update(kw)
    with pytest.raises(ValueError, match=msg):
        cr.convrot_fp8_linear_forward(**args)


@pytest.mark.parametrize("kw,msg", [
    (dict(W=torch.zeros(64)), "2-D"),
    (dict(W=torch.zeros(64, 256, dtype=torch.int8)), "float8_e4m3fn"),
    (dict(src_scale=torch.ones(1, 2)), "src_scale is required"),
    (dict(W=torch.zeros(64, 256).to(torch.float8_e4m3fn)), "src_scale is required"),
    (dict(W=torch.zeros(64, 256).to(torch.float8_e4m3fn), src_scale=torch.ones(2, 2)),
     "src_scale must have shape"),
    (dict(scales="e8"), "scales must be"),
    (dict(layout=2), "layout"),
    (dict(), "must be a GPU tensor"),
])
def test_fp8_prepare_binding_refuses(cr, kw, msg):
    args = dict(W=torch.zeros(64, 256))
    args.update(kw)
    with pytest.raises(ValueError, match=msg):
        cr.convrot_fp8_prepare_weights(**args)


Q = torch.zeros(2, 5, 4, 64, dtype=bf)
P = torch.zeros(5, 2, dtype=torch.int32)


@pytest.mark.parametrize("kw,msg", [
    (dict(q=Q.half()), "q must be float32 or bfloat16"),
    (dict(q=Q[0, 0]), "q must be a tensor"),
    (dict(q=Q[..., :32]), "q must have shape"),
    (dict(q=Q.transpose(2, 3).contiguous().transpose(2, 3)), "contiguous channels"),
    (dict(k=Q.float()), "k must be a torch.bfloat16"),
    (dict(k=Q[:1]), "k must have shape"),
    (dict(k=Q[0]), "k must have as many dimensions"),
    (dict(positions=P.long()), "int32 or float32"),
    (dict(positions=P[:, :1]), "positions must have shape"),
    (dict(positions=P[:4]), "positions must have shape"),
    (dict(positions=P.t().contiguous().t()), "positions must be contiguous"),
    (dict(rope=None), "RopePlan"),
    (dict(), "must be a GPU tensor"),
])
def test_rope_binding_refuses(cr, kw, msg):
    args = dict(q=Q, k=Q, rope=fake_plan(cr), positions=P)
    args.update(kw)
    with pytest.raises(ValueError, match=msg):
        cr.convrot_rope_forward(**args)
    with pytest.raises(ValueError, match=msg):
        cr.convrot_qk_norm_rope_forward(w_q=None, w_k=None, **args)
    with pytest.raises(ValueError, match=msg):
        cr.convrot_qk_norm_rope_backward(g_q=args["q"], g_k=args["k"], w_q=None, w_k=None, **args)


def test_norm_and_qkv_binding_refuse(cr):
    plan = fake_plan(cr)
    with pytest.raises(ValueError, match="w_q must have shape"):
        cr.convrot_qk_norm_rope_forward(Q, Q, torch.ones(63), None, plan, P)
    with pytest.raises(ValueError, match="g_k must be given"):
        cr.convrot_qk_norm_rope_backward(Q, None, Q, Q, None, None, plan, P)
    with pytest.raises(ValueError, match="dw_k given without k"):
        cr.convrot_qk_norm_rope_backward(Q, None, Q, None, None, None, plan, P,
                                         dw_k=torch.ones(64))
    X = torch.zeros(10, 256, dtype=bf)
    w = fake_fp8(cr, N=256)
    pos = torch.zeros(10, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="RopePlan"):
        cr.convrot_qkv_forward(X, w, 2, 1, None, None, None, pos)
    with pytest.raises(ValueError, match="X must have shape"):
        cr.convrot_qkv_forward(X[:, :128].contiguous(), w, 2, 1, None, None, plan, pos)
    with pytest.raises(ValueError, match="positions must have shape"):
        cr.convrot_qkv_forward(X, w, 2, 1, None, None, plan, pos[:5])
    with pytest.raises(ValueError, match="must be a GPU tensor"):
        cr.convrot_qkv_forward(X, w, 2, 1, None, None, plan, pos)
    with pytest.raises(ValueError, match="even"):
        cr.convrot_rope_prepare((15,), 64)
    with pytest.raises(ValueError, match="device must be a GPU"):
        cr.convrot_rope_prepare((16,), 64, device="cpu")


def test_gemm_dequant_rows_kind_refusals(cr):
    lib = cr.library()
    g = lambda d, kind=0, M=4, qx=FAKE, s=FAKE, y=0: lib.convrot_fp8_gemm_dequant_scales(
        qx, s, kind, M, ctypes.byref(d), None, FAKE, y, None)
    for kind in (0, 1):
        for d in (fp8_desc(cr), fp8_desc(cr, scales=1)):
            assert g(d, kind, M=0, qx=None) == cr.OK
            assert g(d, kind, M=-1) == cr.EINVAL and g(d, kind, s=None) == cr.EINVAL
            assert g(d, kind, s=ODD) == cr.EALIGN and g(d, kind, y=cr.I8) == cr.EUNSUPPORTED
    assert g(fp8_desc(cr), 2) == cr.EINVAL and g(fp8_desc(cr), -1, M=0) == cr.EINVAL
    assert g(fp8_desc(cr, magic=1), 2) == cr.ELAYOUT
    q, s = torch.zeros(16, 256, dtype=torch.uint8), torch.zeros(2, 16)
    with pytest.raises(ValueError, match="scales must be"):
        cr.convrot_fp8_gemm_dequant(q, s, 4, fake_fp8(cr), scales="e8")
    with pytest.raises(ValueError, match="GPU tensor"):
        cr.convrot_fp8_gemm_dequant(q, s, 4, fake_fp8(cr), scales="pow2")


def test_stream_of_another_device_refused(cr):
    class Stream:
        device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        cr.convrot_rope_prepare((16,), 64, device="cuda:0", stream=Stream())
    X, plan = torch.zeros(32, 256, dtype=bf), fake_plan(cr)
    for call in (lambda: cr.convrot_fp8_linear_forward(X, fake_fp8(cr), stream=Stream()),
                 lambda: cr.convrot_fp8_prepare_weights(X, stream=Stream()),
                 lambda: cr.convrot_fp8_quantize(X, stream=Stream()),
                 lambda: cr.convrot_rope_forward(Q, Q, plan, P, stream=Stream())):
        with pytest.raises(ValueError, match="GPU tensor on cuda:1"):
            call()


@pytest.mark.parametrize("N,K", [(64, 192), (24, 256), (64, 65664)])
def test_fp8_import_refuses_shapes_before_values(cr, N, K):
    """A shape that the library does not take is refused as such, whatever the scales."""
    W = torch.zeros(N, K).to(torch.float8_e4m3fn)
    for scales in ("f32", "pow2"):
        with pytest.raises(cr.ConvRotError, match="convrot_fp8_prepare_weights"):
            cr.convrot_fp8_prepare_weights(W, src_scale=torch.zeros(-(-N // 128), K // 128),
                                           scales=scales)
