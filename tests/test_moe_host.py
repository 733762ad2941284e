"""Host-side refusals of the mixture-of-experts layer: the C ABI with fake pointers (never
dereferenced) and the Python binding with host tensors.  Nothing is launched."""
import ctypes
import os

import pytest
import torch

A = 0x7f0000000000                  # fake device addresses, far apart
PTR = [A + (i << 40) for i in range(12)]
ODD = A + 8


@pytest.fixture(scope="module")
def cr():
    from w8a8_int8_rotated_amd import convrot
    if not os.path.exists(convrot.LIB_PATH):
        pytest.fail("libconvrot.so not built (run __graft_entry__.build())")
    convrot.library()
    return convrot


def desc(cr, **kw):
    d = cr.convrot_moe_weights()
    d.magic, d.version = cr.MOE_MAGIC, cr.MOE_VERSION
    d.experts, d.shared, d.K, d.F = 16, 1, 512, 256
    d.gate_up, d.gate_up_scale, d.down, d.down_scale = PTR[:4]
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_sizes(cr):
    lib = cr.library()
    p, s = lib.convrot_moe_packed_bytes, lib.convrot_moe_scale_bytes
    assert p(64, 2 * 1408, 5376) == 64 * 2 * 1408 * 5376
    assert s(64, 2 * 1408, 5376) == 64 * 22 * 42 * 4
    for n, R, C in ((0, 256, 256), (529, 256, 256), (4, 200, 256), (4, 256, 64), (-1, 256, 256),
                    (4, 131072, 65536), (4, 256, 65664), (4, 1 << 62, 1 << 62)):
        assert p(n, R, C) == 0 and s(n, R, C) == 0
    w = lambda T=1, k=2, **kw: lib.convrot_moe_workspace_bytes(T, ctypes.byref(desc(cr, **kw)), k)  # noqa: E731
    assert w() > 0 and w(64) == w(65) == w(1 << 40) > w(1)
    assert w(0) == 0 and w(-1) == 0 and w(k=0) == 0 and w(k=17) == 0 and w(magic=1) == 0
    assert lib.convrot_moe_workspace_bytes(1, None, 2) == 0


def test_forward_refusals(cr):
    lib = cr.library()

    def f(T=4, X=PTR[4], r=PTR[5], rt=0, bias=None, k=2, score=0, flags=1, scale=1.0, Y=PTR[6],
          yt=1, ids=PTR[7], w=PTR[8], ws=PTR[9], wsb=1 << 40, **kw):
        return lib.convrot_moe_forward(X, T, r, rt, bias, ctypes.byref(desc(cr, **kw)), k, score,
                                       flags, scale, Y, yt, ids, w, ws, wsb, None)

    assert lib.convrot_moe_forward(A, 1, A, 0, None, None, 1, 0, 0, 1.0, A, 1, A, A, A, 1,
                                   None) == cr.EINVAL
    assert f(T=0, X=None, Y=None, ws=None, wsb=0) == cr.OK
    assert f(T=-1) == cr.EINVAL and f(T=1 << 31) == cr.EUNSUPPORTED
    for bad in (dict(magic=0), dict(version=2)):
        assert f(**bad) == cr.ELAYOUT
    for bad in (dict(experts=0), dict(shared=-1), dict(K=0), dict(F=-128), dict(gate_up=None),
                dict(down_scale=None)):
        assert f(**bad) == cr.EINVAL
    for bad in (dict(experts=513), dict(shared=17), dict(K=320), dict(F=192), dict(K=65664),
                dict(K=65536, F=32768)):
        assert f(**bad) == cr.EUNSUPPORTED
    assert f(down=ODD) == cr.EALIGN
    for k in (0, -1, 17):
        assert f(k=k) == cr.EINVAL
    assert f(k=33, experts=40) == cr.EINVAL
    assert f(rt=2) == cr.EUNSUPPORTED and f(yt=4) == cr.EUNSUPPORTED
    assert f(flags=2) == cr.EUNSUPPORTED and f(score=2) == cr.EINVAL
    assert f(scale=float("nan")) == cr.EINVAL and f(scale=float("inf")) == cr.EINVAL
    for name in ("X", "r", "Y", "ids", "w"):
        assert f(**{name: None}) == cr.EINVAL
        assert f(**{name: ODD}) == cr.EALIGN
    assert f(bias=ODD) == cr.EALIGN and f(ws=ODD) == cr.EALIGN
    assert f(ws=None) == cr.EWORKSPACE and f(wsb=100) == cr.EWORKSPACE
    assert f(Y=PTR[4]) == cr.EINVAL and f(Y=PTR[5] + 16 * 512 * 4 - 16) == cr.EINVAL
    assert f(ids=PTR[6] + 16) == cr.EINVAL and f(w=PTR[7]) == cr.EINVAL
    assert f(bias=PTR[8], w=PTR[8] + 48) == cr.EINVAL


def test_prepare_refusals(cr):
    lib = cr.library()

    def f(gu=PTR[4], dn=PTR[5], dt=0, s1=None, s2=None, scales=0, **kw):
        d = desc(cr, magic=0, version=0, **kw)
        rc = lib.convrot_moe_prepare_weights(gu, dn, dt, s1, s2, scales, ctypes.byref(d), None)
        assert d.magic == 0                                          # nothing written on error
        return rc

    assert lib.convrot_moe_prepare_weights(A, A, 0, None, None, 0, None, None) == cr.EINVAL
    assert f(gu=None) == cr.EINVAL and f(dn=None) == cr.EINVAL
    assert f(dt=cr.I8) == cr.EUNSUPPORTED and f(K=320) == cr.EUNSUPPORTED
    assert f(dt=cr.F8E4M3) == cr.EINVAL and f(s1=PTR[6], s2=PTR[7]) == cr.EINVAL
    assert f(dt=cr.F8E4M3, s1=PTR[6]) == cr.EINVAL and f(scales=2) == cr.EINVAL
    assert f(gu=ODD) == cr.EALIGN and f(dt=cr.F8E4M3, s1=ODD, s2=PTR[7]) == cr.EALIGN
    assert f(down=None) == cr.EINVAL and f(experts=600) == cr.EUNSUPPORTED


def test_binding_refusals(cr):
    gu, dn = torch.zeros(4, 512, 384), torch.zeros(4, 384, 256)
    c = lambda t: t.to(torch.float8_e4m3fn)                          # noqa: E731
    s1, s2 = torch.ones(4, 4, 3), torch.ones(4, 3, 2)
    p = cr.convrot_moe_prepare_weights
    for call in (
            lambda: p(gu[0], dn), lambda: p(gu.half(), dn.half()), lambda: p(gu, dn.bfloat16()),
            lambda: p(gu[:3], dn), lambda: p(gu[:, :256], dn), lambda: p(gu, dn, shared=4),
            lambda: p(gu, dn, shared=-1), lambda: p(gu, dn, scales="f16"),
            lambda: p(c(gu), c(dn)), lambda: p(gu, dn, 0, s1, s2),
            lambda: p(c(gu), c(dn), 0, s1, s2[:3]), lambda: p(c(gu), c(dn), 0, s1, s2.double()),
            lambda: p(gu, dn)):                                      # on the host
        with pytest.raises(ValueError):
            call()
    with pytest.raises(cr.ConvRotError):
        p(torch.zeros(2, 128, 128), torch.zeros(2, 128, 64))
    W = cr.MoEWeights(desc(cr), None, None, dn, None)
    x, r = torch.zeros(3, 512, dtype=torch.bfloat16), torch.zeros(16, 512)
    f = cr.convrot_moe_forward
    for call in (
            lambda: f(x, r, None, 2), lambda: f(x.float(), r, W, 2), lambda: f(x[:, :256], r, W, 2),
            lambda: f(x, r[:15], W, 2), lambda: f(x, r.double(), W, 2),
            lambda: f(x, r, W, 0), lambda: f(x, r, W, 17),
            lambda: f(x, r, W, 2, router_bias=torch.zeros(15)),
            lambda: f(x, r, W, 2, score="relu"), lambda: f(x, r, W, 2, out=x[:2]),
            lambda: f(x, r, W, 2, ids=torch.zeros(3, 2)),
            lambda: f(x, r, W, 2, weights=torch.zeros(3, 3)),
            lambda: f(x, r, W, 2, workspace=torch.zeros(8, dtype=torch.uint8)),
            lambda: f(x, r, W, 2)):                                  # on the host
        with pytest.raises(ValueError):
            call()


def test_forward_overlaps(cr):
    """Outputs and the workspace against every input's whole extent, the experts' codes and
    scales among them, and against each other: the last 16 bytes, and the first ones behind."""
    E, S, K, F, T, k = 16, 1, 512, 256, 4, 2
    need = cr.library().convrot_moe_workspace_bytes(T, ctypes.byref(desc(cr)), k)
    extents = {"gate_up": (E + S) * 2 * F * K, "gate_up_scale": (E + S) * 2 * F // 128 * K // 128 * 4,
               "down": (E + S) * K * F, "down_scale": (E + S) * K // 128 * F // 128 * 4,
               "X": T * K * 2, "r": E * K * 4, "bias": E * 4}
    outs = {"Y": T * K * 2, "ids": T * k * 4, "w": T * k * 4, "ws": need}
    base = {n: PTR[i] for i, n in enumerate((*extents, *outs))}

    def f(**kw):
        a = {**base, **kw}
        d = desc(cr, **{n: a[n] for n in ("gate_up", "gate_up_scale", "down", "down_scale")})
        # a workspace that is a byte short: nothing can be launched
        return cr.library().convrot_moe_forward(
            a["X"], T, a["r"], 0, a["bias"], ctypes.byref(d), k, 0, 1, 1.0, a["Y"], 1, a["ids"],
            a["w"], a["ws"], need - 1, None)

    assert f() == cr.EWORKSPACE
    for o in outs:
        for n, size in {**extents, **outs}.items():
            if n == o:
                continue
            end = (size + 15) // 16 * 16
            assert f(**{o: base[n] + end - 16}) == cr.EINVAL, (o, n)
            assert f(**{o: base[n]}) == cr.EINVAL, (o, n)
            assert f(**{o: base[n] + end}) == cr.EWORKSPACE, (o, n)


def test_workspace_sizes_kept_are_few(cr):
    """A layer called with many batch sizes keeps one size for each up to a pass of 64 tokens, and
    each is the library's."""
    d = desc(cr)
    W = cr.MoEWeights(d, None, None, torch.zeros(1), None)
    r = torch.zeros(16, 512)
    for T in (*range(1, 130), 1000, 38656):
        need = cr.library().convrot_moe_workspace_bytes(T, ctypes.byref(d), 2)
        x = torch.zeros(T, 512, dtype=torch.bfloat16)
        with pytest.raises(ValueError, match=f"{need} needed"):
            cr.convrot_moe_forward(x, r, W, 2, workspace=torch.empty(need - 1, dtype=torch.uint8))
        with pytest.raises(ValueError, match="GPU"):                 # large enough: on the host
            cr.convrot_moe_forward(x, r, W, 2, workspace=torch.empty(need, dtype=torch.uint8))
    assert len(W._workspace) <= 64
