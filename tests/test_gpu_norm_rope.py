"""GPU tests of the rotary positions and the per-head norms with the rotation
against their definitions in 64 bits.

Bounds, with u = 2^-24 (fp32): a rotated channel is a difference of two rounded
products of values with cosines and sines good to 4 u, so it is within
16 u (|a| + |b|) of the definition on its pair (a, b); the norm adds relative
errors below (D/16 + 16) u (sums of D squares in 16-term chains, reciprocal
root, two products).  The rounding to the output type comes on top: 2^-8 of the
value for bf16, 2^-24 for fp32."""
import math

import pytest
import torch

from gpu_util import announce

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def cr():
    from w8a8_int8_rotated_amd import convrot
    convrot.library()
    return convrot


def rates(dims, spectrum, theta):
    R = sum(dims)
    f = ([theta ** (-2.0 * p / R) for p in range(R // 2)] if spectrum == "whole" else
         [theta ** (-2.0 * j / d) for d in dims for j in range(d // 2)])
    axis = [a for a, d in enumerate(dims) for _ in range(d // 2)]
    return torch.tensor(f, dtype=torch.float64), torch.tensor(axis)


def pairs(R, pairing):
    i = torch.arange(R // 2)
    return (i, i + R // 2) if pairing == "half" else (2 * i, 2 * i + 1)


def rotate(x, pos, f, axis, pairing, sign=1.0):
    """x [B, T, H, D] fp64, pos [B, T, axes]."""
    ang = pos.double()[..., axis][:, :, None] * f * sign
    a, b = pairs(2 * len(f), pairing)
    y = x.clone()
    y[..., a] = x[..., a] * ang.cos() - x[..., b] * ang.sin()
    y[..., b] = x[..., b] * ang.cos() + x[..., a] * ang.sin()
    return y


def pair_size(x, R, pairing):
    """|a| + |b| of every channel's pair (|x| for unrotated channels)."""
    a, b = pairs(R, pairing)
    s = x.abs().clone()
    s[..., a] = s[..., b] = (x[..., a].abs() + x[..., b].abs())
    return s


def norm(x, w, eps):
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    return x * r * w, r


class Case:
    def __init__(self, B, T, Hq, Hk, D, dims, pairing="interleaved", spectrum="axis",
                 dtype="bf16", layout="bthd", pos="i32", shared=False, far=1, theta=10000.0):
        self.__dict__.update(locals())
        g = torch.Generator().manual_seed(B * 1000 + T + Hq + D)
        self.dt = DT[dtype]
        axes = len(dims)
        p = torch.randint(0, 50 * far, (1 if shared else B, T, axes), generator=g)
        self.pos = (p * 0.24).float() if pos == "f32" else p.int()
        self.posd = self.pos[0].cuda() if shared else self.pos.cuda()
        self.f, self.axis = rates(dims, spectrum, theta)
        self.R = sum(dims)
        self.q, self.k = self.make(g, 3.0)
        self.wq, self.wk = (1 + 0.3 * torch.randn(D, generator=g) for _ in range(2))

    def make(self, g, gain):
        B, T, D = self.B, self.T, self.D
        out = []
        if self.layout == "qkv":
            row = torch.randn(B, T, (self.Hq + 2 * self.Hk) * D, generator=g).mul(gain)
            row = row.to(self.dt).cuda()
            a, b = self.Hq * D, (self.Hq + self.Hk) * D
            return row[..., :a].unflatten(-1, (self.Hq, D)), row[..., a:b].unflatten(-1, (self.Hk, D))
        for H in (self.Hq, self.Hk):
            if self.layout == "bhtd":
                x = torch.randn(B, H, T, D, generator=g).mul(gain).to(self.dt).cuda().transpose(1, 2)
            else:
                x = torch.randn(B, T, H, D, generator=g).mul(gain).to(self.dt).cuda()
            out.append(x)
        return out

    def plan(self, cr):
        return cr.convrot_rope_prepare(self.dims, self.D, theta=self.theta, pairing=self.pairing,
                                       spectrum=self.spectrum)

    def rot(self, x, sign=1.0):
        return rotate(x, self.pos.expand(self.B, -1, -1), self.f, self.axis, self.pairing, sign)

    def half_step(self, y):
        return y.abs() * (2.0 ** -8 if self.dtype == "bf16" else U)

    def __repr__(self):
        return (f"B{self.B} T{self.T} H{self.Hq}/{self.Hk} D{self.D} {self.dims} {self.pairing} "
                f"{self.spectrum} {self.dtype} {self.layout} {self.pos.dtype} far={self.far}")


def close(got, ref, bound, what):
    err = (got.double().cpu() - ref).abs()
    worst = float((err / bound).max()) if err.numel() else 0.0
    print(f"[parity] {what}: worst error {worst:.3f} of its bound", flush=True)
    assert worst <= 1.0, what


CASES = [
    dict(B=1, T=1, Hq=1, Hk=1, D=8, dims=(2,)),
    dict(B=1, T=1, Hq=32, Hk=8, D=128, dims=(128,), far=20000),
    dict(B=8, T=1, Hq=4, Hk=1, D=64, dims=(64,), pairing="half", far=20000),
    dict(B=2, T=37, Hq=42, Hk=42, D=128, dims=(16, 56, 56), layout="qkv", pos="f32"),
    dict(B=3, T=19, Hq=6, Hk=2, D=96, dims=(32, 32, 32), pairing="half", spectrum="whole",
         dtype="f32"),
    dict(B=2, T=70, Hq=3, Hk=5, D=80, dims=(20, 20), pairing="half", layout="bhtd", shared=True),
    dict(B=1, T=33, Hq=5, Hk=1, D=72, dims=(24, 22, 26), layout="bhtd", dtype="f32"),
    dict(B=2, T=9, Hq=2, Hk=2, D=256, dims=(64, 64, 64, 64), spectrum="whole", pos="f32"),
    dict(B=1, T=11, Hq=3, Hk=2, D=512, dims=(8,), pairing="half"),
    dict(B=1, T=5, Hq=40, Hk=24, D=512, dims=(256, 256), pairing="half", dtype="f32"),
    dict(B=1, T=13, Hq=129, Hk=3, D=32, dims=(10, 6), layout="qkv"),
    dict(B=1, T=9, Hq=7, Hk=7, D=40, dims=(40,), pairing="half", dtype="bf16", layout="qkv"),
    dict(B=1, T=2100, Hq=4, Hk=2, D=64, dims=(24, 40), layout="qkv", pos="f32"),
    # waves that take several tokens, from one batch to the next, or many batches apart
    dict(B=3, T=6007, Hq=2, Hk=2, D=32, dims=(20, 12), pos="f32"),
    dict(B=2500, T=8, Hq=3, Hk=1, D=64, dims=(64,), pairing="half", layout="bhtd", shared=True),
    dict(B=1700, T=11, Hq=2, Hk=1, D=192, dims=(100, 92), dtype="f32"),
]


@pytest.mark.parametrize("kw", CASES, ids=str)
def test_rope(cr, kw):
    c = Case(**kw)
    announce(f"rope {c}")
    plan = c.plan(cr)
    assert torch.equal(plan.axis.cpu().long(), c.axis)
    assert torch.allclose(plan.freq.cpu(), c.f, rtol=1e-14, atol=0)
    oq, ok = cr.convrot_rope_forward(c.q, c.k, plan, c.posd)
    for x, y in ((c.q, oq), (c.k, ok)):
        x64 = x.double().cpu()
        ref = c.rot(x64)
        bound = 16 * U * pair_size(x64, c.R, c.pairing) + c.half_step(ref) + 1e-40
        close(y, ref, bound, f"rope {c}")
        # channels beyond the rotary ones are copied
        assert torch.equal(y[..., c.R:], x[..., c.R:])
    # inverse: the transpose
    bq, bk = cr.convrot_rope_forward(c.q, None, plan, c.posd, inverse=True)
    assert bk is None
    x64 = c.q.double().cpu()
    ref = c.rot(x64, -1.0)
    close(bq, ref, 16 * U * pair_size(x64, c.R, c.pairing) + c.half_step(ref) + 1e-40, "inverse")
    # in place, on the strided tensors themselves
    q2, k2 = c.q, c.k
    cr.convrot_rope_forward(q2, k2, plan, c.posd, out_q=q2, out_k=k2)
    assert torch.equal(q2, oq) and torch.equal(k2, ok)


EPS = 1e-6


@pytest.mark.parametrize("kw", CASES, ids=str)
def test_norm_rope(cr, kw):
    c = Case(**kw)
    announce(f"norm + rope {c}")
    plan = c.plan(cr)
    before = c.q.clone()
    oq, ok = cr.convrot_qk_norm_rope_forward(c.q, c.k, c.wq.cuda(), c.wk.cuda(), plan, c.posd,
                                             eps=EPS)
    assert torch.equal(c.q, before)
    for x, w, y in ((c.q, c.wq, oq), (c.k, c.wk, ok)):
        n, _ = norm(x.double().cpu(), w.double(), EPS)
        ref = c.rot(n)
        bound = (c.D / 16 + 32) * U * pair_size(n, c.R, c.pairing) + c.half_step(ref) + 1e-40
        close(y, ref, bound, f"norm + rope {c}")
    # no weights: ones; queries alone
    y1, none = cr.convrot_qk_norm_rope_forward(c.q, None, None, None, plan, c.posd, eps=EPS)
    y2, _ = cr.convrot_qk_norm_rope_forward(c.q, None, torch.ones(c.D, device="cuda"), None, plan,
                                            c.posd, eps=EPS)
    assert none is None and torch.equal(y1, y2)
    # in place
    q2, k2 = c.q, c.k
    cr.convrot_qk_norm_rope_forward(q2, k2, c.wq.cuda(), c.wk.cuda(), plan, c.posd, eps=EPS,
                                    out_q=q2, out_k=k2)
    assert torch.equal(q2, oq) and torch.equal(k2, ok)


def reference_backward(c, g, x, w):
    """(dx, dw, scale of dx's terms, sum of dw's magnitudes) in fp64."""
    g, x, w = g.double().cpu(), x.double().cpu(), w.double()
    gn = c.rot(g, -1.0)
    _, r = norm(x, w, EPS)
    xh = x * r
    t = gn * w
    m = (t * xh).mean(-1, keepdim=True)
    gs = pair_size(g, c.R, c.pairing)
    # every term's magnitude, for the rounding bound
    mag = r * (gs * w.abs() + xh.abs() * ((gs * w.abs()) * xh.abs()).mean(-1, keepdim=True))
    return r * (t - xh * m), (gn * xh).sum((0, 1, 2)), mag, (gs * xh.abs()).sum((0, 1, 2))


@pytest.mark.parametrize("kw", CASES, ids=str)
def test_norm_rope_backward(cr, kw):
    c = Case(**kw)
    announce(f"norm + rope backward {c}")
    plan = c.plan(cr)
    gq, gk = c.make(torch.Generator().manual_seed(9), 0.1)
    wq, wk = c.wq.cuda(), c.wk.cuda()
    nws = cr.convrot_qk_norm_rope_workspace_bytes(c.B, c.T, c.Hq, c.Hk, c.D)
    ws = torch.full((nws,), 0xFF, dtype=torch.uint8, device="cuda")
    dq, dk, dwq, dwk = cr.convrot_qk_norm_rope_backward(gq, gk, c.q, c.k, wq, wk, plan, c.posd,
                                                        eps=EPS, workspace=ws)
    # a lane adds its rows one after another (at most tokens x heads of them),
    # then lanes, waves and workgroups join in at most 6 + 16 more additions
    chain = min(c.B * c.T * max(c.Hq, c.Hk), 2 * c.B * c.T * max(c.Hq, c.Hk) / 1024 + 64) + 64
    for g, x, w, dx, dw in ((gq, c.q, c.wq, dq, dwq), (gk, c.k, c.wk, dk, dwk)):
        rdx, rdw, mag, dwmag = reference_backward(c, g, x, w)
        close(dx, rdx, (c.D / 8 + 64) * U * mag + c.half_step(rdx) + 1e-40, f"dx {c}")
        close(dw, rdw, (chain + c.D / 16 + 64) * U * dwmag + 1e-40, f"dw {c}")
    # the same call repeats bit for bit; queries alone give the same dq
    again = cr.convrot_qk_norm_rope_backward(gq, gk, c.q, c.k, wq, wk, plan, c.posd, eps=EPS)
    for a, b in zip(again, (dq, dk, dwq, dwk)):
        assert torch.equal(a, b)
    only = cr.convrot_qk_norm_rope_backward(gq, None, c.q, None, wq, None, plan, c.posd, eps=EPS)
    assert torch.equal(only[0], dq) and only[1] is None and only[3] is None
    # in place over the gradients
    cr.convrot_qk_norm_rope_backward(gq, gk, c.q, c.k, wq, wk, plan, c.posd, eps=EPS, dq=gq, dk=gk)
    assert torch.equal(gq, dq) and torch.equal(gk, dk)


@pytest.mark.parametrize("pairing", ["interleaved", "half"])
def test_backward_against_differences(cr, pairing):
    """Directional derivatives of sum(v * forward) by central differences of the
    fp64 definition.  With step h the difference quotient is off by O(h^2)
    (third derivatives, ~1e-7 here) and by 1e-16 / h."""
    c = Case(B=2, T=5, Hq=3, Hk=2, D=48, dims=(16, 12, 20) if pairing == "interleaved" else (24, 24),
             pairing=pairing, dtype="f32")
    announce(f"backward against differences {pairing}")
    g = torch.Generator().manual_seed(3)
    gq, gk = c.make(g, 1.0)
    got = cr.convrot_qk_norm_rope_backward(gq, gk, c.q, c.k, c.wq.cuda(), c.wk.cuda(), c.plan(cr),
                                           c.posd, eps=EPS)
    h = 1e-4
    for i, (g_, x, w) in enumerate(((gq, c.q, c.wq), (gk, c.k, c.wk))):
        g_, x, w = g_.double().cpu(), x.double().cpu(), w.double()
        loss = lambda x, w: (g_ * c.rot(norm(x, w, EPS)[0])).sum()
        dirx, dirw = torch.randn(x.shape, generator=g).double(), torch.randn(w.shape, generator=g).double()
        for d, lp, lm, dir_ in ((got[i], loss(x + h * dirx, w), loss(x - h * dirx, w), dirx),
                                (got[2 + i], loss(x, w + h * dirw), loss(x, w - h * dirw), dirw)):
            want = float((lp - lm) / (2 * h))
            have = float((d.double().cpu() * dir_).sum())
            scale = float((d.double().cpu() * dir_).abs().sum())
            assert abs(have - want) <= 1e-5 * scale + 1e-6, (i, have, want)


def test_zero_rows_and_far_positions(cr):
    """A zero row stays zero (forward and backward finite); at positions of
    10^6 the angles keep fp32's accuracy."""
    c = Case(B=1, T=64, Hq=2, Hk=2, D=128, dims=(128,), dtype="f32", far=20000)
    announce("zero rows, far positions")
    c.q[0, 5] = 0
    plan = c.plan(cr)
    y, _ = cr.convrot_qk_norm_rope_forward(c.q, None, c.wq.cuda(), None, plan, c.posd)
    assert bool((y[0, 5] == 0).all()) and bool(torch.isfinite(y).all())
    dq, _, dw, _ = cr.convrot_qk_norm_rope_backward(torch.ones_like(c.q), None, c.q, None,
                                                    c.wq.cuda(), None, plan, c.posd)
    assert bool(torch.isfinite(dq).all()) and bool(torch.isfinite(dw).all())
    assert int(c.pos.max()) > 900_000


def test_no_tokens(cr):
    plan = cr.convrot_rope_prepare((64,), 64)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.empty(0, 1, dtype=torch.int32, device="cuda")
    w = torch.ones(64, device="cuda")
    announce("no tokens")
    y, _ = cr.convrot_qk_norm_rope_forward(q, None, w, None, plan, pos)
    assert y.shape == q.shape
    dq, _, dw, _ = cr.convrot_qk_norm_rope_backward(q, None, q, None, w, None, plan, pos)
    assert dq.shape == q.shape and bool((dw == 0).all())


def test_non_finite_rows_stay_alone(cr):
    c = Case(B=1, T=20, Hq=4, Hk=2, D=64, dims=(24, 16), pairing="half")
    plan = c.plan(cr)
    clean, _ = cr.convrot_qk_norm_rope_forward(c.q, None, None, None, plan, c.posd)
    plain, _ = cr.convrot_rope_forward(c.q, None, plan, c.posd)
    announce("non-finite rows")
    c.q[0, 3, 1, 50] = float("nan")          # an unrotated channel
    c.q[0, 7, 2, 45] = float("inf")
    y, _ = cr.convrot_qk_norm_rope_forward(c.q, None, None, None, plan, c.posd)
    bad = torch.zeros(20, 4, dtype=torch.bool, device="cuda")
    bad[3, 1] = bad[7, 2] = True
    assert torch.equal(y[0][~bad], clean[0][~bad])
    assert bool(torch.isnan(y[0, 3, 1]).all())
    z, _ = cr.convrot_rope_forward(c.q, None, plan, c.posd)
    same = z == plain
    same[0, 3, 1, 50] = same[0, 7, 2, 45] = True
    assert bool(same.all())                   # other channels of the rows too


def test_custom_tables(cr):
    """Overwritten frequencies and axes are what the rotation uses; axes
    outside the plan's are read as the nearest one."""
    c = Case(B=1, T=30, Hq=2, Hk=2, D=64, dims=(32, 32), dtype="f32")
    announce("custom tables")
    plan = c.plan(cr)
    c.f = c.f * 0.37
    c.axis = torch.arange(32) % 2
    plan.freq.copy_(c.f)
    plan.axis.copy_(torch.where(c.axis == 1, 9, -3))
    y, _ = cr.convrot_rope_forward(c.q, None, plan, c.posd)
    x64 = c.q.double().cpu()
    ref = c.rot(x64)
    close(y, ref, 16 * U * pair_size(x64, c.R, c.pairing) + c.half_step(ref) + 1e-40, "custom")


def test_offsets_beyond_32_bits(cr):
    """Token strides that put rows past 2^32 bytes."""
    D, H, T = 64, 1, 3
    announce("offsets beyond 32 bits")
    st = 1 << 31                               # elements: 4 GiB apart in bf16
    base = torch.zeros(2 * st + D, dtype=torch.bfloat16, device="cuda")
    q = base.as_strided((T, H, D), (st, D, 1))
    q.copy_(torch.randn(T, H, D, device="cuda"))
    plan = cr.convrot_rope_prepare((64,), 64)
    pos = torch.tensor([[0], [1], [2]], dtype=torch.int32, device="cuda")
    want, _ = cr.convrot_rope_forward(q.contiguous(), None, plan, pos)
    cr.convrot_rope_forward(q, None, plan, pos, out_q=q)
    assert torch.equal(q, want)


def test_graph_and_streams(cr):
    """Forward and backward captured together replay to the eager results."""
    c = Case(B=2, T=100, Hq=6, Hk=3, D=128, dims=(32, 48, 48), layout="qkv")
    announce("norm + rope graph")
    plan = c.plan(cr)
    gq, gk = c.make(torch.Generator().manual_seed(4), 0.5)
    wq, wk = c.wq.cuda(), c.wk.cuda()
    ws = torch.empty(cr.convrot_qk_norm_rope_workspace_bytes(2, 100, 6, 3, 128),
                     dtype=torch.uint8, device="cuda")
    fwd = [torch.empty(c.q.shape, dtype=c.dt, device="cuda"),
           torch.empty(c.k.shape, dtype=c.dt, device="cuda")]
    bwd = [torch.empty_like(fwd[0]), torch.empty_like(fwd[1]), torch.empty(128, device="cuda"),
           torch.empty(128, device="cuda")]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cr.convrot_qk_norm_rope_forward(c.q, c.k, wq, wk, plan, c.posd, out_q=fwd[0], out_k=fwd[1])
        cr.convrot_qk_norm_rope_backward(gq, gk, c.q, c.k, wq, wk, plan, c.posd, dq=bwd[0],
                                         dk=bwd[1], dw_q=bwd[2], dw_k=bwd[3], workspace=ws)
    for i in range(3):
        c.q.copy_(torch.randn(c.q.shape, device="cuda"))
        gk.copy_(torch.randn(gk.shape, device="cuda"))
        ef = cr.convrot_qk_norm_rope_forward(c.q, c.k, wq, wk, plan, c.posd)
        eb = cr.convrot_qk_norm_rope_backward(gq, gk, c.q, c.k, wq, wk, plan, c.posd)
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip((*fwd, *bwd), (*ef, *eb)):
            assert torch.equal(a, b), f"replay {i}"
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = cr.convrot_qk_norm_rope_backward(gq, gk, c.q, c.k, wq, wk, plan, c.posd, stream=s)
    s.synchronize()
    for a, b in zip(y, eb):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,T,out", [(1, 1, "bf16"), (2, 75, "bf16"), (1, 300, "f32")])
def test_qkv_path(cr, fp8, B, T, out):
    """The QKV projection with norms and rotation is its three parts: the linear,
    the norm on its Q and K columns, and values left alone; then attention's
    inputs turned back give the normed projections."""
    K, D, Hq, Hk = 512, 64, 6, 2
    N = (Hq + 2 * Hk) * D
    g = torch.Generator().manual_seed(T)
    X = torch.randn(B, T, K, generator=g).to(torch.bfloat16).cuda()
    W = torch.randn(N, K, generator=g).mul(0.05).cuda()
    bias = torch.randn(N, generator=g).cuda()
    wq, wk = (1 + 0.2 * torch.randn(D, generator=g).cuda() for _ in range(2))
    pos = torch.randint(0, 90, (T, 3), generator=g, dtype=torch.int32).cuda()
    plan = cr.convrot_rope_prepare((16, 24, 24), D)
    announce(f"qkv path fp8={fp8} B={B} T={T} {out}")
    if fp8:
        pw = cr.convrot_fp8_prepare_weights(W)
        y = cr.convrot_fp8_linear_forward(X.view(-1, K), pw, bias=bias, out_dtype=DT[out])
    else:
        pw = cr.convrot_linear_prepare_weights(W, 128)
        y = cr.convrot_linear_forward(X.view(-1, K), pw, bias=bias, out_dtype=DT[out])
    got = cr.convrot_qkv_forward(X, pw, Hq, Hk, wq, wk, plan, pos, bias=bias, out_dtype=DT[out])
    y = y.view(B, T, N)
    q = y[..., :Hq * D].unflatten(-1, (Hq, D))
    k = y[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
    eq, ek = cr.convrot_qk_norm_rope_forward(q, k, wq, wk, plan, pos)
    assert torch.equal(got[..., :Hq * D], eq.flatten(-2))
    assert torch.equal(got[..., Hq * D:(Hq + Hk) * D], ek.flatten(-2))
    assert torch.equal(got[..., (Hq + Hk) * D:], y[..., (Hq + Hk) * D:])
    back, _ = cr.convrot_rope_forward(got[..., :Hq * D].unflatten(-1, (Hq, D)), None, plan, pos,
                                      inverse=True)
    n, _ = norm(q.double().cpu(), wq.double().cpu(), 1e-6)
    # two roundings to the type, of values no larger than their pair
    size = pair_size(n, 64, "interleaved")
    half = 2.0 ** -8 if out == "bf16" else U
    close(back, n, 2.1 * half * size + 64 * U * size + 1e-40, "turned back")


def test_broadcast_inputs_and_outputs(cr):
    """Inputs may repeat rows with a zero stride; outputs may not."""
    plan = cr.convrot_rope_prepare((64,), 64)
    base = torch.randn(1, 7, 1, 64, device="cuda").bfloat16()
    q = base.expand(3, 7, 4, 64)
    pos = torch.arange(7, dtype=torch.int32, device="cuda").view(7, 1)
    w = torch.randn(64, device="cuda")
    announce("broadcast inputs")
    y, _ = cr.convrot_qk_norm_rope_forward(q, None, w, None, plan, pos)
    want, _ = cr.convrot_qk_norm_rope_forward(q.contiguous(), None, w, None, plan, pos)
    assert torch.equal(y, want)
    g = torch.randn(3, 7, 4, 64, device="cuda").bfloat16()
    a = cr.convrot_qk_norm_rope_backward(g, None, q, None, w, None, plan, pos)
    b = cr.convrot_qk_norm_rope_backward(g, None, q.contiguous(), None, w, None, plan, pos)
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
    with pytest.raises(cr.ConvRotError):
        cr.convrot_rope_forward(q, None, plan, pos, out_q=q)


def test_two_streams_at_once(cr):
    """Independent calls on two streams, each with its own workspace."""
    c = Case(B=1, T=500, Hq=8, Hk=4, D=128, dims=(64, 64))
    plan = c.plan(cr)
    gq, gk = c.make(torch.Generator().manual_seed(2), 1.0)
    args = (gq, gk, c.q, c.k, c.wq.cuda(), c.wk.cuda(), plan, c.posd)
    want = cr.convrot_qk_norm_rope_backward(*args)
    announce("two streams")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for s in streams:
            got.append(cr.convrot_qk_norm_rope_backward(*args, stream=s))
    torch.cuda.synchronize()
    for y in got:
        for a, b in zip(y, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("pos,axes", [("i32", [24, 20, 20]), ("f32", [64])])
def test_steps_of_a_longer_position_array(cr, pos, axes):
    """One token per call, its positions a slice (at 4 or 12 bytes' offsets) of the
    sequence's: the rows of the call over the whole sequence."""
    c = Case(1, 9, 6, 2, 64, axes, pos=pos)
    announce(f"position slices {c!r}")
    plan, p = c.plan(cr), c.posd.reshape(9, len(axes))
    whole = cr.convrot_qk_norm_rope_forward(c.q, c.k, c.wq.cuda(), c.wk.cuda(), plan, p)
    for t in range(9):
        step = cr.convrot_qk_norm_rope_forward(c.q[:, t:t + 1], c.k[:, t:t + 1], c.wq.cuda(),
                                               c.wk.cuda(), plan, p[t:t + 1])
        for y, z in zip(whole, step):
            assert torch.equal(y[:, t:t + 1], z), t


def test_offsets_past_32_bits(cr):
    """More than 2^31 elements of queries: the last tokens' rows, forward, inverse
    and backward, are those of a call on these tokens alone."""
    T, H, D = 140_000, 128, 128
    announce("norm + rope, 2.3e9 elements")
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(T, H, D, generator=g, device="cuda", dtype=torch.bfloat16)
    pos = torch.randint(0, 1000, (T, 3), generator=g, device="cuda", dtype=torch.int32)
    w = torch.randn(D, generator=g, device="cuda")
    plan = cr.convrot_rope_prepare([16, 56, 56], D)
    for part in (slice(0, 3), slice(131_070, 131_075), slice(T - 5, T)):
        x, p = q[part], pos[part].contiguous()
        for run in (lambda q, pos: cr.convrot_rope_forward(q, None, plan, pos)[0],
                    lambda q, pos: cr.convrot_rope_forward(q, None, plan, pos, inverse=True)[0],
                    lambda q, pos: cr.convrot_qk_norm_rope_forward(q, None, w, None, plan, pos)[0],
                    lambda q, pos: cr.convrot_qk_norm_rope_backward(
                        q.flip(0) if q.shape[0] < T else G, None, q, None, w, None, plan, pos)[0]):
            G = q.clone()
            G[part] = x.flip(0)
            whole = run(q, pos)
            assert torch.equal(whole[part], run(x, p))
            del G, whole


@pytest.mark.parametrize("pairing", ["interleaved", "half"])
@pytest.mark.parametrize("pos", ["i32", "f32"])
def test_far_positions_keep_fp32_accuracy(cr, pairing, pos):
    """fp32 rows at positions to 10^6, with a zero row: rotation, norm with rotation and
    its backward within the bounds of near positions (an fp32 angle would be off by 0.06
    radians here).  fp32 positions are multiples of 0.24, the definition's own inputs."""
    c = Case(B=1, T=64, Hq=2, Hk=1, D=128, dims=(64, 32, 32), pairing=pairing, dtype="f32",
             pos=pos, far=20000 if pos == "i32" else 83000)
    assert float(c.pos.max()) > 900_000
    announce(f"far positions {c}")
    c.q[0, 5] = 0
    plan, wq, wk = c.plan(cr), c.wq.cuda(), c.wk.cuda()
    for inverse, sign in ((False, 1.0), (True, -1.0)):
        y, _ = cr.convrot_rope_forward(c.q, None, plan, c.posd, inverse=inverse)
        x64 = c.q.double().cpu()
        ref = c.rot(x64, sign)
        close(y, ref, 16 * U * pair_size(x64, c.R, c.pairing) + c.half_step(ref) + 1e-40, "rope")
    out = cr.convrot_qk_norm_rope_forward(c.q, c.k, wq, wk, plan, c.posd, eps=EPS)
    for x, w, y in ((c.q, c.wq, out[0]), (c.k, c.wk, out[1])):
        n, _ = norm(x.double().cpu(), w.double(), EPS)
        ref = c.rot(n)
        bound = (c.D / 16 + 32) * U * pair_size(n, c.R, c.pairing) + c.half_step(ref) + 1e-40
        close(y, ref, bound, "norm + rope")
    assert bool((out[0][0, 5] == 0).all())
    gq, gk = c.make(torch.Generator().manual_seed(8), 0.1)
    dq, dk, dwq, dwk = cr.convrot_qk_norm_rope_backward(gq, gk, c.q, c.k, wq, wk, plan, c.posd,
                                                        eps=EPS)
    chain = c.T * c.Hq + 64                  # as in test_norm_rope_backward
    for g, x, w, dx, dw in ((gq, c.q, c.wq, dq, dwq), (gk, c.k, c.wk, dk, dwk)):
        rdx, rdw, mag, dwmag = reference_backward(c, g, x, w)
        close(dx, rdx, (c.D / 8 + 64) * U * mag + c.half_step(rdx) + 1e-40, "dx")
        close(dw, rdw, (chain + c.D / 16 + 64) * U * dwmag + 1e-40, "dw")
