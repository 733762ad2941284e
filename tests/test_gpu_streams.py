"""Calls on a caller's stream while the current stream is busy, with nothing
waiting for either but what a test says: results equal those of the same call
alone, and no memory changes hands before both streams are done with it."""
import pytest
import torch

from gpu_util import announce

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def cr():
    from w8a8_int8_rotated_amd import convrot
    convrot.library()
    return convrot


@pytest.fixture(scope="module")
def busy():
    a = torch.randn(8192, 8192, device="cuda")
    b = torch.empty_like(a)

    def run():
        """Some tens of milliseconds of work on the current stream."""
        for _ in range(4):
            torch.mm(a, a, out=b)
    run()
    torch.cuda.synchronize()
    return run


def calls(cr):
    """(name, call on given inputs and keywords, input) of the entries with outputs."""
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    f8 = cr.convrot_fp8_prepare_weights(rand(1024, 512))
    i8 = cr.convrot_linear_prepare_weights(rand(1024, 512), 128)
    plan = cr.convrot_rope_prepare((64,), 64)
    pos = torch.arange(300, dtype=torch.int32, device="cuda").view(300, 1)
    w = torch.ones(64, device="cuda")
    x, q, gq = rand(300, 512), rand(300, 8, 64), rand(300, 8, 64)
    flat = lambda out: [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]
    up, down = (cr.convrot_linear_prepare_weights(rand(*s), 128) for s in ((512, 512), (1024, 512)))
    gu = cr.convrot_swiglu_prepare(rand(1024, 512), 128)
    fa, fb = cr.convrot_lowrank_prepare(rand(128, 512), rand(1024, 128), 128)
    a, b = rand(128, 512), rand(1024, 128)
    qx, sx = cr.convrot_rotate_quantize(x, 128)
    return [
        ("fp8 linear", lambda x, **k: flat(cr.convrot_fp8_linear_forward(x, f8, **k)), x),
        ("fp8 quantise", lambda x, **k: flat(cr.convrot_fp8_quantize(x, **k))[1:], x[:288]),
        ("rope", lambda q, **k: flat(cr.convrot_rope_forward(q, None, plan, pos, **k)), q),
        ("norm + rope",
         lambda q, **k: flat(cr.convrot_qk_norm_rope_forward(q, None, w, None, plan, pos, **k)), q),
        ("norm + rope backward",
         lambda q, **k: flat(cr.convrot_qk_norm_rope_backward(gq, None, q, None, w, None, plan, pos,
                                                              **k)), q),
        ("qkv int8",
         lambda x, **k: flat(cr.convrot_qkv_forward(x, i8, 8, 4, w, w, plan, pos, **k)), x),
        ("qkv fp8",
         lambda x, **k: flat(cr.convrot_qkv_forward(x, f8, 8, 4, w, w, plan, pos, **k)), x),
        ("int8 linear", lambda x, **k: flat(cr.convrot_linear_forward(x, i8, **k)), x),
        ("int8 mlp", lambda x, **k: flat(cr.convrot_mlp_forward(x, up, down, **k)), x),
        ("swiglu mlp", lambda x, **k: flat(cr.convrot_swiglu_mlp_forward(x, gu, down, **k)), x),
        ("low rank", lambda x, **k: flat(cr.lowrank_convrot_forward(x, fa, fb, **k)), x),
        ("bf16 low rank", lambda x, **k: flat(cr.lowrank_bf16_forward(x, a, b, **k)), x),
        ("rotate + quantise", lambda x, **k: flat(cr.convrot_rotate_quantize(x, 128, **k))[1:], x),
        ("int8 gemm", lambda s, **k: flat(cr.convrot_gemm_dequant(qx, s, i8, **k)), sx),
        ("factor 1", lambda s, **k: flat(cr.convrot_lowrank_factor1(qx, s, fa, **k))[1:], sx),
        ("gelu", lambda x, **k: flat(cr.convrot_gelu_bf16(x, **k)), x),
        ("swiglu", lambda x, **k: flat(cr.convrot_swiglu_bf16(x, **k)), x),
        ("silu", lambda x, **k: flat(cr.convrot_silu_f32(x, **k)), x),
    ]


def same(got, want):
    return len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kind", ["f32", "pow2"])
def test_strided_weight_on_a_side_stream(cr, busy, kind):
    """The contiguous copy of a strided weight is made on the caller's stream."""
    w = torch.randn(2048, 4096, device="cuda")
    want = cr.convrot_fp8_prepare_weights(w.t().contiguous(), scales=kind)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(3):
        announce(f"strided weight on a side stream {kind} {i}")
        busy()
        pw = cr.convrot_fp8_prepare_weights(w.t(), scales=kind, stream=s)
        with torch.cuda.stream(s):
            codes, scale = pw.codes.cpu(), pw.scale.cpu()
        assert torch.equal(codes, want.codes.cpu()) and torch.equal(scale, want.scale.cpu())


@pytest.mark.parametrize("what", ["linear", "low rank", "swiglu"])
def test_strided_int8_weight_on_a_side_stream(cr, busy, what):
    w = torch.randn(2048, 4096, device="cuda")
    b = torch.randn(128, 4096, device="cuda")
    prep = {"linear": lambda w, b, **k: (cr.convrot_linear_prepare_weights(w, 128, **k),),
            "low rank": lambda w, b, **k: cr.convrot_lowrank_prepare(w[:128], b, 128, **k),
            "swiglu": lambda w, b, **k: (cr.convrot_swiglu_prepare(w, 128, **k),)}[what]
    want = prep(w.t().contiguous(), b.t().contiguous())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    announce(f"strided {what} weight on a side stream")
    busy()
    got = prep(w.t(), b.t(), stream=s)
    with torch.cuda.stream(s):
        got = [(p.codes.cpu(), p.scale.cpu()) for p in got]
    for p, (codes, scale) in zip(want, got):
        assert torch.equal(codes, p.codes.cpu()) and torch.equal(scale, p.scale.cpu())


def test_pow2_import_reads_scales_on_the_callers_stream(cr, busy):
    """The check of imported powers of two sees what the stream holds by then."""
    codes = torch.ones(256, 256, device="cuda").to(F8)
    scale = torch.full((2, 2), 3.0, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    announce("pow2 import on a side stream")
    with torch.cuda.stream(s):
        busy()
        scale.fill_(0.5)
    pw = cr.convrot_fp8_prepare_weights(codes, src_scale=scale, scales="pow2", stream=s)
    s.synchronize()
    assert bool((pw.scale == 0.5).all())
    with torch.cuda.stream(s):
        busy()
        scale.fill_(3.0)
    with pytest.raises(ValueError, match="powers of two"):
        cr.convrot_fp8_prepare_weights(codes, src_scale=scale, scales="pow2", stream=s)


def test_plan_on_a_side_stream(cr, busy):
    want = cr.convrot_rope_prepare((16, 24, 24), 64)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    announce("rope plan on a side stream")
    busy()
    junk = [torch.empty_like(want.freq).fill_(7.0), torch.empty_like(want.axis).fill_(7)]
    del junk
    plan = cr.convrot_rope_prepare((16, 24, 24), 64, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(plan.freq, want.freq) and torch.equal(plan.axis, want.axis)


@pytest.mark.parametrize("i", range(18))
def test_memory_of_either_stream(cr, busy, i):
    name, call, x = calls(cr)[i]
    announce(f"streams: {name}")
    neg = -x
    want, other = call(x), call(neg)
    s, cur = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    # memory freed on the current stream, whose work on it is still to come
    busy()
    junk = [torch.empty_like(t).fill_(7) for t in want for _ in range(3)]
    del junk
    got = call(x, stream=s)
    torch.cuda.synchronize()
    assert same(got, want)
    # results dropped while the current stream still has to read them
    got = call(x, stream=s)
    busy()
    cur.wait_stream(s)
    kept = [t.clone() for t in got]
    del got
    later = [call(neg, stream=s) for _ in range(3)]
    torch.cuda.synchronize()
    assert same(kept, want) and all(same(t, other) for t in later)
    # an argument dropped before the stream has come to the call
    y = x.clone()
    s.wait_stream(cur)
    with torch.cuda.stream(s):
        busy()
    got = call(y, stream=s)
    del y
    junk = [torch.full_like(x, float("nan")) for _ in range(3)]
    torch.cuda.synchronize()
    assert same(got, want)


def test_captured_side_stream(cr):
    """A call on a stream forked inside a capture belongs to the graph."""
    for name, call, x in calls(cr):
        announce(f"captured side stream: {name}")
        want, x = call(x), x.clone()
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cur = torch.cuda.current_stream()
            s.wait_stream(cur)
            got = call(x, stream=s)
            cur.wait_stream(s)
            out = [t.clone() for t in got]
        for k in range(3):
            for t in out:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert same(out, want), (name, k)
            other = call(-x)
            torch.cuda.synchronize()
            del other
