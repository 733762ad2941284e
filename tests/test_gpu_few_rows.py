"""The INT8 product for up to 64 rows: equal bits to the integer definition and, row by row,
to the tiled kernel (a call of more rows), over its row tiles a workgroup and ragged ends."""
import numpy as np
import pytest
import torch

from gpu_util import announce, padded_rows, tile, tiled_index, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cr():
    from w8a8_int8_rotated_amd import convrot
    convrot.library()
    return convrot


# N: one, two and four blocks of 16 outputs a workgroup on 256 CUs, and blocks left over in the
# last; K: fewer 64-wide tiles than waves, ragged shares, many
SHAPES = [(16, 128), (48, 256), (4096, 128), (4112, 640), (8208, 384), (16400, 256), (16128, 5376),
          (21520, 128), (528, 65536 // 2),
          (24592, 256)]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("N,K", SHAPES, ids=str)
def test_against_integers_and_the_tiled_kernel(cr, N, K, out, bias):
    rng = np.random.default_rng(N + K)
    g = torch.Generator(device="cuda").manual_seed(N + K)
    codes = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    W = cr.convrot_linear_prepare_weights(codes, 64, src_scale=torch.rand(N, generator=g,
                                                                          device="cuda") * 1e-3)
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    for M in (1, 5, 16, 17, 32, 33, 50, 64):
        announce(f"few rows M={M} N={N} K={K} {out} bias={bias}")
        q = rng.integers(-127, 128, (65, K)).astype(np.int8)
        s = to_dev(rng.random(65).astype(np.float32))
        tiled = to_dev(tile(q))                       # 65 rows: the tiled kernel
        Mp = padded_rows(M)
        few = tiled.reshape(-1)[:Mp * K].clone().view(Mp, K)
        if M < Mp:                                    # padding rows may hold anything
            flat = few.reshape(-1)
            flat[torch.from_numpy(tiled_index(Mp, K)[M:].reshape(-1)).cuda()] = -128
        whole = torch.full((M + 2, N), 7.0, dtype=out, device="cuda")
        y = cr.convrot_gemm_dequant(few, s[:M].contiguous(), W, b, out=whole[:M])
        assert bool((whole[M:] == 7).all())
        full = cr.convrot_gemm_dequant(tiled, s, W, b, out_dtype=out)
        assert torch.equal(y, full[:M])
        acc = (torch.from_numpy(q[:M]).double() @ codes.cpu().double().t()).float().cuda()
        ref = acc * s[:M, None] * W.scale
        ref = (ref + b if bias else ref).to(out)
        assert torch.equal(y, ref)


def test_linear_few_rows(cr):
    """The whole linear: a row alone equals the same row of a larger batch."""
    K, N = 1280, 528
    x = torch.randn(70, K, device="cuda").to(torch.bfloat16)
    W = cr.convrot_linear_prepare_weights(torch.randn(N, K, device="cuda") * 0.02, 128)
    b = torch.randn(N, device="cuda")
    full = cr.convrot_linear_forward(x, W, bias=b)
    for M in (1, 2, 15, 16, 17, 33, 64):
        assert torch.equal(cr.convrot_linear_forward(x[:M].contiguous(), W, bias=b), full[:M])
    assert padded_rows(16) == 16


@pytest.mark.parametrize("N", [2 ** 20, 2 ** 20 + 16])
def test_both_sides_of_the_widest_border(cr, N):
    """17 and 32 rows of the widest outputs that this kernel takes, and of wider ones."""
    K = 128
    g = torch.Generator(device="cuda").manual_seed(N)
    codes = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    W = cr.convrot_linear_prepare_weights(codes, 64, src_scale=torch.rand(N, generator=g,
                                                                          device="cuda") * 1e-3)
    rng = np.random.default_rng(3)
    for M in (16, 17, 32):
        announce(f"few rows M={M} N={N} K={K}")
        q = rng.integers(-127, 128, (M, K)).astype(np.int8)
        s = to_dev(rng.random(M).astype(np.float32))
        whole = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
        y = cr.convrot_gemm_dequant(to_dev(tile(q)), s, W, out=whole[:M])
        assert bool((whole[M:] == 7).all())
        acc = (to_dev(q).float().double() @ codes.double().t()).float()
        assert torch.equal(y, (acc * s[:, None] * W.scale).to(torch.bfloat16))
