"""8-bit floating point with block scales: the quantiser bit for bit, and the
product against its definition in 64 bits."""
import numpy as np
import pytest
import torch

from sparse_mixture_experts_gating_b200 import matmul_fp8, quantize_fp8, status
from tests import _fp8 as F

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def code_values(codes):
    return F.decode(codes.contiguous().view(torch.uint8).cpu().numpy())


def check_quantized(x, codes, scales, block_rows, transpose):
    """codes and scales of x [..., R, K] against the definition, bit for bit."""
    xs = x.float().cpu().numpy().reshape((-1,) + tuple(x.shape[-2:]))
    cs = code_values(codes).reshape((xs.shape[0],) + tuple(codes.shape[-2:]))
    ss = scales.cpu().numpy().reshape((xs.shape[0],) + tuple(scales.shape[-2:]))
    for m, c, s in zip(xs, cs, ss):
        vc, vs = F.quantize(m.T if transpose else m, block_rows)
        np.testing.assert_array_equal(s, vs)
        np.testing.assert_array_equal(c, vc)


SHAPES = [(1, 1), (1, 127), (2, 128), (5, 129), (16, 256), (130, 300), (257, 1000), (128, 4096), (1000, 17)]


@pytest.mark.parametrize("block_rows,transpose", [(1, False), (128, False), (1, True), (128, True)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,K", SHAPES)
def test_quantiser_matches_the_definition(R, K, dtype, block_rows, transpose):
    x = torch.randn((R, K), device="cuda", generator=gen(R * 7 + K)).to(dtype)
    x[0] *= 2.0 ** -90           # near the smallest block maximum
    x[R // 2, : K // 2] = 0.0    # zeros, and with K > 256 a block of nothing else
    x[-1] *= 1e20
    codes, scales = quantize_fp8(x, block_rows=block_rows, transpose=transpose)
    status()
    rows, cols = (K, R) if transpose else (R, K)
    assert codes.shape == (rows, cols) and codes.dtype == torch.float8_e4m3fn
    assert scales.shape == (-(-rows // block_rows), F.blocks(cols)) and scales.dtype == F32
    assert codes.data_ptr() % 16 == 0 and (rows == 1 or codes.stride(0) % 16 == 0)
    check_quantized(x, codes, scales, block_rows, transpose)


def test_quantiser_takes_ties_to_even_and_keeps_zero_blocks():
    x = torch.zeros((3, 256), device="cuda")
    x[0, 0] = 448.0                                                   # scale 1: codes are the values themselves
    x[0, 1:128] = torch.arange(1, 128, device="cuda") * 0.5 + 0.25    # many halves between two codes
    x[1, 5] = 2.0 ** -149                                             # below the smallest block maximum
    codes, scales = quantize_fp8(x)
    check_quantized(x, codes, scales, 1, False)
    assert scales[0, 0].item() == 1.0
    assert code_values(codes)[2].any() == False  # noqa: E712
    assert (scales[2] == np.float32(np.float32(2.0 ** -100) / np.float32(448))).all()


def test_quantiser_reads_views_and_stacks():
    base = torch.randn((4, 40, 333), device="cuda", generator=gen(2))
    for x in (base[:, :, 3:200], base[1, 5:, 1:], base.transpose(1, 2), base[:, ::2], base[0, :1, 7:9]):
        for block_rows in (1, 128):
            codes, scales = quantize_fp8(x, block_rows=block_rows)
            check_quantized(x, codes, scales, block_rows, False)
    e = torch.empty((0, 64), device="cuda")
    codes, scales = quantize_fp8(e)
    assert codes.shape == (0, 64) and scales.shape == (0, 1)


def test_quantiser_marks_what_is_not_finite():
    x = torch.randn((4, 256), device="cuda", generator=gen(3))
    x[1, 3] = float("nan")
    x[2, 130] = float("inf")
    codes, scales = quantize_fp8(x)
    v = code_values(codes) * np.repeat(scales.cpu().numpy(), 128, 1)
    assert np.isnan(v[1, 3]) and np.isfinite(np.delete(v[1], 3)).all()
    assert np.isnan(v[2, 128:]).all() and np.isfinite(v[2, :128]).all()
    assert np.isfinite(v[[0, 3]]).all()


def operands(M, N, K, G, b_rows, seed):
    g = gen(seed)
    x = torch.randn((M, K), device="cuda", generator=g) * (torch.rand((M, 1), device="cuda", generator=g) + 0.1)
    shape = (N, K) if G is None else (G, N, K)
    w = torch.randn(shape, device="cuda", generator=g) * K ** -0.5
    return quantize_fp8(x), quantize_fp8(w, block_rows=b_rows)


def host(pair, block_rows):
    codes, scales = pair
    return F.values(code_values(codes), scales.cpu().numpy(), block_rows)


def check_product(y, av, bv, out_dtype):
    exact = av @ bv.T
    tol = F.product_bound(av, bv) + np.abs(exact) * (torch.finfo(out_dtype).eps / 2) * 1.01 + 1e-30
    err = np.abs(y.double().cpu().numpy() - exact)
    assert (err <= tol).all(), (err / tol).max()


DENSE = [(1, 1, 1), (1, 256, 128), (3, 129, 130), (16, 512, 1024), (33, 300, 257), (65, 64, 2048), (128, 256, 128),
         (129, 257, 129), (200, 1111, 384), (300, 1000, 1104), (1, 4096, 4096), (17, 128, 8200)]


@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", DENSE)
def test_product_matches_64_bits(M, N, K, out_dtype, b_rows):
    a, b = operands(M, N, K, None, b_rows, M + N + K)
    y = matmul_fp8(a, b, out_dtype=out_dtype)
    status()
    check_product(y, host(a, 1), host(b, b_rows), out_dtype)


@pytest.mark.parametrize("M,N,K,cuts", [
    (40, 130, 200, [0, 0, 7, 7, 40]),            # empty groups first and inside
    (300, 256, 384, [0, 129, 129, 300, 300]),    # an empty last group
    (64, 64, 128, [5, 6, 40]),                   # rows before the first group and behind the last
    (517, 200, 300, [0, 1, 128, 256, 390, 517]),
    (10, 100, 64, [10, 10, 10]),                 # no rows at all
])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_grouped_product(M, N, K, cuts, out_dtype):
    G = len(cuts) - 1
    a, b = operands(M, N, K, G, 128, M + N)
    offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    out = torch.full((M, N), 7.0, dtype=out_dtype, device="cuda")
    assert matmul_fp8(a, b, offsets=offsets, out_dtype=out_dtype, out=out) is out
    status()
    av = host(a, 1)
    for g in range(G):
        lo, hi = cuts[g], cuts[g + 1]
        if hi > lo:
            check_product(out[lo:hi], av[lo:hi], host((b[0][g], b[1][g]), 128), out_dtype)
    outside = torch.cat([out[: cuts[0]], out[cuts[-1]:]])
    assert (outside == 7.0).all()
