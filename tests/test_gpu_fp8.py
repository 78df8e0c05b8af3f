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


def test_quantiser_takes_contiguous_tensors_of_any_stride():
    base = torch.randn(4096, device="cuda", generator=gen(12))
    for size, stride in (((4, 1, 200), (200, 999, 1)), ((4, 1, 200), (208, 200, 1)), ((2, 3, 1, 8), (24, 8, 77, 1)), ((3, 1, 1), (1, 5, 7))):
        x = base.as_strided(size, stride)
        for kw in (dict(), dict(block_rows=128), dict(transpose=True), dict(block_rows=128, transpose=True)):
            codes, scales = quantize_fp8(x, **kw)
            check_quantized(x, codes, scales, kw.get("block_rows", 1), kw.get("transpose", False))
    for size in ((2, 0, 8), (2, 5, 0), (0, 5, 8)):
        for tr in (False, True):
            codes, scales = quantize_fp8(torch.empty(size, device="cuda"), transpose=tr)
            assert codes.shape == (size if not tr else (size[0], size[2], size[1])) and scales.shape[0] == size[0]


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


@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(2100, 5000, 200), (1900, 5003, 300)])
def test_more_tiles_than_sms(M, N, K, out_dtype, b_rows):
    """Every CTA makes several tiles, whole and partial ones, with aligned rows and without."""
    a, b = operands(M, N, K, None, b_rows, M)
    y = matmul_fp8(a, b, out_dtype=out_dtype)
    status()
    check_product(y, host(a, 1), host(b, b_rows), out_dtype)


@pytest.mark.parametrize("b_rows", [128, 1])
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K,G", [(20, 300, 5000, 3), (150, 260, 9000, 4), (2000, 1030, 260, 40), (40, 500, 130, 256)])
def test_grouped_product_of_long_rows_and_many_groups(M, N, K, G, out_dtype, b_rows):
    """K cut over the CTAs, and groups of every size, with either scale form of b."""
    a, b = operands(M, N, K, G, b_rows, M + G)
    cuts = np.sort(np.random.default_rng(G).integers(0, M + 1, G + 1))
    out = torch.full((M, N), 7.0, dtype=out_dtype, device="cuda")
    matmul_fp8(a, b, offsets=torch.from_numpy(cuts.astype(np.int32)).cuda(), out_dtype=out_dtype, out=out)
    status()
    av, bc, bs = host(a, 1), code_values(b[0]), b[1].cpu().numpy()
    for g in range(G):
        lo, hi = cuts[g], cuts[g + 1]
        if hi > lo:
            check_product(out[lo:hi], av[lo:hi], F.values(bc[g], bs[g], b_rows), out_dtype)
    assert (out[:cuts[0]] == 7).all() and (out[cuts[-1]:] == 7).all()


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K,G", [(1, 14000, 640, None), (5, 4096, 4100, None), (32, 2001, 2048, None), (64, 4096, 1024, None),
                                     (33, 2900, 2048, None), (64, 777, 1500, None), (20, 4100, 2048, 5), (50, 1024, 1152, 9),
                                     (7, 2000, 4096, 30), (8, 3333, 1025, None), (8, 4100, 2048, 3), (2, 14080, 384, 2),
                                     (3, 3585, 5000, None), (1, 256, 4096, None), (8, 130, 7100, None), (4, 1500, 4096, 2),
                                     (2, 100, 15000, None)])
def test_few_rows_whose_sums_meet_in_a_cluster(M, N, K, G, out_dtype):
    """K cut over the CTAs of a cluster, dense and grouped (with empty groups and rows of none)."""
    a, b = operands(M, N, K, G, 128, M + N)
    out = torch.full((M, N), 7.0, dtype=out_dtype, device="cuda")
    if G is None:
        matmul_fp8(a, b, out_dtype=out_dtype, out=out)
        status()
        check_product(out, host(a, 1), host(b, 128), out_dtype)
        return
    cuts = np.sort(np.random.default_rng(M).integers(0, M + 1, G + 1))
    matmul_fp8(a, b, offsets=torch.from_numpy(cuts.astype(np.int32)).cuda(), out_dtype=out_dtype, out=out)
    status()
    av, bc, bs = host(a, 1), code_values(b[0]), b[1].cpu().numpy()
    for g in range(G):
        lo, hi = cuts[g], cuts[g + 1]
        if hi > lo:
            check_product(out[lo:hi], av[lo:hi], F.values(bc[g], bs[g], 128), out_dtype)
    assert (out[:cuts[0]] == 7).all() and (out[cuts[-1]:] == 7).all()


def test_cluster_products_captured_and_on_two_streams():
    a, b = operands(2, 2000, 4096, None, 128, 21)
    a2, _ = operands(2, 2000, 4096, None, 128, 22)
    x = [t.clone() for t in a]
    ref, ref2 = matmul_fp8(a, b), matmul_fp8(a2, b)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = matmul_fp8(x, b)
    for src, want in ((a, ref), (a2, ref2), (a, ref)):
        for t, s in zip(x, src):
            t.view(torch.uint8).copy_(s.view(torch.uint8))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [matmul_fp8(p, b, stream=s) for _ in range(20) for p, s in zip((a, a2), streams)]
    torch.cuda.synchronize()
    status()
    for i, y in enumerate(got):
        assert torch.equal(y, (ref, ref2)[i % 2])


def test_product_writes_its_columns_only():
    """A result with a wider row stride, and one that starts at an odd element."""
    a, b = operands(140, 77, 256, None, 128, 5)
    for dtype in (BF, F32):
        for first in (0, 1, 8):
            big = torch.full((140, 100), 3.0, dtype=dtype, device="cuda")
            out = big[:, first:first + 77]
            matmul_fp8(a, b, out=out, out_dtype=dtype)
            status()
            check_product(out, host(a, 1), host(b, 128), dtype)
            assert (big[:, :first] == 3).all() and (big[:, first + 77:] == 3).all()


def test_product_with_zero_and_tiny_scales_and_not_a_number():
    M, N, K = 40, 130, 256
    x = torch.randn((M, K), device="cuda", generator=gen(1))
    w = torch.randn((N, K), device="cuda", generator=gen(2))
    x[3] = 0.0
    w[:, 128:] = 0.0
    x[5] *= 1e-20
    x[7, 9] = float("nan")
    a, b = quantize_fp8(x), quantize_fp8(w, block_rows=128)
    y = matmul_fp8(a, b, out_dtype=F32)
    status()
    assert not y[3].any() and torch.isnan(y[7]).all()
    keep = [i for i in range(M) if i != 7]
    av = host(a, 1)[keep]
    check_product(y[keep], av, host(b, 128), F32)


@pytest.mark.parametrize("M", [50, 400])
def test_offsets_out_of_order_stay_inside(M):
    """Offsets that do not ascend or leave [0, M] are clamped and made ascending:
    the rows outside the clamped range are left alone, the buffer's end too."""
    G, N, K = 4, 64, 128
    a, b = operands(M, N, K, G, 128, 3)
    big = torch.full((M + 64, N), 5.0, device="cuda")
    for cuts in ([10, 5, 30, 20, 40], [-7, 3, 1000000, 12, 20], [20, 20, 10, 10, 30]):
        big.fill_(5.0)
        matmul_fp8(a, b, offsets=torch.tensor(cuts, dtype=torch.int32, device="cuda"), out=big[:M], out_dtype=F32)
        status()
        run = np.clip(np.maximum.accumulate(np.clip(cuts, 0, M)), 0, M)
        av = host(a, 1)
        for g in range(G):
            if run[g + 1] > run[g]:
                check_product(big[run[g]:run[g + 1]], av[run[g]:run[g + 1]], host((b[0][g], b[1][g]), 128), F32)
        assert (big[:run[0]] == 5).all() and (big[run[-1]:] == 5).all()


def test_the_three_products_of_a_linear_layer():
    """y = x W^T, dx = dy W and dW = dy^T x on the quantiser's plain and transposed
    forms, against the same products of the numbers they stand for."""
    T, d_in, d_out = 300, 200, 330
    x = torch.randn((T, d_in), device="cuda", generator=gen(1)).to(BF)
    W = torch.randn((d_out, d_in), device="cuda", generator=gen(2)).to(BF) * d_in ** -0.5
    dy = torch.randn((T, d_out), device="cuda", generator=gen(3)).to(BF)
    xq, Wq, dyq = quantize_fp8(x), quantize_fp8(W, block_rows=128), quantize_fp8(dy)
    Wt = quantize_fp8(W, block_rows=128, transpose=True)
    xt, dyt = quantize_fp8(x, transpose=True), quantize_fp8(dy, transpose=True)
    # a weight's blocks are square: its transposed form stands for the same numbers
    np.testing.assert_array_equal(host(Wt, 128), host(Wq, 128).T)
    y = matmul_fp8(xq, Wq)
    dx = matmul_fp8(dyq, Wt, out_dtype=F32)
    dW = matmul_fp8(dyt, xt, out_dtype=F32)
    status()
    check_product(y, host(xq, 1), host(Wq, 128), BF)
    check_product(dx, host(dyq, 1), host(Wt, 128), F32)
    check_product(dW, host(dyt, 1), host(xt, 1), F32)
    # and they are the layer's own within the format's rounding: half a step of 3
    # bits, 2^-4, of each operand (2^-8 more for the two together and for bf16 y),
    # or for numbers below the smallest normal code 2^-10 of a scale, 2^-10 / 448 of
    # the block's largest, against at most 330 others: 7.2e-4 of both's largest
    for got, p, q in ((y, x, W), (dx, dy, W.T), (dW, dy.T, x.T)):
        p, q = p.double().cpu().numpy(), q.double().cpu().numpy()
        tol = (2 * 2.0 ** -4 + 2.0 ** -8) * (np.abs(p) @ np.abs(q).T) + 2.0 ** -8 * np.abs(p @ q.T) + 1e-3 * np.abs(p).max() * np.abs(q).max()
        assert (np.abs(got.double().cpu().numpy() - p @ q.T) <= tol).all()


def test_on_another_stream_and_two_at_once():
    a, b = operands(300, 512, 1024, None, 128, 8)
    c, d = operands(1, 1024, 4096, None, 128, 9)
    first, second = matmul_fp8(a, b), matmul_fp8(c, d)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(8):
        got.append((matmul_fp8(a, b, stream=s1), matmul_fp8(c, d, stream=s2)))
    x = torch.randn((64, 512), device="cuda", generator=gen(4))
    s1.wait_stream(torch.cuda.current_stream())
    q = quantize_fp8(x, stream=s1)
    torch.cuda.synchronize()
    status()
    for y, z in got:
        assert torch.equal(y, first) and torch.equal(z, second)
    check_quantized(x, *q, 1, False)


def test_captured_and_replayed_on_new_inputs():
    """quantise -> product -> quantise -> product in a graph, replayed on other inputs."""
    x = torch.randn((130, 512), device="cuda", generator=gen(1)).to(BF)
    w1 = quantize_fp8(torch.randn((1024, 512), device="cuda", generator=gen(2)) * 0.05, block_rows=128)
    w2 = quantize_fp8(torch.randn((256, 1024), device="cuda", generator=gen(3)) * 0.05, block_rows=128)

    def chain(x):
        return matmul_fp8(quantize_fp8(matmul_fp8(quantize_fp8(x), w1)), w2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(x)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = chain(x)
    for seed in (5, 6):
        x.copy_(torch.randn((130, 512), device="cuda", generator=gen(seed)).to(BF))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, chain(x))
    status()


def test_binding_refusals():
    a, b = operands(8, 64, 128, None, 128, 1)
    g3 = operands(8, 64, 128, 2, 128, 1)[1]
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    bad = [
        lambda: quantize_fp8(torch.zeros(4, device="cuda")),
        lambda: quantize_fp8(torch.zeros((4, 4), dtype=torch.float16, device="cuda")),
        lambda: quantize_fp8(torch.zeros((4, 4), device="cuda"), block_rows=64),
        lambda: matmul_fp8(a, g3),
        lambda: matmul_fp8(a, b, offsets=off),
        lambda: matmul_fp8(a, g3, offsets=off.long()),
        lambda: matmul_fp8(a, g3, offsets=off[:2]),
        lambda: matmul_fp8(a, b, out_dtype=torch.float16),
        lambda: matmul_fp8(a, b, out=torch.empty((8, 63), dtype=BF, device="cuda")),
        lambda: matmul_fp8(a, b, out=torch.empty((8, 64), dtype=F32, device="cuda")),
        lambda: matmul_fp8((a[0].view(torch.uint8), a[1]), b),
        lambda: matmul_fp8((a[0], a[1].double()), b),
        lambda: matmul_fp8((a[0], a[1].cpu()), b),
        lambda: matmul_fp8((a[0][:, :64], a[1]), b),
        lambda: matmul_fp8(a, (b[0], b[1][:, :0])),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    from sparse_mixture_experts_gating_b200 import MoEError
    with pytest.raises(MoEError, match="multiples of 16 bytes"):  # codes of another maker, rows 100 bytes apart
        matmul_fp8((torch.zeros((8, 100), dtype=torch.float8_e4m3fn, device="cuda"), torch.ones((8, 1), device="cuda")),
                   (torch.zeros((8, 100), dtype=torch.float8_e4m3fn, device="cuda"), torch.ones((1, 1), device="cuda")))
    empty = matmul_fp8((a[0][:0], a[1][:0]), b)
    assert empty.shape == (0, 64)
    status()


def test_a_product_summed_in_clusters_takes_no_workspace():
    from sparse_mixture_experts_gating_b200._lib import MOE_ERR_INVALID_ARG, MOE_OK, lib
    N, K = 768, 4096
    a = quantize_fp8(torch.randn((16, K), device="cuda", generator=gen(72)))
    w = torch.randn((N, K), device="cuda", generator=gen(73))
    b, br = quantize_fp8(w, block_rows=128), quantize_fp8(w)

    def call(M, pair, b_rows, ws, n):
        out = torch.full((M, N), float("nan"), device="cuda")
        rc = lib().moe_matmul_fp8(M, N, K, 1, a[0].data_ptr(), K, a[1].data_ptr(), pair[0].data_ptr(), K, pair[1].data_ptr(),
                                  b_rows, None, out.data_ptr(), 0, N, ws, n, torch.cuda.current_stream().cuda_stream)
        return rc, out

    for M, pair, b_rows, clustered in ((1, b, 128, True), (8, b, 128, True), (8, br, 1, False), (16, b, 128, False)):
        n = lib().moe_matmul_fp8_scratch_bytes(M, N, K, 1, b_rows)
        assert (n == 0) == clustered and n <= lib().moe_matmul_fp8_workspace_bytes(M, N, K, 1)
        rc, out = call(M, pair, b_rows, None, 0)
        if clustered:
            assert rc == MOE_OK
        else:
            assert rc == MOE_ERR_INVALID_ARG
            ws = torch.empty(n, dtype=torch.uint8, device="cuda")
            rc, out = call(M, pair, b_rows, ws.data_ptr(), n)
            assert rc == MOE_OK
        status()
        assert torch.equal(out, matmul_fp8((a[0][:M], a[1][:M]), pair, out_dtype=F32))


@pytest.mark.parametrize("groups", [0, 3])
def test_a_row_beside_other_rows_and_in_batches_of_other_sizes(groups):
    """The sizes choose how K is cut: among calls of the same sizes a row has the
    same bits whatever stands beside it; among others it stays within the bound."""
    N, K, most = 1024, 4096, 512
    g = gen(71)
    a = quantize_fp8(torch.randn((most, K), device="cuda", generator=g))
    b = quantize_fp8(torch.randn(((groups,) if groups else ()) + (N, K), device="cuda", generator=g), block_rows=128)
    other = quantize_fp8(torch.randn((most, K), device="cuda", generator=g))
    av = F.values(code_values(a[0]), a[1].cpu().numpy(), 1)[:1]
    b0 = (b[0][0], b[1][0]) if groups else b
    bv = F.values(code_values(b0[0]), b0[1].cpu().numpy(), 128)
    exact, bound = av @ bv.T, F.product_bound(av, bv)
    for M in (1, 8, 16, 64, 65, 128, 129, 256, 512):
        # (groups: the row is the first group's first, the others share what is left)
        off = torch.tensor([0, (M + 1) // 2, M, M], dtype=torch.int32, device="cuda") if groups else None
        mixed = tuple(torch.cat([p[:1].view(torch.uint8), o[1:M].view(torch.uint8)]).view(p.dtype).view(M, -1)
                      for p, o in zip(a, other))
        y = matmul_fp8((a[0][:M], a[1][:M]), b, offsets=off, out_dtype=F32)
        z = matmul_fp8(mixed, b, offsets=off, out_dtype=F32)
        status()
        assert torch.equal(y[0], z[0]), M
        if M >= 8:  # the row elsewhere, the groups begun elsewhere
            moved = tuple(torch.roll(p[:M].view(torch.uint8), 3, 0).view(p.dtype) for p in a)
            off3 = torch.tensor([3, M - 2, M - 2, M], dtype=torch.int32, device="cuda") if groups else None
            assert torch.equal(y[0], matmul_fp8(moved, b, offsets=off3, out_dtype=F32)[3]), M
        assert (np.abs(y[:1].double().cpu().numpy() - exact) <= bound).all(), M
