"""Host side of the 8-bit operators and the balance loss, without a GPU: the
refusals of the C entries (each before any CUDA call) and of the binding, the
workspace sizes, and the definitions that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_mixture_experts_gating_b200 as moe
from sparse_mixture_experts_gating_b200 import _build, _lib
from tests import _balance as D
from tests import _fp8 as F

INVALID, UNSUPPORTED = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED
P, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4097)


@pytest.fixture(scope="module")
def L():
    _build.build()
    return _lib.lib()


# ------------------------------------------------------------------ refusals
def quant(L, x=P, dtype=1, mats=1, rows=8, K=64, ld=64, block=1, tr=0, codes=P, ldc=64, scales=P):
    return L.moe_quantize_fp8(x, dtype, mats, rows, K, ld, block, tr, codes, ldc, scales, None)


@pytest.mark.parametrize("kw", [dict(mats=-1), dict(rows=-1), dict(K=-1), dict(dtype=2), dict(block=64), dict(ld=63),
                                dict(ldc=63), dict(tr=1, ldc=7), dict(x=None), dict(codes=None), dict(scales=None),
                                dict(x=ODD), dict(scales=ODD)])
def test_quantiser_refuses(L, kw):
    assert quant(L, **kw) == INVALID
    assert L.moe_last_error().decode().startswith("moe_quantize_fp8")


def test_quantiser_limits(L):
    assert quant(L, rows=1 << 31) == UNSUPPORTED
    assert quant(L, mats=1 << 20, rows=1 << 20) == UNSUPPORTED
    for empty in (dict(mats=0), dict(rows=0), dict(K=0)):  # nothing to do, whatever the pointers
        assert quant(L, x=None, codes=None, scales=None, **empty) == _lib.MOE_OK


def mm(L, M=8, N=32, K=64, G=1, a=P, lda=64, sa=P, b=P, ldb=64, sb=P, b_rows=128, off=None, out=P, dt=1, ldo=32,
       ws=P, n=1 << 40):
    return L.moe_matmul_fp8(M, N, K, G, a, lda, sa, b, ldb, sb, b_rows, off, out, dt, ldo, ws, n, None)


@pytest.mark.parametrize("kw", [dict(M=-1), dict(N=0), dict(K=0), dict(G=0), dict(G=257), dict(G=2), dict(dt=2),
                                dict(b_rows=2), dict(lda=48), dict(ldb=63), dict(ldo=31), dict(a=None), dict(sa=None),
                                dict(b=None), dict(sb=None), dict(out=None), dict(a=ODD), dict(b=ODD),
                                dict(lda=72), dict(ldb=65), dict(sa=ODD), dict(sb=ODD), dict(out=ODD), dict(off=ODD),
                                dict(K=1 << 14, lda=1 << 14, ldb=1 << 14, ws=None),
                                dict(K=1 << 14, lda=1 << 14, ldb=1 << 14, n=16),
                                dict(K=1 << 14, lda=1 << 14, ldb=1 << 14, ws=ODD)])
def test_product_refuses(L, kw):
    assert mm(L, **kw) == INVALID
    assert L.moe_last_error().decode().startswith("moe_matmul_fp8")


def test_product_limits(L):
    assert mm(L, M=1 << 31) == UNSUPPORTED
    assert mm(L, N=1 << 25, ldo=1 << 25) == UNSUPPORTED
    assert mm(L, M=1 << 30, N=1 << 20, ldo=1 << 20) == UNSUPPORTED
    assert mm(L, M=0, a=None, out=None) == _lib.MOE_OK
    for args in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0), (1, 1, 1, 257)):
        assert L.moe_matmul_fp8_workspace_bytes(*args) == 0
    assert L.moe_matmul_fp8_workspace_bytes(1, 256, 1 << 14, 1) >= 4 * 256  # one tile: K is cut


def test_product_sizes_near_the_limits(L):
    """No size overflows the plan: it is refused, and needs no workspace, or it is planned."""
    for M, N, K, G in ((1 << 62, 1, 1, 1), (1, (1 << 31) - 1, 1, 1), (1, 1, (1 << 31) - 1, 1), ((1 << 31) - 1, 1, 1, 1),
                       (1 << 30, 1 << 20, 64, 1)):
        assert L.moe_matmul_fp8_workspace_bytes(M, N, K, G) == 0
        assert mm(L, M=M, N=N, K=K, G=G, lda=1 << 31, ldb=1 << 31, ldo=1 << 31, off=P) == UNSUPPORTED
    assert mm(L, ldo=1 << 60) == UNSUPPORTED and mm(L, ldb=1 << 39) == UNSUPPORTED
    # 2^23 k-blocks: at most two waves of ranges are looked at, each with its partial
    n = L.moe_matmul_fp8_workspace_bytes(128, 128, 1 << 30, 1)
    assert 0 < n <= 2 * 148 * 128 * 128 * 4


def balance(L, T=8, E=4, k=2, l=P, dt=0, sc=0, B=1, off=None, mask=None, aux=P, z=P, c=P, t=P, ws=P, n=1 << 40):
    return L.moe_router_balance(T, E, k, l, dt, sc, B, off, mask, aux, z, c, t, ws, n, None)


def backward(L, T=8, E=4, k=2, l=P, dt=0, sc=0, B=1, off=None, mask=None, c=P, t=P, da=P, dz=P, d=P):
    return L.moe_router_balance_backward(T, E, k, l, dt, sc, B, off, mask, c, t, da, dz, d, None)


BAD = [dict(T=-1), dict(B=-1, off=P), dict(E=0), dict(E=257, k=2), dict(k=0), dict(k=5), dict(E=16, k=9), dict(dt=2), dict(sc=2),
       dict(B=2), dict(l=None), dict(l=ODD), dict(off=ODD), dict(c=None), dict(t=None), dict(c=ODD), dict(t=ODD)]


@pytest.mark.parametrize("kw", BAD + [dict(aux=None), dict(z=None), dict(ws=None), dict(n=8), dict(ws=ODD), dict(aux=ODD)])
def test_balance_refuses(L, kw):
    assert balance(L, **kw) == INVALID
    assert L.moe_last_error().decode().startswith("moe_router_balance: ")


@pytest.mark.parametrize("kw", BAD + [dict(d=None), dict(d=ODD), dict(da=ODD), dict(dz=ODD)])
def test_balance_backward_refuses(L, kw):
    assert backward(L, **kw) == INVALID
    assert L.moe_last_error().decode().startswith("moe_router_balance_backward: ")


def test_balance_limits(L):
    assert balance(L, T=1 << 31) == UNSUPPORTED
    assert balance(L, B=0, off=P, aux=None) == _lib.MOE_OK      # no sequences: nothing to write
    assert backward(L, T=0, d=None) == _lib.MOE_OK
    assert L.moe_router_balance_workspace_bytes(-1, 4, 1) == 0 and L.moe_router_balance_workspace_bytes(8, 0, 1) == 0
    assert L.moe_router_balance_workspace_bytes(8, 4, -1) == 0
    assert L.moe_router_balance_workspace_bytes(0, 4, 3) >= 0


@pytest.mark.parametrize("n", [(1 << 31) - 255, (1 << 31) - 1, 1 << 31, 1 << 60])
def test_balance_counts_that_no_31_bit_step_passes(L, n):
    assert balance(L, T=n) == UNSUPPORTED and backward(L, T=n) == UNSUPPORTED
    assert balance(L, B=n, off=P) == UNSUPPORTED and backward(L, B=n, off=P) == UNSUPPORTED
    assert L.moe_router_balance_workspace_bytes(n, 4, 1) == 0 and L.moe_router_balance_workspace_bytes(8, 4, n) == 0


def create(L, *args):
    h = ctypes.c_void_p()
    assert L.moe_create(*args, ctypes.byref(h)) == 0
    return h


def layer(L, h, T=4, x=P, W1=P, S1=P, W3=P, S3=P, W2=P, S2=P, y=P, ws=P, n=1 << 40):
    return L.moe_forward_fp8(h, T, x, P, None, W1, S1, W3, S3, W2, S2, y, P, P, P, P, ws, n, None, None)


def test_layer_refuses(L):
    h = create(L, 8, 2, 64, 64, 1, 1, 0.0, 1)
    assert layer(L, None) == INVALID
    for kw in (dict(T=-1), dict(x=None), dict(W1=None), dict(W2=None), dict(W3=None), dict(S1=None), dict(S3=None), dict(S2=None),
               dict(y=None), dict(S1=ODD), dict(x=ODD), dict(W1=ODD), dict(ws=None), dict(n=16), dict(ws=ctypes.c_void_p(4112))):
        assert layer(L, h, **kw) == INVALID, kw
        assert L.moe_last_error().decode().startswith("moe_forward_fp8")
    L.moe_destroy(h)
    h = create(L, 8, 2, 64, 64, 0, 1, 0.0, 1)  # ReLU takes no W3
    assert layer(L, h) == INVALID
    L.moe_destroy(h)
    for args in ((8, 2, 64, 64, 1, 1, 0.0, 0), (8, 2, 72, 64, 1, 1, 0.0, 1), (8, 2, 64, 72, 1, 1, 0.0, 1)):
        h = create(L, *args)  # an fp32 layer; widths that are no multiple of 16
        assert layer(L, h) == UNSUPPORTED, args
        L.moe_destroy(h)


def test_layer_workspace_never_shrinks_as_T_grows(L):
    shapes = [(8, 2, 4096, 14336, 1, 1, 0.0, 1), (64, 1, 768, 2048, 0, 0, 1.25, 1), (128, 4, 2048, 768, 1, 1, 2.0, 1),
              (4, 2, 32, 64, 0, 1, 0.0, 1), (256, 8, 64, 64, 0, 0, 0.5, 1), (3, 2, 1040, 1168, 1, 1, 0.0, 1),
              (2, 1, 4096, 1024, 1, 0, 0.0, 1)]
    for i, args in enumerate(shapes):
        h = create(L, *args)
        assert L.moe_set_shared_experts(h, i % 2 if args[0] < 256 else 0) == 0
        prev = 0
        for T in list(range(0, 700)) + [1023, 1024, 1025, 2047, 2048, 2049, 4096, 8191, 8192]:
            n = L.moe_workspace_bytes_fp8(h, T)
            assert n >= prev and n % 256 == 0, (args, T)
            prev = n
        assert L.moe_workspace_bytes_fp8(h, -1) == 0
        L.moe_destroy(h)
    assert L.moe_workspace_bytes_fp8(None, 1) == 0


def test_binding_refuses_what_is_not_on_a_gpu():
    x = torch.randn(4, 64)
    c, s = torch.empty(4, 64, dtype=torch.float8_e4m3fn), torch.empty(4, 1)
    for call in (lambda: moe.quantize_fp8(x), lambda: moe.matmul_fp8((c, s), (c, s)), lambda: moe.router_balance(x, 2),
                 lambda: moe.router_balance_backward(x, torch.zeros(1, 64, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), None, None, 2)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_rows_of_reads_every_contiguous_tensor():
    """(matrices, rows, columns, row stride), whatever strides torch keeps for dimensions of one or none."""
    from sparse_mixture_experts_gating_b200.layer import _rows_of
    base = torch.zeros(1 << 16)
    assert _rows_of(base.as_strided((4, 1, 8), (8, 100, 1))) == (4, 1, 8, 8)
    assert _rows_of(base.as_strided((4, 1, 8), (16, 8, 1))) == (4, 1, 8, 16)   # one row of each pitch
    assert _rows_of(base.as_strided((1, 1, 8), (3, 5, 1))) == (1, 1, 8, 16)
    assert _rows_of(base.as_strided((2, 3, 1, 8), (24, 8, 999, 1))) == (6, 1, 8, 8)
    assert _rows_of(base.as_strided((2, 5, 8), (80, 16, 1))) == (2, 5, 8, 16)
    assert _rows_of(base.as_strided((2, 5, 8), (100, 16, 1))) is None           # a gap between matrices
    assert _rows_of(base.as_strided((5, 8), (0, 1))) is None                    # one row, five times
    assert _rows_of(base.as_strided((4, 1, 8), (0, 8, 1))) is None
    assert _rows_of(base.as_strided((5, 8), (8, 2))) is None
    for shape in ((2, 0, 8), (2, 5, 0), (0, 5, 8), (2, 3, 0, 8), (1, 1, 1), (3, 1, 1), (2, 1, 7), (1, 0, 8)):
        t = torch.empty(shape)
        mats, rows, cols, ld = _rows_of(t)
        assert (mats * rows * cols, rows, cols) == (t.numel(), shape[-2], shape[-1]) and ld >= cols
    for shape in ((0, 8), (1, 8), (3, 0), (1, 1)):
        assert _rows_of(torch.empty(shape))[:3] == (1,) + shape


# ------------------------------------------------------------------ the definitions the GPU tests use
def test_e4m3_rounding_is_the_formats():
    """The table and the rounding of tests/_fp8.py against torch's conversion, over
    every code, every midpoint of two and the numbers next to them."""
    codes = np.arange(256, dtype=np.uint8)
    mine = F.decode(codes)
    theirs = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(mine, theirs)
    mid = (F.E4M3[1:] + F.E4M3[:-1]) / 2
    v = np.concatenate([F.E4M3, mid, np.nextafter(mid.astype(np.float32), 0), np.nextafter(mid.astype(np.float32), 500)])
    v = np.concatenate([v, -v]).astype(np.float32)
    np.testing.assert_array_equal(F.round_e4m3(v.astype(np.float64)), torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy())


def test_quantised_blocks_have_their_largest_at_448():
    x = np.random.default_rng(0).standard_normal((130, 300)).astype(np.float32)
    for block_rows in (1, 128):
        codes, scales = F.quantize(x, block_rows)
        assert scales.shape == (-(-130 // block_rows), 3)
        top = np.maximum.reduceat(np.abs(codes), [0, 128, 256], axis=1)
        assert (np.maximum.reduceat(top, np.arange(0, 130, block_rows), axis=0) == 448).all()
        # half a step of 3 bits, or of the smallest number
        err = np.abs(F.values(codes, scales, block_rows) - x)
        assert (err <= np.maximum(np.abs(x) * 2.0 ** -4, F.spread(scales, block_rows, 130, 300) * 2.0 ** -10) * 1.0001).all()


def test_balance_definition_closed_forms():
    E, T, k = 8, 40, 2
    even = np.zeros((T, E))
    for t in range(T):  # every expert is chosen equally often, with nearly even scores
        even[t, [(2 * t) % E, (2 * t + 1) % E]] = 1e-9
    aux, z, counts, tokens = D.loss(even, k, [0, T], None, "softmax")
    assert abs(aux[0] - 1) < 1e-6 and (counts == T * k / E).all() and tokens[0] == T
    assert abs(z[0] - np.log(E) ** 2) < 1e-6
    one = np.zeros((T, E))
    one[:, 3] = 100.0  # all on one expert
    aux, *_ = D.loss(one, 1, [0, T], None, "softmax")
    assert abs(aux[0] - E) < 1e-6
    # sigmoid scores, computed as a softmax of their logarithm
    l = np.random.default_rng(1).standard_normal((5, E))
    s = 1 / (1 + np.exp(-l))
    np.testing.assert_allclose(D.scores(l, "sigmoid"), s / s.sum(1, keepdims=True), rtol=1e-12)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_balance_gradient_matches_differences(scoring):
    T, E, k, cuts = 9, 6, 2, [0, 4, 4, 8]
    l = np.random.default_rng(2).standard_normal((T, E))
    mask = np.ones(T, bool)
    mask[1] = False
    daux, dz = np.array([1.0, 2.0, -0.5]), np.array([0.5, 1.0, 0.25])
    hot = D.choices(l, k)
    d, _ = D.gradient(l, k, cuts, mask, scoring, daux, dz)
    assert not d[1].any() and not d[8].any()
    for t in range(T):
        for e in range(E):
            v = []
            for s in (1e-6, -1e-6):
                x = l.copy()
                x[t, e] += s
                a, z, *_ = D.loss(x, k, cuts, mask, scoring, hot)
                v.append((daux * a).sum() + (dz * z).sum())
            assert abs((v[0] - v[1]) / 2e-6 - d[t, e]) < 1e-7


def test_backward_refuses_a_layer_whose_last_forward_was_8_bit():
    """(The refusal is made before anything is read: tensors on the CPU do.)"""
    layer = moe.MoELayer(4, 2, 64, 64)
    x, W_r, W = torch.zeros(8, 64), torch.zeros(4, 64), torch.zeros(4, 64, 64)
    layer._last = torch.zeros(256, dtype=torch.uint8)  # as forward_fp8 leaves it
    with pytest.raises(ValueError, match="forward_fp8"):
        layer.backward(x, W_r, None, W, W, W, x)


def test_a_cut_of_few_rows_stays_within_one_wave(L):
    """Products of at most 64 rows: the K ranges of all tiles together are no more
    than an SM has one of (148); from 75 to 95 tiles there is one range a tile."""
    for groups in (1, 2, 8):
        for M in (1, 3, 8, 16, 64):
            used = min(groups, M)
            for per_group in range(1, 150):
                N, tiles = per_group * 256, per_group * used
                n = L.moe_matmul_fp8_workspace_bytes(M, N, 4096, groups)
                ranges = max(1, n // (4 * M * N))
                assert n == (0 if ranges == 1 else 4 * M * N * ranges)
                assert ranges == 1 or tiles * ranges <= 148, (groups, M, N)
                assert ranges == 1 or tiles < 75, (groups, M, N)


def test_product_scratch_is_what_the_call_writes(L):
    """Up to eight rows with 128-row scales sum their few ranges in clusters, without
    partials; with a scale a row, or with more rows, the partials need their room."""
    both = L.moe_matmul_fp8_workspace_bytes
    scratch = L.moe_matmul_fp8_scratch_bytes
    for M, N, K in ((1, 14336, 4096), (8, 14336, 4096), (8, 768, 2048)):
        assert scratch(M, N, K, 1, 128) == 0 and scratch(M, N, K, 1, 1) == both(M, N, K, 1) > 0
    for M, N, K in ((9, 14336, 4096), (64, 768, 2048), (8, 32, 1 << 14), (300, 256, 8192)):
        assert scratch(M, N, K, 1, 128) == scratch(M, N, K, 1, 1) == both(M, N, K, 1) > 0
    for args in ((0, 1, 1, 1, 1), (1, 1, 1, 257, 128), (1, 256, 1 << 14, 1, 2), (1 << 62, 1, 1, 1, 1)):
        assert scratch(*args) == 0


@pytest.mark.parametrize("act", [0, 1])
def test_backward_refuses_a_logit_gradient_off_its_elements(L, act):
    h = create(L, 8, 2, 64, 64, act, 1, 0.0, 1)
    n, W3 = 1 << 40, P if act else None
    for dl in (ODD, ctypes.c_void_p(4098)):
        assert L.moe_backward_logits(h, 4, P, P, None, P, W3, P, P, 0.0, 0.0, dl, P, P, None, P, W3, P, P, n, P, n, None) == INVALID
        assert b"dlogits" in L.moe_last_error()
    L.moe_destroy(h)
