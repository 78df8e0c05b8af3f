"""The layer's forward with 8-bit expert weights against its definition.

Routing is the oracle's (bit for bit on dyadic router inputs).  The experts
read x quantised, and quantise the hidden activation: a hidden value that lies
within the fp32 error of a border between two codes may take either, so each
output is allowed what those elements can move it by, and nothing more.
"""
import numpy as np
import pytest
import torch

import oracle as O
from sparse_mixture_experts_gating_b200 import MoEError, MoELayer, matmul_fp8, quantize_fp8, status
from sparse_mixture_experts_gating_b200.workloads import (ACT_RELU, ACT_SWIGLU, DTYPE_BF16, GATE_RENORM, GATE_SWITCH,
                                                          Workload, make_inputs)
from tests import _fp8 as F
from tests._parity import assert_gates_and_losses, assert_routing_equal, layer_for, np32

pytestmark = pytest.mark.gpu

R, S, SW, RN = ACT_RELU, ACT_SWIGLU, GATE_SWITCH, GATE_RENORM
ULP = 2.0 ** -23


def quantized(inp):
    return {k: None if inp[k] is None else quantize_fp8(inp[k], block_rows=128) for k in ("W1", "W3", "W2")}


def run(w, inp, q, layer=None, **kw):
    layer = layer or layer_for(w)
    dbg = layer.debug_buffers(w.T, inp["x"].device)
    y, counts, dropped, aux, z = layer.forward_fp8(inp["x"], inp["W_r"], inp["b_r"], q["W1"], q["W3"], q["W2"],
                                                   debug=dbg, **kw)
    status()
    g = {"y_dev": y, "counts": counts.cpu().numpy(), "dropped": int(dropped.item()), "aux": float(aux.item()),
         "z": float(z.item())}
    g.update({k: t.cpu().numpy() for k, t in dbg.items()})
    bl = layer.balance_losses(w.T).cpu().numpy()
    g.update(aux_all_choices=float(bl[0]), cv_counts=float(bl[1]), cv2_probs=float(bl[2]))
    return g


def host_weight(pair, e):
    return F.values(F.decode(pair[0][e].view(torch.uint8).cpu().numpy()), pair[1][e].cpu().numpy(), 128)


def reference(w, inp, q):
    """(the oracle's routing, y, how far a computed y may be off) in 64 bits."""
    x = np32(inp["x"])
    zero = np.zeros((w.E, w.d_ff, w.d), np.float32)
    o = O.moe_forward(x, np32(inp["W_r"]), np32(inp["b_r"]), zero, zero if w.act == S else None,
                      np.zeros((w.E, w.d, w.d_ff), np.float32), k=w.k, gate_mode=w.gate, act=w.act,
                      capacity_factor=w.capacity_factor)
    xv = F.values(*F.quantize(x), 1)
    y, tol = np.zeros((w.T, w.d)), np.zeros((w.T, w.d))
    for e in range(w.E + w.n_shared):
        if e < w.E:
            rows, slot = np.nonzero((o["idx"] == e) & o["kept"])
            gate = o["gate"][rows, slot][:, None]
        else:
            rows, gate = np.arange(w.T), 1.0
        if rows.size == 0:
            continue
        W1, W2 = host_weight(q["W1"], e), host_weight(q["W2"], e)
        a1, e1 = xv[rows] @ W1.T, F.product_bound(xv[rows], W1)
        if w.act == R:
            h, eh = np.maximum(a1, 0), e1
        else:
            W3 = host_weight(q["W3"], e)
            a3, e3 = xv[rows] @ W3.T, F.product_bound(xv[rows], W3)
            s = a1 / (1 + np.exp(-a1))
            h = s * a3
            # |silu'| < 1.1; the fast exponential and divide are off by a few units and one per unit of |a1|
            eh = 1.1 * np.abs(a3) * e1 + (np.abs(s) + 1.1 * e1) * e3 + np.abs(h) * (8 + 1.2 * np.abs(a1)) * ULP
        codes, scales = F.quantize(h)
        sc = F.spread(scales.astype(np.float64), 1, *h.shape)
        top = F.spread(np.stack([np.abs(h[:, c:c + 128]).max(1) for c in range(0, w.d_ff, 128)], 1), 1, *h.shape)
        etop = F.spread(np.stack([eh[:, c:c + 128].max(1) for c in range(0, w.d_ff, 128)], 1), 1, *h.shape)
        # the value that is rounded, h / scale, and how far a computed one may be off
        v = np.abs(h) / sc
        ev = (eh + np.abs(h) * etop / np.maximum(top, F.TINY)) / sc + 8 * ULP * v
        lo, hi = F.round_e4m3(np.maximum(v - ev, 0)), F.round_e4m3(np.minimum(v + ev, 448))
        move = np.maximum(hi - np.abs(codes), np.abs(codes) - lo) * sc
        hv = codes * sc
        move = move + np.abs(hv) * (etop / np.maximum(top, F.TINY) + 2 * ULP)  # the scale's own error
        yr = hv @ W2.T
        er = F.product_bound(hv, W2) + move @ np.abs(W2).T
        y[rows] += gate * yr
        tol[rows] += np.abs(gate) * er + np.abs(yr) * 2e-6 + np.abs(gate * yr) * 4 * ULP
        if w.T > 64:
            # a gated row may lie in fp16 between the second projection and the sum,
            # 128 columns of it scaled so that the largest is at least 2^14: half a
            # unit of 11 bits, or of the smallest number, 2^-25 of 2^14 at least
            big = np.concatenate([np.repeat(np.abs(yr[:, c:c + 128]).max(1, keepdims=True), min(128, w.d - c), 1)
                                  for c in range(0, w.d, 128)], 1)
            tol[rows] += np.abs(gate * yr) * 2.0 ** -12 * 1.001 + np.abs(gate) * big * 2.0 ** -39
    return o, y, tol + np.abs(y) * 8 * ULP + 1e-30


def check(w, inp, q, g):
    o, y, tol = reference(w, inp, q)
    assert_routing_equal(g, o)
    assert_gates_and_losses(g, o)
    err = np.abs(g["y_f32"].astype(np.float64) - y)
    assert (err <= tol).all(), (err / tol).max()
    # few of the elements that may move do: the layer's usual bound of the mean holds as well
    assert err.sum() <= 2e-3 * np.abs(y).sum(), err.sum() / np.abs(y).sum()
    assert torch.equal(torch.from_numpy(g["y_f32"]).to(torch.bfloat16), g["y_dev"].cpu())


CASES = [
    Workload("one_token", T=1, d=256, E=8, k=2, d_ff=512, act=S, gate=RN, capacity_factor=0.0, dtype=DTYPE_BF16,
             dyadic=True, seed=31),
    Workload("decode", T=20, d=384, E=4, k=2, d_ff=640, act=S, gate=RN, capacity_factor=0.0, dtype=DTYPE_BF16,
             bias="normal", dyadic=True, seed=32),
    Workload("ragged_blocks", T=70, d=208, E=3, k=1, d_ff=176, act=S, gate=SW, capacity_factor=0.0, dtype=DTYPE_BF16,
             dyadic=True, seed=33),
    Workload("relu_drops", T=300, d=128, E=8, k=2, d_ff=272, act=R, gate=SW, capacity_factor=0.75, dtype=DTYPE_BF16,
             bias="normal", dyadic=True, seed=34),
    Workload("large_groups", T=700, d=256, E=4, k=2, d_ff=384, act=S, gate=RN, capacity_factor=1.25,
             dtype=DTYPE_BF16, bias="normal", dyadic=True, seed=35),
    Workload("shared", T=150, d=144, E=5, k=3, d_ff=256, act=R, gate=RN, capacity_factor=1.0, dtype=DTYPE_BF16,
             dyadic=True, seed=36, n_shared=2),
    Workload("tiny_rows", T=33, d=16, E=4, k=4, d_ff=16, act=S, gate=RN, capacity_factor=0.0, dtype=DTYPE_BF16,
             dyadic=True, seed=37),
]


@pytest.mark.parametrize("w", CASES, ids=lambda w: w.name)
def test_layer_matches_its_definition(w):
    inp = make_inputs(w, device="cuda")
    q = quantized(inp)
    check(w, inp, q, run(w, inp, q))


CUT = [  # both projections with K cut: few rows, and whole 128-row tiles; scaled fp16 rows; many experts
    Workload("cut_few_rows", T=3, d=2048, E=4, k=2, d_ff=128, act=S, gate=RN, capacity_factor=0.0, dtype=DTYPE_BF16,
             dyadic=True, seed=41),
    Workload("cut_first", T=100, d=2048, E=2, k=1, d_ff=256, act=S, gate=SW, capacity_factor=0.0, dtype=DTYPE_BF16,
             dyadic=True, seed=42),
    Workload("cut_second", T=100, d=128, E=2, k=2, d_ff=2048, act=R, gate=RN, capacity_factor=0.0, dtype=DTYPE_BF16,
             dyadic=True, seed=43),
    Workload("many_experts", T=260, d=64, E=200, k=8, d_ff=48, act=S, gate=RN, capacity_factor=0.0, dtype=DTYPE_BF16,
             dyadic=True, seed=44),
]


@pytest.mark.parametrize("w", CUT, ids=lambda w: w.name)
def test_cut_products_match_the_definition(w):
    inp = make_inputs(w, device="cuda")
    q = quantized(inp)
    check(w, inp, q, run(w, inp, q))


def test_layer_is_its_operators_in_a_row():
    """One expert that every token takes with gate 1: the layer is quantise, product,
    activation, quantise, product with the standalone operators."""
    w = Workload("one_expert", T=200, d=256, E=1, k=1, d_ff=384, act=S, gate=RN, capacity_factor=0.0, dtype=DTYPE_BF16,
                 dyadic=True, seed=51)
    inp = make_inputs(w, device="cuda")
    q = quantized(inp)
    g = run(w, inp, q)
    xq = quantize_fp8(inp["x"])
    first = [(q[n][0][0], q[n][1][0]) for n in ("W1", "W3", "W2")]
    a1, a3 = (matmul_fp8(xq, p, out_dtype=torch.float32) for p in first[:2])
    h = torch.nn.functional.silu(a1) * a3
    y = matmul_fp8(quantize_fp8(h), first[2], out_dtype=torch.float32)
    status()
    o, ref, tol = reference(w, inp, q)
    assert (np.abs(y.double().cpu().numpy() - ref) <= tol).all()
    assert (np.abs(g["y_f32"] - y.cpu().numpy()) <= 2 * tol).all()


@pytest.mark.parametrize("T", [3, 50, 200])
def test_a_closed_gate_of_far_values_is_zero(T):
    """silu(a) b where a is far below zero and a b past fp32's range: 0, not NaN."""
    w = Workload("far_gate", T=T, d=256, E=2, k=1, d_ff=384, act=S, gate=SW, capacity_factor=0.0, dtype=DTYPE_BF16,
                 dyadic=True, seed=52)
    inp = make_inputs(w, device="cuda")
    inp["x"].fill_(1.0)
    inp["W1"].fill_(-2.0 ** 60)
    inp["W3"].fill_(2.0 ** 60)
    q = quantized(inp)
    y, *_ = layer_for(w).forward_fp8(inp["x"], inp["W_r"], inp["b_r"], q["W1"], q["W3"], q["W2"])
    status()
    assert not y.any()


def test_same_inputs_give_the_same_bits_and_calls_share_nothing():
    w = CASES[4]
    inp = make_inputs(w, device="cuda")
    q = quantized(inp)
    layer = layer_for(w)
    args = (inp["x"], inp["W_r"], inp["b_r"], q["W1"], q["W3"], q["W2"])
    first = layer.forward_fp8(*args)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [layer.forward_fp8(*args, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    status()
    for r in got:
        for a, b in zip(first, r):
            assert torch.equal(a, b)


@pytest.mark.parametrize("w", [CASES[1], CASES[4]], ids=lambda w: w.name)
def test_layer_captured_and_replayed_beside_another_graph(w):
    inp = make_inputs(w, device="cuda")
    q = quantized(inp)
    layer = layer_for(w)
    x = inp["x"].clone()

    def call():
        return layer.forward_fp8(x, inp["W_r"], inp["b_r"], q["W1"], q["W3"], q["W2"])

    call()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, call()))
    x.copy_(inp["x"].flip(0))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for s, (g, _) in zip((s1, s2), graphs):
        with torch.cuda.stream(s):
            for _ in range(4):
                g.replay()
    torch.cuda.synchronize()
    ref = call()
    torch.cuda.synchronize()
    status()
    for _, out in graphs:
        for a, b in zip(out, ref):
            assert torch.equal(a, b)


def test_empty_batch_and_refusals():
    w = CASES[1]
    inp = make_inputs(w, device="cuda")
    q = quantized(inp)
    layer = layer_for(w)
    y, counts, dropped, aux, z = layer.forward_fp8(inp["x"][:0], inp["W_r"], None, q["W1"], q["W3"], q["W2"])
    status()
    assert y.shape == (0, w.d) and not counts.any() and dropped.item() == 0 and aux.item() == 0 and z.item() == 0
    x, W_r = inp["x"], inp["W_r"]
    for call in (lambda: layer.forward_fp8(x.float(), W_r, None, q["W1"], q["W3"], q["W2"]),
                 lambda: layer.forward_fp8(x[:, :128], W_r, None, q["W1"], q["W3"], q["W2"]),
                 lambda: layer.forward_fp8(x, W_r, None, None, q["W3"], q["W2"]),
                 lambda: layer.forward_fp8(x, W_r, None, (q["W1"][0], q["W1"][1][:, :1]), q["W3"], q["W2"]),
                 lambda: layer.forward_fp8(x, W_r, None, q["W2"], q["W3"], q["W2"]),
                 lambda: layer.forward_fp8(x, W_r, None, q["W1"], q["W3"], q["W2"], out=torch.empty_like(x).float())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(MoEError):  # a SwiGLU layer without W3
        layer.forward_fp8(x, W_r, None, q["W1"], None, q["W2"])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=["nan", "inf"])
@pytest.mark.parametrize("T,d,d_ff", [(3, 2048, 128), (50, 256, 384), (100, 2048, 256), (200, 128, 272)],
                         ids=["cut_few_rows", "few_rows", "cut_tiles", "whole_tiles"])
@pytest.mark.parametrize("act", [R, S], ids=["relu", "swiglu"])
def test_a_weight_that_is_not_finite_reaches_the_tokens_of_its_expert(act, T, d, d_ff, bad):
    """A NaN of the first projection stays one under both activations: y is NaN for
    the tokens that the expert serves, and for no other."""
    w = Workload("not_finite", T=T, d=d, E=4, k=2, d_ff=d_ff, act=act, gate=RN, capacity_factor=0.0, dtype=DTYPE_BF16,
                 dyadic=True, seed=53)
    inp = make_inputs(w, device="cuda")
    layer = layer_for(w)
    dbg = layer.debug_buffers(T, "cuda")
    q = quantized(inp)
    layer.forward_fp8(inp["x"], inp["W_r"], inp["b_r"], q["W1"], q["W3"], q["W2"], debug=dbg)
    e = int(dbg["topk_idx"][0, 1])  # an expert that some token takes
    inp["W1"][e, d_ff - 3, d // 2 + 1] = bad
    q = quantized(inp)
    y, *_ = layer.forward_fp8(inp["x"], inp["W_r"], inp["b_r"], q["W1"], q["W3"], q["W2"])
    status()
    served = (dbg["topk_idx"] == e).any(1)
    assert served.any()
    assert torch.equal(torch.isnan(y), served[:, None].expand(T, d))
    assert torch.isfinite(y[~served]).all()


def test_backward_after_an_8_bit_forward():
    """Refused without a workspace; with the one of a forward, and after another
    forward, it gives that forward's gradients."""
    w = CASES[1]
    inp = make_inputs(w, device="cuda")
    q = quantized(inp)
    layer = layer_for(w)
    args = [inp[n] for n in ("x", "W_r", "b_r", "W1", "W3", "W2")]
    dy = torch.ones_like(inp["x"])
    layer.forward(*args)
    want = layer.backward(*args, dy)
    ws = torch.empty(layer.workspace_bytes(w.T), dtype=torch.uint8, device="cuda")
    layer.forward(*args, workspace=ws)
    layer.forward_fp8(inp["x"].flip(0), inp["W_r"], inp["b_r"], q["W1"], q["W3"], q["W2"])
    with pytest.raises(ValueError, match="forward_fp8"):
        layer.backward(*args, dy)
    kept = layer.backward(*args, dy, workspace=ws)
    layer.forward(*args)
    again = layer.backward(*args, dy)
    status()
    for name, g in want.items():
        assert g is None or (torch.equal(g, kept[name]) and torch.equal(g, again[name])), name


@pytest.mark.parametrize("T", [65, 700])
def test_hidden_precision_keeps_the_gated_rows_in_fp32(T):
    """Over 64 tokens whose second projection's K is not cut: the gated rows are
    rounded to fp16 (11 bits) unless MOE_HIDDEN_BF16X2 asks for fp32."""
    w = Workload("gated_rows", T=T, d=256, E=1, k=1, d_ff=128, act=R, gate=RN, capacity_factor=0.0, dtype=DTYPE_BF16,
                 dyadic=True, seed=64)
    inp = make_inputs(w, device="cuda")
    q = quantized(inp)
    y16, y32 = (run(w, inp, q, layer_for(w, hidden))["y_f32"] for hidden in ("auto", "bf16x2"))
    assert not (y16.view(np.uint32) & 0x1FFF).any()            # one row of gate 1: 11 bits of 24
    assert ((y32.view(np.uint32) & 0x1FFF) != 0).mean() > 0.9  # all of them
    # half a unit of 11 bits, or of the smallest number of rows whose largest is at least 2^14
    top = np.abs(y32).reshape(T, -1, 128).max(2).repeat(128, 1)
    assert (np.abs(y16.astype(np.float64) - y32) <= np.abs(y32) * 2.0 ** -11 + top * 2.0 ** -39).all()
    w = CASES[4]  # and against the definition
    inp = make_inputs(w, device="cuda")
    q = quantized(inp)
    check(w, inp, q, run(w, inp, q, layer_for(w, "bf16x2")))


TILES = [  # more than two whole 128-row tiles a CTA: each epilogue's shared memory is written again under its stores
    Workload("swiglu_tiles", T=4096, d=128, E=2, k=1, d_ff=1280, act=S, gate=SW, capacity_factor=0.0, dtype=DTYPE_BF16,
             dyadic=True, seed=61),
    Workload("relu_tiles", T=5120, d=128, E=2, k=1, d_ff=2048, act=R, gate=SW, capacity_factor=0.0, dtype=DTYPE_BF16,
             dyadic=True, seed=62),
    Workload("fp16_row_tiles", T=5120, d=2048, E=2, k=1, d_ff=128, act=R, gate=SW, capacity_factor=0.0,
             dtype=DTYPE_BF16, dyadic=True, seed=63),
]


@pytest.mark.parametrize("w", TILES, ids=lambda w: w.name)
def test_many_whole_tiles_a_cta(w):
    inp = make_inputs(w, device="cuda")
    q = quantized(inp)
    layer = layer_for(w)
    g = run(w, inp, q, layer)
    check(w, inp, q, g)
    for _ in range(8):
        y, *_ = layer.forward_fp8(inp["x"], inp["W_r"], inp["b_r"], q["W1"], q["W3"], q["W2"])
        assert torch.equal(y, g["y_dev"])
    status()


def test_refusals_of_results_and_workspaces_of_the_wrong_form():
    """What the kernels write through is checked like what they read."""
    w = CASES[1]
    inp = make_inputs(w, device="cuda")
    q = quantized(inp)
    layer = layer_for(w)
    i32, f32 = torch.int32, torch.float32

    def call(**kw):
        return layer.forward_fp8(inp["x"], inp["W_r"], inp["b_r"], q["W1"], q["W3"], q["W2"], **kw)

    def stats(n=w.E, counts=i32, losses=f32, device="cuda"):
        return tuple(torch.zeros(m, dtype=t, device=device) for m, t in ((n, counts), (1, i32), (1, losses), (1, f32)))

    dbg = layer.debug_buffers(w.T, "cuda")
    n = layer.workspace_bytes_fp8(w.T)
    for kw in (dict(stats=stats(n=w.E - 1)), dict(stats=stats(counts=torch.int16)), dict(stats=stats(losses=torch.bfloat16)),
               dict(stats=stats(device="cpu")), dict(workspace=torch.empty(n, dtype=torch.uint8)),
               dict(workspace=torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]),
               dict(debug=dict(dbg, y_f32=dbg["y_f32"][1:])), dict(debug=dict(dbg, topk_idx=dbg["topk_idx"].short())),
               dict(debug=dict(dbg, y_f32=dbg["y_f32"].t())),
               dict(debug=dict(dbg, lse_out=dbg["lse_out"].cpu())), dict(debug=dict(logits=dbg["logits_out"]))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(MoEError):  # too small
        call(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    given = stats()
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    got = call(stats=given, workspace=ws, debug=dict(dbg, drop_mask=None))
    assert all(a is b for a, b in zip(got[1:], given))
    for a, b in zip(got, call()):
        assert torch.equal(a, b)
    again = call(debug=dict(logits_in=dbg["logits_out"]))  # its own logits handed in
    assert torch.equal(again[0], got[0])
    status()
