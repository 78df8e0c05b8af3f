"""The balance loss and z-loss of each sequence and their gradient, against the
definition in 64 bits, against differences, and with the layer they serve."""
import numpy as np
import pytest
import torch

from sparse_mixture_experts_gating_b200 import MoELayer, router_balance, router_balance_backward, status
from sparse_mixture_experts_gating_b200.workloads import (ACT_RELU, DTYPE_BF16, GATE_SWITCH, Workload, make_inputs)
from tests import _balance as D
from tests._parity import layer_for

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def make(T, E, seed, dtype, mask, minus_inf):
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = torch.randn((T, E), device="cuda", generator=g) * 2 + torch.randn(E, device="cuda", generator=g)
    l = l.to(dtype)
    if minus_inf and T > 0:
        l[torch.rand((T, E), device="cuda", generator=g) < 0.2] = float("-inf")
        l[T // 2] = float("-inf")                      # a token with no expert left
    m = None
    if mask:
        m = torch.rand(T, device="cuda", generator=g) > 0.3
        l[~m] = float("nan")
        if T > 3:
            m[1], m[3] = False, False
            l[1], l[3] = float("inf"), torch.finfo(dtype).min
    return l, m


def run(l, k, offsets, m, scoring, daux, dz, **kw):
    aux, z, counts, tokens = router_balance(l, k, offsets=offsets, mask=m, scoring=scoring, **kw)
    d = router_balance_backward(l, counts, tokens, daux, dz, k, offsets=offsets, mask=m, scoring=scoring, **kw)
    return aux, z, counts, tokens, d


def check(l, k, cuts, m, scoring, seed=0):
    B = len(cuts) - 1
    g = torch.Generator(device="cuda").manual_seed(seed)
    daux, dz = (torch.randn(B, device="cuda", generator=g) for _ in range(2))
    offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    aux, z, counts, tokens, d = run(l, k, offsets, m, scoring, daux, dz)
    status()
    lh, mh = l.double().cpu().numpy(), None if m is None else m.cpu().numpy().astype(bool)
    ra, rz, rc, rt = D.loss(lh, k, cuts, mh, scoring)
    np.testing.assert_array_equal(tokens.cpu().numpy(), rt)
    np.testing.assert_array_equal(counts.cpu().numpy(), rc)
    fin = lh[np.isfinite(lh)]
    spread = 0.0 if fin.size == 0 else float(min(fin.max(), 60) - max(fin.min(), -60))
    # a score: (16 + 4 spread) units; at most 64 fp32 additions in a tile, the tiles in 64 bits
    e = (80 + 4 * spread) * D.ULP
    assert (np.abs(aux.cpu().numpy() - ra) <= e * np.abs(ra) + 1e-37).all()
    assert (np.abs(z.cpu().numpy() - rz) <= 2 * e * (rz + np.sqrt(rz)) + 1e-12).all()
    rd, tol = D.gradient(lh, k, cuts, mh, scoring, daux.double().cpu().numpy(), dz.double().cpu().numpy())
    err = np.abs(d.cpu().numpy() - rd)
    assert (err <= tol).all(), (err / tol).max()


CASES = [  # T, E, k, cuts
    (1, 1, 1, [0, 1]),
    (1, 8, 2, [0, 1]),
    (7, 3, 3, [0, 3, 3, 7]),
    (33, 8, 2, [0, 1, 32, 33]),
    (100, 9, 3, [0, 0, 50, 100, 100]),
    (64, 16, 4, [5, 20, 60]),                       # tokens of no sequence at both ends
    (300, 31, 8, [0, 31, 64, 65, 128, 300]),
    (513, 60, 6, [0, 512, 513]),
    (257, 64, 1, [0, 257]),
    (200, 100, 4, list(range(0, 201, 5))),          # many short sequences in a tile
    (1000, 128, 8, [0, 999, 1000]),
    (130, 129, 2, [0, 64, 130]),
    (700, 255, 8, [0, 100, 400, 700]),
    (96, 256, 5, [0, 32, 64, 96]),
    (40000, 8, 2, [0, 12345, 40000]),               # several tiles a sequence
    (60000, 33, 4, [3, 30, 59990]),
]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,cuts", CASES)
@pytest.mark.parametrize("dtype,mask,minus_inf", [(F32, False, False), (BF, True, False), (F32, True, True),
                                                  (BF, False, True)])
def test_losses_and_gradient_match_64_bits(T, E, k, cuts, scoring, dtype, mask, minus_inf):
    l, m = make(T, E, T + E, dtype, mask, minus_inf)
    check(l, k, cuts, m, scoring)


def test_far_logits_neither_overflow_nor_vanish():
    """Sigmoid scores far below zero: their ratio is still the exponential's."""
    for shift in (-300.0, 80.0):
        l = torch.randn((50, 12), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) + shift
        aux, z, counts, tokens, d = run(l, 3, None, None, "sigmoid", torch.ones(1, device="cuda"), None)
        lh = l.double().cpu().numpy()
        ra, rz, rc, rt = D.loss(lh, 3, [0, 50], None, "sigmoid")
        rd, tol = D.gradient(lh, 3, [0, 50], None, "sigmoid", [1.0], [0.0])
        # logits of this size carry 2^-16 of absolute rounding into every difference of two
        assert abs(aux.item() - ra[0]) <= 1e-4 * ra[0] and abs(z.item() - rz[0]) <= 1e-5 * rz[0]
        np.testing.assert_array_equal(counts.cpu().numpy(), rc)
        assert torch.isfinite(d).all()
        if shift < 0:  # (above, sigmoid(-l) of the logits leaves nothing)
            scale = np.abs(rd).max()
            assert np.abs(d.cpu().numpy() - rd).max() <= 1e-4 * scale


@pytest.mark.parametrize("E", [5, 20, 64, 200])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_rows_of_the_lowest_value_and_other_far_ones(dtype, scoring, E):
    """Experts masked by a huge finite value, all of a token's among them: their
    scores are 0, or all alike."""
    far = [torch.finfo(dtype).min, -1e30, -1e10, -1e9, 70000.0, 1e10, torch.finfo(dtype).max]
    rows = []
    for v in far:
        whole = torch.full((E,), v)
        one = whole.clone()
        one[E // 2] = 1.0                                  # one other: the lowest lose to it, the largest win
        two = torch.zeros(E)
        two[[1, 3]] = v
        rows += [whole, one, two]
    l = torch.stack(rows).to(dtype).cuda().repeat_interleave(3, 0)   # a sequence of three tokens for each
    B, k = len(rows), 2
    cuts = [3 * b for b in range(B + 1)]
    offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    daux = torch.linspace(-1, 2, B, device="cuda")
    aux, z, counts, tokens, d = run(l, k, offsets, None, scoring, daux, None)
    status()
    lh = l.double().cpu().numpy()
    ra, rz, rc, rt = D.loss(lh, k, cuts, None, scoring)
    np.testing.assert_array_equal(counts.cpu().numpy(), rc)
    np.testing.assert_array_equal(tokens.cpu().numpy(), rt)
    # differences of two logits are 0, or far beyond the exponential's range, or (1 against 0) small
    e = 80 * D.ULP
    assert (np.abs(aux.cpu().numpy() - ra) <= e * np.abs(ra)).all()
    with np.errstate(over="ignore"):
        np.testing.assert_allclose(z.cpu().numpy(), rz.astype(np.float32), rtol=2 * e)  # (infinite beyond fp32)
    rd, _ = D.gradient(lh, k, cuts, None, scoring, daux.double().cpu().numpy(), np.zeros(B))
    bound = np.abs(daux.double().cpu().numpy()).repeat(3)[:, None] * E / 3  # |g| <= E |daux| / n, and so is its mean
    assert (np.abs(d.cpu().numpy() - rd) <= 3 * e * 2 * bound * D.scores(lh, scoring) + 1e-37).all()


def test_ties_go_to_the_lower_index():
    l = torch.zeros((40, 20), device="cuda")
    l[:, 7] = 1.0
    aux, z, counts, tokens = router_balance(l, 3)
    expect = torch.zeros((1, 20), dtype=torch.int32, device="cuda")
    expect[0, [0, 1, 7]] = 40
    assert torch.equal(counts, expect) and tokens.item() == 40


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("E,k", [(E, k) for E in (1, 2, 5, 8, 9, 16, 31, 64, 100, 256) for k in (1, 2, 4, 8) if k <= E])
def test_rows_of_few_values(E, k, dtype):
    """Logits all alike, or of two or three values, with some experts at -inf."""
    g = torch.Generator(device="cuda").manual_seed(E * 10 + k)
    l = torch.randint(0, 3, (240, E), device="cuda", generator=g).float()
    l[:80] = 0.0
    l[40:80, ::2] = -0.0
    l[80:160] = l[80:160].clamp(max=1)
    l[torch.rand((240, E), device="cuda", generator=g) < torch.linspace(0, 0.9, 240, device="cuda")[:, None]] = float("-inf")
    check(l.to(dtype), k, [0, 1, 40, 80, 160, 240], None, "softmax")


def test_nothing_to_count():
    l, _ = make(10, 6, 3, F32, False, False)
    off = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    one = torch.ones(1, device="cuda")
    for logits, m in ((l, torch.zeros(10, dtype=torch.bool, device="cuda")), (torch.full_like(l, float("-inf")), None)):
        aux, z, counts, tokens, d = run(logits, 2, off, m, "softmax", one, one)
        assert aux.item() == 0 and z.item() == 0 and tokens.item() == 0 and not counts.any() and not d.any()
    e = torch.empty((0, 6), device="cuda")
    aux, z, counts, tokens, d = run(e, 2, None, None, "softmax", one, one)
    assert aux.item() == 0 and z.item() == 0 and tokens.item() == 0 and d.shape == (0, 6)
    aux, z, counts, tokens, d = run(l, 2, torch.zeros(1, dtype=torch.int32, device="cuda"), None, "softmax", one[:0], one[:0])
    assert aux.shape == (0,) and counts.shape == (0, 6) and not d.any()


def test_a_logit_that_is_nan_shows():
    l, _ = make(64, 8, 4, F32, False, False)
    off = torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda")
    l[40, 2] = float("nan")
    one = torch.ones(2, device="cuda")
    aux, z, counts, tokens, d = run(l, 2, off, None, "softmax", one, one)
    assert torch.isfinite(aux[0]) and torch.isnan(aux[1]) and torch.isnan(z[1])
    assert torch.isnan(d[40]).all() and torch.isfinite(d[:30]).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_gradient_matches_differences(scoring):
    """Central differences of the definition, the choices held fixed."""
    T, E, k, cuts = 12, 5, 2, [0, 4, 9, 12]
    l, _ = make(T, E, 8, F32, False, False)
    lh = l.double().cpu().numpy()
    hot = D.choices(lh, k)
    daux, dz = np.array([1.0, -0.5, 2.0]), np.array([0.3, 1.0, -0.2])
    *_, d = run(l, k, torch.tensor(cuts, dtype=torch.int32, device="cuda"), None, scoring,
                torch.tensor(daux, dtype=F32, device="cuda"), torch.tensor(dz, dtype=F32, device="cuda"))
    h, num = 1e-5, np.zeros((T, E))
    for t in range(T):
        for e in range(E):
            v = []
            for s in (h, -h):
                x = lh.copy()
                x[t, e] += s
                a, z, *_ = D.loss(x, k, cuts, None, scoring, hot)
                v.append((daux * a).sum() + (dz * z).sum())
            num[t, e] = (v[0] - v[1]) / (2 * h)
    assert np.abs(d.cpu().numpy() - num).max() <= 2e-5 * np.abs(num).max()


def test_same_inputs_give_the_same_bits():
    l, m = make(30000, 100, 5, BF, True, False)
    off = torch.tensor([0, 100, 20000, 30000], dtype=torch.int32, device="cuda")
    g = torch.ones(3, device="cuda")
    first = run(l, 4, off, m, "softmax", g, g)
    for _ in range(3):
        for a, b in zip(first, run(l, 4, off, m, "softmax", g, g)):
            assert torch.equal(a, b)


def test_with_the_layer():
    """One sequence without padding is the layer's own batch: the losses are those
    that it reports, and with one choice a token the gradient through
    backward(dlogits=...) is the one of its own coefficients."""
    w = Workload("balance_layer", T=200, d=64, E=8, k=1, d_ff=128, act=ACT_RELU, gate=GATE_SWITCH, capacity_factor=1.0,
                 dtype=DTYPE_BF16, bias="normal", dyadic=True, seed=77)
    inp = make_inputs(w, device="cuda")
    layer = layer_for(w)
    args = [inp[n] for n in ("x", "W_r", "b_r", "W1", "W3", "W2")]
    dbg = layer.debug_buffers(w.T, "cuda")
    y, counts, dropped, aux, z = layer(*args, debug=dbg)
    logits = dbg["logits_out"]
    a, zz, c, n = router_balance(logits, w.k)
    assert n.item() == w.T and torch.equal(c[0], counts)
    assert abs(a.item() - aux.item()) <= 1e-5 * aux.item() and abs(zz.item() - z.item()) <= 1e-5 * z.item()
    assert abs(a.item() - layer.balance_losses(w.T)[0].item()) <= 1e-5 * aux.item()
    dy = torch.randn((w.T, w.d), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(BF)
    own = layer.backward(*args, dy, aux_coef=0.5, z_coef=0.25)
    dl = router_balance_backward(logits, c, n, torch.full((1,), 0.5, device="cuda"),
                                 torch.full((1,), 0.25, device="cuda"), w.k)
    ours = layer.backward(*args, dy, dlogits=dl)
    without = layer.backward(*args, dy)
    status()
    for name in ("dx", "dW_r", "db_r"):
        scale = own[name].abs().max()
        assert (own[name] - ours[name]).abs().max() <= 2e-5 * scale, name
        assert (own[name] - without[name]).abs().max() > 1e-3 * scale, name  # the losses do reach it
    for name in ("dW1", "dW2"):
        assert torch.equal(own[name], ours[name])


def test_offsets_out_of_order_stay_inside():
    """Offsets that leave [0, T] or do not ascend: whatever the sums are, nothing
    outside the results is written, and a gradient is written for every token."""
    T, E, k = 500, 12, 3
    l, _ = make(T, E, 6, F32, False, False)
    one = torch.ones(3, device="cuda")
    for cuts in ([-5, 100, 50, 900], [400, 300, 200, 100], [0, 2 ** 31 - 1, -2 ** 31, 500]):
        off = torch.tensor(cuts, dtype=torch.int64).to(torch.int32).cuda()
        aux, z, counts, tokens, d = run(l, k, off, None, "softmax", one, one)
        status()
        assert d.shape == (T, E)


def test_captured_and_replayed_and_on_another_stream():
    l, m = make(2000, 40, 9, F32, True, False)
    off = torch.tensor([0, 700, 2000], dtype=torch.int32, device="cuda")
    g2 = torch.ones(2, device="cuda")
    first = run(l, 4, off, m, "sigmoid", g2, g2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(l, 4, off, m, "sigmoid", g2, g2)
    g.replay()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = run(l, 4, off, m, "sigmoid", g2, g2, stream=s)
    torch.cuda.synchronize()
    for a, b, c in zip(first, out, other):
        assert torch.equal(a, b) and torch.equal(a, c)
    l.copy_(l.flip(1))  # (NaN where padding stood, still)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, run(l, 4, off, m, "sigmoid", g2, g2)):
        assert torch.equal(a, b)


def test_binding_refusals():
    l, _ = make(10, 6, 3, F32, False, False)
    off = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    c, t = torch.zeros((1, 6), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for call in (lambda: router_balance(l.half(), 2), lambda: router_balance(l[:, ::2], 2), lambda: router_balance(l[0], 2),
                 lambda: router_balance(l, 2, offsets=off.long()), lambda: router_balance(l, 2, offsets=off[:0]),
                 lambda: router_balance(l, 2, mask=torch.ones(9, dtype=torch.bool, device="cuda")),
                 lambda: router_balance(l, 2, scoring="relu"), lambda: router_balance(l, 2, offsets=off.cpu()),
                 lambda: router_balance_backward(l, c[:, :5], t, None, None, 2),
                 lambda: router_balance_backward(l, c, t, torch.ones(2, device="cuda"), None, 2)):
        with pytest.raises(ValueError):
            call()
    from sparse_mixture_experts_gating_b200 import MoEError
    for k in (0, 7, 9):
        with pytest.raises(MoEError):
            router_balance(l, k)
    d = router_balance_backward(l, c, t, None, None, 2)
    assert not d.any()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_infinite_logits_mark_their_sequence_alone(scoring, dtype):
    """A logit of +inf: z is NaN; aux too where scores are a softmax, while its sigmoid
    is a score of 1.  The other sequences and the other tokens' gradients keep their values."""
    cuts, k = [0, 40, 90, 130], 2
    l, _ = make(130, 24, 8, dtype, False, False)
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    one = torch.ones(3, device="cuda")
    clean = run(l, k, off, None, scoring, one, one)
    t, e = 57, 5
    far = l.clone()
    far[t, e] = float("inf")
    aux, z, counts, tokens, d = run(far, k, off, None, scoring, one, one)
    status()
    for i in (0, 2):
        assert aux[i] == clean[0][i] and z[i] == clean[1][i] and torch.equal(counts[i], clean[2][i])
    assert torch.isnan(z[1]) and torch.equal(tokens, clean[3])
    assert torch.isnan(d[t]).all()
    keep = torch.ones(130, dtype=torch.bool, device="cuda")
    keep[cuts[1]:cuts[2]] = False
    assert torch.equal(d[keep], clean[4][keep])
    keep[cuts[1]:cuts[2]] = True
    keep[t] = False
    assert torch.isfinite(d[keep]).all()
    if scoring == "softmax":
        assert torch.isnan(aux[1])
    else:  # the token's score of that expert is that of a logit past fp32's resolution
        far[t, e] = 100.0
        ra, _, rc, _ = D.loss(far.double().cpu().numpy(), k, cuts, None, scoring)
        assert torch.equal(counts.cpu(), torch.from_numpy(rc).to(torch.int32))
        assert abs(aux[1].item() - ra[1]) <= 300 * D.ULP * ra[1]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_nan_logits_mark_their_sequence_alone(scoring, dtype):
    cuts, k = [0, 40, 90, 130], 3
    l, _ = make(130, 24, 9, dtype, False, False)
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    one = torch.ones(3, device="cuda")
    clean = run(l, k, off, None, scoring, one, one)
    for e in (slice(5, 6), slice(0, 24)):  # one of the token's logits, and all
        for sign in (1.0, -1.0):
            bad = l.clone()
            bad[57, e] = torch.tensor(float("nan"), device="cuda").copysign(torch.tensor(sign, device="cuda")).to(dtype)
            aux, z, counts, tokens, d = run(bad, k, off, None, scoring, one, one)
            status()
            for i in (0, 2):
                assert aux[i] == clean[0][i] and z[i] == clean[1][i] and torch.equal(counts[i], clean[2][i])
            assert torch.isnan(aux[1]) and torch.isnan(z[1]) and torch.isnan(d[57]).all()
            assert 50 * k - k <= counts[1].sum().item() <= 50 * k and torch.equal(tokens, clean[3])
            assert torch.equal(d[:40], clean[4][:40]) and torch.equal(d[90:], clean[4][90:])
            assert torch.isfinite(torch.cat([d[40:57], d[58:90]])).all()


def test_offsets_out_of_order_write_every_result_and_nothing_beside_them():
    """The C entries with every output and the workspace between guards: offsets that
    leave [0, T] or do not ascend write no byte outside, and a gradient for every token."""
    from sparse_mixture_experts_gating_b200._lib import MOE_OK, lib
    T, E, k, B, G = 500, 12, 3, 3, 4096
    l, _ = make(T, E, 6, F32, False, False)
    one = torch.ones(B, device="cuda")
    sane = torch.tensor([0, 150, 320, T], dtype=torch.int32, device="cuda")
    _, _, c0, t0, _ = run(l, k, sane, None, "softmax", one, one)
    n = lib().moe_router_balance_workspace_bytes(T, E, B)
    sizes = dict(aux=4 * B, z=4 * B, counts=4 * B * E, tokens=4 * B, ws=n, d=4 * T * E)
    room = {name: torch.full((G + (size + 15) // 16 * 16 + G,), 0xA5, dtype=torch.uint8, device="cuda")
            for name, size in sizes.items()}
    p = {name: t.data_ptr() + G for name, t in room.items()}
    s = torch.cuda.current_stream().cuda_stream
    for cuts in ([-5, 100, 50, 900], [400, 300, 200, 100], [0, 2 ** 31 - 1, -2 ** 31, 500], [500, 500, 500, 0],
                 [-2 ** 31, -1, 2 ** 31 - 1, 2 ** 31 - 1], [7, 7, 500, 501]):
        for t in room.values():
            t.fill_(0xA5)
        off = torch.tensor(cuts, dtype=torch.int64).to(torch.int32).cuda()
        assert lib().moe_router_balance(T, E, k, l.data_ptr(), 0, 0, B, off.data_ptr(), None, p["aux"], p["z"], p["counts"],
                                        p["tokens"], p["ws"], n, s) == MOE_OK
        assert lib().moe_router_balance_backward(T, E, k, l.data_ptr(), 0, 0, B, off.data_ptr(), None, c0.data_ptr(),
                                                 t0.data_ptr(), one.data_ptr(), one.data_ptr(), p["d"], s) == MOE_OK
        status()
        for name, size in sizes.items():
            t = room[name]
            assert (t[:G] == 0xA5).all() and (t[G + size:] == 0xA5).all(), (name, cuts)
        d = room["d"][G:G + sizes["d"]].view(F32)
        assert torch.isfinite(d).all() and not (d == torch.full((4,), 0xA5, dtype=torch.uint8).view(F32).item()).any(), cuts
        for name in ("aux", "z", "counts", "tokens"):  # (whatever they say, they are written)
            words = room[name][G:G + sizes[name]].view(torch.int32)
            assert not (words == torch.full((4,), 0xA5, dtype=torch.uint8).view(torch.int32).item()).any(), (name, cuts)
