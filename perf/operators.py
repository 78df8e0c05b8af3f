"""The 8-bit expert products and the router's balance loss: their measured cases.

Four operators: "quantize" (rows of activations in groups of 128, or 128 x 128
blocks of a weight, to e4m3 codes with fp32 scales), "matmul" (product of two
such operands, dense or grouped by expert), "layer" (the MoE layer's forward
with 8-bit experts) and "balance" (the balance loss of each sequence with the
per-expert counts, and its gradient).  `run` computes them with elementary
torch operations, or through the package where `own` is true.
"""
import math

import torch

own = False

if torch.cuda.is_available():
    DEV = torch.device("cuda")
else:
    DEV = torch.device("cpu")

F8 = torch.float8_e4m3fn
F8_MAX = 448.0
TINY = 2.0 ** -100  # smallest block maximum that sets a scale


def ceil128(n):
    return (n + 127) // 128


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the activations of a small decoding batch, quantised before the experts' products: latency
        dict(name="quantize_decode", op="quantize", G=1, R=16, K=4096, dtype="bf16", block_rows=1, transpose=False),
        # the activations of a prefill batch
        dict(name="quantize_prefill", op="quantize", G=1, R=8192, K=4096, dtype="bf16", block_rows=1, transpose=False),
        # the weights of 128 small experts, once per optimizer step or at load time
        dict(name="quantize_weights", op="quantize", G=128, R=768, K=2048, dtype="bf16", block_rows=128, transpose=False),
        # one token through one wide projection: the weight stream
        dict(name="matmul_token", op="matmul", M=1, N=14336, K=4096, G=0, b_rows=128, out="bf16"),
        # a prefill batch through the same projection: the tensor cores
        dict(name="matmul_prefill", op="matmul", M=8192, N=14336, K=4096, G=0, b_rows=128, out="bf16"),
        # a training batch over 128 small experts, ragged groups
        dict(name="matmul_grouped", op="matmul", M=40961, N=768, K=2048, G=128, b_rows=128, out="bf16"),
        # a weight gradient: both operands in groups along the tokens, odd sizes, fp32 result
        dict(name="matmul_gradient", op="matmul", M=1500, N=1111, K=8200, G=0, b_rows=1, out="fp32"),
        # one token through a whole layer of 8 experts
        dict(name="layer_decode", op="layer", T=1, d=4096, E=8, k=2, d_ff=14336, act="swiglu", gate="renorm", cf=0.0),
        # a training-size batch over 128 small experts with a capacity
        dict(name="layer_fine_grained", op="layer", T=16384, d=2048, E=128, k=4, d_ff=768, act="swiglu", gate="renorm", cf=2.0),
        # a prefill batch through 8 large experts
        dict(name="layer_prefill", op="layer", T=8192, d=4096, E=8, k=2, d_ff=14336, act="swiglu", gate="renorm", cf=0.0),
        # a short padded batch over 8 experts, bf16 logits: latency
        dict(name="balance_short", op="balance", T=300, E=8, k=2, B=5, dtype="bf16", scoring="softmax", mask=True),
        # packed long sequences over 128 experts
        dict(name="balance_long", op="balance", T=131072, E=128, k=4, B=37, dtype="fp32", scoring="softmax", mask=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "layer", "balance"])
    if op == "quantize":
        block_rows = rng.choice([1, 128])
        G = 1 if block_rows == 1 else rng.choice([1, 3, 8])
        K = _log(rng, 100, 14336)
        return dict(op=op, G=G, R=_log(rng, 1, min(16384, 130_000_000 // (G * K))), K=K, dtype=rng.choice(["bf16", "fp32"]),
                    block_rows=block_rows, transpose=rng.random() < 0.4)
    if op == "matmul":
        G = rng.choice([0, 0, rng.randint(2, 128)])
        b_rows = 128 if G else rng.choice([128, 128, 1])
        K = _log(rng, 100, 14336)
        N = _log(rng, 100, min(14336, 200_000_000 // (max(G, 1) * K)))
        M = _log(rng, 1, min(16384, 450_000_000_000 // (K * N)))
        return dict(op=op, M=M, N=N, K=K, G=G, b_rows=b_rows, out=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "layer":
        E = rng.choice([4, 8, 16, 64])
        d = 16 * _log(rng, 8, 256)
        d_ff = 16 * _log(rng, 8, min(512, 40_000_000 // (E * d)))
        return dict(op=op, T=_log(rng, 1, 8192), d=d, E=E, k=rng.choice([1, 2, 4]), d_ff=d_ff, act=rng.choice(["swiglu", "swiglu", "relu"]),
                    gate=rng.choice(["renorm", "switch"]), cf=rng.choice([0.0, 0.0, 1.25, 2.0]))
    E = rng.randint(4, 256)
    T = _log(rng, 1, 16_000_000 // E)
    return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), B=_log(rng, 1, 64), dtype=rng.choice(["bf16", "fp32"]),
                scoring=rng.choice(["softmax", "sigmoid"]), mask=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _codes(shape, gen):
    """Codes of a quantised normal tensor: a block's largest value, about 4 standard deviations, has code 448."""
    out = torch.empty(shape, dtype=F8, device=DEV)
    flat = out.view(-1)
    n, step = flat.numel(), 1 << 27
    for i in range(0, n, step):
        m = min(step, n - i)
        flat[i:i + m] = torch.randn(m, generator=gen, device=DEV).mul_(105.0).clamp_(-F8_MAX, F8_MAX).to(F8)
    return out


def _pitched(codes):
    """The same codes in rows of a multiple of 16 bytes, as the quantiser lays them out."""
    K = codes.shape[-1]
    if K % 16 == 0:
        return codes
    wide = torch.zeros(codes.shape[:-1] + (K + 16 - K % 16,), dtype=F8, device=DEV)
    wide.view(torch.uint8)[..., :K] = codes.view(torch.uint8)
    return wide[..., :K]


def _scales(shape, sigma, gen):
    return torch.rand(shape, generator=gen, device=DEV).add_(0.5).mul_(sigma / 105.0)


def _cuts(total, parts, gen):
    """parts + 1 ascending offsets of ragged parts (some may be empty) of `total` rows, on the CPU."""
    w = torch.rand(parts, generator=gen, device=DEV).double().square().cpu() + 0.02
    cum = (w.cumsum(0) / w.sum() * total).round().long()
    cum[-1] = total
    return torch.cat([torch.zeros(1, dtype=torch.long), cum])


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op == "quantize":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        shape = (case["R"], case["K"]) if case["G"] == 1 else (case["G"], case["R"], case["K"])
        s["x"] = torch.randn(shape, generator=gen, device=DEV).to(dt)
    elif op == "matmul":
        M, N, K, G = case["M"], case["N"], case["K"], case["G"]
        lead = (G,) if G else ()
        sb_rows = N if case["b_rows"] == 1 else ceil128(N)
        s["a"] = (_pitched(_codes((M, K), gen)), _scales((M, ceil128(K)), 1.0, gen))
        s["b"] = (_pitched(_codes(lead + (N, K), gen)), _scales(lead + (sb_rows, ceil128(K)), K ** -0.5, gen))
        s["offsets"] = None
        if G:
            cuts = _cuts(M, G, gen)
            s["offsets"] = cuts.to(torch.int32).to(DEV)
            s["group"] = torch.repeat_interleave(torch.arange(G), cuts[1:] - cuts[:-1]).to(DEV)
            s["most"] = int((cuts[1:] - cuts[:-1]).max())
    elif op == "layer":
        T, d, E, d_ff = case["T"], case["d"], case["E"], case["d_ff"]
        # x on a 2^-6 grid and the router on a 2^-10 grid, so that fp32 logits are exact in any order
        s["x"] = (torch.randn((T, d), generator=gen, device=DEV).clamp_(-3.9, 3.9) * 64).round().div(64).to(torch.bfloat16)
        s["W_r"] = (torch.randn((E, d), generator=gen, device=DEV) * d ** -0.5 * 1024).round().div(1024)
        names = ("W1", "W3", "W2") if case["act"] == "swiglu" else ("W1", "W2")
        s["W3"] = None
        for n in names:
            rows, cols = (d, d_ff) if n == "W2" else (d_ff, d)
            s[n] = (_codes((E, rows, cols), gen), _scales((E, ceil128(rows), ceil128(cols)), cols ** -0.5, gen))
        if own:
            from sparse_mixture_experts_gating_b200 import MoELayer
            s["layer"] = MoELayer(E, case["k"], d, d_ff, act=case["act"], gate_mode=case["gate"], capacity_factor=case["cf"],
                                  dtype=torch.bfloat16)
    else:
        T, E, B = case["T"], case["E"], case["B"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        skew = torch.randn(E, generator=gen, device=DEV)  # some experts are liked better
        s["logits"] = (torch.randn((T, E), generator=gen, device=DEV) + skew).to(dt)
        cuts = _cuts(T, B, gen)
        s["offsets"] = cuts.to(torch.int32).to(DEV)
        s["mask"] = None
        if case["mask"]:  # padding: about one token in eight
            s["mask"] = torch.rand(T, generator=gen, device=DEV) > 0.125
            s["logits"][~s["mask"]] = float("nan")  # whatever stood there
        s["daux"] = torch.rand(B, generator=gen, device=DEV) * 0.02
        s["dz"] = torch.rand(B, generator=gen, device=DEV) * 0.002
    return s


# ------------------------------------------------------------------ one pass
def _quantize(x, block_rows):
    """Codes [.., R, K] and scales [.., ceil(R / block_rows), ceil(K / 128)] of x [.., R, K]."""
    R, K = x.shape[-2:]
    rb = (R + block_rows - 1) // block_rows
    lead = x.shape[:-2]
    f = torch.nn.functional.pad(x.float(), (0, ceil128(K) * 128 - K, 0, rb * block_rows - R))
    f = f.view(lead + (rb, block_rows, ceil128(K), 128))
    a = f.abs().amax(dim=(-3, -1), keepdim=True).clamp_min(TINY)
    most = torch.full_like(a, F8_MAX)  # a tensor: with a number, torch multiplies by a reciprocal, which rounds twice
    codes = (f * (most / a)).to(F8).view(lead + (rb * block_rows, ceil128(K) * 128))
    return codes[..., :R, :K].contiguous(), (a / most).view(lead + (rb, ceil128(K)))


def _values(codes, scales):
    """What codes and scales stand for, in 32 bits; a scale covers 128 rows where there are fewer scales than rows."""
    R, K = codes.shape[-2:]
    if scales.shape[-2] != R:
        scales = scales.repeat_interleave(128, -2)[..., :R, :]
    return codes.float() * scales.repeat_interleave(128, -1)[..., :K]


def _route(logits, k, gate):
    """The k chosen experts of each token (ties to the lower index) and their gates."""
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    idx = order.indices[:, :k]
    if gate == "renorm":
        g = torch.softmax(order.values[:, :k], 1)
    else:
        g = torch.softmax(logits, 1).gather(1, idx)
    return idx, g


def _layer(s):
    c, x = s["case"], s["x"]
    T, E, k = c["T"], c["E"], c["k"]
    logits = x.float() @ s["W_r"].T
    idx, g = _route(logits, k, c["gate"])
    hot = torch.zeros((T, E), dtype=torch.int32, device=x.device).scatter_(1, idx, 1)
    counts = hot.sum(0, dtype=torch.int32)
    cap = math.ceil(c["cf"] * T * k / E) if c["cf"] > 0 else T
    kept = hot.bool() & (hot.cumsum(0) <= cap)  # slots go in token order
    dropped = (hot.sum() - kept.sum()).to(torch.int32).view(1)
    gates = torch.zeros((T, E), device=x.device).scatter_(1, idx, g)
    p = torch.softmax(logits, 1)
    first = torch.zeros(E, device=x.device).index_add_(0, idx[:, 0], torch.ones(T, device=x.device))
    aux = (E * (first / T * p.mean(0)).sum()).view(1)
    z = torch.logsumexp(logits, 1).square().mean().view(1)
    xv = _values(*_quantize(x, 1))
    y = torch.zeros((T, c["d"]), device=x.device)
    for e in range(E):
        rows = kept[:, e].nonzero().view(-1)
        a = xv[rows] @ _values(s["W1"][0][e], s["W1"][1][e]).T
        if s["W3"] is None:
            h = a.clamp_min(0)
        else:
            h = a * torch.sigmoid(a) * (xv[rows] @ _values(s["W3"][0][e], s["W3"][1][e]).T)
        h = _values(*_quantize(h, 1))
        y[rows] += gates[rows, e, None] * (h @ _values(s["W2"][0][e], s["W2"][1][e]).T)
    return {"y": y.to(torch.bfloat16), "counts": counts, "dropped": dropped, "aux": aux, "z": z}


def _balance(s):
    c = s["case"]
    T, E, k, B = c["T"], c["E"], c["k"], c["B"]
    l = s["logits"].float()
    seg = torch.bucketize(torch.arange(T, device=l.device), s["offsets"][1:].long(), right=True)
    live = torch.ones(T, dtype=torch.bool, device=l.device) if s["mask"] is None else s["mask"]
    l = torch.where(live[:, None], l, torch.zeros_like(l))
    w = live.float()[:, None]
    n = torch.zeros(B, dtype=torch.float64, device=l.device).index_add_(0, seg, live.double())
    idx = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :k]
    hot = torch.zeros((T, E), device=l.device).scatter_(1, idx, 1.0) * w
    counts = torch.zeros((B, E), dtype=torch.float64, device=l.device).index_add_(0, seg, hot.double())
    q = torch.softmax(l, 1)
    sg = torch.sigmoid(l)
    p = q if c["scoring"] == "softmax" else sg / sg.sum(1, keepdim=True)
    lse = torch.logsumexp(l, 1)
    m = n.clamp_min(1)
    P = torch.zeros((B, E), dtype=torch.float64, device=l.device).index_add_(0, seg, (p * w).double()) / m[:, None]
    aux = E / (k * m) * (counts * P).sum(1)
    z = torch.zeros(B, dtype=torch.float64, device=l.device).index_add_(0, seg, (lse.double().square() * live)) / m
    ge = (s["daux"] * E / (k * m * m))[:, None] * counts
    ge = ge[seg].float()
    d = p * (ge - (p * ge).sum(1, keepdim=True))
    if c["scoring"] == "sigmoid":
        d = d * (1 - sg)
    d = d + (s["dz"] * 2 / m)[seg].float()[:, None] * lse[:, None] * q
    return {"aux": aux.float(), "z": z.float(), "counts": counts.to(torch.int32), "tokens": n.to(torch.int32), "dlogits": d * w}


def run(s):
    c, op = s["case"], s["op"]
    if own:
        import sparse_mixture_experts_gating_b200 as moe
        if op == "quantize":
            codes, scales = moe.quantize_fp8(s["x"], block_rows=c["block_rows"], transpose=c["transpose"])
            return {"codes": codes, "scales": scales}
        if op == "matmul":
            dt = torch.bfloat16 if c["out"] == "bf16" else torch.float32
            return {"y": moe.matmul_fp8(s["a"], s["b"], offsets=s["offsets"], out_dtype=dt)}
        if op == "layer":
            y, counts, dropped, aux, z = s["layer"].forward_fp8(s["x"], s["W_r"], None, s["W1"], s["W3"], s["W2"])
            return {"y": y, "counts": counts, "dropped": dropped, "aux": aux, "z": z}
        aux, z, counts, tokens = moe.router_balance(s["logits"], c["k"], offsets=s["offsets"], mask=s["mask"], scoring=c["scoring"])
        d = moe.router_balance_backward(s["logits"], counts, tokens, s["daux"], s["dz"], c["k"], offsets=s["offsets"], mask=s["mask"],
                                        scoring=c["scoring"])
        return {"aux": aux, "z": z, "counts": counts, "tokens": tokens, "dlogits": d}
    if op == "quantize":
        x = s["x"].transpose(-2, -1) if c["transpose"] else s["x"]
        codes, scales = _quantize(x, c["block_rows"])
        return {"codes": codes, "scales": scales}
    if op == "matmul":
        dt = torch.bfloat16 if c["out"] == "bf16" else torch.float32
        a, b = _values(*s["a"]), _values(*s["b"])
        if not c["G"]:
            return {"y": (a @ b.T).to(dt)}
        # every group's rows, padded to the largest group
        at = s["offsets"][:-1].long()[:, None] + torch.arange(s["most"], device=a.device)
        y = torch.bmm(a[at.clamp_max(c["M"] - 1)], b.transpose(1, 2))
        row = torch.arange(c["M"], device=a.device) - s["offsets"].long()[s["group"]]
        return {"y": y[s["group"], row].to(dt)}
    if op == "layer":
        return _layer(s)
    return _balance(s)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["G"] * case["R"] * case["K"]
        r, k = (case["K"], case["R"]) if case["transpose"] else (case["R"], case["K"])
        groups = case["G"] * -(-r // case["block_rows"]) * ceil128(k)
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + n + 4 * groups, "flops": 3 * n}
    if op == "matmul":
        M, N, K, G = case["M"], case["N"], case["K"], max(1, case["G"])
        sb = N if case["b_rows"] == 1 else ceil128(N)
        used = min(G, M)  # no more groups than rows have any
        return {"bytes": M * K + used * N * K + 4 * ceil128(K) * (M + used * sb) + M * N * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * M * N * K}
    if op == "layer":
        T, d, E, k, d_ff = (case[n] for n in ("T", "d", "E", "k", "d_ff"))
        nw = 3 if case["act"] == "swiglu" else 2
        cap = math.ceil(case["cf"] * T * k / E) if case["cf"] > 0 else T
        rows = min(T * k, E * cap)
        used = E * (1 - (1 - k / E) ** T)  # experts that are chosen at all, for an even router
        return {"bytes": used * nw * d * d_ff + 4 * E * d + 2 * 2 * T * d, "flops": 2 * nw * rows * d * d_ff + 2 * T * d * E}
    T, E, B = case["T"], case["E"], case["B"]
    return {"bytes": T * E * (2 * (2 if case["dtype"] == "bf16" else 4) + 4) + 12 * B + 4 * B * E, "flops": 20 * T * E}


# ------------------------------------------------------------------ the definitions, in 64 bits
def _quantized64(x, block_rows, axis_groups=128):
    """(codes as 64-bit numbers, scales) of a 64-bit x [R][K]; the definition's own roundings to 32 bits are made one by one."""
    R, K = x.shape
    x = x.to(torch.float32).double()
    rb, kb = -(-R // block_rows), -(-K // axis_groups)
    m = torch.zeros((rb * block_rows, kb * axis_groups), dtype=torch.float64, device=x.device)
    m[:R, :K] = x.abs()
    top = m.reshape(rb, block_rows, kb, axis_groups).permute(0, 2, 1, 3).reshape(rb, kb, -1).max(-1).values
    top = torch.maximum(top, torch.full_like(top, TINY))
    inv = (448.0 / top).float().double()
    at_r = torch.arange(R, device=x.device) // block_rows
    at_k = torch.arange(K, device=x.device) // axis_groups
    v = (x * inv[at_r][:, at_k]).float().double()
    # the nearest e4m3 number: 3 bits after the leading one, exponents from -6 up, ties to even
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -30))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0), (top / 448.0).float()


def _spread64(codes, scales, block_rows):
    at_r = torch.arange(codes.shape[0], device=codes.device) // block_rows
    at_k = torch.arange(codes.shape[1], device=codes.device) // 128
    return codes.double() * scales.double()[at_r][:, at_k]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].reshape(case["G"], case["R"], case["K"])
        both = [_quantized64((m.T if case["transpose"] else m).double(), case["block_rows"]) for m in x]
        codes, scales = torch.stack([b[0] for b in both]), torch.stack([b[1] for b in both])
        return {"codes": codes[0] if case["G"] == 1 else codes, "scales": scales[0] if case["G"] == 1 else scales}
    if op == "matmul":
        M, N, K, G = case["M"], case["N"], case["K"], case["G"]
        a = _spread64(*s["a"], 1)
        if not G:
            return {"y": a @ _spread64(*s["b"], case["b_rows"]).T}
        y = torch.zeros((M, N), dtype=torch.float64, device=a.device)
        cuts = s["offsets"].tolist()
        for g in range(G):
            lo, hi = cuts[g], cuts[g + 1]
            y[lo:hi] = a[lo:hi] @ _spread64(s["b"][0][g], s["b"][1][g], 128).T
        return {"y": y}
    if op == "layer":
        return _layer64(case, s)
    return _balance64(case, s)


def _layer64(case, s):
    T, d, E, k, d_ff = (case[n] for n in ("T", "d", "E", "k", "d_ff"))
    x = s["x"].double()
    h = (x @ s["W_r"].double().T).float().double()  # a logit is rounded once
    rest, idx = h.clone(), []
    for _ in range(k):  # the largest that is left, the first of equals
        best = rest.max(1, keepdim=True).values
        at = (rest == best).double().argmax(1)
        idx.append(at)
        rest.scatter_(1, at[:, None], -math.inf)
    idx = torch.stack(idx, 1)
    full = torch.exp(h - h.max(1, keepdim=True).values)
    full = full / full.sum(1, keepdim=True)
    if case["gate"] == "renorm":
        g = torch.exp(h.gather(1, idx) - h.gather(1, idx[:, :1]))
        g = g / g.sum(1, keepdim=True)
    else:
        g = full.gather(1, idx)
    lse = torch.log(torch.exp(h - h.max(1, keepdim=True).values).sum(1)) + h.max(1).values
    counts = torch.bincount(idx.reshape(-1), minlength=E)
    aux = E * (torch.bincount(idx[:, 0], minlength=E).double() / T * full.mean(0)).sum()
    cap = math.ceil(case["cf"] * T * k / E) if case["cf"] > 0 else T
    xv = _spread64(*_quantized64(x, 1), 1)
    y = torch.zeros((T, d), dtype=torch.float64, device=x.device)
    dropped = 0
    for e in range(E):
        rows, slot = (idx == e).nonzero(as_tuple=True)
        dropped += max(0, rows.numel() - cap)
        rows, slot = rows[:cap], slot[:cap]
        if rows.numel() == 0:
            continue
        a = xv[rows] @ _spread64(s["W1"][0][e], s["W1"][1][e], 128).T
        if case["act"] == "relu":
            hid = torch.relu(a)
        else:
            hid = a / (1 + torch.exp(-a)) * (xv[rows] @ _spread64(s["W3"][0][e], s["W3"][1][e], 128).T)
        hid = _spread64(*_quantized64(hid, 1), 1)
        y[rows] += g[rows, slot][:, None] * (hid @ _spread64(s["W2"][0][e], s["W2"][1][e], 128).T)
    return {"y": y, "counts": counts.to(torch.int32), "dropped": torch.tensor([dropped], dtype=torch.int32), "aux": aux.view(1),
            "z": lse.square().mean().view(1)}


def _balance64(case, s):
    T, E, k, B = case["T"], case["E"], case["k"], case["B"]
    cuts = s["offsets"].tolist()
    aux, z, counts, tokens = [], [], [], []
    dl = torch.zeros((T, E), dtype=torch.float64, device=s["logits"].device)
    for b in range(B):
        at = torch.arange(cuts[b], cuts[b + 1], device=dl.device)
        if s["mask"] is not None:
            at = at[s["mask"][at]]
        n = at.numel()
        tokens.append(n)
        if n == 0:
            counts.append(torch.zeros(E, dtype=torch.int32, device=dl.device))
            aux.append(0.0)
            z.append(0.0)
            continue
        l = s["logits"][at].double()
        rest, c = l.clone(), torch.zeros(E, dtype=torch.float64, device=dl.device)
        for _ in range(k):
            pick = (rest == rest.max(1, keepdim=True).values).double().argmax(1)
            c += torch.bincount(pick, minlength=E)
            rest.scatter_(1, pick[:, None], -math.inf)
        counts.append(c.to(torch.int32))
        top = l.max(1, keepdim=True).values
        ex = torch.exp(l - top)
        q = ex / ex.sum(1, keepdim=True)
        lse = (top + ex.sum(1, keepdim=True).log()).squeeze(1)
        if case["scoring"] == "softmax":
            p, inner = q, 1.0
        else:
            sg = 1 / (1 + torch.exp(-l))
            p, inner = sg / sg.sum(1, keepdim=True), 1 / (1 + torch.exp(l))
        f = c / (k * n)
        aux.append(float(E * (f * p.mean(0)).sum()))
        z.append(float(lse.square().mean()))
        # d aux / d p[t, e] = E f[e] / n
        gp = float(s["daux"][b]) * E * f / n
        dl[at] = p * (gp - (p @ gp)[:, None]) * inner + float(s["dz"][b]) * 2 / n * lse[:, None] * q
    f64 = dict(dtype=torch.float64)
    return {"aux": torch.tensor(aux, **f64), "z": torch.tensor(z, **f64), "counts": torch.stack(counts),
            "tokens": torch.tensor(tokens, dtype=torch.int32), "dlogits": dl}
