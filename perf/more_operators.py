"""Cases for timing and checking more operators of a training step of the expert layer's block.

Three families, each with a plain torch form in 32 bits, the framework's calls, and the definition in 64 bits:

* ``gated`` / ``gated_grad``: gate and up products by expert with the activation and their product, and the way back from
  the down product's answer to the gate and up rows;
* ``ortho`` / ``muon``: matrices orthogonalised by Newton-Schulz products, and a step of Muon over a stack of them;
* ``layer`` / ``layer_grad``: layer norm with the residual stream's addition, and its gradients.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5                        # layer norm
NS_EPS, NS_STEPS, NS_COEFFICIENTS = 1e-7, 5, (3.4445, -4.7750, 2.0315)
LR, MOMENTUM, DECAY = 2e-4, 0.95, 0.1
BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}


# ---------------------------------------------------------------------------------------------------- cases

def _gated(name, op, P, I, H, E, skew=0.0, dropped=0, keep=True, weighted=True, act="silu"):
    return {"name": name, "op": op, "P": P, "I": I, "H": H, "E": E, "skew": skew, "dropped": dropped, "keep": keep,
            "weighted": weighted, "act": act}


def _matrices(name, op, E, N, K, p="bf16", g="bf16", nesterov=True, clip=False):
    return {"name": name, "op": op, "E": E, "N": N, "K": K, "p": p, "g": g, "nesterov": nesterov, "clip": clip}


def _layer(name, op, T, H, x="bf16", w="f32", add=True, bias=True):
    return {"name": name, "op": op, "T": T, "H": H, "x": x, "w": w, "add": add, "bias": bias}


def listed():
    return [
        # one token of the small-expert decode (top-8 of 256): the eight experts' gate and up weights stream by once
        _gated("gated one token", "gated", 8, 512, 2048, 256, keep=False),
        # gate and up of a skewed training batch (2048 tokens, top-8 of 64), with the rows that the way back needs
        _gated("gated skewed", "gated", 16384, 2048, 7168, 64, skew=1.2),
        # the way back over many small experts (1000 tokens, top-8 of 256)
        _gated("gated gradient small experts", "gated_grad", 8000, 512, 2048, 256, dropped=5),
        # the way back of the skewed batch
        _gated("gated gradient skewed", "gated_grad", 16384, 2048, 7168, 64, skew=1.2),
        # the tiny layer's down projections: launches and latency
        _matrices("orthogonalise tiny layer", "ortho", 8, 256, 128),
        # gate and up of 64 small experts
        _matrices("orthogonalise small experts", "ortho", 64, 1024, 2048),
        # matrices that no tile divides, BF16 parameters, clipped
        _matrices("muon odd matrices", "muon", 8, 1000, 520, p="bf16", g="f32", clip=True),
        # the down projections of 8 large experts, with float32 masters and their copies
        _matrices("muon large experts", "muon", 8, 7168, 2048, p="f32"),
        # before a layer while decoding
        _layer("layer norm decode", "layer", 8, 2048),
        # the same in a prefill
        _layer("layer norm prefill", "layer", 8192, 7168),
        # its gradients in training, joined with the stream's
        _layer("layer norm gradient", "layer_grad", 4096, 7168),
        # a float32 stream of odd sizes without anything to join
        _layer("layer norm gradient f32", "layer_grad", 1000, 1000, x="f32", add=False),
    ]


def _log(rng, low, high, step=1):
    return max(low, min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))) / step) * step))


def draw(rng):
    op = rng.choice(["gated", "gated_grad", "ortho", "muon", "layer", "layer_grad"])
    if op in ("gated", "gated_grad"):
        while True:
            c = _gated("", op, _log(rng, 1, 16384), _log(rng, 16, 2048, 8), _log(rng, 64, 7168, 8), _log(rng, 1, 256),
                       rng.choice([0.0, 0.6, 1.2]), 0, rng.random() < 0.7, rng.random() < 0.7, rng.choice(["silu", "silu", "gelu"]))
            c["dropped"] = rng.choice([0, 0, min(7, c["P"] // 2)])
            longest = c["P"] * float(_popularity(c).max()) + 8
            if c["E"] * c["I"] * c["H"] <= 9e8 and c["E"] * longest * c["I"] * c["H"] <= 1.8e12:
                break
    elif op in ("ortho", "muon"):
        while True:
            c = _matrices("", op, _log(rng, 1, 64), _log(rng, 24, 4096), _log(rng, 24, 4096), rng.choice(["bf16", "f32"]),
                          rng.choice(["bf16", "f32"]), rng.random() < 0.7, rng.random() < 0.5)
            n, k = sorted((c["N"], c["K"]))
            if c["E"] * n * n * k <= 2e11:
                break
        if op == "ortho":
            c["nesterov"] = c["clip"] = False
    else:
        c = _layer("", op, _log(rng, 1, 4096 if op == "layer_grad" else 8192), _log(rng, 64, 7168, 8), rng.choice(["bf16", "f32"]),
                   rng.choice(["bf16", "f32"]), rng.random() < 0.6, rng.random() < 0.7)
        if c["x"] == "f32":
            c["T"] = min(c["T"], 2048)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------------- inputs

def _popularity(case):
    p = np.arange(1, case["E"] + 1, dtype=np.float64) ** -case["skew"]
    return p / p.sum()


def _counts(case, seed):
    """Rows of each expert: the routing of P - dropped pairs with a Zipf popularity."""
    rng = np.random.RandomState(seed % (1 << 31))
    return rng.multinomial(case["P"] - case["dropped"], _popularity(case))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=BF16, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(scale).to(dtype)

    s = {"case": case}
    op = case["op"]
    if op in ("gated", "gated_grad"):
        P, I, H, E = (case[k] for k in "PIHE")
        counts = _counts(case, seed)
        s["longest"] = max(1, int(counts.max()))
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
        # the router's renormalised weights of top-k pairs
        s["row_w"] = torch.rand(P, generator=gen, device="cuda").mul_(0.25).add_(0.02) if case["weighted"] else None
        zeros = lambda *shape, dtype=BF16: torch.zeros(*shape, dtype=dtype, device="cuda")      # noqa: E731
        s["h"] = zeros(P, I) if op == "gated" or case["keep"] else None
        if op == "gated":
            s["x"] = randn(P, H)
            s["w"] = torch.empty(E, 2 * I, H, dtype=BF16, device="cuda").normal_(0.0, 0.02, generator=gen)
            s["a"] = zeros(P, 2 * I) if case["keep"] else None
        else:
            s["dy"] = randn(P, H, scale=0.1)
            s["w"] = torch.empty(E, H, I, dtype=BF16, device="cuda").normal_(0.0, 0.02, generator=gen)
            s["a"] = randn(P, 2 * I, scale=1.5)
            s["da"] = zeros(P, 2 * I)
            s["drow_w"] = zeros(P, dtype=F32) if case["weighted"] else None
    elif op in ("ortho", "muon"):
        shape = (case["E"], case["N"], case["K"])
        s["g"] = randn(*shape, dtype=TYPES[case["g"]], scale=1e-3)
        if op == "ortho":
            s["out"] = torch.empty(shape, dtype=BF16, device="cuda")
        else:
            s["p"] = randn(*shape, dtype=TYPES[case["p"]], scale=0.02)
            s["m"] = randn(*shape, dtype=F32, scale=3e-4)
            s["copy"] = s["p"].to(BF16) if case["p"] == "f32" else None
            s["clip"] = torch.full((1,), 0.5, device="cuda") if case["clip"] else None
    else:
        T, H = case["T"], case["H"]
        xt, wt = TYPES[case["x"]], TYPES[case["w"]]
        s["x"] = (randn(T, H, dtype=F32, scale=1.5) + 0.3).to(xt)     # the stream; for the gradient the one that was normed
        s["w"] = randn(H, dtype=F32, scale=0.2).add_(1.0).to(wt)
        s["bias"] = randn(H, dtype=F32, scale=0.2).to(wt) if case["bias"] else None
        if op == "layer":
            s["b"] = randn(T, H, scale=2.0) if case["add"] else None  # what the layer before answered
        else:
            s["dn"] = randn(T, H, scale=0.1)
            s["ds"] = randn(T, H, dtype=xt, scale=0.1) if case["add"] else None
    return s


# ---------------------------------------------------------------------------------------------------- plain forms

def _by_expert(rows, s):
    """[rows, C] -> [E, longest, C] in 32 bits, zero where an expert has no such row."""
    start, end = s["offsets"][:-1, None].long(), s["offsets"][1:, None].long()
    at = start + torch.arange(s["longest"], device="cuda")
    return torch.where((at < end)[..., None], rows.float()[at.clamp(max=rows.shape[0] - 1)], 0.0)


def _by_row(blocks, s, P):
    """[E, longest, C] -> ([P, C], which rows an expert has), zero in the others."""
    row = torch.arange(P, device="cuda")
    e = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    has = e < blocks.shape[0]
    e = e.clamp(max=blocks.shape[0] - 1)
    at = (row - s["offsets"].long()[e]).clamp(0, s["longest"] - 1)
    return torch.where(has[:, None], blocks[e, at], 0.0), has


_ROOT = math.sqrt(2 / math.pi)


def _activation(z, act):
    """The activation and its derivative."""
    if act == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return z * sig, sig * (1 + z * (1 - sig))
    t = torch.tanh(_ROOT * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * _ROOT * (1 + 3 * 0.044715 * z * z)


def _gated_plain(s):
    case = s["case"]
    w, row_w = s["w"].float(), 1.0 if s["row_w"] is None else s["row_w"][:, None]
    if case["op"] == "gated":
        a, _ = _by_row(torch.bmm(_by_expert(s["x"], s), w.transpose(1, 2)), s, case["P"])
        gate, up = a.split(case["I"], 1)
        out = {"h": (_activation(gate, case["act"])[0] * up * row_w).to(BF16)}
        if case["keep"]:
            out["a"] = a.to(BF16)
        return out
    dh, has = _by_row(torch.bmm(_by_expert(s["dy"], s), w), s, case["P"])
    gate, up = torch.where(has[:, None], s["a"].float(), 0.0).split(case["I"], 1)
    f, df = _activation(gate, case["act"])
    out = {"da": torch.cat([dh * row_w * up * df, dh * row_w * f], 1).to(BF16)}
    if case["keep"]:
        out["h"] = (f * up * row_w).to(BF16)
    if case["weighted"]:
        out["drow_w"] = (dh * f * up).sum(1)
    return out


def _orthogonal(u):
    """Newton-Schulz iterations over the shorter side of each matrix [E, N, K]."""
    a, b, c = NS_COEFFICIENTS
    x = u / u.square().sum((1, 2), keepdim=True).sqrt().clamp(min=NS_EPS)
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    for _ in range(NS_STEPS):
        y = torch.bmm(x, x.transpose(1, 2))
        x = a * x + torch.bmm(b * y + c * torch.bmm(y, y), x)
    return x.transpose(1, 2) if tall else x


def _muon_plain(s):
    case = s["case"]
    g = s["g"].float()
    if s["clip"] is not None:
        g = g * s["clip"]
    m = MOMENTUM * s["m"] + (1 - MOMENTUM) * g
    u = (1 - MOMENTUM) * g + MOMENTUM * m if case["nesterov"] else m
    rate = LR * 0.2 * math.sqrt(max(case["N"], case["K"]))
    p = s["p"].float() * (1 - LR * DECAY) - rate * _orthogonal(u)
    s["m"].copy_(m)
    s["p"].copy_(p)
    if s["copy"] is not None:
        s["copy"].copy_(p)


def _muon_out(s):
    return {k: s[k] for k in ("p", "m", "copy") if s[k] is not None}


def _layer_plain(s):
    case = s["case"]
    w = s["w"].float()
    x = s["x"].float()
    if case["op"] == "layer":
        if s["b"] is not None:
            x = x + s["b"].float()
        d = x - x.mean(1, keepdim=True)
        n = d * torch.rsqrt(d.square().mean(1, keepdim=True) + EPS) * w
        if s["bias"] is not None:
            n = n + s["bias"].float()
        out = {"n": n.to(BF16)}
        if s["b"] is not None:
            out["s"] = x.to(s["x"].dtype)
        return out
    d = x - x.mean(1, keepdim=True)
    r = torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    h, dn = d * r, s["dn"].float()
    dh = dn * w
    dx = r * (dh - dh.mean(1, keepdim=True) - h * (dh * h).mean(1, keepdim=True))
    if s["ds"] is not None:
        dx = dx + s["ds"].float()
    out = {"dx": dx.to(s["x"].dtype), "dw": (dn * h).sum(0)}
    if s["bias"] is not None:
        out["dbias"] = dn.sum(0)
    return out


def _plain(s):
    op = s["case"]["op"]
    if op in ("gated", "gated_grad"):
        return _gated_plain(s)
    if op == "ortho":
        return _orthogonal(s["g"].float()).to(BF16)
    if op == "muon":
        _muon_plain(s)
        return _muon_out(s)
    return _layer_plain(s)


# ---------------------------------------------------------------------------------------------------- the framework's calls

def _own(s):
    import moe_expert_layer_counting_gb300 as M
    case = s["case"]
    op = case["op"]
    if op in ("gated", "gated_grad"):
        if "ws" not in s:
            s["ws"] = torch.empty(M.moe_gated_workspace_size(*(case[k] for k in "PHIE")), dtype=torch.uint8, device="cuda")
        act = {"silu": M.ACT_SILU, "gelu": M.ACT_GELU_TANH}[case["act"]]
        if op == "gated":
            M.moe_gated_forward(s["x"], s["w"], s["offsets"], s["h"], s["ws"], a=s["a"], row_w=s["row_w"], activation=act)
            return {k: s[k] for k in ("h", "a") if s[k] is not None}
        M.moe_gated_dgrad(s["dy"], s["w"], s["offsets"], s["a"], s["da"], s["ws"], h=s["h"], row_w=s["row_w"],
                          drow_w=s["drow_w"], activation=act)
        return {k: s[k] for k in ("da", "h", "drow_w") if s[k] is not None}
    if op == "ortho":
        if "ws" not in s:
            s["ws"] = torch.empty(M.moe_muon_workspace_size(*s["g"].shape), dtype=torch.uint8, device="cuda")
        M.moe_orthogonalize(s["g"], s["out"], s["ws"], steps=NS_STEPS, coefficients=NS_COEFFICIENTS, eps=NS_EPS)
        return s["out"]
    if op == "muon":
        if "muon" not in s:
            s["muon"] = M.Muon([s["p"]], lr=LR, momentum=MOMENTUM, nesterov=case["nesterov"], weight_decay=DECAY,
                               adjust="rms", ns_steps=NS_STEPS, ns_coefficients=NS_COEFFICIENTS, eps=NS_EPS,
                               copies=None if s["copy"] is None else [s["copy"]], state=([s["m"]],))
        s["muon"].step([s["g"]], grad_scale=s["clip"])
        return _muon_out(s)
    if "norm" not in s:
        s["norm"] = M.LayerNorm(s["w"], s["bias"], eps=EPS)
    if op == "layer":
        y, n = s["norm"].forward(s["x"], s["b"])
        return {"n": n} if s["b"] is None else {"n": n, "s": y}
    d = s["norm"].backward(s["x"], s["dn"], s["ds"])
    return {k: v for k, v in d.items() if v is not None}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("gated", "gated_grad"):
        P, I, H, E = case["P"] - case["dropped"], case["I"], case["H"], case["E"]
        hit = int((_counts(case, 0) > 0).sum())
        small = 4 * (E + 1) + 4 * P * case["weighted"]
        if op == "gated":
            return {"bytes": 2 * P * (H + I) + 4 * P * I * case["keep"] + 4 * hit * I * H + small, "flops": 4 * P * I * H}
        return {"bytes": 2 * P * H + 8 * P * I + 2 * P * I * case["keep"] + 2 * hit * I * H + small + 4 * P * case["weighted"],
                "flops": 2 * P * I * H}
    if op in ("ortho", "muon"):
        n, k = sorted((case["N"], case["K"]))
        # x x^T and its square are symmetric: half of each; then their product with x
        flops = case["E"] * NS_STEPS * (n * n * k + n ** 3 + 2 * n * n * k)
        g = 2 if case["g"] == "bf16" else 4
        per = g + 2 if op == "ortho" else g + 8 + (4 if case["p"] == "bf16" else 10)
        return {"bytes": case["E"] * n * k * per, "flops": flops}
    T, H = case["T"], case["H"]
    xb, w = 2 if case["x"] == "bf16" else 4, H * (2 if case["w"] == "bf16" else 4)
    if op == "layer":
        return {"bytes": T * H * (xb + 2 + (2 + xb) * case["add"]) + w * (1 + case["bias"]), "flops": 9 * T * H}
    return {"bytes": T * H * (2 * xb + 2 + xb * case["add"]) + w + 4 * H * (1 + case["bias"]), "flops": 17 * T * H}


# ---------------------------------------------------------------------------------------------------- the definitions in 64 bits

def _exact_gated(s):
    case = s["case"]
    at = s["offsets"].tolist()
    I, w = case["I"], None if s["row_w"] is None else s["row_w"].double()

    def act(z):
        return z * torch.sigmoid(z) if case["act"] == "silu" else 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))

    out = {k: torch.zeros(s[k].shape, dtype=torch.float64, device="cuda") for k in ("h", "a", "da", "drow_w") if s.get(k) is not None}
    if case["op"] == "gated_grad":
        out.pop("a")
    for e in range(case["E"]):
        r = slice(at[e], at[e + 1])
        if at[e] == at[e + 1]:
            continue
        if case["op"] == "gated":
            a = s["x"][r].double() @ s["w"][e].double().T
            h = act(a[:, :I]) * a[:, I:]
            out["h"][r] = h if w is None else h * w[r, None]
            if "a" in out:
                out["a"][r] = a
            continue
        # torch's own differentiation of dy . (h W^T)
        a = s["a"][r].double().requires_grad_()
        rw = (torch.ones(at[e + 1] - at[e], dtype=torch.float64, device="cuda") if w is None else w[r].clone()).requires_grad_()
        h = act(a[:, :I]) * a[:, I:] * rw[:, None]
        da, drw = torch.autograd.grad(h, [a, rw], s["dy"][r].double() @ s["w"][e].double())
        out["da"][r] = da
        if "h" in out:
            out["h"][r] = h.detach()
        if "drow_w" in out:
            out["drow_w"][r] = drw
    return out


def _exact_orthogonal(u):
    """One matrix in 64 bits: the polynomial of its Gram matrix over the shorter side, from the right where that is the columns."""
    a, b, c = NS_COEFFICIENTS
    norm = math.sqrt(float((u * u).sum()))
    x = u / max(norm, NS_EPS)
    n = min(x.shape)
    one = torch.eye(n, dtype=torch.float64, device=u.device)
    for _ in range(NS_STEPS):
        gram = x @ x.T if x.shape[0] == n else x.T @ x
        q = a * one + b * gram + c * gram @ gram
        x = q @ x if x.shape[0] == n else x @ q
    return x


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("gated", "gated_grad"):
        return _exact_gated(s)
    if op in ("ortho", "muon"):
        g = s["g"].double()
        if op == "ortho":
            return torch.stack([_exact_orthogonal(u) for u in g])
        if s["clip"] is not None:
            g = g * s["clip"].double()
        m = s["m"].double() + (1 - MOMENTUM) * (g - s["m"].double())
        u = m + (1 - MOMENTUM) * (g - m) if case["nesterov"] else m
        o = torch.stack([_exact_orthogonal(v) for v in u])
        p = s["p"].double()
        p = p - LR * DECAY * p - LR * 0.2 * max(case["N"], case["K"]) ** 0.5 * o
        out = {"p": p, "m": m}
        if s["copy"] is not None:
            out["copy"] = p
        return out
    # the gradients are those of torch's own differentiation of the definition
    x, w = s["x"].double().requires_grad_(), s["w"].double().requires_grad_()
    bias = torch.zeros_like(w) if s["bias"] is None else s["bias"].double().requires_grad_()
    stream = x if s.get("b") is None else x + s["b"].double()
    mean = stream.sum(1, keepdim=True) / case["H"]
    var = (stream - mean).pow(2).sum(1, keepdim=True) / case["H"]
    n = (stream - mean) / torch.sqrt(var + EPS) * w + bias
    if op == "layer":
        out = {"n": n.detach()}
        if s["b"] is not None:
            out["s"] = stream.detach()
        return out
    loss = (n * s["dn"].double()).sum()
    if s["ds"] is not None:
        loss = loss + (stream * s["ds"].double()).sum()
    grads = torch.autograd.grad(loss, [x, w] + ([bias] if s["bias"] is not None else []))
    return dict(zip(("dx", "dw", "dbias"), grads))
