"""Cases for timing and checking the operators of a training step of the expert layer.

Three families, each with a plain torch form in 32 bits, the framework's calls, and the definition in 64 bits:

* ``forward`` / ``rows`` / ``weights``: products grouped by expert with ragged sizes, and their two gradients;
* ``norm`` / ``norm_grad``: the norms before and after the layer with gate and residual scale, and their gradient;
* ``adamw``: one AdamW step over many tensors, with states in 32 or in 8 bits.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
SCALE = 0.75                      # residual scale of the norm cases
LR, BETA1, BETA2, ADAM_EPS, DECAY = 1e-3, 0.9, 0.95, 1e-8, 0.1
BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}


# ---------------------------------------------------------------------------------------------------- cases

def _grouped(name, op, P, N, K, E, skew=0.0, dropped=0, out="bf16"):
    return {"name": name, "op": op, "P": P, "N": N, "K": K, "E": E, "skew": skew, "dropped": dropped, "out": out}


def _norm(name, op, T, H, x="bf16", w="f32", gate="none", sigmoid=False, post=True, pre=True):
    return {"name": name, "op": op, "T": T, "H": H, "x": x, "w": w, "gate": gate, "sigmoid": sigmoid, "post": post,
            "pre": pre}


def _adamw(name, bits, E, H, I, p="f32", g="bf16", clip=True, odd=0):
    return {"name": name, "op": "adamw", "bits": bits, "E": E, "H": H, "I": I, "p": p, "g": g, "clip": clip, "odd": odd}


def listed():
    return [
        # the gate and up rows of the tiny layer (64 tokens, top-2 of 8): a call whose time is its launch
        _grouped("products, tiny layer", "forward", 128, 256, 256, 8),
        # gate and up of the small-expert decode (8 tokens, top-8 of 256): the touched experts' weights stream by once
        _grouped("products, decode", "forward", 64, 1024, 2048, 256),
        # gate and up of a skewed prefill (2048 tokens, top-8 of 64): the hottest expert has 4000 rows, the coldest a few
        _grouped("products, skewed prefill", "forward", 16384, 4096, 7168, 64, skew=1.2),
        # the gradient of the down product's rows for the same tokens
        _grouped("gradient of rows, skewed", "rows", 16384, 7168, 2048, 64, skew=1.2),
        # the gradient of gate and up's weights, 512 tokens, top-8 of 32, a few pairs dropped
        _grouped("gradient of weights", "weights", 4096, 4096, 7168, 32, dropped=5),
        # the same for many small experts, held in 32 bits for accumulation over micro-batches
        _grouped("gradient of weights, f32", "weights", 8000, 1024, 2048, 256, out="f32"),
        # between two layers while decoding: norm after, sigmoid gate of each token, norm before the next
        _norm("norms, decode", "norm", 8, 2048, gate="token", sigmoid=True),
        # the same in a prefill, with a gate of each channel
        _norm("norms, prefill", "norm", 8192, 7168, gate="channel"),
        # its gradient in training
        _norm("norms, gradient", "norm_grad", 4096, 7168, gate="channel"),
        # the tiny layer's 19 tensors
        _adamw("adamw, tiny layer", 32, 8, 256, 128),
        # 64 small experts, each two tensors, the router and the norms
        _adamw("adamw, 32-bit states", 32, 64, 2048, 512),
        # 8 large experts, states in 8 bits
        _adamw("adamw, 8-bit states", 8, 8, 7168, 2048),
    ]


def _log(rng, low, high, step=1):
    return max(low, min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))) / step) * step))


def draw(rng):
    op = rng.choice(["forward", "rows", "weights", "norm", "norm_grad", "adamw"])
    if op in ("forward", "rows", "weights"):
        while True:
            c = _grouped("", op, _log(rng, 1, 16384), _log(rng, 64, 7168, 8), _log(rng, 64, 7168, 8), _log(rng, 1, 256),
                         rng.choice([0.0, 0.6, 1.2]), 0, rng.choice(["bf16", "f32"]) if op == "weights" else "bf16")
            c["dropped"] = rng.choice([0, 0, min(7, c["P"] // 2)])
            longest = c["P"] * float(_popularity(c).max()) + 8
            if c["E"] * c["N"] * c["K"] <= 1e9 and c["E"] * longest * c["N"] * c["K"] <= 2e12:
                break
    elif op in ("norm", "norm_grad"):
        c = _norm("", op, _log(rng, 1, 4096 if op == "norm_grad" else 8192), _log(rng, 64, 7168, 8), rng.choice(["bf16", "f32"]),
                  rng.choice(["bf16", "f32"]), rng.choice(["none", "token", "channel", "full"]), rng.random() < 0.5,
                  rng.random() < 0.7, rng.random() < 0.7)
        if op == "norm_grad" and c["x"] == "f32":
            c["T"] = min(c["T"], 2048)
    else:
        c = _adamw("", rng.choice([8, 32]), _log(rng, 1, 48), _log(rng, 64, 2048, 8), _log(rng, 32, 512, 8),
                   rng.choice(["f32", "f32", "bf16"]), rng.choice(["bf16", "f32"]), rng.random() < 0.5, rng.randrange(1, 32))
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


def _tensor_sizes(case):
    """Values of each tensor: two for each expert, the router, two norms, and (odd) one of a size that nothing divides."""
    E, H, I = case["E"], case["H"], case["I"]
    return [2 * I * H] * E + [H * I] * E + [E * H, H, H] + ([1000 * case["odd"] + 1] if case["odd"] else [])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=BF16, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(scale).to(dtype)

    s = {"case": case}
    op = case["op"]
    if op in ("forward", "rows", "weights"):
        P, N, K, E = (case[k] for k in "PNKE")
        counts = _counts(case, seed)
        s["longest"] = max(1, int(counts.max()))
        s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
        if op != "rows":
            s["x"] = randn(P, K)
        if op != "forward":
            s["dy"] = randn(P, N, scale=0.1)
        if op != "weights":
            s["w"] = torch.empty(E, N, K, dtype=BF16, device="cuda").normal_(0.0, 0.02, generator=gen)
            s["out"] = torch.zeros(P, N if op == "forward" else K, dtype=BF16, device="cuda")
        else:
            s["out"] = torch.zeros(E, N, K, dtype=TYPES[case["out"]], device="cuda")
    elif op in ("norm", "norm_grad"):
        T, H = case["T"], case["H"]
        xt, wt = TYPES[case["x"]], TYPES[case["w"]]
        shape = {"none": None, "token": (T, 1), "channel": (1, H), "full": (T, H)}[case["gate"]]
        s["b"] = randn(T, H, scale=2.0)
        s["gate"] = None if shape is None else randn(*shape, dtype=BF16 if case["gate"] == "full" else F32)
        s["w_post"] = randn(H, dtype=F32, scale=0.2).add_(1.0).to(wt) if case["post"] else None
        s["w_pre"] = randn(H, dtype=F32, scale=0.2).add_(1.0).to(wt) if case["pre"] else None
        s["x"] = randn(T, H, dtype=xt, scale=1.5)            # the stream before the layer; for the gradient the one after it
        if op == "norm_grad":
            s["dy"] = randn(T, H, dtype=xt, scale=0.1)
            s["dn"] = randn(T, H, scale=0.1) if case["pre"] else None
    else:
        sizes = _tensor_sizes(case)
        starts = np.concatenate([[0], np.cumsum([-(-n // 32) * 32 for n in sizes])])
        total = int(starts[-1])
        s["sizes"], s["starts"], s["step"] = sizes, starts[:-1].tolist(), 1000
        live = torch.ones(total, device="cuda")
        for n, a, b in zip(sizes, starts[:-1], starts[1:]):
            live[int(a) + n:int(b)] = 0
        s["p"] = (randn(total, dtype=F32, scale=0.02) * live).to(TYPES[case["p"]])
        s["g"] = (randn(total, dtype=F32, scale=1e-3) * live).to(TYPES[case["g"]])
        m = randn(total, dtype=F32, scale=3e-4) * live
        r = randn(total, dtype=F32, scale=1e-3).abs_() * live
        if case["p"] == "f32":
            s["copy"] = s["p"].to(BF16)
        if case["bits"] == 32:
            s["m"], s["v"] = m, r * r
        else:
            s["m"], s["m_scale"] = _to_8_bits(m, False)
            s["v"], s["v_scale"] = _to_8_bits(r, True)
        s["clip"] = torch.full((1,), 0.5, device="cuda") if case["clip"] else None
    return s


# ---------------------------------------------------------------------------------------------------- plain forms

def _by_expert(rows, s):
    """[rows, C] -> [E, longest, C] in 32 bits, zero where an expert has no such row."""
    start, end = s["offsets"][:-1, None].long(), s["offsets"][1:, None].long()
    at = start + torch.arange(s["longest"], device="cuda")
    return torch.where((at < end)[..., None], rows.float()[at.clamp(max=rows.shape[0] - 1)], 0.0)


def _by_row(blocks, s, like):
    """[E, longest, C] -> [P, C], zero in the rows that no expert has."""
    row = torch.arange(like.shape[0], device="cuda")
    e = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    has = e < blocks.shape[0]
    e = e.clamp(max=blocks.shape[0] - 1)
    at = (row - s["offsets"].long()[e]).clamp(0, s["longest"] - 1)
    return torch.where(has[:, None], blocks[e, at], 0.0).to(like.dtype)


def _norm_of(v, w):
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    return r, v * r if w is None else v * r * w


def _up(t, dtype=F32):
    return None if t is None else t.to(dtype)


def _norm_forward(case, x, b, gate, w_post, w_pre):
    u = _norm_of(b, w_post)[1] if case["post"] else b
    if gate is not None:
        u = (torch.sigmoid(gate) if case["sigmoid"] else gate) * u
    y = SCALE * x + u
    return y, _norm_of(y, w_pre)[1] if case["pre"] else None


def _norm_back(v, w, d):
    """Gradients of v * rsqrt(mean v^2 + eps) * w in v and w."""
    r, _ = _norm_of(v, w)
    h = v * r
    dh = d * w
    return r * (dh - h * (dh * h).mean(-1, keepdim=True)), (d * h).sum(0)


def _norm_backward(case, y, b, gate, w_post, w_pre, dy, dn):
    out = {}
    d = dy
    if case["pre"]:
        more, out["dw_pre"] = _norm_back(y, w_pre, dn)
        d = d + more
    out["dx"] = SCALE * d
    du = d
    if gate is not None:
        u = _norm_of(b, w_post)[1] if case["post"] else b
        g = torch.sigmoid(gate) if case["sigmoid"] else gate
        dg = d * u
        if case["gate"] == "token":
            dg = dg.sum(1, keepdim=True)
        elif case["gate"] == "channel":
            dg = dg.sum(0, keepdim=True)
        out["dgate"] = dg * g * (1 - g) if case["sigmoid"] else dg
        du = g * d
    out["db"] = du
    if case["post"]:
        out["db"], out["dw_post"] = _norm_back(b, w_post, du)
    return out


def _to_8_bits(v, positive):
    """E4M3 codes and the bytes of a power of two for each 32 values: the smallest with amax <= 448 * 2^e. A value of `positive`
    that is not zero takes the smallest code at least."""
    v = v.view(-1, 32)
    amax = v.abs().amax(1)
    f, e = torch.frexp(amax)                                    # amax = f * 2^e, f in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e - 9 + (f > 0.875).int(), -127).clamp(-127, 127)
    scaled = torch.ldexp(v, -e[:, None].float().clamp(max=126).int())
    if positive:
        scaled = torch.where(v > 0, scaled.clamp(min=2.0 ** -9), scaled)
    return scaled.to(torch.float8_e4m3fn).view(torch.uint8).view(-1), (e + 127).to(torch.uint8)


def _from_8_bits(code, byte):
    return torch.ldexp(code.view(torch.float8_e4m3fn).float().view(-1, 32), byte[:, None].int() - 127).view(-1)


def _adamw_plain(s):
    case = s["case"]
    s["step"] += 1
    g = s["g"].float()
    if s["clip"] is not None:
        g = g * s["clip"]
    small = case["bits"] == 8
    m = _from_8_bits(s["m"], s["m_scale"]) if small else s["m"]
    v = _from_8_bits(s["v"], s["v_scale"]).square() if small else s["v"]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    root = torch.sqrt(v)
    c1, c2 = 1 - BETA1 ** s["step"], 1 - BETA2 ** s["step"]
    p = s["p"].float() * (1 - LR * DECAY) - (LR / c1) * (m / (root * (1 / math.sqrt(c2)) + ADAM_EPS))
    s["p"].copy_(p)
    if "copy" in s:
        s["copy"].copy_(p)
    if small:
        for name, value in (("m", m), ("v", root)):
            code, byte = _to_8_bits(value, name == "v")
            s[name].copy_(code)
            s[name + "_scale"].copy_(byte)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)


def _adamw_out(s):
    out = {k: s[k] for k in ("p", "copy", "m_scale", "v_scale") if k in s}
    for k in ("m", "v"):
        out[k] = s[k].view(torch.float8_e4m3fn) if s["case"]["bits"] == 8 else s[k]
    return out


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "forward":
        return _by_row(torch.bmm(_by_expert(s["x"], s), s["w"].float().transpose(1, 2)), s, s["out"])
    if op == "rows":
        return _by_row(torch.bmm(_by_expert(s["dy"], s), s["w"].float()), s, s["out"])
    if op == "weights":
        return torch.bmm(_by_expert(s["dy"], s).transpose(1, 2), _by_expert(s["x"], s)).to(TYPES[case["out"]])
    if op == "norm":
        y, n = _norm_forward(case, s["x"].float(), s["b"].float(), _up(s["gate"]), _up(s["w_post"]), _up(s["w_pre"]))
        out = {"y": y.to(s["x"].dtype)}
        if n is not None:
            out["n"] = n.to(BF16)
        return out
    if op == "norm_grad":
        out = _norm_backward(case, s["x"].float(), s["b"].float(), _up(s["gate"]), _up(s["w_post"]), _up(s["w_pre"]),
                             s["dy"].float(), _up(s["dn"]))
        out["dx"] = out["dx"].to(s["x"].dtype)
        out["db"] = out["db"].to(BF16)
        if "dgate" in out:
            out["dgate"] = out["dgate"].to(s["gate"].dtype)
        return out
    _adamw_plain(s)
    return _adamw_out(s)


# ---------------------------------------------------------------------------------------------------- the framework's calls

def _own(s):
    import moe_expert_layer_counting_gb300 as M
    case = s["case"]
    op = case["op"]
    if op in ("forward", "rows", "weights"):
        if "ws" not in s:
            s["ws"] = torch.empty(M.moe_grouped_workspace_size(*(case[k] for k in "PNKE")), dtype=torch.uint8, device="cuda")
        if op == "forward":
            M.moe_grouped_forward(s["x"], s["w"], s["offsets"], s["out"], s["ws"])
        elif op == "rows":
            M.moe_grouped_dgrad(s["dy"], s["w"], s["offsets"], s["out"], s["ws"])
        else:
            M.moe_grouped_wgrad(s["dy"], s["x"], s["offsets"], s["out"], s["ws"])
        return s["out"]
    if op in ("norm", "norm_grad") and "norm" not in s:
        s["norm"] = M.BlockNorm(s["w_post"], s["w_pre"], residual_scale=SCALE, eps=EPS, gate_sigmoid=case["sigmoid"])
    if op == "norm":
        y, n = s["norm"].forward(s["x"], s["b"], s["gate"])
        return {"y": y, "n": n} if n is not None else {"y": y}
    if op == "norm_grad":
        g = s["norm"].backward(s["x"], s["b"], s["gate"], s["dy"], s["dn"])
        return {k: v for k, v in g.items() if v is not None}
    if "adamw" not in s:
        def parts(name, per=1):
            return [s[name][a // per:-(-(a + n) // per)] for a, n in zip(s["starts"], s["sizes"])] if name in s else None
        s["adamw"] = M.AdamW(parts("p"), lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS, weight_decay=DECAY, state_bits=case["bits"],
                             copies=parts("copy"), step=s["step"],
                             state=(parts("m"), parts("v"), parts("m_scale", 32), parts("v_scale", 32)))
        s["grads"] = parts("g")
    s["adamw"].step(s["grads"], grad_scale=s["clip"])
    return _adamw_out(s)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("forward", "rows", "weights"):
        P, N, K, E = case["P"] - case["dropped"], case["N"], case["K"], case["E"]
        rows = 2 * P * (N + K) + 4 * (E + 1)
        if op == "weights":
            weights = E * N * K * (2 if case["out"] == "bf16" else 4)
        else:
            weights = 2 * int((_counts(case, 0) > 0).sum()) * N * K
        return {"bytes": rows + weights, "flops": 2 * P * N * K}
    if op in ("norm", "norm_grad"):
        T, H = case["T"], case["H"]
        xb = 2 if case["x"] == "bf16" else 4
        gate = {"none": 0, "token": 4 * T, "channel": 4 * H, "full": 2 * T * H}[case["gate"]]
        w = H * (2 if case["w"] == "bf16" else 4) * (case["post"] + case["pre"])
        if op == "norm":
            return {"bytes": T * H * (2 * xb + 2 + 2 * case["pre"]) + gate + w, "flops": 12 * T * H}
        return {"bytes": T * H * (3 * xb + 4 + 2 * case["pre"]) + 2 * gate + w + 4 * H * (case["post"] + case["pre"]),
                "flops": 30 * T * H}
    n = sum(_tensor_sizes(case))
    p = 2 * (2 if case["p"] == "bf16" else 4) + (2 if case["p"] == "f32" else 0)
    g = 2 if case["g"] == "bf16" else 4
    state = 16 if case["bits"] == 32 else 4 + 4 / 32
    return {"bytes": n * (p + g + state), "flops": 15 * n}


# ---------------------------------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("forward", "rows", "weights"):
        at = s["offsets"].tolist()
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            a, b = at[e], at[e + 1]
            if op == "forward":
                out[a:b] = s["x"][a:b].double() @ s["w"][e].double().T
            elif op == "rows":
                out[a:b] = s["dy"][a:b].double() @ s["w"][e].double()
            else:
                out[e] = s["dy"][a:b].double().T @ s["x"][a:b].double()
        return out
    if op in ("norm", "norm_grad"):
        # the gradients are those of torch's own differentiation of the definition
        leaf = {k: s[k].double().requires_grad_() for k in ("x", "b", "gate", "w_post", "w_pre") if s.get(k) is not None}
        gate = leaf.get("gate")
        g = 1.0 if gate is None else 1 / (1 + torch.exp(-gate)) if case["sigmoid"] else gate

        def normed(v, w):
            return v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / v.shape[-1] + EPS) * w

        u = normed(leaf["b"], leaf["w_post"]) if case["post"] else leaf["b"]
        if op == "norm":
            y = SCALE * leaf["x"] + g * u
            out = {"y": y.detach()}
            if case["pre"]:
                out["n"] = normed(y, leaf["w_pre"]).detach()
            return out
        # y is the given stream; the layer's answer enters it with g * u, x with SCALE
        y = leaf["x"]
        loss = (y * s["dy"].double()).sum()
        if case["pre"]:
            loss = loss + (normed(y, leaf["w_pre"]) * s["dn"].double()).sum()
        total, *dw_pre = torch.autograd.grad(loss, [y] + ([leaf["w_pre"]] if case["pre"] else []))
        out = {"dx": SCALE * total}
        if case["pre"]:
            out["dw_pre"] = dw_pre[0]
        wanted = [k for k in ("b", "gate") if k in leaf] + (["w_post"] if case["post"] else [])
        names = {"b": "db", "gate": "dgate", "w_post": "dw_post"}
        grads = torch.autograd.grad((g * u * total).sum(), [leaf[k] for k in wanted])
        out.update({names[k]: d for k, d in zip(wanted, grads)})
        return out
    g, step = s["g"].double(), s["step"] + 1
    if s["clip"] is not None:
        g = g * s["clip"].double()

    def held(name):
        if case["bits"] == 32:
            return s[name].double()
        scale = torch.pow(2.0, s[name + "_scale"].double() - 127)
        v = (s[name].view(torch.float8_e4m3fn).double().view(-1, 32) * scale[:, None]).view(-1)
        return v * v if name == "v" else v

    m = BETA1 * held("m") + (1 - BETA1) * g
    v = BETA2 * held("v") + (1 - BETA2) * g * g
    p = s["p"].double()
    p = p - LR * DECAY * p - LR * (m / (1 - BETA1 ** step)) / (torch.sqrt(v / (1 - BETA2 ** step)) + ADAM_EPS)
    out = {"p": p, "copy": p if "copy" in s else None}
    # codes of 8 bits have no value in 64 bits of their own
    out.update({"m": m, "v": v} if case["bits"] == 32 else {"m": None, "v": None, "m_scale": None, "v_scale": None})
    if out["copy"] is None:
        del out["copy"]
    return out
