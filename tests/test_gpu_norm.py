"""The norms around the layer, forward and backward, against float64.

Tolerance.  Every output is a sum of terms computed in float32.  With `mag`
the sum of the terms' magnitudes (the same formula on absolute values), the
row sums (H terms) and column sums (T terms) give a relative error of at most
(H + T + 64) * 2^-23 of `mag`, the 64 standing for the products, roots,
quotients and exponentials on the way (each at most 4 units of 2^-24); a BF16
output adds one rounding, 2^-8 of its value, a float32 one 2^-24.
"""
import itertools

import pytest
import torch

from tests import helpers as Hp

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    Hp.lib()
    import moe_expert_layer_counting_gb300
    return moe_expert_layer_counting_gb300


class Case:
    def __init__(self, T, H, xt=BF16, wt=F32, gate=None, gt=F32, sigmoid=False, post=True, pre=True, scale=0.75,
                 offset=0.0, eps=1e-6, seed=0, layer=True):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape, dtype, scale=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

        self.T, self.H, self.eps, self.scale, self.offset, self.sigmoid = T, H, eps, scale, offset, sigmoid
        self.x = randn(T, H, dtype=xt, scale=1.5)
        self.b = randn(T, H, dtype=BF16, scale=2.0) if layer else None
        shape = {None: None, "token": (T, 1), "channel": (1, H), "full": (T, H)}[gate]
        self.kind, self.gate = gate, None if shape is None else randn(*shape, dtype=gt)
        self.w_post = (randn(H, dtype=F32, scale=0.2) + 1 - offset).to(wt) if post and layer else None
        self.w_pre = (randn(H, dtype=F32, scale=0.2) + 1 - offset).to(wt) if pre else None
        self.dy = randn(T, H, dtype=xt)
        self.dn = randn(T, H, dtype=BF16) if pre else None

    def module(self, M):
        return M.BlockNorm(self.w_post, self.w_pre, self.scale, self.offset, self.eps, self.sigmoid)

    def g64(self):
        if self.gate is None:
            return torch.ones(1, 1, dtype=F64, device="cuda")
        z = self.gate.double()
        return 1 / (1 + torch.exp(-z)) if self.sigmoid else z


def up(t):
    return None if t is None else t.double()


def forward64(c):
    """{name: (value, magnitude)} of y and n."""
    x = up(c.x)
    if c.b is None:
        y, y_mag = x, x.abs()
    else:
        u = up(c.b)
        if c.w_post is not None:
            u = u * torch.rsqrt(u.pow(2).mean(-1, keepdim=True) + c.eps) * (c.offset + up(c.w_post))
        u = c.g64() * u
        y, y_mag = c.scale * x + u, (c.scale * x).abs() + u.abs()
    out = {"y": (y, y_mag)}
    if c.w_pre is not None:
        r = torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + c.eps)
        w = c.offset + up(c.w_pre)
        n = y * r * w
        worse = y_mag.norm(dim=-1, keepdim=True) / y.norm(dim=-1, keepdim=True).clamp(min=1e-30)
        out["n"] = (n, (y_mag * r * w).abs() + n.abs() * worse)
    return out


def backward64(c, y):
    """{name: (value, magnitude)} of the gradients, written out (not differentiated by torch)."""
    y, out = y.double(), {}
    zero = torch.zeros_like(y)
    d, d_mag = (up(c.dy), up(c.dy).abs()) if c.dy is not None else (zero, zero)
    if c.w_pre is not None and c.dn is not None:
        r = torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + c.eps)
        h, dh = y * r, up(c.dn) * (c.offset + up(c.w_pre))
        d = d + r * (dh - h * (dh * h).mean(-1, keepdim=True))
        d_mag = d_mag + r * (dh.abs() + h.abs() * (dh * h).abs().mean(-1, keepdim=True))
        out["dw_pre"] = ((up(c.dn) * h).sum(0), (up(c.dn) * h).abs().sum(0))
    s = c.scale if c.b is not None else 1.0
    out["dx"] = (s * d, abs(s) * d_mag)
    if c.b is None:
        return out
    b, g = up(c.b), c.g64()
    rb = torch.rsqrt(b.pow(2).mean(-1, keepdim=True) + c.eps) if c.w_post is not None else torch.ones_like(b[:, :1])
    w = c.offset + up(c.w_post) if c.w_post is not None else torch.ones(c.H, dtype=F64, device="cuda")
    hb = b * rb
    if c.gate is not None:
        dg, dg_mag = d * hb * w, d_mag * (hb * w).abs()
        dim = {"token": 1, "channel": 0, "full": None}[c.kind]
        if dim is not None:
            dg, dg_mag = dg.sum(dim, keepdim=True), dg_mag.sum(dim, keepdim=True)
        slope = g * (1 - g) if c.sigmoid else 1.0
        # 1 - g is a difference: an error of 2^-23 in g is one of 2^-23 of 1, not of 1 - g
        out["dgate"] = (dg * slope, dg_mag * (g.abs() if c.sigmoid else 1.0))
    du, du_mag = g * d, g.abs() * d_mag
    if c.w_post is not None:
        dh, dh_mag = du * w, du_mag * w.abs()
        out["db"] = (rb * (dh - hb * (dh * hb).mean(-1, keepdim=True)),
                     rb * (dh_mag + hb.abs() * (dh_mag * hb.abs()).mean(-1, keepdim=True)))
        out["dw_post"] = ((du * hb).sum(0), (du_mag * hb.abs()).sum(0))
    else:
        out["db"] = (du, du_mag)
    return out


def close(name, got, want, H, T):
    ref, mag = want
    rounding = 2.0 ** -8 if got.dtype == BF16 else 2.0 ** -24
    bound = rounding * ref.abs() + (1 + rounding) * (H + T + 64) * 2.0 ** -23 * mag + 1e-37
    off = (got.double() - ref).abs()
    assert bool((off <= bound).all()), f"{name}: worst {float((off / bound).max()):.3f} of the bound"


def check(M, c):
    m = c.module(M)
    y, n = m.forward(c.x, c.b, c.gate)
    want = forward64(c)
    close("y", y, want["y"], c.H, 0)
    if n is not None:
        close("n", n, want["n"], c.H, 0)
    else:
        assert "n" not in want
    got, want = m.backward(y, c.b, c.gate, c.dy, c.dn), backward64(c, y)
    assert {k for k, v in got.items() if v is not None} == set(want)
    for k in want:
        close(k, got[k].reshape(want[k][0].shape), want[k], c.H, c.T)


@pytest.mark.parametrize("T,H", [(1, 8), (1, 2048), (2, 264), (3, 7168), (5, 16384), (40, 64), (33, 1000), (700, 2048),
                                 (613, 8200), (1300, 7168)])
@pytest.mark.parametrize("xt", [BF16, F32])
def test_sizes(M, T, H, xt):
    check(M, Case(T, H, xt, gate="token", sigmoid=True, seed=T + H))


@pytest.mark.parametrize("gate,gt,sigmoid", [(None, F32, False), *itertools.product(("token", "channel", "full"), (BF16, F32),
                                                                                    (False, True))])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_gates_and_norms(M, gate, gt, sigmoid, post, pre):
    check(M, Case(350, 328, gate=gate, gt=gt, sigmoid=sigmoid, post=post, pre=pre))


@pytest.mark.parametrize("gate,gt", [(None, F32), ("token", F32), ("channel", BF16), ("full", F32)])
@pytest.mark.parametrize("H,xt,post,pre", [(8200, BF16, True, True), (16376, F32, True, True), (16384, BF16, False, True),
                                           (9000, F32, True, False)])
def test_rows_split_over_two_blocks(M, H, xt, gate, gt, post, pre):
    check(M, Case(170, H, xt, gate=gate, gt=gt, sigmoid=True, post=post, pre=pre))


@pytest.mark.parametrize("T,H", [(3000, 512), (5000, 248)])
def test_many_short_rows(M, T, H):
    check(M, Case(T, H, F32, gate="full", gt=F32))


@pytest.mark.parametrize("wt", [BF16, F32])
@pytest.mark.parametrize("offset", [0.0, 1.0])
@pytest.mark.parametrize("scale", [0.0, 1.0, -2.5])
def test_weights_offset_and_scale(M, wt, offset, scale):
    check(M, Case(37, 520, F32, wt, gate="channel", offset=offset, scale=scale, eps=1e-3))


@pytest.mark.parametrize("xt", [BF16, F32])
def test_first_norm_alone(M, xt):
    c = Case(19, 1032, xt, layer=False)
    y, n = c.module(M).forward(c.x)
    assert y is c.x
    close("n", n, forward64(c)["n"], c.H, 0)
    got, want = c.module(M).backward(c.x, None, None, c.dy, c.dn), backward64(c, c.x)
    for k in want:
        close(k, got[k], want[k], c.H, c.T)


def test_first_norm_alone_of_split_rows(M):
    c = Case(160, 8208, F32, layer=False)
    close("n", c.module(M).forward(c.x)[1], forward64(c)["n"], c.H, 0)
    got, want = c.module(M).backward(c.x, None, None, c.dy, c.dn), backward64(c, c.x)
    for k in want:
        close(k, got[k], want[k], c.H, c.T)


def test_one_of_the_two_gradients(M):
    for drop in ("dy", "dn"):
        c = Case(45, 264, gate="full", gt=BF16)
        setattr(c, drop, None)
        y, _ = c.module(M).forward(c.x, c.b, c.gate)
        got, want = c.module(M).backward(y, c.b, c.gate, c.dy, c.dn), backward64(c, y)
        assert {k for k, v in got.items() if v is not None} == set(want)
        for k in want:
            close(k, got[k].reshape(want[k][0].shape), want[k], c.H, c.T)


def test_zero_rows(M):
    """Rows of zeros: the norm is 0 and the gradients finite (1 / sqrt(eps) times theirs)."""
    c = Case(6, 512, gate="token")
    c.x[2:4] = 0
    c.b[1:4] = 0
    check(M, c)


def test_infinities_and_nan_stay_in_their_row(M):
    c = Case(9, 512, gate="token")
    c.x[1, 5], c.b[3, 0], c.gate[5] = float("nan"), float("inf"), float("nan")
    m = c.module(M)
    y, n = m.forward(c.x, c.b, c.gate)
    g = m.backward(y, c.b, c.gate, c.dy, c.dn)
    fine = torch.tensor([0, 2, 4, 6, 7, 8], device="cuda")
    for t in (y, n, g["dx"], g["db"], g["dgate"]):
        assert bool(t[fine].isfinite().all())
    for r in (1, 3, 5):
        assert not bool(n[r].isfinite().all()) and not bool(g["dx"][r].isfinite().all())


def test_row_strides_and_in_place(M):
    """Tensors that are column ranges of wider ones; y over x, n over b, dx over dy, db over dn."""
    B = M.binding
    c = Case(50, 264, gate="full", gt=BF16)
    want, wide = forward64(c), {}
    for k in ("x", "b", "gate", "dy", "dn"):
        t = getattr(c, k)
        wide[k] = torch.full((c.T, c.H + 32), 9.0, dtype=t.dtype, device="cuda")
        wide[k][:, 8:8 + c.H] = t
        setattr(c, k, wide[k][:, 8:8 + c.H])
    kept_b = c.b.clone()
    ws = torch.empty(B.moe_norm_workspace_size(c.T, c.H), dtype=torch.uint8, device="cuda")
    how = dict(residual_scale=c.scale, eps=c.eps)
    B.moe_norm_forward(c.x, c.b, c.gate, c.w_post, c.w_pre, c.x, c.b, **how)
    close("y", c.x, want["y"], c.H, 0)
    close("n", c.b, want["n"], c.H, 0)
    c.b.copy_(kept_b)
    want = backward64(c, c.x)
    dgate = torch.empty_like(c.gate)
    dw_post, dw_pre = torch.empty(c.H, device="cuda"), torch.empty(c.H, device="cuda")
    B.moe_norm_backward(c.x, c.b, c.gate, c.w_post, c.w_pre, c.dy, c.dn, ws, c.dy, c.dn, dgate, dw_post, dw_pre, **how)
    for k, t in (("dx", c.dy), ("db", c.dn), ("dgate", dgate), ("dw_post", dw_post), ("dw_pre", dw_pre)):
        close(k, t, want[k], c.H, c.T)
    for t in wide.values():
        assert bool((t[:, :8] == 9).all()) and bool((t[:, 8 + c.H:] == 9).all())


def test_gradients_against_differences(M):
    """Central differences of the float64 forward along random directions (error of the difference: h^2, 1e-8 here)
    against the gradients' products with them; the stream in float32, so that the BF16 rounding of db alone counts."""
    for gate, sigmoid in (("token", True), ("channel", False), ("full", True)):
        c = Case(24, 136, F32, gate=gate, sigmoid=sigmoid, eps=1e-2)
        y, _ = c.module(M).forward(c.x, c.b, c.gate)
        got = c.module(M).backward(y, c.b, c.gate, c.dy, c.dn)
        names = {"x": "dx", "b": "db", "gate": "dgate", "w_post": "dw_post", "w_pre": "dw_pre"}
        base = {k: getattr(c, k).double() for k in names}

        def loss():
            f = forward64(c)
            return float((f["y"][0] * c.dy.double()).sum() + (f["n"][0] * c.dn.double()).sum())

        for k, name in names.items():
            v = torch.randn(base[k].shape, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").double()
            ends = []
            for sign in (1, -1):
                setattr(c, k, base[k] + sign * 1e-4 * v)
                ends.append(loss())
            setattr(c, k, base[k].to(BF16 if k == "b" else F32))
            terms = got[name].double() * v
            diff = (ends[0] - ends[1]) / 2e-4
            rel = 2.0 ** -8 if name == "db" else 1e-5
            assert abs(float(terms.sum()) - diff) <= rel * float(terms.abs().sum()) + 1e-5 * abs(diff), name


def test_same_bits_again_on_another_stream_and_in_a_graph(M):
    c = Case(600, 1024, gate="channel")
    m = c.module(M)

    def call(stream=None):
        y, n = m.forward(c.x, c.b, c.gate, stream=stream)
        return [y, n, *m.backward(y, c.b, c.gate, c.dy, c.dn, stream=stream).values()]

    first = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = call(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = call()
    for t in third:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, d in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, d)


def test_no_rows(M):
    c = Case(0, 64, gate="channel")
    m = c.module(M)
    y, n = m.forward(c.x, c.b, c.gate)
    g = m.backward(y, c.b, c.gate, c.dy, c.dn)
    assert y.shape == n.shape == (0, 64)
    for k in ("dw_pre", "dw_post", "dgate"):
        assert not bool(g[k].any())


def test_offsets_beyond_2_pow_31_values(M):
    """A float32 stream of 2.2e9 values: the last rows are where they should be."""
    T, H = 135_000, 16384
    x = torch.zeros(T, H, device="cuda")
    w = torch.ones(H, device="cuda")
    x[-3:] = torch.randn(3, H, device="cuda")
    n = M.BlockNorm(w_pre=w).forward(x)[1]
    ref = x[-3:].double()
    ref = ref * torch.rsqrt(ref.pow(2).mean(-1, keepdim=True) + 1e-6)
    close("n", n[-3:], (ref, 2 * ref.abs()), H, 0)
    assert not bool(n[:-3].any())
