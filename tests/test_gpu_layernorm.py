"""Layer norm and its gradients against float64.

Tolerance, for every element.  With s32 = 2^-23, A = max |s| of a row, D its root variance (with eps): the mean is a sum of H
terms, off by at most (H / 32 + 12) s32 A / 2 (a thread adds 16 in pairs, then trees; bounded by that count), call it m; the differences
s - mean by m + s32 A; relative to D that is e = (m + s32 A) / D.  The variance's relative error is at most 2 e (worst
sign) + (H / 32 + 12) s32, rsqrt's 2 units, so h is off by e + |h| (e + (H / 32 + 16) s32), and n by |w| times that, 3 s32 of its
size, and its rounding.  Row means of gradients are sums of the same length; column sums add T terms.
"""
import pytest
import torch

from tests import helpers as Hp

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U, S32 = 2.0 ** -8, 2.0 ** -23


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return Hp.lib()


def randn(*shape, seed=0, scale=1.0, dtype=BF16, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(dtype)


def rounding(dtype):
    return U if dtype == BF16 else 2.0 ** -24


def stats(s, eps):
    """h, rsqrt(var + eps), and the bound of h's error, in float64."""
    H = s.shape[1]
    d = s - s.mean(1, keepdim=True)
    r = 1 / torch.sqrt(d.square().mean(1, keepdim=True) + eps)
    h = d * r
    e = (((H / 32 + 12) / 2 + 1) * S32 * s.abs().amax(1, keepdim=True)) * r
    return h, r, e + h.abs() * (e + (H / 32 + 16) * S32), e + (H / 32 + 16) * S32


def close(got, ref, bound, what):
    off = (got.double() - ref).abs()
    assert bool((off <= bound + 1e-37).all()), f"{what}: worst {float((off / (bound + 1e-37)).max()):.3f} of the bound"


def check_forward(s, n, x, b, w, bias, eps):
    ref_s = x.double() if b is None else x.double() + b.double()
    if b is not None:
        close(s, ref_s, rounding(s.dtype) * ref_s.abs() + S32 * ref_s.abs(), "s")
    h, _, eh, _ = stats(ref_s, eps)
    if b is not None:
        eh = eh + 2 * S32 * ref_s.abs().amax(1, keepdim=True) * (1 / torch.sqrt((ref_s - ref_s.mean(1, keepdim=True)).square().mean(1, keepdim=True) + eps))
    W = 1.0 if w is None else w.double()
    ref = h * W + (0.0 if bias is None else bias.double())
    size = (h * W).abs() + ref.abs()
    close(n, ref, U * ref.abs() + (1 + U) * (eh * (abs(W) if w is None else W.abs()) + 3 * S32 * size), "n")


def check_backward(out, s, w, dn, ds, eps):
    s, dn = s.double(), dn.double()
    T, H = s.shape
    h, r, eh, rel = stats(s, eps)
    g = dn * (1.0 if w is None else w.double())
    mg, mgh = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    a = g - mg - h * mgh
    ref = r * a + (0.0 if ds is None else ds.double())
    terms = (H / 32 + 16) * S32
    mean_abs = g.abs().mean(1, keepdim=True)
    e_mgh = (g.abs() * eh).mean(1, keepdim=True) + terms * (g * h).abs().mean(1, keepdim=True)
    err = S32 * (g.abs() * 3 + (h * mgh).abs() * 4) + terms * mean_abs + eh * mgh.abs() + (h.abs() + eh) * e_mgh
    bound = r * (err + a.abs() * rel) + 2 * S32 * ref.abs()
    if ds is not None:
        bound = bound + S32 * ds.double().abs()
    close(out["dx"], ref, rounding(out["dx"].dtype) * ref.abs() + (1 + U) * bound, "dx")
    column = (T + 16) * S32
    if out["dw"] is not None:
        close(out["dw"], (dn * h).sum(0), (dn.abs() * eh).sum(0) + column * (dn * h).abs().sum(0), "dw")
    if out["dbias"] is not None:
        close(out["dbias"], dn.sum(0), column * dn.abs().sum(0), "dbias")


SIZES = [(1, 8), (3, 16), (5, 64), (2, 248), (17, 256), (40, 264), (9, 512), (33, 520), (700, 1000), (8, 2048), (310, 4096), (161, 7168),
         (7, 8192), (5, 8200), (311, 16384), (5000, 64)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forward(B, T, H, dtype):
    from moe_expert_layer_counting_gb300 import LayerNorm
    x, b = randn(T, H, seed=1, scale=1.5, dtype=dtype, shift=0.3), randn(T, H, seed=2, scale=2.0)
    for w, bias in ((randn(H, seed=3, dtype=F32, shift=1.0), randn(H, seed=4, dtype=F32)), (randn(H, seed=3), None), (None, randn(H, seed=4)),
                    (None, None)):
        norm = LayerNorm(w, bias, eps=1e-5)
        s, n = norm.forward(x, b)
        check_forward(s, n, x, b, w, bias, 1e-5)
        s, n = norm.forward(x)
        assert s is x
        check_forward(s, n, x, None, w, bias, 1e-5)


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_backward(B, T, H, dtype):
    from moe_expert_layer_counting_gb300 import LayerNorm
    s, dn, ds = randn(T, H, seed=1, scale=1.5, dtype=dtype, shift=0.3), randn(T, H, seed=2, scale=0.1), randn(T, H, seed=3, scale=0.1, dtype=dtype)
    for w, bias, stream in ((randn(H, seed=3, dtype=F32, shift=1.0), randn(H, seed=4, dtype=F32), ds), (randn(H, seed=3), None, None), (None, randn(H, seed=4), ds)):
        norm = LayerNorm(w, bias, eps=1e-5)
        out = norm.backward(s, dn, stream)
        assert (out["dw"] is None) == (w is None) and (out["dbias"] is None) == (bias is None)
        check_backward(out, s, w, dn, stream, 1e-5)
        again = norm.backward(s, dn, stream)
        assert all(v is None or torch.equal(v, again[k]) for k, v in out.items())


SHORT = [(1, 128), (2, 120), (3, 136), (7, 256), (63, 72), (65, 64), (2500, 24), (9729, 128), (20001, 64), (4867, 248), (40000, 8), (19457, 104)]


@pytest.mark.parametrize("T,H", SHORT)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_short_rows(B, T, H, dtype):
    """Several rows of a warp: numbers of rows around one, two and more rounds of all groups, and between them."""
    from moe_expert_layer_counting_gb300 import LayerNorm
    wide = lambda t: torch.cat([t, torch.full_like(t[:, :8], float("nan"))], 1)[:, :H]       # noqa: E731
    x, b = wide(randn(T, H, seed=1, scale=1.5, dtype=dtype, shift=0.3)), wide(randn(T, H, seed=2, scale=2.0))
    dn, ds = wide(randn(T, H, seed=3, scale=0.1)), wide(randn(T, H, seed=4, scale=0.1, dtype=dtype))
    w, bias = randn(H, seed=5, dtype=F32, shift=1.0), randn(H, seed=6)
    ws = torch.empty(B.moe_layernorm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    for other in (b, None):
        keep = torch.full((T + 1, H + 8), 7.0, dtype=dtype, device="cuda"), torch.full((T + 1, H + 8), 7.0, dtype=BF16, device="cuda")
        s, n = (t[:T, :H] for t in keep)
        B.moe_layernorm_forward(x, other, w, bias.float(), s if other is not None else None, n)
        check_forward(s, n, x, other, w, bias.float(), 1e-5)
        assert all(bool((t[T] == 7).all()) and bool((t[:, H:] == 7).all()) for t in keep)
    norm = LayerNorm(w, bias.float(), eps=1e-5)
    for stream in (ds, None):
        keep = torch.full((T + 1, H + 8), 7.0, dtype=dtype, device="cuda")
        out = {"dx": keep[:T, :H], "dw": torch.empty(H, device="cuda"), "dbias": torch.empty(H, device="cuda")}
        B.moe_layernorm_backward(x, w, dn, stream, ws, out["dx"], out["dw"], out["dbias"])
        check_backward(out, x, w, dn, stream, 1e-5)
        assert bool((keep[T] == 7).all()) and bool((keep[:, H:] == 7).all())
        again = norm.backward(x.contiguous(), dn.contiguous(), None if stream is None else stream.contiguous())
        assert all(torch.equal(out[k], again[k]) for k in out)


@pytest.mark.parametrize("T,H", [(1, 8200), (2, 8208), (75, 12288), (77, 9000), (153, 16376), (400, 16384), (310, 10240)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_long_rows(B, T, H, dtype):
    """Rows that two SMs share: numbers of rows around one, two and more rounds, columns that do not divide into two equal
    halves of eight, outputs in place of inputs, and the same bits again."""
    from moe_expert_layer_counting_gb300 import LayerNorm
    wide = lambda t: torch.cat([t, torch.full_like(t[:, :8], float("nan"))], 1)[:, :H]       # noqa: E731
    s, dn, ds = wide(randn(T, H, seed=1, scale=1.5, dtype=dtype, shift=0.3)), wide(randn(T, H, seed=2, scale=0.1)), \
        wide(randn(T, H, seed=3, scale=0.1, dtype=dtype))
    ws = torch.empty(B.moe_layernorm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    for w, stream in ((randn(H, seed=5, dtype=F32, shift=1.0), ds), (randn(H, seed=6), None), (None, ds)):
        keep = torch.full((T + 1, H + 8), 7.0, dtype=dtype, device="cuda")
        out = {"dx": keep[:T, :H], "dw": None if w is None else torch.empty(H, device="cuda"), "dbias": torch.empty(H, device="cuda")}
        B.moe_layernorm_backward(s, w, dn, stream, ws, out["dx"], out["dw"], out["dbias"])
        check_backward(out, s, w, dn, stream, 1e-5)
        assert bool((keep[T] == 7).all()) and bool((keep[:, H:] == 7).all())
        place = s.clone()
        B.moe_layernorm_backward(place, w, dn, stream, ws, place)
        assert torch.equal(place, out["dx"])
        again = LayerNorm(w, torch.zeros(H, device="cuda") if w is None or w.dtype == F32 else torch.zeros_like(w)).backward(s, dn, stream)
        assert all(v is None or torch.equal(v, again[k]) for k, v in out.items())


def test_long_rows_infinities_and_nan_stay_in_their_row(B):
    from moe_expert_layer_counting_gb300 import LayerNorm
    s, dn = randn(200, 9000, seed=1), randn(200, 9000, seed=2)
    norm = LayerNorm(randn(9000, seed=3), None)
    dx = norm.backward(s, dn)["dx"]
    y, d = s.clone(), dn.clone()
    y[3, 5], y[79, 8999], d[152, 4600], d[199, 0] = float("nan"), float("inf"), float("nan"), float("-inf")
    dx2 = norm.backward(y, d)["dx"]
    fine = torch.ones(200, dtype=torch.bool, device="cuda")
    fine[[3, 79, 152, 199]] = False
    # row 199: mean(g) and mean(g h) are infinite, so that g - mean(g) - h mean(g h) is infinite or, where they cancel, NaN
    assert torch.equal(dx2[fine], dx[fine]) and bool(dx2[[3, 79, 152]].isnan().all()) and not bool(dx2[199].isfinite().any())


@pytest.mark.parametrize("H", [64, 200])
def test_short_rows_infinities_and_nan_stay_in_their_row(B, H):
    from moe_expert_layer_counting_gb300 import LayerNorm
    x, b, dn = randn(130, H, seed=1), randn(130, H, seed=2), randn(130, H, seed=3)
    norm = LayerNorm(randn(H, seed=4), randn(H, seed=5))
    s, n = norm.forward(x, b)
    dx = norm.backward(s, dn)["dx"]
    y, d = x.clone(), dn.clone()
    y[3, 5], y[129, 0], d[20, 7] = float("nan"), float("inf"), float("nan")
    s2, n2 = norm.forward(y, b)
    dx2 = norm.backward(s2, d)["dx"]
    fine = torch.ones(130, dtype=torch.bool, device="cuda")
    fine[[3, 129]] = False
    assert torch.equal(n2[fine], n[fine]) and bool(n2[~fine].isnan().all())
    fine[20] = False
    assert torch.equal(dx2[fine], dx[fine]) and bool(dx2[~fine].isnan().all())


@pytest.mark.parametrize("shift", [0.0, 1e3])
def test_rows_far_from_zero(B, shift):
    """A mean far above the spread: the variance is that of the differences, not of squares that cancel."""
    from moe_expert_layer_counting_gb300 import LayerNorm
    x, dn = randn(20, 1000, seed=1, dtype=F32, shift=shift), randn(20, 1000, seed=2)
    w, bias = randn(1000, seed=3, dtype=F32), randn(1000, seed=4, dtype=F32)
    norm = LayerNorm(w, bias)
    _, n = norm.forward(x)
    check_forward(None, n, x, None, w, bias, 1e-5)
    check_backward(norm.backward(x, dn), x, w, dn, None, 1e-5)


def test_strides_and_in_place(B):
    T, H = 37, 520

    def wide(t, ld):
        v = torch.full((T, ld), float("nan"), dtype=t.dtype, device="cuda")[:, :H]
        return v.copy_(t)

    x, b, dn = wide(randn(T, H, seed=1), H + 8), wide(randn(T, H, seed=2), H + 24), wide(randn(T, H, seed=3), H + 16)
    w, bias = randn(H, seed=4), randn(H, seed=5)
    s, n = torch.empty(T, H, dtype=BF16, device="cuda"), torch.empty(T, H, dtype=BF16, device="cuda")
    B.moe_layernorm_forward(x.contiguous(), b.contiguous(), w, bias, s, n)
    x2, b2 = x.clone(), wide(b, H + 24)
    x2 = wide(x, H + 8)
    B.moe_layernorm_forward(x2, b2, w, bias, x2, b2)                 # s into x, n into b
    assert torch.equal(x2, s) and torch.equal(b2, n)
    ws = torch.empty(B.moe_layernorm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    dx, dw, dbias = torch.empty_like(s), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    B.moe_layernorm_backward(s, w, dn, x, ws, dx, dw, dbias)
    check_backward({"dx": dx, "dw": dw, "dbias": dbias}, s, w, dn, x, 1e-5)
    for place in ("s", "dn", "ds"):
        t = {"s": s.clone(), "dn": wide(dn, H + 16), "ds": wide(x, H + 8)}
        B.moe_layernorm_backward(t["s"], w, t["dn"], t["ds"], ws, t[place])
        assert torch.equal(t[place], dx)
    only = torch.zeros(H, device="cuda")
    B.moe_layernorm_backward(s, w, dn, None, ws, dbias=only)
    assert torch.equal(only, dbias)


def test_infinities_and_nan_stay_in_their_row(B):
    from moe_expert_layer_counting_gb300 import LayerNorm
    x, b, dn = randn(30, 264, seed=1), randn(30, 264, seed=2), randn(30, 264, seed=3)
    norm = LayerNorm(randn(264, seed=4), randn(264, seed=5))
    s, n = norm.forward(x, b)
    dx = norm.backward(s, dn)["dx"]
    y, d = x.clone(), dn.clone()
    y[3, 5], y[11, 0], d[20, 7] = float("nan"), float("inf"), float("nan")
    s2, n2 = norm.forward(y, b)
    dx2 = norm.backward(s2, d)["dx"]
    fine = torch.ones(30, dtype=torch.bool, device="cuda")
    fine[[3, 11]] = False
    assert torch.equal(n2[fine], n[fine]) and bool(n2[3].isnan().all()) and bool(n2[11].isnan().all())
    fine[20] = False
    assert torch.equal(dx2[fine], dx[fine]) and bool(dx2[~fine].isnan().all())


def test_equal_values_and_no_rows(B):
    """A row of one value has no spread: n is the bias, and gradients are finite."""
    from moe_expert_layer_counting_gb300 import LayerNorm
    w, bias = randn(72, seed=1, dtype=F32), randn(72, seed=2, dtype=F32)
    norm = LayerNorm(w, bias)
    x = torch.full((3, 72), 2.5, dtype=BF16, device="cuda")
    _, n = norm.forward(x)
    assert torch.equal(n, bias.bfloat16().expand(3, 72))
    assert bool(norm.backward(x, randn(3, 72, seed=3))["dx"].isfinite().all())
    none = torch.zeros(0, 72, dtype=BF16, device="cuda")
    s, n = norm.forward(none, none)
    assert s.shape == n.shape == (0, 72)
    d = norm.backward(none, none)
    assert d["dx"].shape == (0, 72) and bool((d["dw"] == 0).all()) and bool((d["dbias"] == 0).all())


def test_gradient_against_differences(B):
    from moe_expert_layer_counting_gb300 import LayerNorm
    T, H = 6, 136
    s, dn, ds = randn(T, H, seed=1, dtype=F32), randn(T, H, seed=2), randn(T, H, seed=3, dtype=F32)
    w, bias = randn(H, seed=4, dtype=F32), randn(H, seed=5, dtype=F32)
    out = LayerNorm(w, bias).backward(s, dn, ds)

    def loss(x, a, c):
        d = x - x.mean(1, keepdim=True)
        return ((d / torch.sqrt(d.square().mean(1, keepdim=True) + 1e-5) * a + c) * dn.double()).sum() + (x * ds.double()).sum()

    base, step = [t.double() for t in (s, w, bias)], 1e-5
    for i, k in enumerate(("dx", "dw", "dbias")):
        v = torch.randn(base[i].shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda").double()
        up, down = ([t + sign * step * v if j == i else t for j, t in enumerate(base)] for sign in (1, -1))
        diff = float((loss(*up) - loss(*down)) / (2 * step))
        # float32's sums of T H terms, and the difference's own error of order step^2
        assert abs(float((out[k].double() * v).sum()) - diff) <= 1e-5 * float(out[k].double().norm() * v.norm()) + 1e-6


def test_streams_and_graphs(B):
    from moe_expert_layer_counting_gb300 import LayerNorm
    T, H = 400, 1032
    w, bias = randn(H, seed=4), randn(H, seed=5)
    norm = LayerNorm(w, bias)
    xs, dn = [randn(T, H, seed=s) for s in (1, 2)], randn(T, H, seed=3)

    def both(x, stream=None):
        s, n = norm.forward(x, dn, stream)
        return {"s": s, "n": n, **norm.backward(s, dn, x, stream)}

    want = [both(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(10):
        got = [both(x, st) for x, st in zip(xs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(g[k], v[k]) for g, v in zip(got, want) for k in v)
    # two graphs captured with one object, replayed side by side on new rows
    places, graphs, outs = [x.clone() for x in xs], [], []
    for x in places:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(both(x))
        graphs.append(graph)
    for x, new in zip(places, xs[::-1]):
        x.copy_(new)
    torch.cuda.synchronize()
    for _ in range(10):
        for st, graph in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g[k], v[k]) for g, v in zip(outs, want[::-1]) for k in v)
