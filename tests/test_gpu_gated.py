"""The gated feed-forward block's kernels against float64.

Tolerance, for every element.  With u = 2^-8 half a step of BF16, s32 = 2^-23:
a product's float32 sum is within (terms + 1) s32 of the sum M of its terms'
magnitudes (one truncation per addition).  An activation is f(z) = z s(q), with
s(q) = 1 / (1 + exp(-q)).  Relative to s: exp's argument has up to three roundings
(GELU's polynomial), which exp turns into 1.5 |q| s32, the fast exp is within
2 + 1.2 |q| units of 2^-24, the sum and the quotient within 3; in all (6 + 3 |q|) s32,
called e below.  f takes one rounding more, and an error of z times max |f'| (1.13).
f' = s + f (1 - s) q': s is within e s, f (1 - s) q' within (2 e + 8 s32) |f q'| (the error
of 1 - s is s's own, at most e).  A product of factors adds their
relative errors, and the output one rounding.
"""
import numpy as np
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


def offsets_of(counts, first=0):
    return torch.tensor([first, *(first + np.cumsum(counts))], dtype=torch.int32, device="cuda")


def randn(*shape, seed=0, scale=1.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def workspace(B, P, H, I, E):
    return torch.empty(B.moe_gated_workspace_size(P, H, I, E), dtype=torch.uint8, device="cuda")


def act(z, activation):
    """f, f', the relative error e of s, and the bound of the error of f', in float64; GELU as z s(2u), because
    1 + tanh(u) loses all its digits where u is far below zero."""
    q, dq = z, torch.ones_like(z)
    if activation == 1:
        r = 2 * (2 / np.pi) ** 0.5
        q, dq = r * (z + 0.044715 * z ** 3), r * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(q)
    e = (6 + 3 * q.abs()) * S32
    return z * s, s + z * s * torch.sigmoid(-q) * dq, e, e * s + (2 * e + 8 * S32) * (z * s * dq).abs()


def close(got, ref, bound, what):
    off = (got.double() - ref).abs()
    bad = off > bound + 1e-37
    assert not bool(bad.any()), f"{what}: worst {float((off / (bound + 1e-37)).max()):.3f} of the bound"


def check_forward(h, a, x, w, row_w, counts, activation, first=0):
    I, H = w.shape[1] // 2, w.shape[2]
    at = first
    for e, c in enumerate(counts):
        r = slice(at, at + c)
        at += c
        ref = x[r].double() @ w[e].double().T
        err = (H + 1) * S32 * (x[r].double().abs() @ w[e].double().abs().T)
        if a is not None:
            close(a[r], ref, U * ref.abs() + (1 + U) * err, "a")
        f, _, e_f, _ = act(ref[:, :I], activation)
        up = ref[:, I:]
        v = torch.ones(c, 1, dtype=torch.float64, device="cuda") if row_w is None else row_w[r].double()[:, None]
        df = 1.13 * err[:, :I] + (e_f + S32) * f.abs()
        ref_h = f * up * v
        more = (df * (up.abs() + err[:, I:]) + f.abs() * err[:, I:]) * v.abs() + 3 * S32 * ref_h.abs()
        close(h[r], ref_h, U * ref_h.abs() + (1 + U) * more, "h")


def check_back(out, dy, w, a, row_w, counts, activation, first=0):
    H, I = w.shape[1:]
    at = first
    for e, c in enumerate(counts):
        r = slice(at, at + c)
        at += c
        d = dy[r].double() @ w[e].double()
        err = (H + 1) * S32 * (dy[r].double().abs() @ w[e].double().abs())
        gate, up = a[r].double().split(I, 1)
        f, df, e_f, e_df = act(gate, activation)
        v = torch.ones(c, 1, dtype=torch.float64, device="cuda") if row_w is None else row_w[r].double()[:, None]
        want = {"da": torch.cat([d * v * up * df, d * v * f], 1), "h": f * up * v, "drow_w": (d * f * up).sum(1)}
        dv, ev = (d * v).abs(), err * v.abs()
        more = torch.cat([ev * up.abs() * (df.abs() + e_df) + dv * up.abs() * (e_df + 5 * S32 * df.abs()),
                          (ev * (1 + e_f) + dv * (e_f + 5 * S32)) * f.abs()], 1)
        close(out["da"][r], want["da"], U * want["da"].abs() + (1 + U) * more, "da")
        if "h" in out:
            close(out["h"][r], want["h"], (U + (1 + U) * (e_f + 4 * S32)) * want["h"].abs(), "h")
        if "drow_w" in out:
            bound = ((err * (1 + e_f) + d.abs() * (e_f + (I + 4) * S32)) * (f * up).abs()).sum(1)
            close(out["drow_w"][r], want["drow_w"], bound, "drow_w")


CASES = [
    # counts, I, H
    ([1], 8, 8),
    ([1], 512, 2048),
    ([0, 1, 0, 1], 72, 136),
    ([16, 32, 64, 128, 256], 128, 256),
    ([15, 17, 31, 33, 63, 65, 127, 129, 255, 257], 136, 200),
    ([0, 0, 700, 0, 1, 1025], 264, 1032),
    ([256, 257, 288, 289, 320, 321, 576, 577, 641, 769], 24, 328),
    ([3] * 100 + [0] * 28, 64, 72),
    ([40] * 16, 512, 512),
    ([2, 0, 5] * 341 + [1], 16, 64),          # 1024 experts
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("activation", [0, 1])
def test_forward(B, case, activation):
    counts, I, H = CASES[case]
    E, P = len(counts), sum(counts)
    x, w = randn(P, H, seed=1), randn(E, 2 * I, H, seed=2, scale=1.5 * H ** -0.5)
    row_w = randn(P, seed=3, dtype=F32) if case % 2 else None
    h = torch.full((P, I), 3.0, dtype=BF16, device="cuda")
    a = torch.full((P, 2 * I), 3.0, dtype=BF16, device="cuda") if case != 1 else None
    ws = workspace(B, P, H, I, E)
    B.moe_gated_forward(x, w, offsets_of(counts), h, ws, a=a, row_w=row_w, activation=activation)
    assert B.moe_get_device_status(ws) == B.MOE_OK
    check_forward(h, a, x, w, row_w, counts, activation)


FEW = [
    # counts, first, rows behind the last, I, H
    ([1], 0, 0, 8, 8), ([2], 0, 0, 40, 264), ([1], 0, 1, 512, 2048), ([3, 5], 0, 0, 72, 136), ([0, 8, 0], 0, 0, 24, 520),
    ([1] * 8, 0, 0, 512, 2048), ([0, 1, 0, 4, 0], 2, 1, 136, 4104), ([0, 0, 0], 3, 4, 16, 64), ([0] * 1020 + [1, 0, 2, 1], 1, 2, 16, 64),
    ([7, 0], 1, 0, 64, 7168), ([0, 2, 2, 2, 0, 2], 0, 0, 33 * 8, 256),
]


@pytest.mark.parametrize("case", range(len(FEW)))
@pytest.mark.parametrize("activation", [0, 1])
def test_few_rows(B, case, activation):
    """Up to eight rows, of any number of experts; the others keep what they held."""
    counts, first, behind, I, H = FEW[case]
    E, n = len(counts), sum(counts)
    P = first + n + behind
    x, w = randn(P, H, seed=1), randn(E, 2 * I, H, seed=2, scale=1.5 * H ** -0.5)
    own = torch.zeros(P, dtype=torch.bool, device="cuda")
    own[first:first + n] = True
    x[~own] = float("nan")
    row_w = randn(P, seed=3, dtype=F32) if case % 2 else None
    wide_x = torch.full((P, H + 8), float("nan"), dtype=BF16, device="cuda")
    wide_x[:, :H] = x
    h, a = torch.full((P, I), 7.0, dtype=BF16, device="cuda"), torch.full((P, 2 * I), 7.0, dtype=BF16, device="cuda")
    ws = workspace(B, P, H, I, E)
    ws.fill_(255)
    B.moe_gated_forward(wide_x[:, :H], w, offsets_of(counts, first), h, ws, a=a if case % 3 else None, row_w=row_w, activation=activation)
    assert B.moe_get_device_status(ws) == B.MOE_OK
    check_forward(h, a if case % 3 else None, x, w, row_w, counts, activation, first)
    assert bool((h[~own] == 7).all()) and bool((a[~own if case % 3 else own | True] == 7).all())


MORE = [
    # counts, first, rows behind the last, I, H: runs of more than eight rows, a warp's share of the sum that ends inside or
    # is empty, several rounds of columns
    ([9], 0, 0, 8, 8), ([16], 0, 0, 40, 248), ([3, 10, 0, 2], 0, 1, 72, 1000), ([1] * 16, 0, 0, 512, 1032), ([12], 2, 2, 2048, 1544),
    ([8, 8], 0, 0, 136, 40), ([0, 15, 1], 0, 0, 24, 2056), ([0] * 500 + [11], 3, 0, 16, 264), ([1], 0, 7, 4096, 6152), ([5], 0, 0, 4104, 1288),
]


@pytest.mark.parametrize("case", range(len(MORE)))
def test_up_to_sixteen_rows(B, case):
    """As above, on both sides of eight rows, and bit by bit the same from a second call."""
    counts, first, behind, I, H = MORE[case]
    E, n, activation = len(counts), sum(counts), case % 2
    P = first + n + behind
    x, w = randn(P, H, seed=11), randn(E, 2 * I, H, seed=12, scale=1.5 * H ** -0.5)
    own = torch.zeros(P, dtype=torch.bool, device="cuda")
    own[first:first + n] = True
    x[~own] = float("nan")
    row_w, got = randn(P, seed=13, dtype=F32) if case % 3 else None, []
    for _ in range(2):
        wide = [torch.full((P, k + 8 * (1 + case % 2)), 7.0, dtype=BF16, device="cuda") for k in (I, 2 * I)]
        h, a = wide[0][:, :I], wide[1][:, :2 * I]
        ws = workspace(B, P, H, I, E)
        B.moe_gated_forward(x, w, offsets_of(counts, first), h, ws, a=a, row_w=row_w, activation=activation)
        assert B.moe_get_device_status(ws) == B.MOE_OK
        check_forward(h, a, x, w, row_w, counts, activation, first)
        assert bool((h[~own] == 7).all()) and bool((a[~own] == 7).all())
        assert bool((wide[0][:, I:] == 7).all()) and bool((wide[1][:, 2 * I:] == 7).all())
        got.append((h, a))
    assert all(torch.equal(u, v) for u, v in zip(*got))


@pytest.mark.parametrize("rows", [5, 12])
def test_few_rows_infinities_and_nan_stay_in_their_row_and_column(B, rows):
    x, w = randn(rows, 264, seed=1), randn(1, 144, 264, seed=2, scale=0.1)
    offsets, ws = offsets_of([rows]), workspace(B, rows, 264, 72, 1)
    fine, h = (torch.empty(rows, 72, dtype=BF16, device="cuda") for _ in range(2))
    B.moe_gated_forward(x, w, offsets, fine, ws)
    x[3, 7], x[4, 263] = float("nan"), float("inf")
    w[0, 72 + 10, 100] = float("nan")
    B.moe_gated_forward(x, w, offsets, h, ws)
    good = torch.ones(rows, 72, dtype=torch.bool, device="cuda")
    good[[3, 4]] = False
    good[:, 10] = False
    assert torch.equal(h[good], fine[good]) and bool(h[3].isnan().all()) and bool(h[:, 10].isnan().all())
    assert bool(((~h[4].isfinite()) | (h[4] == 0)).all())


@pytest.mark.parametrize("bad", [[0, 5, 3, 8], [0, 4, 8, 9], [-1, 4, 8, 8], [0, -3, 8, 8]])
def test_few_rows_with_bad_offsets(B, bad):
    offsets = torch.tensor(bad, dtype=torch.int32, device="cuda")
    x, w, h = randn(8, 64), randn(3, 80, 64), torch.full((8, 40), 7.0, dtype=BF16, device="cuda")
    ws = workspace(B, 8, 64, 40, 3)
    B.moe_gated_forward(x, w, offsets, h, ws)
    assert B.moe_get_device_status(ws) == B.MOE_ERR_DEVICE_INDEX and bool((h == 7).all())


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("activation", [0, 1])
def test_back(B, case, activation):
    counts, I, H = CASES[case]
    E, P = len(counts), sum(counts)
    dy, w = randn(P, H, seed=4), randn(E, H, I, seed=5, scale=H ** -0.5)
    a = randn(P, 2 * I, seed=6, scale=1.5)
    row_w = randn(P, seed=3, dtype=F32) if case % 2 else None
    out = {"da": torch.full((P, 2 * I), 3.0, dtype=BF16, device="cuda"), "h": torch.full((P, I), 3.0, dtype=BF16, device="cuda"),
           "drow_w": torch.full((P,), 3.0, device="cuda")}
    if case == 2:
        del out["h"]
    if case == 3:
        del out["drow_w"]
    ws = workspace(B, P, H, I, E)
    B.moe_gated_dgrad(
        dy, w, offsets_of(counts), a, out["da"], ws, h=out.get("h"), row_w=row_w, drow_w=out.get("drow_w"),
        activation=activation)
    assert B.moe_get_device_status(ws) == B.MOE_OK
    check_back(out, dy, w, a, row_w, counts, activation)


def test_strides_rows_of_no_expert_and_repeats(B):
    """Row strides, a first offset above 0, rows behind the last: those keep what they held (NaN in them goes nowhere),
    and two calls give the same bits."""
    counts, first, I, H = [70, 0, 5, 300], 3, 72, 136
    E, P = len(counts), 3 + sum(counts) + 9
    own = torch.zeros(P, dtype=torch.bool, device="cuda")
    own[first:first + sum(counts)] = True

    def wide(t, ld, fill=None):
        w = torch.full((P, ld), float("nan"), dtype=t.dtype, device="cuda")
        v = w[:, :t.shape[1]]
        v.copy_(t) if fill is None else v.fill_(fill)
        return v

    x, w1, w2 = randn(P, H, seed=1), randn(E, 2 * I, H, seed=2, scale=H ** -0.5), randn(E, H, I, seed=3, scale=H ** -0.5)
    x[~own] = float("nan")
    row_w = randn(P, seed=4, dtype=F32)
    row_w[~own] = float("inf")
    xs, offsets = wide(x, H + 8), offsets_of(counts, first)
    results = []
    for _ in range(2):
        h, a = wide(x[:, :I], I + 24, 7.0), wide(torch.cat([x, x], 1)[:, :2 * I], 2 * I + 8, 7.0)
        ws = workspace(B, P, H, I, E)
        B.moe_gated_forward(xs, w1, offsets, h, ws, a=a, row_w=row_w)
        check_forward(h, a, x, w1, row_w, counts, 0, first)
        assert bool((h[~own] == 7).all()) and bool((a[~own] == 7).all())
        before = a.clone()
        dv, h2 = torch.full((P,), 7.0, device="cuda"), wide(x[:, :I], I + 8, 7.0)
        B.moe_gated_dgrad(xs, w2, offsets, a, a, ws, h=h2, row_w=row_w, drow_w=dv)       # da may be a
        assert B.moe_get_device_status(ws) == B.MOE_OK
        check_back({"da": a, "h": h2, "drow_w": dv}, x, w2, before, row_w, counts, 0, first)
        assert bool((a[~own] == 7).all()) and bool((dv[~own] == 7).all()) and bool((h2[~own] == 7).all())
        results.append([t.clone() for t in (h, before, a, h2, dv)])
    assert all(torch.equal(p, q) for p, q in zip(*results))


@pytest.mark.parametrize("bad", [[0, 5, 3, 16], [0, 4, 8, 17], [-1, 4, 8, 16]])
def test_bad_offsets_are_reported_and_nothing_is_written(B, bad):
    E, P, I, H = 3, 16, 40, 64
    offsets = torch.tensor(bad, dtype=torch.int32, device="cuda")
    x, w1, w2 = randn(P, H), randn(E, 2 * I, H), randn(E, H, I)
    a, h, da = (torch.full((P, n), 7.0, dtype=BF16, device="cuda") for n in (2 * I, I, 2 * I))
    dv, ws = torch.full((P,), 7.0, device="cuda"), workspace(B, P, H, I, E)
    B.moe_gated_forward(x, w1, offsets, h, ws, a=a)
    assert B.moe_get_device_status(ws) == B.MOE_ERR_DEVICE_INDEX
    B.moe_gated_dgrad(x, w2, offsets, a, da, ws, h=h, drow_w=dv)
    assert B.moe_get_device_status(ws) == B.MOE_ERR_DEVICE_INDEX
    assert all(bool((t == 7).all()) for t in (a, h, da, dv))


def test_infinities_and_nan_stay_in_their_row_and_expert(B):
    counts, I, H = [20, 20], 64, 64
    x, w1, w2 = randn(40, H, seed=1), randn(2, 2 * I, H, seed=2, scale=0.1), randn(2, H, I, seed=3, scale=0.1)
    outs = []
    for spoil in (False, True):
        y, v = x.clone(), w1.clone()
        if spoil:
            y[4, 3], y[25, 7] = float("nan"), float("inf")
            v[1, 5] = float("nan")                         # a gate column of the second expert
        h, a, ws = torch.zeros(40, I, dtype=BF16, device="cuda"), torch.zeros(40, 2 * I, dtype=BF16, device="cuda"), workspace(B, 40, H, I, 2)
        B.moe_gated_forward(y, v, offsets_of(counts), h, ws, a=a)
        da, dv = torch.zeros_like(a), torch.zeros(40, device="cuda")
        B.moe_gated_dgrad(y, w2, offsets_of(counts), a, da, ws, drow_w=dv)
        outs.append((h, a, da, dv))
    fine = torch.ones(40, dtype=torch.bool, device="cuda")
    fine[4] = fine[25] = False
    cols = torch.ones(2 * I, dtype=torch.bool, device="cuda")
    cols[5] = cols[I + 5] = False
    (h0, a0, da0, dv0), (h1, a1, da1, dv1) = outs
    assert torch.equal(h0[:20][fine[:20]], h1[:20][fine[:20]]) and torch.equal(a0[fine][:, cols], a1[fine][:, cols])
    assert torch.equal(da0[fine][:, cols], da1[fine][:, cols]) and torch.equal(dv0[:20][fine[:20]], dv1[:20][fine[:20]])
    assert bool(h1[4].isnan().all()) and bool(h1[20:, 5].isnan().all())


def test_activations_far_out(B):
    """Gates of any finite size: f and f' go to 0 and to z, 1, without infinities on the way."""
    I = H = 64
    z = torch.tensor([0.0, 1e-30, -1e-30, 20, -20, 88, -88, 95, -95, 1e4, -1e4, 1e19, -1e19, 3e38, -3e38, 12, -12],
                     device="cuda").to(BF16)
    P = len(z)
    a = torch.ones(P, 2 * I, dtype=BF16, device="cuda")
    a[:, :I] = z[:, None]
    dy = torch.zeros(P, H, dtype=BF16, device="cuda")
    dy[:, 0] = 1
    w2 = torch.zeros(1, H, I, dtype=BF16, device="cuda")
    w2[0, 0] = 1
    for activation in (0, 1):
        da, h, ws = torch.empty_like(a), torch.empty(P, I, dtype=BF16, device="cuda"), workspace(B, P, H, I, 1)
        B.moe_gated_dgrad(dy, w2, offsets_of([P]), a, da, ws, h=h, activation=activation)
        f, df, _, _ = act(z.double().clamp(-1e6, 1e6), activation)
        f, df = torch.where(z.double().abs() > 1e6, z.double().clamp(min=0), f), torch.where(z.double().abs() > 1e6, (z > 0).double(), df)
        for got, ref in ((h, f), (da[:, I:], f), (da[:, :I], df)):
            off = (got.double() - ref[:, None]).abs()
            # quotients beyond 2^126 flush to 0: up to 88 * 2^-126 of f and f'
            assert bool((off <= (U + 300 * S32) * ref.abs()[:, None] + 1e-34).all())


def test_streams_and_graphs(B):
    """Two calls at once on two streams, and a captured call replayed on new rows, give the eager call's bits."""
    counts, I, H = [33, 100, 0, 7], 136, 264
    E, P = len(counts), sum(counts)
    w1, w2, offsets = randn(E, 2 * I, H, seed=2, scale=0.05), randn(E, H, I, seed=3, scale=0.05), offsets_of(counts)

    def call(x, o):
        B.moe_gated_forward(x, w1, offsets, o["h"], o["ws"], a=o["a"])
        B.moe_gated_dgrad(x, w2, offsets, o["a"], o["da"], o["ws"], drow_w=o["dv"])

    def outs():
        return {"h": torch.zeros(P, I, dtype=BF16, device="cuda"), "a": torch.zeros(P, 2 * I, dtype=BF16, device="cuda"),
                "da": torch.zeros(P, 2 * I, dtype=BF16, device="cuda"), "dv": torch.zeros(P, device="cuda"),
                "ws": workspace(B, P, H, I, E)}

    xs = [randn(P, H, seed=s) for s in (7, 8)]
    want = []
    for x in xs:
        o = outs()
        call(x, o)
        want.append(o)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in xs], [outs() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, x, o in zip(streams, xs, got):
            with torch.cuda.stream(st):
                call(x, o)
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert all(torch.equal(o[k], w[k]) for k in ("h", "a", "da", "dv"))
    x, o, graph = xs[0].clone(), outs(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(x, o)
    for y, w in zip(xs[::-1], want[::-1]):
        x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o[k], w[k]) for k in ("h", "a", "da", "dv"))


def test_a_wait_that_runs_out_is_reported(B, monkeypatch):
    counts, I, H = [40, 60], 64, 128
    x, w1, w2 = randn(100, H), randn(2, 2 * I, H), randn(2, H, I)
    a, h, da = (torch.zeros(100, n, dtype=BF16, device="cuda") for n in (2 * I, I, 2 * I))
    dv, ws = torch.full((100,), 7.0, device="cuda"), workspace(B, 100, H, I, 2)
    monkeypatch.setenv("MOE_MXQ_DEBUG_INJECT_WAIT", "1")
    B.moe_gated_forward(x, w1, offsets_of(counts), h, ws, a=a)
    assert B.moe_get_device_status(ws) == B.MOE_ERR_TIMEOUT
    B.moe_gated_dgrad(x, w2, offsets_of(counts), a, da, ws, drow_w=dv)
    assert B.moe_get_device_status(ws) == B.MOE_ERR_TIMEOUT
    monkeypatch.delenv("MOE_MXQ_DEBUG_INJECT_WAIT")
    B.moe_gated_forward(x, w1, offsets_of(counts), h, ws, a=a)
    assert B.moe_get_device_status(ws) == B.MOE_OK
    check_forward(h, a, x, w1, None, counts, 0)


def test_no_rows(B):
    w1, w2 = randn(2, 64, 64), randn(2, 64, 32)
    new = lambda n: torch.zeros(0, n, dtype=BF16, device="cuda")      # noqa: E731
    ws = workspace(B, 0, 64, 32, 2)
    ws.fill_(255)
    B.moe_gated_forward(new(64), w1, offsets_of([0, 0]), new(32), ws)
    assert B.moe_get_device_status(ws) == B.MOE_OK
    ws.fill_(255)
    B.moe_gated_dgrad(new(64), w2, offsets_of([0, 0]), new(64), new(64), ws, drow_w=torch.zeros(0, device="cuda"))
    assert B.moe_get_device_status(ws) == B.MOE_OK


def leaf_gradients(n, l1, l2, activation, db):
    """b and the gradients in float64 by torch's differentiation."""
    leaf = [t.double().requires_grad_() for t in (n, l1, l2)]
    gate, up = (leaf[0] @ leaf[1].T).split(l2.shape[1], 1)
    q = gate if activation == 0 else 2 * (2 / np.pi) ** 0.5 * (gate + 0.044715 * gate ** 3)
    out = (gate * torch.sigmoid(q) * up) @ leaf[2].T
    return out.detach(), torch.autograd.grad((out * db.double()).sum(), leaf)


@pytest.mark.parametrize("T,H,I,activation", [(0, 64, 32, 0), (1, 256, 128, 1), (37, 136, 72, 0), (700, 264, 520, 1)])
def test_block_and_gradients(B, T, H, I, activation):
    """Every tensor rounded to BF16 on the way (h, da) carries at most 2^-8 of its values, and no result passes more
    than three: 3 * 2^-8 in norm."""
    from moe_expert_layer_counting_gb300 import GatedFeedForward
    n, db = randn(T, H, seed=1), randn(T, H, seed=2)
    l1, l2 = randn(2 * I, H, seed=3, scale=H ** -0.5), randn(H, I, seed=4, scale=I ** -0.5)
    block = GatedFeedForward(l1, l2, activation)
    b, s = block.forward(n)
    dl1, dl2 = torch.full((2 * I, H), 9.0, device="cuda"), torch.full((H, I), 9.0, device="cuda")
    dn = block.backward(db, s, dl1, dl2)
    assert block.status() == 0
    ref, grads = leaf_gradients(n, l1, l2, activation, db)
    for got, want in ((b, ref), (dn, grads[0]), (dl1, grads[1]), (dl2, grads[2])):
        assert float((got.double() - want).norm()) <= 3 * U * float(want.norm())
    served, kept = block.forward(n, keep=False)
    assert kept is None and torch.equal(served, b)
    again = dl1.clone()
    block.backward(db, s, dl1, dl2, accumulate=True)
    assert torch.allclose(dl1, 2 * again)


def test_block_against_differences(B):
    """The gradient along a direction against the loss's difference, computed in float64 with the block's formula."""
    from moe_expert_layer_counting_gb300 import GatedFeedForward
    T, H, I = 19, 72, 40
    n, db = randn(T, H, seed=1), randn(T, H, seed=2)
    l1, l2 = randn(2 * I, H, seed=3, scale=H ** -0.5), randn(H, I, seed=4, scale=I ** -0.5)
    block = GatedFeedForward(l1, l2)
    _, s = block.forward(n)
    dl1, dl2 = torch.empty(2 * I, H, device="cuda"), torch.empty(H, I, device="cuda")
    dn = block.backward(db, s, dl1, dl2)

    def loss(a, b, c):
        gate, up = (a @ b.T).split(I, 1)
        return ((gate * torch.sigmoid(gate) * up) @ c.T * db.double()).sum()

    base = [t.double() for t in (n, l1, l2)]
    step = 1e-4
    for i, grad in enumerate((dn, dl1, dl2)):
        d = torch.randn(grad.shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda").double()
        up, down = ([t + sign * step * d if j == i else t for j, t in enumerate(base)] for sign in (1, -1))
        diff = (loss(*up) - loss(*down)) / (2 * step)
        # the gradient's own error in norm (3 * 2^-8), along the direction; the difference's is of order step^2
        assert abs(float((grad.double() * d).sum() - diff)) <= 3 * U * float(grad.double().norm() * d.norm())


@pytest.mark.parametrize("T,E,H,I,k", [(1, 4, 64, 32, 1), (50, 6, 136, 64, 3)])
def test_expert_layer_with_fused_activation(B, T, E, H, I, k):
    """TrainableExperts(fused=True) against the layer of separate operations: no result of either is more than
    6 * 2^-8 in norm from the definition (test_gpu_training.py)."""
    from moe_expert_layer_counting_gb300 import TrainableExperts
    n, db = randn(T, H, seed=1), randn(T, H, seed=2)
    l1, l2 = randn(E, 2 * I, H, seed=3, scale=H ** -0.5), randn(E, H, I, seed=4, scale=I ** -0.5)
    g = torch.Generator(device="cuda").manual_seed(5)
    idx = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]).int()
    idx[::3, 0] = -1
    w = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
    got = []
    for fused in (False, True):
        layer = TrainableExperts(l1, l2, fused=fused)
        b, s = layer.forward(n, idx, w)
        dl1, dl2 = torch.empty(E, 2 * I, H, device="cuda"), torch.empty(E, H, I, device="cuda")
        dn, dw = layer.backward(db, s, dl1, dl2)
        assert layer.status() == 0
        got.append((b, dn, dl1, dl2, dw))
    for x, y in zip(*got):
        assert float((x.double() - y.double()).norm()) <= 12 * U * float(x.double().norm())
