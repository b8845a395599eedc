"""The BF16 products grouped by expert and their gradients against float64.

Tolerance.  A product of two BF16 values is exact in float32, so an output
carries the error of its float32 sum, at most (terms + 1) * 2^-23 of the sum
of the terms' magnitudes (the tensor core truncates: one unit in the last
place per addition), and for a BF16 output one rounding, at most 2^-8 of its
value (8 significant bits).  Both bounds are applied to every element.
"""
import numpy as np
import pytest
import torch

from tests import helpers as Hp

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return Hp.lib()


def offsets_of(counts, first=0):
    return torch.tensor([first, *(first + np.cumsum(counts))], dtype=torch.int32, device="cuda")


def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF16)


def workspace(B, P, N, K, E):
    return torch.empty(B.moe_grouped_workspace_size(P, N, K, E), dtype=torch.uint8, device="cuda")


def close(got, ref, magnitude, terms):
    """Every element within the bound of the file's comment."""
    rounding = 2.0 ** -8 if got.dtype == BF16 else 0.0
    bound = rounding * ref.abs() + (1 + rounding) * (terms + 1) * 2.0 ** -23 * magnitude + 1e-38
    off = (got.double() - ref).abs()
    assert bool((off <= bound).all()), f"worst {float((off / bound).max()):.3f} of the bound"


def reference(op, counts, rows, other, first=0):
    """(result, sum of the magnitudes) per expert segment in float64: list of (a, b, ref, mag, terms)."""
    out, a = [], first
    for e, c in enumerate(counts):
        b = a + c
        if op == "forward":
            l, r = rows[a:b].double(), other[e].double().T
        elif op == "dgrad":
            l, r = rows[a:b].double(), other[e].double()
        else:
            l, r = rows[a:b].double().T, other[a:b].double()
        out.append((a, b, l @ r, l.abs() @ r.abs(), l.shape[1]))
        a = b
    return out


CASES = [
    # counts, N, K
    ([1], 8, 8),
    ([1], 256, 2048),
    ([0, 1, 0], 64, 128),
    ([16, 32, 64, 128, 256], 256, 256),
    ([15, 17, 31, 33, 63, 65, 127, 129, 255, 257], 264, 200),
    ([0, 0, 700, 0, 1, 1025], 520, 1032),
    ([256, 257, 288, 289, 320, 321, 384, 512, 513, 576, 577, 640, 641, 768, 769], 136, 328),
    ([2300, 64, 65, 1], 392, 456),
    ([3] * 100 + [0] * 28, 128, 72),
    ([40] * 16, 1024, 512),
    ([2, 0, 5] * 341 + [1], 16, 64),          # 1024 experts
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("op", ["forward", "dgrad"])
def test_rows(B, op, case):
    counts, N, K = CASES[case]
    E, P = len(counts), sum(counts)
    R, M = (K, N) if op == "forward" else (N, K)
    x, w = randn(P, R, seed=1), randn(E, N, K, seed=2, scale=0.1)
    out = torch.full((P, M), 3.0, dtype=BF16, device="cuda")
    ws = workspace(B, P, N, K, E)
    call = B.moe_grouped_forward if op == "forward" else B.moe_grouped_dgrad
    call(x, w, offsets_of(counts), out, ws)
    assert B.moe_get_device_status(ws) == B.MOE_OK
    for a, b, ref, mag, terms in reference(op, counts, x, w):
        close(out[a:b], ref, mag, terms)


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_weights(B, dtype, case):
    counts, N, K = CASES[case]
    E, P = len(counts), sum(counts)
    dy, x = randn(P, N, seed=3), randn(P, K, seed=4)
    dw = torch.full((E, N, K), 3.0, dtype=dtype, device="cuda")
    ws = workspace(B, P, N, K, E)
    B.moe_grouped_wgrad(dy, x, offsets_of(counts), dw, ws)
    assert B.moe_get_device_status(ws) == B.MOE_OK
    for e, (_, _, ref, mag, terms) in enumerate(reference("wgrad", counts, dy, x)):
        close(dw[e], ref, mag, terms)            # an expert without rows: zeros


@pytest.mark.parametrize("counts", [[5, 0, 90], [64, 64], [0]])
def test_weights_accumulate(B, counts):
    E, P, N, K = len(counts), sum(counts), 72, 136
    dy, x = randn(P, N, seed=5), randn(P, K, seed=6)
    base = torch.randn(E, N, K, device="cuda")
    dw = base.clone()
    ws = workspace(B, P, N, K, E)
    B.moe_grouped_wgrad(dy, x, offsets_of(counts), dw, ws, accumulate=True)
    for e, (_, _, ref, mag, terms) in enumerate(reference("wgrad", counts, dy, x)):
        close(dw[e], base[e].double() + ref, base[e].double().abs() + mag, terms + 1)
        if counts[e] == 0:
            assert torch.equal(dw[e], base[e])


def test_long_segment_in_float32(B):
    """16 384 rows of one expert: a float32 gradient keeps float32's precision over a long sum (error in norm at
    most 2e-6, which truncation over the whole length would pass several times over)."""
    P, N, K = 16384, 128, 256
    dy, x = randn(P, N, seed=7), randn(P, K, seed=8)
    dw = torch.empty(1, N, K, device="cuda")
    ws = workspace(B, P, N, K, 1)
    B.moe_grouped_wgrad(dy, x, offsets_of([P]), dw, ws)
    ref = dy.double().T @ x.double()
    assert float((dw[0].double() - ref).norm() / ref.norm()) <= 2e-6


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_weights_of_more_items_than_pairs_of_sms(B, dtype):
    """Experts of more than 4096 rows, short and empty ones, 280 tiles of dw, two calls at a time on two streams."""
    counts, N, K = [4100, 0, 3, 70, 0, 5000, 129, 17], 1032, 1544
    E, P = len(counts), sum(counts)
    dy, x, off = randn(P, N, seed=3), randn(P, K, seed=4), offsets_of(counts)
    dws = [torch.full((E, N, K), 3.0, dtype=dtype, device="cuda") for _ in range(2)]
    spaces, streams = [workspace(B, P, N, K, E) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for dw, ws, stream in zip(dws, spaces, streams):
            B.moe_grouped_wgrad(dy, x, off, dw, ws, stream=stream)
    torch.cuda.synchronize()
    assert all(B.moe_get_device_status(ws) == B.MOE_OK for ws in spaces)
    for e, (_, _, ref, mag, terms) in enumerate(reference("wgrad", counts, dy, x)):
        close(dws[0][e], ref, mag, terms)
    assert torch.equal(dws[0], dws[1])


def test_many_items_with_bad_offsets_or_a_wait_that_runs_out(B, monkeypatch):
    """What is left of the launch is dropped: the call ends, reports, and the next one is right."""
    E, P, N, K = 400, 800, 256, 264
    dy, x, ws = randn(P, N, seed=1), randn(P, K, seed=2), workspace(B, P, N, K, E)
    dw = torch.full((E, N, K), 3.0, dtype=BF16, device="cuda")
    bad = offsets_of([2] * E).clone()
    bad[7] = 900
    B.moe_grouped_wgrad(dy, x, bad, dw, ws)
    assert B.moe_get_device_status(ws) == B.MOE_ERR_DEVICE_INDEX and bool((dw == 3.0).all())
    monkeypatch.setenv("MOE_MXQ_DEBUG_INJECT_WAIT", "1")
    B.moe_grouped_wgrad(dy, x, offsets_of([2] * E), dw, ws)
    assert B.moe_get_device_status(ws) == B.MOE_ERR_TIMEOUT
    monkeypatch.delenv("MOE_MXQ_DEBUG_INJECT_WAIT")
    B.moe_grouped_wgrad(dy, x, offsets_of([2] * E), dw, ws)
    assert B.moe_get_device_status(ws) == B.MOE_OK
    for e, (_, _, ref, mag, terms) in enumerate(reference("wgrad", [2] * E, dy, x)):
        close(dw[e], ref, mag, terms)


@pytest.mark.parametrize("first,last", [(0, 9), (6, 0), (5, 4)])
def test_rows_of_no_expert_are_left_alone(B, first, last):
    """Rows outside [offsets[0], offsets[E]) are not written, whatever they hold (NaN here), and reach no result."""
    counts, N, K = [19, 0, 70], 136, 200
    E, P = len(counts), first + sum(counts) + last
    x, dy, w = randn(P, K, seed=1), randn(P, N, seed=2), randn(E, N, K, seed=3)
    for t in (x, dy):
        t[:first] = float("nan")
        t[P - last:] = float("nan")
    off = offsets_of(counts, first)
    y = torch.full((P, N), 3.0, dtype=BF16, device="cuda")
    dx = torch.full((P, K), 3.0, dtype=BF16, device="cuda")
    dw = torch.empty(E, N, K, device="cuda")
    ws = workspace(B, P, N, K, E)
    B.moe_grouped_forward(x, w, off, y, ws)
    B.moe_grouped_dgrad(dy, w, off, dx, ws)
    B.moe_grouped_wgrad(dy, x, off, dw, ws)
    end = P - last
    for out in (y, dx):
        assert bool((out[:first] == 3.0).all()) and bool((out[end:] == 3.0).all())
        assert bool(out[first:end].isfinite().all())
    for e, (_, _, ref, mag, terms) in enumerate(reference("wgrad", counts, dy, x, first)):
        close(dw[e], ref, mag, terms)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_infinities_and_nan_stay_with_their_expert(B, bad):
    counts, N, K = [5, 30, 3, 17, 64], 128, 192
    E, P = len(counts), sum(counts)
    x, dy, w = randn(P, K, seed=1), randn(P, N, seed=2), randn(E, N, K, seed=3)
    off = offsets_of(counts)
    a, b = int(off[2]), int(off[3])
    x[a:b], dy[a:b], w[2] = bad, bad, bad
    y = torch.empty(P, N, dtype=BF16, device="cuda")
    dx = torch.empty(P, K, dtype=BF16, device="cuda")
    dw = torch.empty(E, N, K, dtype=BF16, device="cuda")
    ws = workspace(B, P, N, K, E)
    B.moe_grouped_forward(x, w, off, y, ws)
    B.moe_grouped_dgrad(dy, w, off, dx, ws)
    B.moe_grouped_wgrad(dy, x, off, dw, ws)
    for out, seg in ((y, slice(a, b)), (dx, slice(a, b)), (dw, slice(2, 3))):
        fine = out.isfinite().flatten(1).all(1)
        assert not bool(fine[seg].any())
        fine[seg] = True
        assert bool(fine.all())


def test_row_strides(B):
    """Row tensors that are column ranges of wider ones."""
    counts, N, K = [33, 7, 260], 264, 136
    E, P = len(counts), sum(counts)
    wide = {n: randn(P, c + 48, seed=i) for i, (n, c) in enumerate((("x", K), ("dy", N), ("y", N), ("dx", K)))}
    kept = {n: t.clone() for n, t in wide.items()}
    x, dy, y, dx = (wide[n][:, 16:16 + c] for n, c in (("x", K), ("dy", N), ("y", N), ("dx", K)))
    w, off, ws = randn(E, N, K, seed=9), offsets_of(counts), workspace(B, P, N, K, E)
    dw = torch.empty(E, N, K, device="cuda")
    B.moe_grouped_forward(x, w, off, y, ws)
    B.moe_grouped_dgrad(dy, w, off, dx, ws)
    B.moe_grouped_wgrad(dy, x, off, dw, ws)
    for op, src, out in (("forward", x, y), ("dgrad", dy, dx)):
        for a, b, ref, mag, terms in reference(op, counts, src, w):
            close(out[a:b], ref, mag, terms)
    for e, (_, _, ref, mag, terms) in enumerate(reference("wgrad", counts, dy, x)):
        close(dw[e], ref, mag, terms)
    for n, c in (("y", N), ("dx", K)):             # nothing beside the columns is touched
        assert torch.equal(wide[n][:, :16], kept[n][:, :16]) and torch.equal(wide[n][:, 16 + c:], kept[n][:, 16 + c:])


def test_outputs_beyond_2_pow_31_values(B):
    """A row tensor of 2.2e9 values: the last rows are where they should be."""
    P, N, K = 270_000, 8192, 64
    counts = [P - 300, 300]
    x, w = randn(P, K, seed=1), randn(2, N, K, seed=2)
    y = torch.empty(P, N, dtype=BF16, device="cuda")
    ws = workspace(B, P, N, K, 2)
    B.moe_grouped_forward(x, w, offsets_of(counts), y, ws)
    for a, b, e in ((0, 64, 0), (P - 364, P - 300, 0), (P - 300, P, 1)):
        l, r = x[a:b].double(), w[e].double().T
        close(y[a:b], l @ r, l.abs() @ r.abs(), K)
    # and as an input: the gradient of those rows
    dx = torch.empty(P, K, dtype=BF16, device="cuda")
    B.moe_grouped_dgrad(y, w, offsets_of(counts), dx, ws)
    l, r = y[P - 300:].double(), w[1].double()
    close(dx[P - 300:], l @ r, l.abs() @ r.abs(), N)


def test_gradients_against_differences(B):
    """L(x, w) = sum c * y is linear in x and in w, so a central difference of the float64 forward along a direction
    is its derivative; it has to be the gradients' product with that direction (their BF16 rounding, 2^-8 of each
    term, is the tolerance)."""
    counts, N, K = [9, 0, 40], 72, 104
    E, P = len(counts), sum(counts)
    x, w, c = randn(P, K, seed=1), randn(E, N, K, seed=2), randn(P, N, seed=3)
    off, ws = offsets_of(counts), workspace(B, P, N, K, E)
    dx, dw = torch.empty(P, K, dtype=BF16, device="cuda"), torch.empty(E, N, K, dtype=BF16, device="cuda")
    B.moe_grouped_dgrad(c, w, off, dx, ws)
    B.moe_grouped_wgrad(c, x, off, dw, ws)

    def loss(x, w):
        return sum((c[a:b].double() * (x[a:b] @ w[e].T)).sum()
                   for e, (a, b) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())))

    xd, wd = x.double(), w.double()
    for seed in range(3):
        vx, vw = randn(P, K, seed=10 + seed).double(), randn(E, N, K, seed=20 + seed).double()
        for got, v, diff in ((dx, vx, (loss(xd + vx, wd) - loss(xd - vx, wd)) / 2),
                             (dw, vw, (loss(xd, wd + vw) - loss(xd, wd - vw)) / 2)):
            terms = got.double() * v
            assert abs(float(terms.sum() - diff)) <= float(terms.abs().sum()) * 2.0 ** -8


def test_same_bits_again_on_another_stream_and_in_a_graph(B):
    counts, N, K = [100, 0, 37, 300], 512, 384
    E, P = len(counts), sum(counts)
    x, dy, w = randn(P, K, seed=1), randn(P, N, seed=2), randn(E, N, K, seed=3)
    off, ws = offsets_of(counts), workspace(B, P, N, K, E)

    def outputs():
        return (torch.zeros(P, N, dtype=BF16, device="cuda"), torch.zeros(P, K, dtype=BF16, device="cuda"),
                torch.zeros(E, N, K, device="cuda"))

    def call(out, stream=None):
        B.moe_grouped_forward(x, w, off, out[0], ws, stream=stream)
        B.moe_grouped_dgrad(dy, w, off, out[1], ws, stream=stream)
        B.moe_grouped_wgrad(dy, x, off, out[2], ws, stream=stream)

    first = outputs()
    call(first)
    torch.cuda.synchronize()
    second, side = outputs(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(second, stream=side)
    torch.cuda.synchronize()
    third = outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(third)
    for t in third:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("offsets", [[0, 5, 4, 10], [-1, 2, 4, 10], [0, 5, 8, 11], [0, 2 ** 31 - 1, 8, 10]])
def test_bad_offsets_are_reported_and_write_nothing(B, offsets):
    E, P, N, K = 3, 10, 64, 64
    x, w = randn(P, K), randn(E, N, K)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    ws = workspace(B, P, N, K, E)
    y = torch.full((P, N), 3.0, dtype=BF16, device="cuda")
    dw = torch.full((E, N, K), 3.0, device="cuda")
    B.moe_grouped_forward(x, w, off, y, ws)
    assert B.moe_get_device_status(ws) == B.MOE_ERR_DEVICE_INDEX
    B.moe_grouped_dgrad(x, w, off, y, ws)
    assert B.moe_get_device_status(ws) == B.MOE_ERR_DEVICE_INDEX
    B.moe_grouped_wgrad(x, x, off, dw, ws)
    assert B.moe_get_device_status(ws) == B.MOE_ERR_DEVICE_INDEX
    assert bool((y == 3.0).all()) and bool((dw == 3.0).all())
    B.moe_grouped_forward(x, w, offsets_of([4, 0, 6]), y, ws)          # the next call resets the status
    assert B.moe_get_device_status(ws) == B.MOE_OK and not bool((y == 3.0).all())


def test_no_rows(B):
    E, N, K = 2, 64, 64
    x, y = torch.empty(0, K, dtype=BF16, device="cuda"), torch.empty(0, N, dtype=BF16, device="cuda")
    w, off = randn(E, N, K), torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    ws = workspace(B, 0, N, K, E)
    B.moe_grouped_forward(x, w, off, y, ws)
    B.moe_grouped_dgrad(y, w, off, x, ws)
    for dtype in (BF16, torch.float32):
        dw = torch.ones(E, N, K, dtype=dtype, device="cuda")
        B.moe_grouped_wgrad(y, x, off, dw, ws)
        assert not bool(dw.any())
    dw = torch.ones(E, N, K, device="cuda")
    B.moe_grouped_wgrad(y, x, off, dw, ws, accumulate=True)
    assert bool((dw == 1).all()) and B.moe_get_device_status(ws) == B.MOE_OK


def test_a_wait_that_runs_out_is_reported(B, monkeypatch):
    """The debug wait of moe_get_device_status's description: status, site, and a context that still works."""
    counts, N, K = [70, 3], 128, 128
    E, P = 2, 73
    x, w, off, ws = randn(P, K, seed=1), randn(E, N, K, seed=2), offsets_of(counts), workspace(B, P, N, K, E)
    y = torch.empty(P, N, dtype=BF16, device="cuda")
    dw = torch.empty(E, N, K, device="cuda")
    monkeypatch.setenv("MOE_MXQ_DEBUG_INJECT_WAIT", "1")
    for call in (lambda: B.moe_grouped_forward(x, w, off, y, ws), lambda: B.moe_grouped_wgrad(x, x, off, dw, ws)):
        call()
        assert B.moe_get_device_status(ws) == B.MOE_ERR_TIMEOUT
        assert ws[:12].view(torch.int32).tolist()[1:] == [1, 7]
    monkeypatch.delenv("MOE_MXQ_DEBUG_INJECT_WAIT")
    B.moe_grouped_forward(x, w, off, y, ws)
    assert B.moe_get_device_status(ws) == B.MOE_OK
    for a, b, ref, mag, terms in reference("forward", counts, x, w):
        close(y[a:b], ref, mag, terms)
