"""Matrices orthogonalised by Newton-Schulz products, and Muon's step, against float64.

Tolerance, in norm.  The kernels round each iterate, S and Q to FP16 (half a step is 2^-12 of a value), and what that
does to the result depends on the matrix: the polynomial's derivative is up to 3.4 an iteration where singular values are
small.  ``rounded`` below is the definition in float64 with the same roundings; the kernels' sums in float32 change which
way a value is rounded, not how far, so that their error is as large as ``rounded``'s up to the draw: within 1.5 times
of it for many values, and four half steps (1e-3) more for few.  The output's own rounding is 2^-8 (BF16) or 2^-24.
A sum in the tensor core truncates (2^-23 of the running sum a term): 4096 terms add 5e-4 at the very most, which the same
1e-3 covers.
"""
import math

import pytest
import torch

from tests import helpers as Hp

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -8
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return Hp.lib()


def randn(*shape, seed=0, scale=1.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def fp16(x):
    return (x * 4096).half().double() / 4096


def orthogonal(x, steps=5, coefficients=COEFFICIENTS, eps=1e-7, rounded=False):
    """Of one matrix, in float64; rounded: with the kernels' roundings to FP16."""
    a, b, c = coefficients
    x = x.double()
    norm = max(float(x.square().sum().sqrt()), eps)
    x = x / norm if norm else x
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    one = torch.eye(x.shape[0], dtype=torch.float64, device=x.device)
    if rounded:
        x = fp16(x)
    for _ in range(steps):
        gram = x @ x.T
        if rounded and c:
            s = fp16(gram + b / (2 * c) * one)
            x = fp16(fp16(c * s @ s + (a - b * b / (4 * c)) * one) @ x)
        elif rounded:
            x = fp16(fp16(a * one + b * gram) @ x)
        else:
            x = a * x + (b * gram + c * gram @ gram) @ x
    return x.T if tall else x


def error(got, ref):
    return float((got.double() - ref).norm()) / max(float(ref.norm()), 1e-300)


def check(got, x, **how):
    for o, m in zip(got, x):
        ref = orthogonal(m, **how)
        emulated = error(orthogonal(m, rounded=True, **how), ref)
        assert error(o, ref) <= 1.5 * emulated + 1e-3 + (U if got.dtype == BF16 else 0), (error(o, ref), emulated)


def ortho(B, x, dtype=BF16, **how):
    out = torch.full(x.shape, 9.0, dtype=dtype, device="cuda")
    E, N, K = x.shape if x.dim() == 3 else (1, *x.shape)
    ws = torch.empty(B.moe_muon_workspace_size(E, N, K), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    B.moe_orthogonalize(x, out, ws, **how)
    assert B.moe_get_device_status(ws) == B.MOE_OK
    return out


SHAPES = [(1, 1, 1), (1, 1, 7), (2, 5, 3), (3, 2, 300), (2, 64, 64), (2, 256, 128), (1, 300, 1000), (1, 1000, 300), (5, 40, 72),
          (1, 257, 513), (2, 520, 264), (1, 31, 4100), (2, 128, 384), (2, 385, 128), (1, 127, 3070), (3, 800, 24), (1, 129, 129),
          (2, 2000, 128), (1, 17, 1600), (1, 1024, 2048), (1, 2050, 700), (90, 16, 24), (3, 513, 513)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_orthogonalize(B, shape, dtype):
    x = randn(*shape, seed=sum(shape), scale=1e-3, dtype=dtype)
    check(ortho(B, x, F32 if dtype == BF16 else BF16), x)


def kept_diagonals(x):
    """As orthogonal(rounded=True), but for what FP16 leaves of the diagonals: of S it goes into Q's, of Q into a factor of X's
    row."""
    a, b, c = COEFFICIENTS
    x = x.double()
    x = x / x.square().sum().sqrt()
    x = fp16(x.T if x.shape[0] > x.shape[1] else x)
    one = torch.eye(x.shape[0], dtype=torch.float64, device=x.device)
    for _ in range(5):
        s = x @ x.T + b / (2 * c) * one
        r = fp16(s)
        q = c * r @ r + (a - b * b / (4 * c)) * one + torch.diag(2 * c * r.diag() * (s - r).diag())
        x = fp16((q.diag() / fp16(q).diag())[:, None] * (fp16(q) @ x))
    return x


@pytest.mark.parametrize("shape", [(3, 897, 32), (2, 31, 2660), (40, 40, 600), (2, 128, 384), (5, 562, 40), (1, 48, 256), (160, 500, 60)])
def test_small_matrices_keep_their_diagonals(B, shape):
    """Of matrices of 12 000 values and more the draw of the roundings plays no part but for 1.5 times, and sums of up to 2660
    terms in the tensor core add 2660 * 2^-23 = 3.2e-4 at most; the results' own rounding (float32) nothing."""
    x = randn(*shape, seed=sum(shape), scale=1e-3, dtype=F32)
    for o, m in list(zip(ortho(B, x, F32), x))[:6]:
        ref, tall = orthogonal(m), m.shape[0] > m.shape[1]
        emulated = kept_diagonals(m)
        assert error(o, ref) <= 1.5 * error(emulated.T if tall else emulated, ref) + 3.2e-4


def test_matrix_in_place_and_repeats(B):
    x = randn(200, 136, seed=3)
    first, second = ortho(B, x), ortho(B, x)
    assert torch.equal(first, second)
    ws = torch.empty(B.moe_muon_workspace_size(1, 200, 136), dtype=torch.uint8, device="cuda")
    B.moe_orthogonalize(x, x, ws)
    assert torch.equal(x, first)


@pytest.mark.parametrize("how", [dict(steps=0), dict(steps=1), dict(steps=8), dict(coefficients=(1.5, -0.5, 0.0), steps=12),
                                 dict(coefficients=(1.875, -1.25, 0.375), steps=7), dict(eps=1.0)])
@pytest.mark.parametrize("shape", [(2, 96, 160), (2, 160, 96), (2, 96, 800), (2, 160, 240), (2, 240, 160)])
def test_other_polynomials(B, shape, how):
    x = randn(*shape, seed=5, scale=1e-3, dtype=F32)
    check(ortho(B, x, F32, **how), x, **how)


def test_orthogonal_rows(B):
    """After enough steps of a polynomial that converges (1.875, -1.25, 0.375), the rows are orthonormal: o o^T is I within
    the roundings of the last iterate and of o o^T itself."""
    o = ortho(B, randn(1, 128, 512, seed=6), F32, coefficients=(1.875, -1.25, 0.375), steps=12)[0].double()
    assert float((o @ o.T - torch.eye(128, device="cuda")).abs().max()) <= 8 * 2.0 ** -11


def test_few_large_singular_values(B):
    x = (randn(1, 256, 8, seed=1, dtype=F32) @ randn(1, 8, 640, seed=2, dtype=F32) + 0.1 * randn(1, 256, 640, seed=3, dtype=F32))
    check(ortho(B, x, F32), x)


@pytest.mark.parametrize("scale", [1e-15, 1e15])
def test_far_scales(B, scale):
    """The squares stay within float32: the result is that of the matrix at scale 1 (eps aside)."""
    x = randn(1, 64, 96, seed=4, dtype=F32)
    check(ortho(B, x * scale, F32, eps=0.0), x * scale, eps=0.0)


@pytest.mark.parametrize("shape", [(5, 72, 136), (5, 72, 1360), (5, 200, 136)])
def test_zeros_infinities_and_nan_stay_in_their_matrix(B, shape):
    x = randn(*shape, seed=8)
    want = ortho(B, x)
    y = x.clone()
    y[1] = 0
    y[2, 3, 5] = float("nan")
    y[4, 0, 0] = float("inf")
    got = ortho(B, y)
    assert torch.equal(got[0], want[0]) and torch.equal(got[3], want[3])
    assert bool((got[1] == 0).all()) and bool(got[2].isnan().all()) and not bool(got[4].isfinite().all())
    assert bool((ortho(B, torch.zeros_like(x), eps=0.0) == 0).all())


def emulate(p, g, m, clip, lr, mu, wd, scale, nesterov):
    g = g.double() * (1 if clip is None else float(clip))
    m = mu * m.double() + (1 - mu) * g
    u = mu * m + (1 - mu) * g if nesterov else m
    o = torch.stack([orthogonal(v) for v in u])
    worst = max(error(orthogonal(v, rounded=True), w) for v, w in zip(u, o))
    return p.double() * (1 - lr * wd) - lr * scale * o, m, lr * scale * o, worst


@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 65, 33), (3, 128, 72), (2, 72, 264), (2, 100, 900), (2, 901, 100), (2, 136, 264), (2, 265, 133)])
@pytest.mark.parametrize("ptype,gtype,nesterov", [(F32, BF16, True), (BF16, F32, False), (BF16, BF16, True), (F32, F32, True)])
def test_step(B, shape, ptype, gtype, nesterov):
    from moe_expert_layer_counting_gb300 import Muon
    p, m = randn(*shape, seed=1, scale=0.02, dtype=ptype), randn(*shape, seed=2, scale=1e-3, dtype=F32)
    gs = [randn(*shape, seed=3 + i, scale=1e-3, dtype=gtype) for i in range(2)]
    clip = torch.full((1,), 0.37, device="cuda") if nesterov else None
    copy = torch.zeros(shape, dtype=BF16, device="cuda") if ptype == F32 else None
    opt = Muon([p], lr=0.01, momentum=0.9, nesterov=nesterov, weight_decay=0.2, adjust="shape",
               copies=None if copy is None else [copy], state=([m],))
    scale = max(1.0, shape[1] / shape[2]) ** 0.5
    for g in gs:
        want_p, want_m, update, worst = emulate(p, g, m, clip, 0.01, 0.9, 0.2, scale, nesterov)
        opt.step([g], grad_scale=clip)
        assert opt.device_status() == 0
        # m: a product and a fused sum; p the same, and in BF16 one rounding
        assert bool(((m.double() - want_m).abs() <= 4 * 2.0 ** -24 * (want_m.abs() + 1e-3)).all())
        off = float((p.double() - want_p).norm())
        rounding = U if ptype == BF16 else 2.0 ** -23
        assert off <= (1.5 * worst + 1e-3) * float(update.norm()) + 2 * rounding * float(want_p.norm())
        assert copy is None or torch.equal(copy, p.bfloat16())


def test_several_parameters(B):
    """Matrices, stacks and a stack of stacks in one object, against one object each."""
    from moe_expert_layer_counting_gb300 import Muon
    shapes = [(40, 24), (3, 16, 72), (2, 2, 33, 20), (0, 8, 8), (2, 200, 136)]
    make = lambda: [randn(*s, seed=i, scale=0.02, dtype=F32) for i, s in enumerate(shapes)]      # noqa: E731
    grads = [randn(*s, seed=9 + i, scale=1e-3) for i, s in enumerate(shapes)]
    together, apart = make(), make()
    copies = [None, torch.zeros(shapes[1], dtype=BF16, device="cuda"), None, None, None]
    opt = Muon(together, lr=0.01, copies=copies)
    singles = [Muon([p], lr=0.01) for p in apart]
    for _ in range(3):
        opt.step(grads)
        for single, g in zip(singles, grads):
            single.step([g])
    assert opt.device_status() == 0
    assert all(torch.equal(p, q) for p, q in zip(together, apart)) and torch.equal(copies[1], together[1].bfloat16())


def test_state_resumes(B):
    from moe_expert_layer_counting_gb300 import Muon
    grads = [randn(2, 24, 40, seed=i, scale=1e-3) for i in range(4)]
    p, q = (randn(2, 24, 40, seed=9, scale=0.02, dtype=F32) for _ in range(2))
    whole, first = Muon([p], lr=0.01), Muon([q], lr=0.01)
    for g in grads:
        whole.step([g])
    for g in grads[:2]:
        first.step([g])
    second = Muon([q], lr=0.01, state=(first.state["m"],))
    for g in grads[2:]:
        second.step([g])
    assert torch.equal(p, q) and torch.equal(whole.state["m"][0], second.state["m"][0])


@pytest.mark.parametrize("shape", [(2, 300, 136), (3, 100, 40), (2, 64, 1000)])
def test_streams_and_graphs(B, shape):
    from moe_expert_layer_counting_gb300 import Muon
    grads = [randn(*shape, seed=i, scale=1e-3) for i in range(3)]
    p = randn(*shape, seed=9, scale=0.02, dtype=F32)
    start = p.clone()
    opt = Muon([p], lr=0.01)
    for g in grads:
        opt.step([g])
    want = p.clone()
    # two objects on two streams at once
    ps, streams = [start.clone() for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    opts = [Muon([q], lr=0.01) for q in ps]
    torch.cuda.synchronize()
    for g in grads:
        for o, st in zip(opts, streams):
            o.step([g], stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(q, want) for q in ps) and all(o.device_status(st) == 0 for o, st in zip(opts, streams))
    # captured: each replay is a step with the gradients that lie there
    q, g = start.clone(), grads[0].clone()
    captured = Muon([q], lr=0.01)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step([g])
    for new in grads:
        g.copy_(new)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q, want)


@pytest.mark.parametrize("shape", [(2, 300, 136), (1, 136, 300), (2, 72, 40), (1, 100, 2000)])
def test_a_wait_that_runs_out_is_reported(B, monkeypatch, shape):
    x, out = randn(*shape), torch.zeros(shape, dtype=BF16, device="cuda")
    ws = torch.empty(B.moe_muon_workspace_size(*shape), dtype=torch.uint8, device="cuda")
    monkeypatch.setenv("MOE_MXQ_DEBUG_INJECT_WAIT", "1")
    B.moe_orthogonalize(x, out, ws, steps=1)
    assert B.moe_get_device_status(ws) == B.MOE_ERR_TIMEOUT
    monkeypatch.delenv("MOE_MXQ_DEBUG_INJECT_WAIT")
    words = torch.full((64,), 255, dtype=torch.uint8, device="cuda")
    B.moe_orthogonalize(x, out, ws, status=words)
    assert B.moe_get_device_status(words) == B.MOE_OK
    check(out, x)
