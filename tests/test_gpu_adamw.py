"""AdamW over many tensors against float64, and its 8-bit states bit for bit.

Tolerance.  m and v are two rounded products and a rounded sum, p a handful of
float32 operations: each output is within 2^-21 of the sum of its terms'
magnitudes (8 roundings of 2^-24; the root, the quotient and the product of
the update count 2 each), a BF16 output within one rounding, 2^-8 of its
value, more.  The codes of 8-bit states depend on m and sqrt(v) as float32
rounds each operation, which NumPy restates exactly: they are compared bit for
bit, with the E4M3 and UE8M0 rules of the oracle.
"""
import itertools

import numpy as np
import pytest
import torch

from oracle import formats as F
from tests import helpers as Hp

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HOW = dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
SIZES = [1, 7, 8, 31, 32, 33, 0, 255, 4096, 4097, 20_011, 100_000]


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    Hp.lib()
    import moe_expert_layer_counting_gb300
    return moe_expert_layer_counting_gb300


def tensors(sizes, dtype, scale, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(dtype) for n in sizes]


def close(got, ref, magnitude):
    rounding = 2.0 ** -8 if got.dtype == BF16 else 0.0
    bound = rounding * ref.abs() + (1 + rounding) * 2.0 ** -21 * magnitude + 1e-37
    off = (got.double() - ref).abs()
    assert bool((off <= bound).all()), f"worst {float((off / bound).max()):.3f} of the bound"


def expected(p, m, v, g, t, lr, betas, eps, weight_decay):
    """(p, its magnitude, m, its magnitude, v) in float64 from the state before the step."""
    b1, b2 = betas
    p, g = p.double(), g.double()
    m_new, m_mag = b1 * m + (1 - b1) * g, b1 * m.abs() + (1 - b1) * g.abs()
    v_new = b2 * v + (1 - b2) * g * g
    root = torch.sqrt(v_new / (1 - b2 ** t)) + eps
    rate = lr / (1 - b1 ** t)
    return p * (1 - lr * weight_decay) - rate * m_new / root, p.abs() + rate * m_mag / root, m_new, m_mag, v_new


@pytest.mark.parametrize("pt,gt,clip", list(itertools.product((F32, BF16), (F32, BF16), (False, True))))
def test_float32_states(M, pt, gt, clip):
    params, grads = tensors(SIZES, pt, 0.5, 1), [tensors(SIZES, gt, 1e-2, s) for s in (2, 3, 4)]
    copies = tensors(SIZES, BF16, 1.0, 5) if pt == F32 else None
    opt = M.AdamW(params, copies=copies, **HOW)
    scale = torch.tensor([0.37], device="cuda") if clip else None
    for t, gs in enumerate(grads, 1):
        before = [(p.clone(), m.double(), v.double()) for p, m, v in zip(params, opt.state["m"], opt.state["v"])]
        opt.step(gs, grad_scale=scale)
        for i, (p, m, v) in enumerate(before):
            g = gs[i].double() * (scale.double() if clip else 1.0)
            p_ref, p_mag, m_ref, m_mag, v_ref = expected(p, m, v, g, t, **HOW)
            close(params[i], p_ref, p_mag)
            close(opt.state["m"][i], m_ref, m_mag)
            close(opt.state["v"][i], v_ref, v_ref)
            if copies:
                assert torch.equal(copies[i], params[i].to(BF16))
    assert opt.steps == 3


def group_codes(x, root):
    """E4M3 codes and UE8M0 bytes of float32 x in groups of 32 by the oracle's rules."""
    n = x.size
    pad = np.zeros(-(-n // 32) * 32, np.float32)
    pad[:n] = x
    groups = pad.reshape(-1, 32)
    e = np.array([F.ue8m0_exponent(float(a), 448.0) for a in np.abs(groups).max(1)], np.int64)
    scaled = np.ldexp(groups.astype(np.float64), -e[:, None])
    if root:
        scaled = np.where(groups > 0, np.maximum(scaled, 2.0 ** -9), scaled)
    return F.encode_e4m3(scaled).reshape(-1)[:n].astype(np.uint8), np.array([F.scale_byte(int(v)) for v in e], np.uint8)


def values(codes, scales):
    """float32 values of codes and scales (both NumPy)."""
    s = np.repeat(np.ldexp(1.0, scales.astype(np.int64) - 127), 32)[:codes.size]
    return (F.decode_e4m3(codes).astype(np.float64) * s).astype(np.float32)


@pytest.mark.parametrize("pt,gt,clip", [(F32, BF16, True), (F32, F32, False), (BF16, BF16, False)])
def test_8_bit_states(M, pt, gt, clip):
    params, grads = tensors(SIZES, pt, 0.5, 1), [tensors(SIZES, gt, 1e-2, s) for s in (2, 3, 4)]
    for gs in grads:                                    # a wide spread inside a group, and zeros
        for g in gs:
            g[::5] *= 1e-4
            g[3::7] = 0
    opt = M.AdamW(params, state_bits=8, **HOW)
    scale = torch.tensor([0.37], device="cuda") if clip else None
    b1, b2 = (np.float32(b) for b in HOW["betas"])
    c1, c2 = (np.float32(1 - b) for b in HOW["betas"])
    for t, gs in enumerate(grads, 1):
        before = [p.clone() for p in params]
        held = {k: [x.cpu().numpy().copy() for x in s] for k, s in opt.state.items()}
        opt.step(gs, grad_scale=scale)
        for i, n in enumerate(SIZES):
            if n == 0:
                continue
            g = gs[i].float().cpu().numpy() * (np.float32(0.37) if clip else np.float32(1))
            m = values(held["m"][i], held["m_scale"][i])
            r = values(held["v"][i], held["v_scale"][i])
            p_ref, p_mag, *_ = expected(before[i], torch.from_numpy(m).cuda().double(), torch.from_numpy(r).cuda().double() ** 2,
                                        torch.from_numpy(g).cuda(), t, **HOW)
            close(params[i], p_ref, p_mag)
            m = m * b1 + g * c1                          # float32, each operation rounded
            v = (r * r) * b2 + (g * g) * c2
            for name, x, root in (("m", m, False), ("v", np.sqrt(v), True)):
                codes, scales = group_codes(x, root)
                assert np.array_equal(opt.state[name + "_scale"][i].cpu().numpy(), scales), (name, t, n)
                assert np.array_equal(opt.state[name][i].cpu().numpy(), codes), (name, t, n)


@pytest.mark.parametrize("low,high", [(-23, 0), (-23, -17), (-21, -18), (-4, 4), (10, 17)])
@pytest.mark.parametrize("bits", [8, 32])
def test_gradients_over_the_whole_range(M, bits, low, high):
    """Magnitudes from 10^low to 10^high in every group, squares that are subnormal or round to 0 among them: the codes
    bit for bit, and p from m and v as float32 rounds them (a sum of eps alone where v is 0)."""
    n, eps = 5000, 1e-30
    rng = np.random.RandomState(7)
    g = (10.0 ** rng.uniform(low, high, n) * rng.choice([-1.0, 1.0], n)).astype(np.float32)
    p = torch.zeros(n, device="cuda")
    b1, b2 = HOW["betas"]
    opt = M.AdamW([p], state_bits=bits, lr=1e-2, betas=(b1, b2), eps=eps, weight_decay=0.0)
    opt.step([torch.from_numpy(g).cuda()])
    m, v = g * np.float32(1 - b1), (g * g) * np.float32(1 - b2)
    m64, root = m.astype(np.float64), np.sqrt(v.astype(np.float64) / (1 - b2)) + eps
    want = torch.from_numpy(-1e-2 / (1 - b1) * m64 / root).cuda()
    close(p, want, want.abs())
    for name, x, is_root in (("m", m, False), ("v", np.sqrt(v) if bits == 8 else v, True)):
        if bits == 8:
            codes, scales = group_codes(x, is_root)
            assert np.array_equal(opt.state[name + "_scale"][0].cpu().numpy(), scales), name
            assert np.array_equal(opt.state[name][0].cpu().numpy(), codes), name
        else:
            assert np.array_equal(opt.state[name][0].cpu().numpy(), x), name


def test_a_small_gradient_beside_a_large_one_does_not_jump(M):
    """8-bit states: sqrt(v) of a value far below its group's largest would round to 0 and the next step divide by
    eps; it is held at the smallest code instead, and no step moves a value by more than a few rates."""
    n = 64
    p = torch.zeros(n, device="cuda")
    g = torch.full((n,), 1e-6, device="cuda")
    g[0], g[40] = 1e3, 1e4
    opt = M.AdamW([p], state_bits=8, lr=1e-3, betas=(0.9, 0.95), eps=1e-12, weight_decay=0.0)
    for _ in range(20):
        before = p.clone()
        opt.step([g])
        # |m| / sqrt(v) without bias is at most sqrt((1 - b1)^2 / (1 - b2)) / sqrt(1 - b1^2 / b2) = 1.2; E4M3 adds 1/16 twice
        assert float((p - before).abs().max()) <= 1e-3 * 1.2 * (1 + 1 / 8) / (1 - 0.9)
    assert bool(p.isfinite().all())


def test_nan_and_infinity_stay_in_their_value(M):
    for bits in (32, 8):
        p, g = tensors([200], F32, 1.0, 1)[0], tensors([200], F32, 1.0, 2)[0]
        g[70], g[100] = float("nan"), float("inf")
        opt = M.AdamW([p], state_bits=bits)
        opt.step([g])
        opt.step([g])
        fine = p.isfinite()
        assert not bool(fine[70]) and not bool(fine[100])
        fine[[70, 100]] = True
        assert bool(fine.all())


def test_many_tensors_and_shapes(M):
    """More tensors than one launch's table holds, of several dimensions, each at a place of its own."""
    sizes = [(3, 5 + i % 40) for i in range(1000)]
    params = [torch.randn(*s, device="cuda") for s in sizes]
    grads = [torch.randn(*s, device="cuda") for s in sizes]
    before = [p.clone() for p in params]
    M.AdamW(params, **HOW).step(grads)
    for p, b, g in zip(params, before, grads):
        z = torch.zeros_like(b, dtype=torch.float64)
        p_ref, p_mag, *_ = expected(b, z, z, g, 1, **HOW)
        close(p, p_ref, p_mag)


def test_beyond_2_pow_31_values(M):
    n = 2 ** 31 + 4099
    p, g = torch.ones(n, dtype=BF16, device="cuda"), torch.ones(n, dtype=BF16, device="cuda")
    g[:-5000] = 0
    opt = M.AdamW([p], state_bits=8, lr=0.5, weight_decay=0.0)
    opt.step([g])
    # first step: m / c1 = g and sqrt(v / c2) = |g|, so p falls by lr where g is 1 and stays where it is 0
    assert bool((p[-5000:] == 0.5).all()) and bool((p[-9000:-5000] == 1).all()) and bool((p[:9000] == 1).all())


def test_another_stream_and_resuming(M):
    """A run of three steps, and one whose state is handed on after two, on another stream: the same bits."""
    sizes = [33, 4096, 70_001]
    for bits in (32, 8):
        grads = [tensors(sizes, BF16, 1e-2, s) for s in (2, 3, 4)]
        first, second = tensors(sizes, F32, 0.5, 1), tensors(sizes, F32, 0.5, 1)
        opt = M.AdamW(first, state_bits=bits, **HOW)
        for gs in grads:
            opt.step(gs)
        a = M.AdamW(second, state_bits=bits, **HOW)
        a.step(grads[0])
        a.step(grads[1])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        b = M.AdamW(second, state_bits=bits, step=a.steps, state=tuple(a.state.values()), **HOW)
        b.step(grads[2], stream=side)
        torch.cuda.synchronize()
        for x, y in zip(first, second):
            assert torch.equal(x, y)
        for k in opt.state:
            for x, y in zip(opt.state[k], b.state[k]):
                assert torch.equal(x, y)
