"""TrainableExperts where its input is not the usual: expert indices that do not exist, no tokens, strides and types."""
import pytest
import torch

from tests import helpers as Hp

pytestmark = pytest.mark.gpu

E, H, I, k = 6, 136, 64, 3


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    Hp.lib()
    import moe_expert_layer_counting_gb300
    return moe_expert_layer_counting_gb300


def inputs(T, seed=0):
    """n, l1, l2, topk_idx, topk_w, db."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()

    idx = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].int().contiguous()
    return (randn(T, H), randn(E, 2 * I, H, scale=H ** -0.5), randn(E, H, I, scale=I ** -0.5), idx,
            torch.softmax(randn(T, k).float(), 1), randn(T, H))


def step(M, n, l1, l2, idx, w, db, dl=None, accumulate=False):
    """(status, b, dn, dtopk_w, dl1, dl2)."""
    from moe_expert_layer_counting_gb300.training import TrainableExperts
    layer = TrainableExperts(l1, l2)
    b, s = layer.forward(n, idx, w)
    dl1, dl2 = dl or (torch.full(l1.shape, 3.0, device="cuda"), torch.full(l2.shape, 3.0, device="cuda"))
    dn, dw = layer.backward(db, s, dl1, dl2, accumulate)
    return layer.status(), b, dn, dw, dl1, dl2


@pytest.mark.parametrize("bad", [E, E + 1, 2 ** 31 - 1])
def test_an_index_that_no_expert_has_is_reported_and_its_pair_dropped(M, bad):
    n, l1, l2, idx, w, db = inputs(50)
    at = torch.zeros_like(idx, dtype=torch.bool)
    at[::7, 1] = True
    at[11] = True
    dropped = step(M, n, l1, l2, torch.where(at, -1, idx), w, db)
    got = step(M, n, l1, l2, torch.where(at, bad, idx), w, db)
    assert dropped[0] == M.binding.MOE_OK and got[0] == M.binding.MOE_ERR_DEVICE_INDEX
    for a, b in zip(got[1:], dropped[1:]):
        assert torch.equal(a, b)
    assert not bool(got[1][11].any()) and not bool(got[2][11].any()) and not bool(got[3][at].any())


def test_no_tokens(M):
    n, l1, l2, idx, w, db = inputs(0)
    status, b, dn, dw, dl1, dl2 = step(M, n, l1, l2, idx, w, db)
    assert status == M.binding.MOE_OK and b.shape == dn.shape == (0, H) and dw.shape == (0, k)
    assert not bool(dl1.any()) and not bool(dl2.any())
    dl = torch.ones_like(l1, dtype=torch.float32), torch.ones_like(l2, dtype=torch.float32)
    step(M, n, l1, l2, idx, w, db, dl, accumulate=True)
    assert all(bool((t == 1).all()) for t in dl)


def test_strides(M):
    """Inputs that are parts of wider tensors: the same bits as their copies."""
    n, l1, l2, idx, w, db = inputs(30)
    wide = torch.full((30, k + 2), E, dtype=torch.int32, device="cuda")
    wide[:, 1:1 + k] = idx
    rows = torch.zeros(30, 2, H, dtype=torch.bfloat16, device="cuda")
    rows[:, 0], rows[:, 1] = n, db
    want = step(M, n, l1, l2, idx, w, db)
    got = step(M, rows[:, 0], l1, l2, wide[:, 1:1 + k], w.T.contiguous().T, rows[:, 1])
    assert want[0] == got[0] == M.binding.MOE_OK
    for a, b in zip(want[1:], got[1:]):
        assert torch.equal(a, b)
