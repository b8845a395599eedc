"""Which tensors a step of AdamW works on: those that its lists hold at that time.  The call into the library is replaced by
one that keeps the table, so no GPU is needed."""
import copy
import pickle

import numpy as np
import pytest
import torch

from tests import helpers as Hp


@pytest.fixture
def steps(monkeypatch):
    """(AdamW, the tables of the steps taken so far)."""
    B = Hp.lib()
    from moe_expert_layer_counting_gb300 import AdamW
    tables = []

    def keep(table, p_dtype, g_dtype, *how, address=None, **more):
        assert address is None or address == table.ctypes.data
        tables.append(table.copy())

    monkeypatch.setattr(B, "moe_adamw_step", keep)
    return AdamW, tables


SIZES = (40, 0, 7)


def tensors(dtype=torch.float32, sizes=SIZES):
    return [torch.zeros(n, dtype=dtype) for n in sizes]


def make(AdamW, bits):
    return AdamW(tensors(), state_bits=bits, copies=tensors(torch.bfloat16))


def of_lists(opt, grads):
    """The table that these lists make."""
    lists = {"p": opt.params, "g": grads, **opt.state, "copy": opt.copies}
    return {name: [t.data_ptr() for t in ts] for name, ts in lists.items()}


def check(table, opt, grads):
    assert table["n"].tolist() == list(SIZES)
    for name, want in of_lists(opt, grads).items():
        assert table[name].tolist() == want, name


@pytest.mark.parametrize("bits", [8, 32])
def test_a_parameter_of_another_storage(steps, bits):
    AdamW, tables = steps
    opt, grads = make(AdamW, bits), tensors(torch.bfloat16)
    opt.step(grads)
    check(tables[-1], opt, grads)
    opt.params[0].data = torch.zeros(40)
    opt.step(grads)
    check(tables[-1], opt, grads)
    opt.params[2].untyped_storage().resize_(4096)                 # moves the values of 7 x 4 bytes
    opt.step(grads)
    check(tables[-1], opt, grads)
    assert opt.steps == 3


@pytest.mark.parametrize("bits", [8, 32])
def test_another_tensor_in_a_list(steps, bits):
    AdamW, tables = steps
    opt, grads = make(AdamW, bits), tensors(torch.bfloat16)
    opt.step(grads)
    for ts in (opt.params, opt.copies, *opt.state.values()):
        ts[0] = ts[0].clone()
        opt.step(grads)
        check(tables[-1], opt, grads)
    for name in list(opt.state):
        opt.state[name] = [t.clone() for t in opt.state[name]]
        opt.step(grads)
        check(tables[-1], opt, grads)


def test_tensors_that_no_longer_fit_are_refused(steps):
    AdamW, tables = steps
    grads = tensors(torch.bfloat16)

    def shorter(opt):
        opt.params[0].data = torch.zeros(39)

    def of_another_type(opt):
        opt.params[2].data = torch.zeros(7, dtype=torch.bfloat16)

    def strided(opt):
        opt.state["m"][0] = torch.zeros(80)[::2]

    def a_longer_list(opt):
        opt.copies.append(torch.zeros(1, dtype=torch.bfloat16))

    def a_shorter_list(opt):
        del opt.state["v"][2]

    for change in (shorter, of_another_type, strided, a_longer_list, a_shorter_list):
        opt = make(AdamW, 32)
        opt.step(grads)
        change(opt)
        for _ in range(2):                                        # and again
            with pytest.raises(ValueError):
                opt.step(grads)
        assert len(tables) == 1 and opt.steps == 1
        tables.clear()


def test_memory_of_the_old_storage_is_not_handed_on(steps):
    """A smaller parameter at the address of the old one would pass for it: the old storage is kept until the next look."""
    AdamW, tables = steps
    p = torch.zeros(4096)
    opt = AdamW([p])
    opt.step([torch.zeros(4096)])
    old = p.data_ptr()
    for _ in range(20):
        p.data = torch.zeros(1)
        p.data = torch.zeros(4000)
        assert p.data_ptr() != old
    with pytest.raises(ValueError):
        opt.step([torch.zeros(4096)])
    assert np.array_equal(tables[-1]["p"], [old])


@pytest.mark.parametrize("copied", [copy.deepcopy, copy.copy, lambda o: pickle.loads(pickle.dumps(o))])
@pytest.mark.parametrize("bits", [8, 32])
def test_a_copied_object_has_a_table_of_its_own(steps, copied, bits):
    """deepcopy and pickle: the copy's tensors, through the copy's table (the fake call compares its address); copy: the same."""
    AdamW, tables = steps
    opt, grads = make(AdamW, bits), tensors(torch.bfloat16)
    opt.step(grads)
    other = copied(opt)
    for which in (other, opt, other):
        which.step(grads)
        check(tables[-1], which, grads)
    assert (other.steps, opt.steps) == (3, 2)
    other.params = tensors()
    for which in (other, opt):
        which.step(grads)
        check(tables[-1], which, grads)
    if copied is not copy.copy:
        assert all(a.data_ptr() != b.data_ptr() for a, b in zip(opt.params, other.params) if a.numel())
        del opt                                                   # nothing of the original is needed
        other.step(grads)
        check(tables[-1], other, grads)


def test_a_step_in_a_capture_is_refused(steps, monkeypatch):
    AdamW, tables = steps
    opt, grads = make(AdamW, 32), tensors(torch.bfloat16)
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "is_initialized", lambda: True)
        m.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
        with pytest.raises(RuntimeError):
            opt.step(grads)
        assert not tables and opt.steps == 0
        m.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
        opt.step(grads)
    assert len(tables) == opt.steps == 1


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
def test_a_step_in_a_real_capture_is_refused(given):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    Hp.lib()
    from moe_expert_layer_counting_gb300 import AdamW
    p, g = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    opt, graph, side = AdamW([p]), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        g += 1
        with pytest.raises(RuntimeError):
            if given:
                with torch.cuda.stream(torch.cuda.Stream()):       # not the one that captures
                    opt.step([g], stream=side)
            else:
                opt.step([g])
    graph.replay()
    torch.cuda.synchronize()
    assert opt.steps == 0 and bool((p == 1).all()) and bool((g == 2).all())
    opt.step([g])
    assert opt.steps == 1 and bool((p < 1).all())


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_values_of_another_storage_are_updated(bits):
    """Two steps, the values moved in between: the same bits as two steps where they lay, and the old storage untouched."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    Hp.lib()
    from moe_expert_layer_counting_gb300 import AdamW
    g = torch.Generator(device="cuda").manual_seed(1)
    start, grads = (torch.randn(3, 1000, generator=g, device="cuda") for _ in range(2))
    runs = []
    for move in (False, True):
        p = start.clone()
        opt = AdamW([p], state_bits=bits, copies=[p.bfloat16()])
        opt.step([grads])
        if move:
            old = [p.detach(), opt.copies[0], *(s[0] for s in opt.state.values())]
            kept = [t.clone() for t in old]
            p.data = p.data.clone()
            opt.copies = [t.clone() for t in opt.copies]
            opt.state = {k: [t.clone() for t in s] for k, s in opt.state.items()}
        opt.step([grads])
        runs.append([p, *opt.copies, *(s[0] for s in opt.state.values())])
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    for a, b in zip(old, kept):
        assert torch.equal(a, b)
