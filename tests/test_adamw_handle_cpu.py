"""The AdamW handle's bookkeeping, without a GPU: tensors that say they are on one, and a library that writes
down what it is given."""
import ctypes

import numpy as np
import pytest
import torch

import async_rl_b200 as bi
from async_rl_b200 import optim


class Fake(torch.Tensor):
    """A CPU tensor that passes for the device's."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.device.index


def fake(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Fake)


class Library:
    def __init__(self):
        self.tables = []

    def bi_adamw_step(self, table, n, cfg, grad_scale, step_dev, status, stream):
        rows = (ctypes.c_int64 * (8 * n)).from_address(table)
        self.tables.append(np.array(rows).reshape(n, 8))
        return 0


@pytest.fixture
def lib(monkeypatch):
    got = Library()
    monkeypatch.setattr(optim._lib, "load", lambda: got)
    monkeypatch.setattr(optim, "_stream", lambda dev: 0)
    return got


def handle(*shapes, dtype=torch.float32):
    p, m, v = ([fake(*s, dtype=d) for s in shapes] for d in (dtype, torch.float32, torch.float32))
    return bi.AdamWState(p, None, m, v)


def step(st, grads, lib):
    bi.adamw_step(st, grads, 1, 1e-3)
    return lib.tables[-1]


@pytest.mark.parametrize("other", [lambda: fake(299), lambda: fake(300, dtype=torch.float64),
                                   lambda: fake(20, 15).t(), lambda: fake(300, dtype=torch.bfloat16)])
def test_a_refused_binding_leaves_the_handle_as_it_was(other, lib):
    """The storage is replaced by one that is refused, and put back: the next step is the first one's again."""
    st = handle((300,), (40, 3))
    g = [fake(300), fake(40, 3)]
    first = step(st, g, lib)
    old = st.params[0].data
    st.params[0].data = other()
    with pytest.raises(ValueError):
        step(st, g, lib)
    st.params[0].data = old
    assert st.sizes == [300, 120] and st.shapes == [(300,), (40, 3)] and not st.param_bf16 and st.state_bits == 32
    assert np.array_equal(step(st, g, lib), first)


def test_gradients_are_held_to_the_tensors_of_this_step(lib):
    """Every tensor replaced by a larger one: gradients of the old size would be read past their end."""
    st = handle((300,))
    step(st, [fake(300)], lib)
    for t in st.tensors():
        t.data = fake(5000)
    with pytest.raises(ValueError, match="shape"):
        step(st, [fake(300)], lib)
    assert step(st, [fake(5000)], lib)[0, 7] == 5000


HALF, EVERY_OTHER = (lambda t: t[:100]), (lambda t: t[::2])


@pytest.mark.parametrize("other,which", [(HALF, 0), (HALF, 1), (HALF, 2), (EVERY_OTHER, 0), (EVERY_OTHER, 1),
                                         (lambda t: t.view(torch.int32), 0), (lambda t: t.view(20, 15).t(), 0)])
def test_another_size_type_or_layout_at_the_same_address_is_refused(other, which, lib):
    """Of a param, exp_avg or exp_avg_sq."""
    st = handle((300,), (40, 3))
    g = [fake(300), fake(40, 3)]
    step(st, g, lib)
    t = st.tensors()[2 * which]
    old = t.data
    t.data = other(old)
    assert t.data_ptr() == old.data_ptr()
    n = len(lib.tables)
    for _ in range(2):
        with pytest.raises(ValueError):
            step(st, g, lib)
    assert len(lib.tables) == n
    t.data = old
    step(st, g, lib)


def test_all_tensors_shrunk_or_reshaped_in_place_are_followed(lib):
    st = handle((300,), (40, 3))
    step(st, [fake(300), fake(40, 3)], lib)
    for t in st.tensors()[::2]:
        t.data = t.data[:100]
    st.params[1].data = st.params[1].data.view(3, 40)
    with pytest.raises(ValueError, match="shape"):
        step(st, [fake(300), fake(40, 3)], lib)
    assert step(st, [fake(100), fake(3, 40)], lib)[:, 7].tolist() == [100, 120]


@pytest.mark.parametrize("grads", [
    lambda st, flat: [st.params[0], fake(40, 3)], lambda st, flat: [fake(300), st.exp_avg_sq[1]],
    lambda st, flat: [flat[10:310], fake(40, 3)], lambda st, flat: [fake(300), flat[299:419].view(40, 3)]])
def test_gradients_may_not_overlap_what_the_step_writes(grads, lib):
    """A gradient that is written while other threads still read it gives results that depend on timing."""
    flat = fake(900)
    p = [flat[:300], flat[500:620].view(40, 3)]
    st = bi.AdamWState(p, None, [fake(300), fake(40, 3)], [fake(300), fake(40, 3)])
    good = [flat[620:720].expand(3, 100).reshape(300), flat[300:420].view(40, 3)]
    for _ in range(2):
        step(st, good, lib)
        n = len(lib.tables)
        with pytest.raises(ValueError, match="overlap"):
            step(st, grads(st, flat), lib)
        assert len(lib.tables) == n


def test_gradients_may_share_memory_and_be_empty(lib):
    st = handle((300,), (0,), (300,))
    g = fake(400)
    assert step(st, [g[:300], g[:0], g[100:]], lib)[:, 7].tolist() == [300, 0, 300]
