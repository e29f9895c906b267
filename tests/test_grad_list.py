"""GradList reads its tensors at each call: addresses, sizes and types are those of the tensors as they are then
(CPU only: the table that a call would pass, nothing is launched)."""

import pytest
import torch

import fp8_transformer_gb300 as te

b = te.binding
BF = torch.bfloat16


def table(plan):
    t, _ = plan._table()
    return [(t[i].data, t[i].out, t[i].numel, t[i].dtype) for i in range(len(plan.grads))]


def of(t, out=None):
    return t.data_ptr(), None if out is None else out.data_ptr(), t.numel(), b._DTYPE[t.dtype]


def changes(n=1000):
    """Ways in which a tensor of n float32 keeps its address and changes its size or its type."""
    def resize(t):
        t.resize_(10)

    def shorter(t):
        t.data = t.data[:10]

    def other_shape(t):
        t.data = t.data.view(n // 10, 10)[:3]

    def other_type(t):
        t.data = t.data.view(BF)[:n]

    def longer(t):
        t.data = t.data.view(BF)

    return [resize, shorter, other_shape, other_type, longer]


@pytest.mark.parametrize("change", changes(), ids=lambda f: f.__name__)
def test_same_address_other_size_or_type(change):
    a, p = torch.ones(7), torch.ones(1000)
    plan = te.GradList([a, p])
    assert table(plan) == [of(a), of(p)]
    at = p.data_ptr()
    change(p)
    assert p.data_ptr() == at
    assert table(plan) == [of(a), of(p)]


@pytest.mark.parametrize("change", changes(), ids=lambda f: f.__name__)
def test_an_out_of_another_size_or_type(change):
    p, o = torch.ones(1000), torch.ones(1000)
    plan = te.GradList([p], [o])
    assert table(plan) == [of(p, o)]
    change(o)
    with pytest.raises(ValueError):
        plan._table()
    change(p)
    assert table(plan) == [of(p, o)]


@pytest.mark.parametrize("other", [lambda t: t[::2], lambda t: t[:1].expand(500), lambda t: t.view(20, 50).t(),
                                   lambda t: t.view(torch.int32), lambda t: t.view(torch.float16)],
                         ids=["strided", "expanded", "transposed", "int32", "float16"])
def test_same_address_no_longer_dense_or_of_a_type(other):
    p = torch.ones(1000)
    plan = te.GradList([torch.ones(3), p])
    at = p.data_ptr()
    if other(p.data).dtype != torch.float32:  # .data keeps to floating types of its own; the list does not
        plan.grads[1] = other(p.data)
    else:
        p.data = other(p.data)
    assert plan.grads[1].data_ptr() == at
    with pytest.raises(ValueError):
        plan._table()


def test_moved_and_emptied():
    p = torch.nn.Parameter(torch.ones(50))
    plan = te.GradList([p])
    p.data = torch.full((200,), 2.0, dtype=BF)
    assert table(plan) == [of(p)]
    p.data = torch.empty(0)
    assert table(plan)[0][2:] == (0, b.TE_F32)


def test_lists():
    a, c = torch.ones(5), torch.ones(6)
    plan = te.GradList(iter([a]))
    plan.grads.append(c)  # the list is the object's own, and may grow
    assert table(plan) == [of(a), of(c)]
    assert te.GradList([]).device is None and te.GradList([a]).device == -1
    plan = te.GradList([a, c], [c.clone().resize_(5), c])
    plan.outs.pop()
    with pytest.raises(ValueError):
        plan._table()
    for grads, outs in (((a, c), None), ([a, c], (a, c)), ((), None)):
        plan = te.GradList([a, c])
        plan.grads, plan.outs = grads, outs
        with pytest.raises(ValueError):
            plan._table()
    for bad in ([a, None], [a, 3.0], [a, torch.ones(3, dtype=torch.float64)], [torch.ones(4).to_sparse()],
                [a, torch.ones(3, device="meta")]):
        with pytest.raises((ValueError, AttributeError)):
            te.GradList(bad)
