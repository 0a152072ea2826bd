"""What the op hands to the library, and refuses, for the layer's products (host only)."""
import pytest
import torch

from combine_routing_histogram_amd import binding as B
from combine_routing_histogram_amd import layer as L
from test_layer_abi import _host_op

BF = torch.bfloat16


@pytest.fixture
def op(monkeypatch):
    """An op of 8 experts, top-4, whose last dispatch had 10 tokens; the library's
    calls leave their arguments in op.calls."""
    op = _host_op()
    op._op, op.calls = 0, []
    op._stream = lambda: 0
    monkeypatch.setattr(B, "epdc_get_offsets", lambda op: (4096, 4096))
    for name in ("epdc_expert_product", "epdc_expert_backward"):
        monkeypatch.setattr(L, name, lambda *a: op.calls.append(a))
    return op


def test_backward_takes_a_buffer_for_the_rows_gradient(op):
    x, w, g = torch.zeros(40, 256, dtype=BF), torch.zeros(8, 64, 256, dtype=BF), \
        torch.zeros(40, 64, dtype=BF)
    ok = torch.empty(45, 256, dtype=BF)
    assert op.expert_product_backward(g, x, w, grad_input=ok)[0] is ok
    assert ok.data_ptr() in op.calls[0]
    for bad in (ok[:39], ok.float(), torch.empty(40, 128, dtype=BF), ok.t()):
        with pytest.raises(ValueError):
            op.expert_product_backward(g, x, w, grad_input=bad)
    with pytest.raises(ValueError):
        op.expert_product_backward(g, x, w, grad_input=ok, need_input=False)
    assert len(op.calls) == 1


@pytest.mark.parametrize("first,n,expected", [(0, 8, 40), (0, 4, 20), (7, 1, 5)])
def test_expected_rows(op, first, n, expected):
    x, w = torch.zeros(40, 256, dtype=BF), torch.zeros(n, 64, 256, dtype=BF)
    op.expert_product(x, w, first_expert=first, out=torch.empty(40, 64, dtype=BF))
    assert op.calls[0][0].expected_rows == expected


def test_expected_rows_of_fewer_than_one(op):
    """0 would mean all of the rows, and the form for many."""
    op._tokens = 1
    x, w = torch.zeros(4, 256, dtype=BF), torch.zeros(1, 64, 256, dtype=BF)
    op.expert_product(x, w, first_expert=3, out=torch.empty(4, 64, dtype=BF))
    assert op.calls[0][0].expected_rows == 1
