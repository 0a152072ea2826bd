"""The experts of single ranks: gradients of the parts against the whole."""
import numpy as np
import pytest
import torch

from layer_common import DEV, draw_indices, ints, layout, routed_op

pytestmark = pytest.mark.gpu


def _case(T, K=4, E=16, H=64, N=40, R=4):
    rng = np.random.default_rng(T)
    idx = draw_indices(rng, T, K, E)
    idx[::5, 0] = -1
    _, off = layout(idx, E)
    op = routed_op(idx, E, hidden=H, ranks=R)
    return op, off, ints(rng, (T * K, H)), ints(rng, (E, N, H)), ints(rng, (T * K, N))


@pytest.mark.parametrize("T", [5, 400])
def test_ranks_write_one_buffer(T):
    op, off, x, w, dy = _case(T)
    whole, gw, gb = op.expert_product_backward(dy, x, w, bias=True)
    buf = torch.full_like(x, 7.0)
    for r in range(4):
        mine = slice(4 * r, 4 * r + 4)
        part = op.expert_product_backward(dy, x, w[mine].contiguous(), bias=True,
                                          first_expert=4 * r, grad_input=buf)
        assert part[0] is buf
        assert torch.equal(part[1], gw[mine]) and torch.equal(part[2], gb[mine])
    n = off[-1]
    assert torch.equal(buf[:n], whole[:n]) and bool((buf[n:] == 7.0).all())


@pytest.mark.parametrize("T", [5, 400])
def test_a_ranks_own_gradient_is_zero_elsewhere(T):
    """Each rank's gradient goes through dispatch_backward as it is: the tokens'
    gradients of the ranks add up to the whole's (small integers: exactly)."""
    op, off, x, w, dy = _case(T)
    whole = op.dispatch_backward(op.expert_product_backward(dy, x, w)[0]).double()
    total = torch.zeros_like(whole)
    for r in range(4):
        # what a fresh tensor may hold: the allocator hands this block out again
        torch.full((T * 4, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
        gx, _, _ = op.expert_product_backward(dy, x, w[4 * r:4 * r + 4].contiguous(),
                                              first_expert=4 * r)
        a, b = off[4 * r], off[4 * r + 4]
        assert not gx[:a].any() and not gx[b:].any()
        total += op.dispatch_backward(gx).double()
    assert torch.equal(total, whole)
