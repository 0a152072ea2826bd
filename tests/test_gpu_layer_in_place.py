"""Outputs in the place of an input where the header allows it give the same bits
as outputs of their own."""
import numpy as np
import pytest
import torch

from combine_routing_histogram_amd import binding as B
from combine_routing_histogram_amd import layer as L
from layer_common import DEV, draw_indices, normal, routed_op

pytestmark = pytest.mark.gpu


def _stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("T", [6, 300])
@pytest.mark.parametrize("act,place", [("silu", "preact"), ("swiglu", "preact"),
                                       ("gelu", "grad_out")])
def test_dz_in_place_of_a_factor(T, act, place):
    from combine_routing_histogram_amd.op import ACTIVATIONS
    rng = np.random.default_rng(T)
    E, K, fin, fout = 4, 2, 72, 80
    op, n = routed_op(draw_indices(rng, T, K, E), E), T * K
    x, w = normal(rng, (n, fin)), normal(rng, (E, fout, fin))
    dy = normal(rng, (n, fout // 2 if act == "swiglu" else fout))
    z = normal(rng, (n, fout))
    gx, gw, _ = op.expert_product_backward(dy, x, w, activation=act, preact=z)
    off, _ = B.epdc_get_offsets(op._op)
    args = L.make_product_args(n, E, fin, fout, activation=ACTIVATIONS[act], expected_rows=n,
                               input=x.data_ptr(), weight=w.data_ptr(), expert_off=off)
    hx, hw = torch.zeros_like(gx), torch.zeros_like(gw)
    dz = {"preact": z, "grad_out": dy}[place]
    L.epdc_expert_backward(args, _stream(), dy.data_ptr(), z.data_ptr(), dz.data_ptr(),
                           hx.data_ptr(), hw.data_ptr(), L.EPDC_DT_BF16, 0)
    assert torch.equal(hx, gx) and torch.equal(hw, gw)


@pytest.mark.parametrize("T,K,H", [(1, 1, 8), (50, 6, 264), (300, 8, 4104)])
def test_combine_gradient_in_place_of_its_rows(T, K, H):
    rng = np.random.default_rng(T)
    op = routed_op(draw_indices(rng, T, K, 16), 16, hidden=H)
    x, dy = normal(rng, (T * K, H)), normal(rng, (T, H))
    w = normal(rng, (T * K, K), dtype=torch.float32)
    gx, gw = op.combine_backward(dy, x, w)
    _, _, slot_of = B.epdc_get_routing(op._op)
    hw = torch.zeros_like(gw)
    L.epdc_combine_backward(_stream(), T, K, H, slot_of, dy.data_ptr(), x.data_ptr(),
                            w.data_ptr(), x.data_ptr(), hw.data_ptr())
    assert torch.equal(x, gx) and torch.equal(hw, gw)
