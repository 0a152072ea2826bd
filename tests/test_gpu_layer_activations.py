"""gelu and its gradient where the normal distribution's tail is small.

The weight is the identity, so the activation's argument is the bf16 input
itself.  1 + erf would cancel there; a tail taken from e^(-x^2 / 2) is off by
that argument's rounding, 2 a^2 2^-23 with a = 8 / sqrt 2, and a few ulp of
what else it takes, together below 2^-15, and by one rounding to bf16, 2^-8,
all relative.  The gradient's density adds the same once more: below 2^-14.
"""
import numpy as np
import pytest
import torch

from layer_common import DEV, layout, routed_op

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


def _case(T, act):
    F = 64
    op = routed_op(np.zeros((T, 1), np.int32), 1)
    z = torch.linspace(-8, -3, T * F, dtype=torch.float64, device=DEV).reshape(T, F)
    z = z[:, torch.randperm(F, generator=torch.Generator().manual_seed(T)).to(DEV)].bfloat16()
    eye = torch.eye(F, device=DEV)
    w = (torch.cat([eye, -512 * eye]) if act == "geglu" else eye).bfloat16()[None].contiguous()
    return op, z, w


# the streamed form (16 rows a tile, then 32), 64-row tiles, 256-row tiles
@pytest.mark.parametrize("T", [8, 20, 50, 300])
@pytest.mark.parametrize("act", ["gelu", "geglu"])
def test_forward_tail(T, act):
    op, z, w = _case(T, act)
    x = z.double()
    y = 0.5 * x * torch.special.erfc(-x * 0.5 ** 0.5)
    if act == "geglu":
        y = y * (-512 * x)
    got = op.expert_product(z, w, activation=act).double()
    assert bool(((got - y).abs() <= (U + 2.0 ** -15) * y.abs()).all())


@pytest.mark.parametrize("T", [8, 300])
@pytest.mark.parametrize("act", ["gelu", "geglu"])
def test_gradient_tail(T, act):
    """dy 1 everywhere; geglu: up 4, so that both halves of dz show the tail."""
    op, z, _ = _case(T, "gelu")
    x = z.double()
    phi = torch.exp(-0.5 * x * x) / (2 * np.pi) ** 0.5
    cdf = 0.5 * torch.special.erfc(-x * 0.5 ** 0.5)
    dz = cdf + x * phi
    pre = z
    if act == "geglu":
        pre = torch.cat([z, torch.full_like(z, 4.0)], 1)
        dz = torch.cat([4 * dz, x * cdf], 1)
    n = dz.shape[1]
    w = torch.eye(n, device=DEV).bfloat16()[None].contiguous()
    gx, _, gb = op.expert_product_backward(torch.ones_like(z), torch.zeros_like(pre), w,
                                           activation=act, preact=pre, bias=True)
    assert bool(((gx.double() - dz).abs() <= (U + 2.0 ** -14) * dz.abs()).all())
    ref = dz.sum(0)   # of one sign
    assert bool(((gb[0].double() - ref).abs() <= (2.0 ** -14 + T * 2.0 ** -24) * ref.abs()).all())
