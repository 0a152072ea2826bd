"""The gate far from zero: sigmoid scores too small or too near 1 for fp32.

Tolerances as in test_gpu_layer_gate.py: differences of logits inside a row stay
below 30, so a share, a ratio of two sums of exponentials, is off by at most
2 REL of itself, the balance loss (a mean of them times counts) by 8 REL, and a
gradient entry by 16 REL of its terms' absolute values.
"""
import numpy as np
import pytest
import torch

from combine_routing_histogram_amd.op import GateConfig
from layer_common import DEV
from test_gpu_layer_gate import REL, _gradient, _op, _reference

pytestmark = pytest.mark.gpu


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


# experts beside empty slots of a lane (5, 24, 300) and without (256); tokens of
# both forms, a wave per token (T <= 16 E) and four tokens to a wave
@pytest.mark.parametrize("base", [-40.0, -60.0, -75.0, -90.0, -200.0, -500.0])
@pytest.mark.parametrize("T,E,K", [(6, 5, 2), (100, 5, 2), (40, 24, 4), (400, 24, 4),
                                   (20, 256, 8), (4100, 256, 8), (33, 300, 6)])
def test_sigmoid_shares_far_below_zero(T, E, K, base):
    """p = s / sum(s) in the balance loss and its gradient, with and without
    experts at -inf and tokens whose logits straddle the border."""
    print(f"far T={T} E={E} base={base}", flush=True)
    rng = np.random.default_rng(T + E)
    l = (base + 3 * rng.standard_normal((T, E))).astype(np.float32)
    l[::3, rng.permutation(E)[:E // 2]] = -np.inf
    l[1::4, 0] = base + 12
    cfg = GateConfig("sigmoid", True, 1.0)
    op, logits = _op(T, E, K), _dev(l)
    w, idx, counts, losses = [t.cpu().numpy() for t in op.gate(logits, cfg, balance=True)]
    rw, ridx, rcounts, rlosses = _reference(l.astype(np.float64), K, cfg)
    assert np.array_equal(idx, ridx) and np.array_equal(counts, rcounts)
    np.testing.assert_allclose(losses, rlosses, rtol=8 * REL)
    gl = np.array([0.5, 0.0], np.float32)
    got = op.gate_backward(logits, _dev(idx), cfg, counts=_dev(counts), grad_losses=_dev(gl))
    ref, mag = _gradient(l.astype(np.float64), K, cfg, idx, None, counts, gl)
    assert (np.abs(got.double().cpu().numpy() - ref) <= 16 * REL * mag + 1e-37).all()


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("base", [6.0, 10.0, 14.0, 18.0, 30.0])
@pytest.mark.parametrize("T,E,K", [(40, 24, 4), (400, 24, 4), (20, 256, 8)])
def test_sigmoid_slope_far_above_zero(T, E, K, base, renormalize):
    """Gradients carry the factor 1 - s = sigma(-l), which 1 minus a rounded s
    loses.  Every entry is a product with that factor (the rest of it bounded as
    in _gradient), so the bound is relative to the product."""
    rng = np.random.default_rng(T + E)
    l = (base + rng.standard_normal((T, E))).astype(np.float32)
    cfg = GateConfig("sigmoid", renormalize, 1.5)
    op, logits = _op(T, E, K), _dev(l)
    _, idx, counts, _ = [t.cpu().numpy() for t in op.gate(logits, cfg, balance=True)]
    gw = rng.standard_normal((T, K)).astype(np.float32)
    gl = np.array([0.5, 0.0], np.float32)
    got = op.gate_backward(logits, _dev(idx), cfg, grad_weights=_dev(gw), counts=_dev(counts),
                           grad_losses=_dev(gl)).double().cpu().numpy()
    x = l.astype(np.float64)
    s, slope = 1 / (1 + np.exp(-x)), 1 / (1 + np.exp(x))   # s and 1 - s
    f = counts[:E] / (T * K)
    p = s / s.sum(1, keepdims=True)
    fp = (f * p).sum(1, keepdims=True)
    ref = gl[0] * E / T * p * (f - fp) * slope
    mag = gl[0] * E / T * p * (f + fp) * slope
    sc, g = np.take_along_axis(s, idx, 1), 1.5 * gw.astype(np.float64)
    if renormalize:
        r = sc / sc.sum(1, keepdims=True)
        gr = (g * r).sum(1, keepdims=True)
        d, dm = r * (g - gr), r * (np.abs(g) + (np.abs(g) * r).sum(1, keepdims=True))
    else:
        d, dm = g * sc, np.abs(g) * sc
    for t in range(T):
        ref[t, idx[t]] += d[t] * slope[t, idx[t]]
        mag[t, idx[t]] += dm[t] * slope[t, idx[t]]
    assert (np.abs(got - ref) <= 16 * REL * mag + 1e-37).all()


@pytest.mark.parametrize("T", [100, 8200])   # a wave per token, four tokens to a wave
def test_order_where_the_softmax_sum_is_at_its_worst(T):
    """Exact order of keys although the fp32 sum of the row is off as far as it can
    be: beside e^0 = 1 every other term is just below half an ulp of 1 and is lost
    from the lane's sum, so the one large score comes out too large, and its
    rival's key lies between its true and its rounded one."""
    E = 512
    l = np.full(E, -16.6356, np.float32)   # e^l = 0.99996 * 2^-24
    l[0] = 0.0
    x = np.exp(l.astype(np.float64))
    s = x / x.sum()
    rival = 300
    bias = np.full(E, -8.0, np.float32)
    bias[0] = -1.0 + 2.0 ** -15
    for above in (1e-7, 3e-7, 6e-7, 1e-6, -1e-7):   # of the rival's key over the exact one
        bias[rival] = s[0] + float(bias[0]) + above - s[rival]
        key = s + bias.astype(np.float64)
        best = int(np.argmax(key))
        assert best == (rival if above > 0 else 0)
        op = _op(T, E, 1)
        logits = _dev(np.tile(l, (T, 1)))
        for balance in (False, True):
            idx = op.gate(logits, GateConfig(), bias=_dev(bias), balance=balance)[1]
            assert bool((idx == best).all()), (above, balance)
