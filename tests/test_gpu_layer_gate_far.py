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
