"""Products of few rows over long contractions: the loop that keeps several steps in flight, for
every type, one and two row blocks of an expert, gated or not, and weights whose rows are whole
128-byte lines or not.  The bounds are those of test_gpu_layer_int8.py, and for the other types
of test_gpu_layer_product.py.
"""
import numpy as np
import pytest
import torch

from layer_common import DEV, draw_indices, layout, normal, routed_op
from test_gpu_layer_int8 import _codes, _reference, _scales
from test_gpu_layer_product import _close, _forward

pytestmark = pytest.mark.gpu


def _inside_a_line(w):
    """The same weight, its first byte 16 past a line's, NaN (int8: -1) before and behind."""
    n = w.numel() * w.element_size()
    raw = torch.full((n + 256,), 0xff, dtype=torch.uint8, device=DEV)
    raw[16:16 + n] = w.view(torch.uint8).flatten()
    return raw[16:16 + n].view(w.dtype).view(w.shape)


# rows of an expert in the mean: 1 to 12 are one block of 16 (bf16 10), 13 to 20 (24) two
@pytest.mark.parametrize("act", ["none", "swiglu", "geglu"])
@pytest.mark.parametrize("T,K,E", [(1, 8, 8), (4, 2, 8), (40, 2, 8), (48, 2, 8), (52, 2, 8),
                                   (80, 2, 8)])
@pytest.mark.parametrize("fin", [1664, 2048, 2064, 4096, 4112])
def test_int8(fin, T, K, E, act):
    print(f"int8 T={T} K={K} E={E} in={fin} {act}", flush=True)
    rng = np.random.default_rng(T + fin)
    idx, fout = draw_indices(rng, T, K, E), 144
    _, off = layout(idx, E)
    op, n = routed_op(idx, E), T * K
    x, w = _codes(rng, (n, fin)), _codes(rng, (E, fout, fin))
    sx, sw = _scales(rng, (n, 1)) / 64, _scales(rng, (E, fout)) / 64
    ref, tol = _reference(x, sx, w, sw, off, act, None, None)
    for weight in (w, _inside_a_line(w)):
        _close(op.expert_product(x, weight, scales=sx, weight_scales=sw, activation=act),
               ref[:n], tol[:n])


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("T,K,E", [(1, 8, 8), (40, 2, 8), (44, 2, 8), (96, 2, 8)])
@pytest.mark.parametrize("fin", [1024, 1032, 2048, 2056])
def test_bf16(fin, T, K, E, act):
    print(f"bf16 T={T} K={K} E={E} in={fin} {act}", flush=True)
    rng = np.random.default_rng(T + fin)
    idx = draw_indices(rng, T, K, E)
    _, off = layout(idx, E)
    op, n = routed_op(idx, E), T * K
    x, w = normal(rng, (n, fin)), normal(rng, (E, 144, fin), fin ** -0.5)
    ref, tol = _forward(x.double(), w.double(), off, act)
    for weight in (w, _inside_a_line(w)):
        _close(op.expert_product(x, weight, activation=act), ref, tol)


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("T,K,E", [(1, 8, 8), (48, 2, 8)])
@pytest.mark.parametrize("fin", [1024, 2176])
def test_e4m3(fin, T, K, E, act):
    print(f"e4m3 T={T} K={K} E={E} in={fin} {act}", flush=True)
    rng = np.random.default_rng(T + fin)
    idx, blocks = draw_indices(rng, T, K, E), fin // 128
    _, off = layout(idx, E)
    op, n = routed_op(idx, E), T * K
    x, w = (normal(rng, s).to(torch.float8_e4m3fn) for s in ((n, fin), (E, 144, fin)))
    unit = lambda *s: torch.from_numpy(rng.uniform(0.5, 2, s).astype(np.float32)).to(DEV)
    sx, sw = unit(n, blocks), unit(E, 2, blocks) * fin ** -0.5
    xd = x.double() * sx.double().repeat_interleave(128, 1)
    wd = w.double() * sw.double().repeat_interleave(128, 1)[:, :144].repeat_interleave(128, 2)
    ref, tol = _forward(xd, wd, off, act, e4m3=True)
    for weight in (w, _inside_a_line(w)):
        _close(op.expert_product(x, weight, scales=sx, weight_scales=sw, activation=act), ref, tol)
