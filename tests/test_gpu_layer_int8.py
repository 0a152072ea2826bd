"""The experts' products in 8-bit integers.

Sums of products of codes are whole numbers that the kernel adds exactly; the
test's come from 64-bit sums.  Behind them z takes four roundings in fp32 (the sum's
conversion, the scales' product, the product with it, the bias), 2^-22 of its
parts; activations are Lipschitz with constant 1.13 and evaluated to 2^-19; the result
is rounded once to bf16, 2^-8.
"""
import numpy as np
import pytest
import torch

from layer_common import DEV, draw_indices, layout, normal, routed_op

pytestmark = pytest.mark.gpu
U, LIP = 2.0 ** -8, 1.13


def _codes(rng, shape, lo=-128):
    return torch.from_numpy(rng.integers(lo, 128, shape).astype(np.int8)).to(DEV)


def _scales(rng, shape):
    return torch.from_numpy(np.exp(rng.normal(-8, 1, shape)).astype(np.float32)).to(DEV)


def _act(z, name):
    F = torch.nn.functional
    if name in ("swiglu", "geglu"):
        g, u = z.chunk(2, dim=1)
        return (F.silu if name == "swiglu" else F.gelu)(g) * u
    return {"none": lambda v: v, "relu": F.relu, "gelu": F.gelu, "silu": F.silu}[name](z)


def _reference(x, sx, w, sw, off, act, bias, residual):
    """(result, bound) in 64 bits; sums of up to 2^17 products are exact there."""
    gated = act in ("swiglu", "geglu")
    cols = w.shape[1] // 2 if gated else w.shape[1]
    out = torch.zeros(x.shape[0], cols, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(out)
    for e in range(w.shape[0]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        z = torch.mm(x[a:b].double(), w[e].double().t().contiguous())
        z = z * sx[a:b].double() * sw[e].double()
        dz = 2.0 ** -22 * z.abs()
        if bias is not None:
            z = z + bias[e].double()
            dz = dz + 2.0 ** -23 * z.abs()
        y = _act(z, act)
        if gated:
            g, u = z.chunk(2, dim=1)
            dg, du = dz.chunk(2, dim=1)
            d = LIP * dg * (u.abs() + du) + (LIP * g.abs() + dg) * du + 2.0 ** -19 * y.abs()
        else:
            d = LIP * dz + (2.0 ** -19 * (y.abs() + z.abs()) if act != "none" else 0)
        if residual is not None:
            y = y + residual[a:b].double()
            d = d + 2.0 ** -23 * y.abs()
        out[a:b], tol[a:b] = y, d + U * (y.abs() + d)
    return out, tol + 1e-30


def _check(got, ref, tol, n):
    err = (got[:n].double() - ref[:n]).abs()
    assert bool((err <= tol[:n]).all()), float((err - tol[:n]).max())


# (T, K, E, in, out): streamed past 16 and 32 rows, tiles of 64 and 256 rows, ragged
# rows, columns and contractions
SHAPES = [(1, 1, 1, 16, 8), (1, 8, 64, 272, 144), (3, 2, 2, 144, 24), (17, 1, 1, 128, 264),
          (45, 2, 4, 304, 104), (63, 1, 1, 400, 72), (65, 1, 1, 2064, 520), (257, 1, 1, 16, 8),
          (256, 2, 2, 528, 512), (700, 2, 3, 208, 1048)]


@pytest.mark.parametrize("T,K,E,fin,fout", SHAPES)
def test_products(T, K, E, fin, fout):
    print(f"int8 T={T} K={K} E={E} in={fin} out={fout}", flush=True)
    rng = np.random.default_rng(T + fin)
    idx = draw_indices(rng, T, K, E)
    _, off = layout(idx, E)
    op, n = routed_op(idx, E), T * K
    x, w = _codes(rng, (n, fin)), _codes(rng, (E, fout, fin))
    sx, sw = _scales(rng, (n, 1)), _scales(rng, (E, fout))
    ref, tol = _reference(x, sx, w, sw, off, "none", None, None)
    _check(op.expert_product(x, w, scales=sx, weight_scales=sw), ref, tol, n)
    bias, res = normal(rng, (E, fout), dtype=torch.float32), normal(rng, (n, fout))
    ref, tol = _reference(x, sx, w, sw, off, "relu", bias, res)
    got = op.expert_product(x, w, scales=sx, weight_scales=sw, bias=bias, activation="relu",
                            residual=res)
    _check(got, ref, tol, n)


@pytest.mark.parametrize("act", ["gelu", "silu", "swiglu", "geglu"])
@pytest.mark.parametrize("T,K,E,fin,fout", [(2, 4, 8, 272, 80), (33, 2, 4, 592, 112),
                                            (400, 2, 3, 336, 304)])
def test_activations(T, K, E, fin, fout, act):
    rng = np.random.default_rng(T)
    idx = draw_indices(rng, T, K, E)
    _, off = layout(idx, E)
    op, n = routed_op(idx, E), T * K
    x, w = _codes(rng, (n, fin)), _codes(rng, (E, fout, fin))
    sx, sw = _scales(rng, (n, 1)), _scales(rng, (E, fout))
    bias = normal(rng, (E, fout), dtype=torch.float32)
    ref, tol = _reference(x, sx, w, sw, off, act, bias, None)
    z = torch.empty(n, fout, dtype=torch.bfloat16, device=DEV)
    got = op.expert_product(x, w, scales=sx, weight_scales=sw, bias=bias, activation=act,
                            preact=z)
    _check(got, ref, tol, n)
    ref, tol = _reference(x, sx, w, sw, off, "none", bias, None)
    _check(z, ref, tol, n)


@pytest.mark.parametrize("T", [2, 20, 40, 100])
def test_longest_contraction(T):
    """All products at their largest, 2^14, as many as may be: just below 2^31."""
    fin, op = (1 << 17) - 16, routed_op(np.zeros((T, 1), np.int32), 1)
    x = torch.full((T, fin), -128, dtype=torch.int8, device=DEV)
    w = torch.full((1, 8, fin), -128, dtype=torch.int8, device=DEV)
    w[0, 1::2] = 127
    one = torch.ones(T, 1, device=DEV)
    got = op.expert_product(x, w, scales=one, weight_scales=torch.ones(1, 8, device=DEV))
    for c, want in ((0, fin * 16384.0), (1, fin * -128.0 * 127)):
        assert bool((got[:, c::2].double() - want).abs().max() <= (U + 2.0 ** -22) * abs(want))


@pytest.mark.parametrize("T", [3, 50, 600])
def test_rows_outside_stay(T):
    """Some of the experts, dropped pairs, an expert twice: rows that belong to no expert of
    the call keep what they held, whatever their codes and scales are."""
    rng = np.random.default_rng(T)
    K, E, fin, fout, first, ne = 4, 8, 144, 40, 2, 3
    idx = draw_indices(rng, T, K, E)
    idx[:, 3] = idx[:, 0]
    idx[::3, 1] = -1
    _, off = layout(idx, E)
    op, n = routed_op(idx, E), T * K
    x, w = _codes(rng, (n, fin)), _codes(rng, (ne, fout, fin))
    sx, sw = _scales(rng, (n, 1)), _scales(rng, (ne, fout))
    a, b = off[first], off[first + ne]
    sx[:a] = sx[b:] = float("nan")
    keep = torch.full((n, fout), 3.5, dtype=torch.bfloat16, device=DEV)
    got = op.expert_product(x, w, scales=sx, weight_scales=sw, first_expert=first,
                            out=keep.clone())
    ref, tol = _reference(x[a:b], sx[a:b], w, sw, off[first:first + ne + 1] - a, "none", None,
                          None)
    _check(got[a:b], ref, tol, b - a)
    assert torch.equal(got[:a], keep[:a]) and torch.equal(got[b:], keep[b:])
