"""The experts' products and their gradients against 64 bits.

Two kinds of check.  With operands that are small integers every product and
partial sum is an integer below 2^24, exact in fp32, and the result is kept
below 257 so that bf16 holds it: bits must be equal.  With normal operands the
bound is the sum of what the format and the order of additions allow: a
product of K terms accumulated in fp32 is off by at most K * 2^-23 of the sum
of the terms' absolute values (one rounding or truncation per addition), the
activations are Lipschitz with constant 1.13 and evaluated to 2^-19 of their
value, and the result is rounded once to bf16, 2^-8 of itself.  Gradients
behind an activation also carry dz's own rounding, 2^-8 of every term.
"""
import numpy as np
import pytest
import torch

from layer_common import DEV, draw_indices, ints, layout, normal, routed_op

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
LIP = 1.13


def _act(z, name):
    F = torch.nn.functional
    if name in ("swiglu", "geglu"):
        g, u = z.chunk(2, dim=1)
        return (F.silu if name == "swiglu" else F.gelu)(g) * u
    return {"none": lambda v: v, "relu": F.relu, "gelu": F.gelu, "silu": F.silu}[name](z)


def _group_max(x, w):
    """[rows, out]: over the groups of 8 features, the sum of the largest |product|."""
    n, K = x.shape
    xg, wg = x.abs().float().reshape(n, K // 8, 8), w.abs().float().reshape(-1, K // 8, 8)
    out = torch.empty(n, w.shape[0], dtype=torch.float64, device=DEV)
    for a in range(0, n, 16):
        p = xg[a:a + 16, None] * wg[None]
        out[a:a + 16] = p.amax(-1).double().sum(-1)
    return out


def _forward(x, w, off, act="none", bias=None, residual=None, e4m3=False):
    """(result, bound on the difference) in 64 bits, expert by expert."""
    n = x.shape[0]
    K = x.shape[1]
    gated = act in ("swiglu", "geglu")
    cols = w.shape[1] // 2 if gated else w.shape[1]
    out = torch.zeros(n, cols, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(out)
    for e in range(w.shape[0]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        wt = w[e].t().contiguous()
        z = torch.mm(x[a:b], wt)
        dz = K * 2.0 ** -23 * torch.mm(x[a:b].abs(), wt.abs())
        if e4m3:
            dz = dz + 7 * 2.0 ** -13 * _group_max(x[a:b], w[e])
        if bias is not None:
            z = z + bias[e]
            dz = dz + 2.0 ** -23 * z.abs()
        y = _act(z, act)
        if gated:
            g, u = z.chunk(2, dim=1)
            dg, du = dz.chunk(2, dim=1)
            d = LIP * dg * (u.abs() + du) + (LIP * g.abs() + dg) * du + 2.0 ** -19 * y.abs()
        else:
            d = LIP * dz + (2.0 ** -19 * (y.abs() + z.abs()) if act != "none" else 0)
        if residual is not None:
            y = y + residual[a:b]
        out[a:b] = y
        tol[a:b] = d + U * (y.abs() + d)
    return out, tol + 1e-30


def _close(got, ref, tol, what=""):
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), \
        f"{what}: off by {float((err - tol).max())} beyond the bound, worst {float(err.max())}"


def _rows_case(rng, T, K, E, hot=None, drop=0.0):
    idx = draw_indices(rng, T, K, E, hot)
    if drop:
        idx = np.where(rng.random(idx.shape) < drop, -1, idx)
    pair, off = layout(idx, E)
    return routed_op(idx, E), off, T * K


# (T, K, E, in, out): few rows per expert (weights streamed past 16 or 32 rows)
# and many (tiles), one token, ragged columns, contractions that end inside a
# step or are shorter
# than one, and rows around a tile's edge
SHAPES = [(1, 1, 1, 8, 8), (1, 2, 4, 64, 16), (1, 8, 64, 264, 136), (3, 2, 2, 72, 24),
          (16, 2, 8, 520, 200), (17, 1, 1, 128, 264), (45, 2, 4, 152, 104), (63, 1, 1, 192, 72), (64, 2, 2, 136, 256),
          (65, 1, 1, 1032, 520), (200, 4, 8, 56, 312), (255, 1, 1, 320, 296), (257, 1, 1, 8, 8),
          (256, 2, 2, 264, 512), (700, 2, 3, 200, 1048)]


@pytest.mark.parametrize("T,K,E,fin,fout", SHAPES)
def test_forward_exact_integers(T, K, E, fin, fout):
    print(f"forward T={T} K={K} E={E} in={fin} out={fout}", flush=True)
    rng = np.random.default_rng(T + fin)
    op, off, n = _rows_case(rng, T, K, E)
    x, w = ints(rng, (n, fin)), ints(rng, (E, fout, fin))
    ref, _ = _forward(x.double(), w.double(), off)
    assert float(ref.abs().max()) <= 256
    got = op.expert_product(x, w)
    assert torch.equal(got.double(), ref)
    # with bias and residual in fp32 before the one rounding: still integers
    bias, res = ints(rng, (E, fout), -9, 9, torch.float32), ints(rng, (n, fout), -9, 9)
    ref, _ = _forward(x.double(), w.double(), off, "relu", bias.double(), res.double())
    got = op.expert_product(x, w, bias=bias, residual=res, activation="relu")
    assert float(ref.abs().max()) <= 256 and torch.equal(got.double(), ref)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "swiglu", "geglu"])
@pytest.mark.parametrize("T,K,E,fin,fout", [(2, 4, 8, 264, 80), (33, 2, 4, 584, 112), (60, 2, 4, 200, 176),
                                            (400, 2, 3, 328, 304)])
def test_forward_activations(T, K, E, fin, fout, act):
    rng = np.random.default_rng(T)
    op, off, n = _rows_case(rng, T, K, E)
    x, w = normal(rng, (n, fin)), normal(rng, (E, fout, fin), fin ** -0.5)
    bias = normal(rng, (E, fout), dtype=torch.float32)
    cols = fout // 2 if act in ("swiglu", "geglu") else fout
    res = normal(rng, (n, cols))
    preact = torch.full((n, fout), 7.0, dtype=torch.bfloat16, device=DEV)
    got = op.expert_product(x, w, bias=bias, activation=act, residual=res, preact=preact)
    ref, tol = _forward(x.double(), w.double(), off, act, bias.double(), res.double())
    _close(got, ref, tol, act)
    zref, ztol = _forward(x.double(), w.double(), off, "none", bias.double())
    _close(preact, zref, ztol, "preact")
    # without the extras, and into a given buffer; the residual may be it
    assert torch.equal(op.expert_product(x, w, bias=bias, activation=act, residual=res, out=res),
                       got)


def test_forward_large_and_skewed():
    """A busy expert of many tiles beside idle and small ones, long contraction."""
    rng = np.random.default_rng(1)
    T, K, E, fin, fout = 1500, 2, 5, 1544, 784
    idx = draw_indices(rng, T, K, E - 1, hot=0.9)     # the last expert gets no row
    pair, off = layout(idx, E)
    op, n = routed_op(idx, E), T * K
    x, w = normal(rng, (n, fin)), normal(rng, (E, fout, fin), fin ** -0.5)
    ref, tol = _forward(x.double(), w.double(), off, "swiglu")
    _close(op.expert_product(x, w, activation="swiglu"), ref, tol)


@pytest.mark.parametrize("T", [3, 50, 600])
def test_rows_outside_stay(T):
    """A subset of the experts, dropped pairs, repeated experts: rows that belong
    to no expert of the call keep what they held, in outputs and gradients."""
    rng = np.random.default_rng(T)
    K, E, fin, fout, first, ne = 4, 8, 72, 40, 2, 3
    idx = draw_indices(rng, T, K, E)
    idx[:, 3] = idx[:, 0]                         # the same expert twice: two rows
    idx[::3, 1] = -1
    pair, off = layout(idx, E)
    op, n = routed_op(idx, E), T * K
    x = ints(rng, (n, fin))
    x[off[-1]:] = float("nan")                    # rows behind the last: never read into a result
    w = ints(rng, (ne, fout, fin))
    keep = torch.full((n, fout), 3.5, dtype=torch.bfloat16, device=DEV)
    out = op.expert_product(x, w, first_expert=first, out=keep.clone())
    a, b = off[first], off[first + ne]
    ref, _ = _forward(x[a:b].double(), w.double(), off[first:first + ne + 1] - a)
    assert torch.equal(out[a:b].double(), ref)
    assert torch.equal(out[:a], keep[:a]) and torch.equal(out[b:], keep[b:])
    dy = ints(rng, (n, fout))
    dy[:a], dy[b:] = float("nan"), float("nan")
    gx, gw, gb = op.expert_product_backward(dy, x, w, first_expert=first, bias=True,
                                            weight_dtype=torch.float32)
    off2 = off[first:first + ne + 1]
    for e in range(ne):
        s = slice(off2[e], off2[e + 1])
        d = dy[s].double()
        assert torch.equal(gx[s].double(), torch.mm(d, w[e].double()))
        assert torch.equal(gw[e].double(), torch.mm(d.t().contiguous(), x[s].double()))
        assert torch.equal(gb[e].double(), d.sum(0))


@pytest.mark.parametrize("T,K,E,fin,fout", SHAPES)
def test_backward_exact_integers(T, K, E, fin, fout):
    print(f"backward T={T} K={K} E={E} in={fin} out={fout}", flush=True)
    rng = np.random.default_rng(T + fin + 1)
    op, off, n = _rows_case(rng, T, K, E)
    x, w, dy = ints(rng, (n, fin)), ints(rng, (E, fout, fin)), ints(rng, (n, fout))
    gx, gw, gb = op.expert_product_backward(dy, x, w, bias=True)
    gx32, gw32, none = op.expert_product_backward(dy, x, w, weight_dtype=torch.float32,
                                                  need_input=False)
    assert gx32 is None and none is None
    for e in range(E):
        s = slice(off[e], off[e + 1])
        d = dy[s].double()
        rx, rw = torch.mm(d, w[e].double()), torch.mm(d.t().contiguous(), x[s].double())
        assert max(float(rx.abs().max()) if rx.numel() else 0, float(rw.abs().max())) <= 256
        assert torch.equal(gx[s].double(), rx)
        assert torch.equal(gw[e].double(), rw) and torch.equal(gw32[e].double(), rw)
        assert torch.equal(gb[e].double(), d.sum(0))


@pytest.mark.parametrize("act", ["relu", "gelu", "silu", "swiglu", "geglu"])
@pytest.mark.parametrize("T,K,E,fin,fout", [(5, 2, 4, 72, 80), (300, 2, 4, 264, 336)])
def test_backward_activations(T, K, E, fin, fout, act):
    rng = np.random.default_rng(T)
    op, off, n = _rows_case(rng, T, K, E)
    cols = fout // 2 if act in ("swiglu", "geglu") else fout
    x, w = normal(rng, (n, fin)), normal(rng, (E, fout, fin), fin ** -0.5)
    z, dy = normal(rng, (n, fout), 2.0), normal(rng, (n, cols))
    gx, gw, gb = op.expert_product_backward(dy, x, w, activation=act, preact=z, bias=True,
                                            weight_dtype=torch.float32)
    zz = z.double().requires_grad_(True)
    dz, = torch.autograd.grad(_act(zz, act), zz, dy.double())
    # an act' of size up to LIP, off by 2^-19; then bf16: U of every entry
    mag = dz.abs() * U + 2.0 ** -18 * (dy.double().abs().repeat(1, fout // cols)
                                       * (1 + z.double().abs().amax()) ** 2)
    for e in range(E):
        s = slice(off[e], off[e + 1])
        m, d, rows = mag[s], dz[s], off[e + 1] - off[e]
        W, X = w[e].double(), x[s].double()
        r = torch.mm(d, W)
        t = torch.mm(m, W.abs()) + fout * 2.0 ** -23 * torch.mm(d.abs() + m, W.abs())
        _close(gx[s], r, t + U * (r.abs() + t) + 1e-30, "input")
        r = torch.mm(d.t().contiguous(), X)
        t = torch.mm(m.t().contiguous(), X.abs()) + \
            rows * 2.0 ** -23 * torch.mm((d.abs() + m).t().contiguous(), X.abs())
        _close(gw[e], r, t + 1e-30, "weight")
        r = d.sum(0)
        t = (m - U * d.abs()).sum(0) + rows * 2.0 ** -23 * (d.abs() + m).sum(0)
        _close(gb[e], r, t + 1e-30, "bias")


def test_backward_against_differences():
    """The forward's own change along a direction, in the products alone (no
    activation, integers: the product is bilinear and every step exact)."""
    rng = np.random.default_rng(4)
    op, off, n = _rows_case(rng, 40, 2, 4)
    x, w, dy = ints(rng, (n, 64)), ints(rng, (4, 48, 64)), ints(rng, (n, 48))
    dx, dw = ints(rng, (n, 64)), ints(rng, (4, 48, 64))
    gx, gw, _ = op.expert_product_backward(dy, x, w, weight_dtype=torch.float32)
    base, moved = op.expert_product(x, w), op.expert_product(x, w + dw)
    lhs = ((moved.double() - base.double()) * dy.double()).sum()
    assert float(lhs) == float((gw.double() * dw.double()).sum())
    lhs = ((op.expert_product(x + dx, w).double() - base.double()) * dy.double()).sum()
    assert float(lhs) == float((gx.double() * dx.double()).sum())


def _e4m3(rng, shape):
    codes = rng.integers(0, 256, shape).astype(np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x38          # no NaN
    return torch.from_numpy(codes).to(DEV).view(torch.float8_e4m3fn)


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("T,K,E,fin,fout", [(1, 4, 16, 128, 32), (2, 2, 4, 640, 144),
                                            (40, 2, 2, 256, 80), (300, 2, 2, 384, 272),
                                            (520, 1, 1, 1152, 560)])
def test_forward_e4m3(T, K, E, fin, fout, act):
    """Every code but NaN, scales over a wide range, up rows that start inside a
    scale block."""
    rng = np.random.default_rng(T)
    op, off, n = _rows_case(rng, T, K, E)
    x8, w8 = _e4m3(rng, (n, fin)), _e4m3(rng, (E, fout, fin))
    sx = torch.from_numpy(np.exp(rng.uniform(-9, -5, (n, fin // 128))).astype(np.float32)).to(DEV)
    sw = torch.from_numpy(np.exp(rng.uniform(-9, -5, (E, (fout + 127) // 128, fin // 128)))
                          .astype(np.float32)).to(DEV)
    bias = normal(rng, (E, fout), dtype=torch.float32)
    got = op.expert_product(x8, w8, scales=sx, weight_scales=sw, bias=bias, activation=act)
    x = (x8.double().reshape(n, -1, 128) * sx.double()[..., None]).reshape(n, fin)
    w = w8.double() * sw.double().repeat_interleave(128, 1)[:, :fout].repeat_interleave(128, 2)
    ref, tol = _forward(x, w, off, act, bias.double(), e4m3=True)
    _close(got, ref, tol, "e4m3")


def test_e4m3_dispatch_feeds_the_product():
    """Rows and scales as the quantizing dispatch writes them."""
    from combine_routing_histogram_amd.op import EpDispatchCombineConfig, EpDispatchCombineOp
    rng = np.random.default_rng(8)
    T, H, K, E, fout = 96, 512, 4, 8, 144
    idx = draw_indices(rng, T, K, E)
    pair, off = layout(idx, E)
    op = EpDispatchCombineOp(EpDispatchCombineConfig(T, H, K, E, 2, quant="fp8_e4m3_b128"), DEV)
    out, _, scales, _, _ = op.dispatch(normal(rng, (T, H)), None, None,
                                       torch.from_numpy(idx).to(DEV))
    w8, sw = _e4m3(rng, (E, fout, H)), torch.full((E, 2, 4), 2.0 ** -9, device=DEV)
    got = op.expert_product(out, w8, scales=scales, weight_scales=sw)
    x = (out.double().reshape(T * K, -1, 128) * scales.double()[..., None]).reshape(T * K, H)
    ref, tol = _forward(x, w8.double() * 2.0 ** -9, off, e4m3=True)
    _close(got, ref, tol)


def test_not_a_number_stays_in_its_row():
    rng = np.random.default_rng(6)
    for T in (4, 300):
        op, off, n = _rows_case(rng, T, 1, 2)
        x, w = ints(rng, (n, 72)), ints(rng, (2, 40, 72))
        clean = op.expert_product(x, w)
        x[n // 2, 71] = float("nan")
        got = op.expert_product(x, w)
        rows = torch.arange(n, device=DEV) != n // 2
        assert torch.equal(got[rows], clean[rows]) and bool(got[n // 2].isnan().all())
        assert bool(op.expert_product(x, w, activation="relu")[n // 2].isnan().all())


def test_no_rows():
    op = routed_op(np.full((3, 2), -1), 4)       # every pair dropped
    x, w = torch.zeros(6, 64, device=DEV).bfloat16(), torch.ones(4, 16, 64, device=DEV).bfloat16()
    keep = torch.full((6, 16), 2.0, device=DEV).bfloat16()
    assert torch.equal(op.expert_product(x, w, out=keep.clone()), keep)
    _, gw, gb = op.expert_product_backward(keep, x, w, bias=True)
    assert not gw.any() and not gb.any()
    op.dispatch(torch.zeros(0, 8, dtype=torch.bfloat16, device=DEV), None, None,
                torch.zeros(0, 2, dtype=torch.int32, device=DEV))       # no token at all
    _, gw, gb = op.expert_product_backward(keep[:0], x[:0], w, bias=True)
    assert op.expert_product(x[:0], w).shape == (0, 16) and not gw.any() and not gb.any()


@pytest.mark.parametrize("T,K,H,E", [(1, 1, 8, 1), (5, 3, 2056, 7), (64, 8, 512, 16),
                                     (33, 16, 4104, 32), (200, 2, 7168, 8)])
def test_combine_backward(T, K, H, E):
    """grad rows are one rounding of w * dy (2^-8; w dy itself exact in fp32 to
    2^-24); grad weights a sum of H fp32 products, H * 2^-24 of their absolute
    values.  Dropped pairs, repeated experts and rows without a pair included."""
    rng = np.random.default_rng(T + H)
    idx = rng.integers(0, E, (T, K)).astype(np.int32)
    if T > 1:
        idx[rng.random((T, K)) < 0.1] = -1
    pair, off = layout(idx, E)
    op = routed_op(idx, E, hidden=H)
    n = T * K
    x, dy = normal(rng, (n, H)), normal(rng, (T, H))
    wr = normal(rng, (n, K), dtype=torch.float32)
    x[len(pair):] = float("nan")
    tok = torch.from_numpy(pair // K).to(DEV)
    k = torch.from_numpy(pair % K).to(DEV)
    for w in (wr, None):
        gx, gw = op.combine_backward(dy, x, w)
        ww = w[torch.arange(len(pair), device=DEV), k].double()[:, None] if w is not None else 1.0
        ref = ww * dy[tok].double()
        _close(gx[:len(pair)], ref, (U + 2.0 ** -23) * ref.abs() + 1e-38, "rows")
        d = dy[tok].double() * x[:len(pair)].double()
        rw = torch.zeros(n, dtype=torch.float64, device=DEV)
        tw = torch.zeros_like(rw)
        at = torch.from_numpy(pair).to(DEV)
        rw[at], tw[at] = d.sum(1), H * 2.0 ** -24 * d.abs().sum(1)
        _close(gw.reshape(-1), rw, tw, "weights")
    # dispatch's own gradient: each token's rows added in fp32
    rows = ints(rng, (n, H))
    rows[len(pair):] = float("nan")
    ref = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    ref.index_add_(0, tok, rows[:len(pair)].double())
    assert torch.equal(op.dispatch_backward(rows).double(), ref)
