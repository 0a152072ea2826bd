"""The gate, its losses and its gradient against the definitions in 64 bits.

Tolerances.  Logits here stay within 30 of each other, so an exponent's
argument (a difference of logits, rounded once) is off by at most 30 * 2^-24
and every score by that, plus a few ulp of exp, sum and division: relative
errors below REL = (30 + 34) * 2^-24 ~ 4e-6.  A weight is a ratio of two such
sums (2 REL), a loss a mean of products of them.  A gradient entry is a sum of
terms, each below the terms' absolute values times a few REL; the bound is
taken on those absolute values.  bf16 gradients are rounded once: 2^-8.
"""
import numpy as np
import pytest
import torch

from combine_routing_histogram_amd.op import (EpDispatchCombineConfig, EpDispatchCombineOp,
                                              GateConfig)
from layer_common import DEV

pytestmark = pytest.mark.gpu
REL = 64 * 2.0 ** -24


def _op(T, E, K):
    return EpDispatchCombineOp(EpDispatchCombineConfig(max(T, 1), 8, K, E, 1), DEV)


def _reference(l, K, cfg, bias=None, mask=None):
    """(weights, indices, counts, losses) in 64 bits from a [T, E] float64 array."""
    T, E = l.shape
    w, idx = np.zeros((T, K)), np.full((T, K), -1, np.int32)
    counts, P, z, n = np.zeros(E + 1, np.int64), np.zeros(E), 0.0, 0
    for t in range(T):
        row = l[t]
        if mask is not None and not mask[t]:
            continue
        if np.isnan(row).any() or np.isposinf(row).any():
            w[t] = np.nan
            P[:], z, n = np.nan, np.nan, n + 1
            continue
        if np.isneginf(row).all():
            continue
        n += 1
        x = np.exp(row - row.max())
        soft = x / x.sum()
        s = soft if cfg.score == "softmax" else 1 / (1 + np.exp(-row))
        key = row if bias is None else np.where(np.isneginf(row), -np.inf, s + bias)
        order = np.argsort(-key, kind="stable")[:K]
        order = order[~np.isneginf(key[order])]
        idx[t, :order.size] = order
        counts[order] += 1
        r = s[order]
        if cfg.renormalize:   # through the logarithms: no sum of scores underflows
            ls = row[order] if cfg.score == "softmax" else -np.logaddexp(0, -row[order])
            r = np.exp(ls - ls.max()) if order.size else r
            r = r / r.sum()
        w[t, :order.size] = cfg.scale * r
        P += s / s.sum()
        z += (row.max() + np.log(x.sum())) ** 2
    counts[E] = n
    m = max(n, 1)
    losses = np.array([E * (counts[:E] / (m * K) * P / m).sum(), z / m])
    return w, idx, counts, losses


def _gradient(l, K, cfg, idx, gw, counts, gl, mask=None):
    """(gradient, bound of its terms' absolute values) from the formulas, 64 bits."""
    T, E = l.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    n = max(counts[E], 1) if counts is not None else 1
    for t in range(T):
        row = l[t]
        if (mask is not None and not mask[t]) or np.isneginf(row).all():
            continue
        if np.isnan(row).any() or np.isposinf(row).any():
            out[t] = np.nan
            continue
        x = np.exp(row - row.max())
        soft = x / x.sum()
        sig = 1 / (1 + np.exp(-row))
        s = soft if cfg.score == "softmax" else sig
        if gw is not None:
            c = idx[t][idx[t] >= 0]
            g = cfg.scale * gw[t][:c.size]
            if cfg.renormalize:
                ls = row[c] if cfg.score == "softmax" else -np.logaddexp(0, -row[c])
                r = np.exp(ls - ls.max())
                r /= r.sum()
                d = r * (g - (g * r).sum())
                dm = r * (np.abs(g) + (np.abs(g) * r).sum())
                if cfg.score == "sigmoid":
                    d, dm = d * (1 - sig[c]), dm   # 1 - sigma is exact to an ulp of 1
                np.add.at(out[t], c, d)
                np.add.at(mag[t], c, dm)
            elif cfg.score == "softmax":
                np.add.at(out[t], c, g * soft[c])
                np.add.at(mag[t], c, np.abs(g) * soft[c])
                out[t] -= soft * (g * soft[c]).sum()
                mag[t] += soft * (np.abs(g) * soft[c]).sum()
            else:
                np.add.at(out[t], c, g * sig[c] * (1 - sig[c]))
                np.add.at(mag[t], c, np.abs(g) * sig[c])
        if gl is not None:
            f = counts[:E] / (n * K)
            p = s / s.sum()
            b = gl[0] * E / n * p * (f - (f * p).sum())
            bm = abs(gl[0]) * E / n * p * (f + (f * p).sum())
            if cfg.score == "sigmoid":
                b = b * (1 - sig)
            lse = row.max() + np.log(x.sum())
            out[t] += b + gl[1] * 2 / n * lse * soft
            mag[t] += bm + abs(gl[1]) * 2 / n * (abs(lse) + abs(row.max()) + 30) * soft
        out[t][np.isneginf(row)] = 0
    return out, mag


def _check(op, logits, K, cfg, bias=None, mask=None, seed=0, T=None):
    l = logits.double().cpu().numpy()
    T, E = l.shape
    rng = np.random.default_rng(seed)
    b = None if bias is None else bias.double().cpu().numpy()
    m = None if mask is None else mask.cpu().numpy() != 0
    w, idx, counts, losses = [t.cpu().numpy() for t in
                              op.gate(logits, cfg, bias=bias, mask=mask, balance=True)]
    w2, idx2 = [t.cpu().numpy() for t in op.gate(logits, cfg, bias=bias, mask=mask)]
    assert np.array_equal(w, w2, equal_nan=True) and np.array_equal(idx, idx2)
    rw, ridx, rcounts, rlosses = _reference(l, K, cfg, b, m)
    assert np.array_equal(idx, ridx)
    assert np.array_equal(counts, rcounts)
    np.testing.assert_allclose(w, rw, rtol=4 * REL, atol=1e-37)
    # the z loss: lse is off by REL of the largest logit's size
    top = np.abs(l[np.isfinite(l)]).max() + 6 if np.isfinite(l).any() else 1
    np.testing.assert_allclose(losses, rlosses, rtol=8 * REL, atol=4 * REL * top * top)
    gw = rng.standard_normal((T, K)).astype(np.float32)
    gl = np.array([0.5, 0.25], np.float32)
    dev = lambda a: torch.from_numpy(a).to(DEV)
    for use_w, use_l in ((True, True), (True, False), (False, True)):
        grad = op.gate_backward(logits, dev(idx), cfg, grad_weights=dev(gw) if use_w else None,
                                mask=mask, counts=dev(counts) if use_l else None,
                                grad_losses=dev(gl) if use_l else None)
        assert grad.dtype == logits.dtype
        ref, mag = _gradient(l, K, cfg, idx, gw if use_w else None, counts if use_l else None,
                             gl if use_l else None, m)
        got = grad.double().cpu().numpy()
        tol = 16 * REL * mag + 1e-37
        if logits.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(ref)
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        ok = np.abs(got - ref) <= tol
        assert ok[~np.isnan(ref)].all(), np.abs(got - ref)[~ok].max()


CONFIGS = [GateConfig(), GateConfig(renormalize=False, scale=2.5),
           GateConfig("sigmoid", True, 2.5), GateConfig("sigmoid", False, 1.0)]


# experts around every boundary of the lanes' slots (64, 128, 256, 512), odd
# counts (unaligned rows), one expert; tokens around a block's pass (32)
@pytest.mark.parametrize("cfg", CONFIGS, ids=lambda c: f"{c.score}-{c.renormalize}")
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 256, 8), (31, 8, 2), (32, 64, 8), (33, 65, 16),
                                   (100, 127, 6), (64, 128, 8), (65, 129, 3), (40, 255, 8),
                                   (37, 256, 1), (35, 257, 16), (70, 511, 5), (33, 512, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_gate_matches_the_definition(T, E, K, cfg, dtype):
    print(f"gate T={T} E={E} K={K} {cfg} {dtype}", flush=True)
    rng = np.random.default_rng(T * 1000 + E)
    logits = torch.from_numpy(2 * rng.standard_normal((T, E))).to(DEV).to(dtype)
    bias = torch.from_numpy(0.2 * rng.standard_normal(E).astype(np.float32)).to(DEV)
    mask = torch.from_numpy((rng.random(T) < 0.8).astype(np.uint8)).to(DEV)
    op = _op(T, E, K)
    _check(op, logits, K, cfg)
    _check(op, logits, K, cfg, bias=bias, mask=mask, seed=1)


# more than 16 tokens per expert: four tokens share a wave
@pytest.mark.parametrize("cfg", [CONFIGS[0], CONFIGS[2], CONFIGS[3]],
                         ids=lambda c: f"{c.score}-{c.renormalize}")
@pytest.mark.parametrize("T,E,K", [(17, 1, 1), (130, 8, 2), (1030, 64, 8), (1043, 65, 16),
                                   (2049, 128, 8), (2070, 129, 6), (4113, 257, 5)])
def test_gate_many_tokens(T, E, K, cfg):
    print(f"gate T={T} E={E} K={K} {cfg}", flush=True)
    rng = np.random.default_rng(T)
    dtype = torch.bfloat16 if T % 2 else torch.float32
    logits = torch.from_numpy(2 * rng.standard_normal((T, E))).to(DEV).to(dtype)
    bias = torch.from_numpy(0.2 * rng.standard_normal(E).astype(np.float32)).to(DEV)
    mask = torch.from_numpy((rng.random(T) < 0.8).astype(np.uint8)).to(DEV)
    _check(_op(T, E, K), logits, K, cfg, bias=bias if T % 3 else None, mask=mask)


# 24 experts: up to 384 tokens a wave each, then four to a wave
@pytest.mark.parametrize("T", [40, 400])
@pytest.mark.parametrize("cfg", CONFIGS, ids=lambda c: f"{c.score}-{c.renormalize}")
def test_masked_and_missing(cfg, T):
    """Masked tokens whatever they hold, rows without experts, fewer experts than
    K, and logits that are not numbers."""
    rng = np.random.default_rng(3)
    E, K = 24, 4
    l = 2 * rng.standard_normal((T, E)).astype(np.float32)
    inf = np.inf
    l[0] = -inf                 # no expert
    l[1, 3:] = -inf             # three of four
    l[2, 1:] = -inf             # one
    l[3], l[4, 5] = np.nan, inf  # masked below
    l[5, ::2] = -inf
    l[6] = 0.25                 # all equal: the lowest indices
    l[7, 10:] = l[7, 0]
    mask = np.ones(T, np.uint8)
    mask[[3, 4, 9, 39]] = 0
    op = _op(T, E, K)
    logits, mk = torch.from_numpy(l).to(DEV), torch.from_numpy(mask).to(DEV)
    bias = torch.from_numpy(0.3 * rng.standard_normal(E).astype(np.float32)).to(DEV)
    for b in (None, bias, torch.zeros_like(bias)):
        _check(op, logits, K, cfg, bias=b, mask=mk)
        _check(op, logits, K, cfg, bias=b, mask=mk.bool())
    _check(op, logits, K, cfg, mask=torch.zeros_like(mk))       # nothing but padding
    l[20, 3], l[21, 0] = np.nan, inf                            # not masked: they show
    logits = torch.from_numpy(l).to(DEV)
    _check(op, logits, K, cfg, bias=bias, mask=mk)


@pytest.mark.parametrize("T", [256, 2100])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_and_near_ties_with_a_bias(score, T):
    """Keys that agree in 32 bits are ordered as in 64; equal ones by index."""
    rng = np.random.default_rng(5)
    E, K = 128, 8
    l = np.round(4 * rng.standard_normal((T, E)) / 2) / 2          # many equal logits
    l[::2] += rng.integers(0, 3, (T // 2, E)) * 2.0 ** -22         # or nearly equal
    logits = torch.from_numpy(l.astype(np.float32)).to(DEV)
    bias = torch.zeros(E, device=DEV)
    _check(_op(T, E, K), logits, K, GateConfig(score, True, 1.0), bias=bias)
    _check(_op(T, E, K), logits, K, GateConfig(score, True, 1.0),
           bias=torch.full((E,), 0.5, device=DEV))
    _check(_op(T, E, K), logits.bfloat16(), K, GateConfig(score, True, 1.0), bias=bias)


def test_far_scores_renormalize_without_underflow():
    """Chosen scores far below the smallest float still give their ratios."""
    op = _op(4, 16, 4)
    l = torch.full((4, 16), -200.0)
    l[:, 3], l[:, 7] = -199.0, -198.0
    w, idx = op.gate(l.to(DEV), GateConfig("sigmoid", True, 1.0))
    r = np.exp(np.array([0.0, -1.0, -2.0, -2.0]))
    assert idx[0].tolist() == [7, 3, 0, 1]
    np.testing.assert_allclose(w[0].cpu().numpy(), r / r.sum(), rtol=1e-4)  # 200 * 2^-23 and exp


# block counts around the last-block sum: 1, 2, the cap of 256 and several passes
@pytest.mark.parametrize("T", [32, 64, 8191, 8192, 8193, 20000])
def test_counts_and_losses_over_many_blocks(T):
    E, K = 96, 6
    rng = np.random.default_rng(T)
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
    op = _op(T, E, K)
    first = [t.clone() for t in op.gate(logits, balance=True)]
    l = logits.double()
    p = torch.softmax(l, 1)
    idx = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :K]
    assert torch.equal(first[1].long(), idx)
    c = torch.bincount(idx.reshape(-1), minlength=E)
    assert torch.equal(first[2][:E].long(), c) and int(first[2][E]) == T
    bal = E * (c.double() / (T * K) * p.mean(0)).sum()
    z = torch.logsumexp(l, 1).square().mean()
    # sums of T terms in fp32, at most T / 8192 + 40 additions deep
    tol = (8 * REL + (T / 8192 + 40) * 2.0 ** -24)
    assert abs(float(first[3][0]) - float(bal)) <= tol * float(bal)
    assert abs(float(first[3][1]) - float(z)) <= 2 * tol * float(z)
    for _ in range(3):   # the scratch is ready again, the result the same bits
        again = op.gate(logits, balance=True)
        for a, b in zip(first, again):
            assert torch.equal(a, b)


def test_no_tokens():
    op = _op(4, 8, 2)
    empty = torch.zeros(0, 8, device=DEV)
    w, i, c, l = op.gate(empty, balance=True)
    assert w.shape == (0, 2) and c.tolist() == [0] * 9 and l.tolist() == [0.0, 0.0]
    g = op.gate_backward(empty, i, grad_losses=torch.ones(2, device=DEV), counts=c)
    assert g.shape == (0, 8)


@pytest.mark.parametrize("cfg", CONFIGS, ids=lambda c: f"{c.score}-{c.renormalize}")
def test_gradient_against_differences(cfg):
    """The gradient predicts the change of the forward's own outputs in 64 bits."""
    rng = np.random.default_rng(11)
    T, E, K = 6, 20, 4
    l = rng.standard_normal((T, E))
    logits = torch.from_numpy(l.astype(np.float32)).to(DEV)
    l = logits.double().cpu().numpy()
    op = _op(T, E, K)
    _, idx, counts, _ = op.gate(logits, cfg, balance=True)
    gw = rng.standard_normal((T, K)).astype(np.float32)
    gl = np.array([0.7, 0.3], np.float32)
    grad = op.gate_backward(logits, idx, cfg, grad_weights=torch.from_numpy(gw).to(DEV),
                            counts=counts, grad_losses=torch.from_numpy(gl).to(DEV))
    got = grad.double().cpu().numpy()
    ids, cnt = idx.cpu().numpy(), counts.cpu().numpy()

    def total(v):   # with the choice and the counts held fixed
        x = np.exp(v - v.max(1, keepdims=True))
        soft = x / x.sum(1, keepdims=True)
        s = soft if cfg.score == "softmax" else 1 / (1 + np.exp(-v))
        r = np.take_along_axis(s, ids, 1)
        if cfg.renormalize:
            r = r / r.sum(1, keepdims=True)
        p = s / s.sum(1, keepdims=True)
        bal = E * (cnt[:E] / (T * K) * p.mean(0)).sum()
        z = ((v.max(1) + np.log(x.sum(1))) ** 2).mean()
        return (cfg.scale * r * gw).sum() + gl[0] * bal + gl[1] * z

    h = 1e-5
    for t in range(T):
        for e in range(E):
            d = np.zeros_like(l)
            d[t, e] = h
            num = (total(l + d) - total(l - d)) / (2 * h)
            # central difference: h^2 of the third derivative (below 100) and
            # 2^-52 * |total| / h; the kernel's fp32 terms are below 10
            assert abs(num - got[t, e]) <= 1e-8 + 1e-9 + 10 * 16 * REL


def test_gate_capture_replays_with_new_logits():
    """A captured forward and backward, replayed on changed inputs between eager
    calls of the same op (which share its scratch, in stream order)."""
    T, E, K = 500, 64, 4
    rng = np.random.default_rng(2)
    op = _op(T, E, K)
    cfg = GateConfig()
    logits = torch.zeros(T, E, device=DEV)
    gw = torch.ones(T, K, device=DEV)
    gl = torch.tensor([1.0, 0.1], device=DEV)

    def step(x):
        w, i, c, l = op.gate(x, cfg, balance=True)
        return w, i, c, l, op.gate_backward(x, i, cfg, grad_weights=gw, counts=c, grad_losses=gl)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(logits)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step(logits)
    for k in range(4):
        x = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
        want = [t.clone() for t in step(x)]
        torch.cuda.synchronize()
        logits.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), k
