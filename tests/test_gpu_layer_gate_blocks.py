"""A balance over every number of blocks, on one op: the wave-per-token form up to
its 256 blocks and in several passes, the change to four tokens a wave, and
calls of fewer tokens than the op's scratch was sized for.

Bounds as in test_gpu_layer_gate.py: sums of T terms in fp32, at most
T / 2048 + 60 additions deep here.
"""
import numpy as np
import pytest
import torch

from combine_routing_histogram_amd.op import GateConfig
from layer_common import DEV
from test_gpu_layer_gate import REL, _op

pytestmark = pytest.mark.gpu
E, K, MOST = 256, 8, 9000


def _expected(logits, cfg, bias):
    l = logits.double()
    T = l.shape[0]
    s = torch.softmax(l, 1) if cfg.score == "softmax" else torch.sigmoid(l)
    key = l if bias is None else s + bias.double()
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :K]
    counts = torch.bincount(idx.reshape(-1), minlength=E)
    p = s / s.sum(1, keepdim=True)
    bal = E * (counts.double() / (T * K) * p.mean(0)).sum()
    return idx, counts, float(bal), float(torch.logsumexp(l, 1).square().mean())


@pytest.mark.parametrize("cfg", [GateConfig(), GateConfig("sigmoid", True, 2.5)],
                         ids=lambda c: c.score)
@pytest.mark.parametrize("order", ["up", "down"])
def test_one_op_over_all_token_counts(order, cfg):
    sizes = [1, 9, 2047, 2048, 2049, 3000, 4096, 4097, 8192, MOST]
    g = torch.Generator(device=DEV).manual_seed(7)
    op = _op(MOST, E, K)
    all_logits = torch.randn(MOST, E, generator=g, device=DEV)
    bias = 0.1 * torch.randn(E, generator=g, device=DEV)
    first = {}
    for T in sizes if order == "up" else sizes[::-1]:
        print(f"gate T={T} {cfg.score} {order}", flush=True)
        logits = all_logits[:T]
        got = [t.clone() for t in op.gate(logits, cfg, bias=bias, balance=True)]
        idx, counts, bal, z = _expected(logits, cfg, bias)
        assert torch.equal(got[1].long(), idx)
        assert torch.equal(got[2][:E].long(), counts) and int(got[2][E]) == T
        tol = 8 * REL + (T / 2048 + 60) * 2.0 ** -24
        assert abs(float(got[3][0]) - bal) <= tol * bal
        assert abs(float(got[3][1]) - z) <= 2 * tol * z
        first[T] = got
    for T in sizes:   # the same bits whatever ran before
        for a, b in zip(op.gate(all_logits[:T], cfg, bias=bias, balance=True), first[T]):
            assert torch.equal(a, b)
