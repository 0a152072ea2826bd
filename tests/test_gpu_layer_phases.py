"""The layer operators with the split phases, the routing replay and the
rank-deduplicated dispatch."""
import numpy as np
import pytest
import torch

from combine_routing_histogram_amd.op import EpDispatchCombineConfig, EpDispatchCombineOp
from layer_common import DEV, layout, normal

pytestmark = pytest.mark.gpu


def test_gate_between_send_and_recv():
    """gate, dispatch_send, gate of other logits, dispatch_recv: the dispatch has
    the first gate's routing and weights, the views hold the second's."""
    rng = np.random.default_rng(0)
    T, H, E, K = 4096, 2048, 64, 8
    op = EpDispatchCombineOp(EpDispatchCombineConfig(T, H, K, E, 2), DEV)
    x = normal(rng, (T, H))
    first, second = (normal(rng, (T, E), dtype=torch.float32) for _ in range(2))
    want = [t.clone() for t in op.gate(second)]
    keep = [t.clone() for t in op.gate(first)]
    pair, off = layout(keep[1].cpu().numpy(), E)
    w, idx = op.gate(first)
    op.dispatch_send(x, w, None, idx)
    got = op.gate(second)
    rows, row_w, _, _, _ = op.dispatch_recv()
    tok = torch.from_numpy(pair // K).to(DEV)
    assert torch.equal(rows, x[tok]) and torch.equal(row_w, keep[0][tok])
    assert op.get_offsets()[0].tolist() == off.tolist()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_gate_between_send_and_recv_captured():
    """The same inside one graph, replayed on new logits."""
    rng = np.random.default_rng(1)
    T, H, E, K = 256, 256, 16, 2
    op = EpDispatchCombineOp(EpDispatchCombineConfig(T, H, K, E, 2), DEV)
    x = normal(rng, (T, H))
    a, b = (normal(rng, (T, E), dtype=torch.float32) for _ in range(2))

    def step():
        w, idx = op.gate(a)
        op.dispatch_send(x, w, None, idx)
        w2, i2 = op.gate(b)
        rows, row_w, _, _, _ = op.dispatch_recv()
        return rows.clone(), row_w.clone(), w2.clone(), i2.clone()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for _ in range(3):
        a.copy_(normal(rng, (T, E), dtype=torch.float32))
        b.copy_(normal(rng, (T, E), dtype=torch.float32))
        want = step()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for p, q in zip(outs, want):
            assert torch.equal(p, q)


def _case(seed, T=300, H=256, E=16, K=4, R=4):
    rng = np.random.default_rng(seed)
    op = EpDispatchCombineOp(EpDispatchCombineConfig(T, H, K, E, R), DEV)
    logits = normal(rng, (T, E), dtype=torch.float32)
    w, idx = [t.clone() for t in op.gate(logits)]
    return rng, op, w, idx, normal(rng, (T, H)), normal(rng, (E, 64, H), H ** -0.5)


def _layer(op, rows, row_w, w1, dy):
    """A product, its gradients and combine's and dispatch's, over given rows."""
    z = torch.empty(rows.shape[0], w1.shape[1], dtype=torch.bfloat16, device=DEV)
    h = op.expert_product(rows, w1, activation="silu", preact=z)
    gx, gw, gb = op.expert_product_backward(h, rows, w1, activation="silu", preact=z, bias=True)
    do, dw = op.combine_backward(dy, rows, row_w)
    n = op.n_cap
    return [t[:n].clone() for t in (h, gx, gw, gb, do, dw, op.dispatch_backward(gx))]


@pytest.mark.parametrize("how", ["split", "replay", "dedup"])
def test_products_behind_every_kind_of_dispatch(how):
    """Split phases, a replay of the routing and the expanded unit rows leave the
    rows and the routing of a plain dispatch, so everything behind is equal."""
    rng, op, w, idx, x, w1 = _case(5)
    dy = normal(rng, tuple(x.shape))
    rows, row_w, _, _, _ = op.dispatch(x, w, None, idx)
    want = _layer(op, rows, row_w, w1, dy)
    if how == "split":
        op.dispatch(torch.zeros_like(x), w, None, torch.zeros_like(idx))
        op.dispatch_send(x, w, None, idx)
        got = op.dispatch_recv()
    elif how == "replay":
        op.dispatch(torch.zeros_like(x), w, None, idx)
        got = op.dispatch_replay(x, w)
    else:
        op.dispatch_dedup(x, w, None, idx)
        got = op.units_to_experts()
    for a, b in zip(_layer(op, got[0], got[1], w1, dy), want):
        assert torch.equal(a, b)
