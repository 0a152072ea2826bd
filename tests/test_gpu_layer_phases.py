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
