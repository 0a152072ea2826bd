"""The layer operators at sizes where their own or a launch's limits show."""
import numpy as np
import pytest
import torch

from combine_routing_histogram_amd import layer as L
from combine_routing_histogram_amd.op import GateConfig
from layer_common import DEV, ints, layout, routed_op
from test_gpu_layer_gate import _check, _op

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("topk", [1, 3])
def test_combine_backward_of_more_tokens_than_blocks(topk):
    """A launch holds fewer than 2^32 threads, 2^23 blocks of 512; small integers,
    so every product and sum is exact."""
    T, H = (1 << 23) + 5, 8
    g = torch.Generator(device=DEV).manual_seed(topk)
    n = T * topk
    slot = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    slot[::1001] = -1
    dy = torch.randint(-4, 5, (T, H), generator=g, device=DEV).to(torch.bfloat16)
    x = torch.randint(-4, 5, (n, H), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randint(-4, 5, (n, topk), generator=g, device=DEV).float()
    dx = torch.full((n, H), 9.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.full((T, topk), 9.0, device=DEV)
    L.epdc_combine_backward(torch.cuda.current_stream().cuda_stream, T, topk, H, slot.data_ptr(),
                            dy.data_ptr(), x.data_ptr(), w.data_ptr(), dx.data_ptr(),
                            dw.data_ptr())
    have = slot >= 0
    s, pair = slot[have].long(), torch.arange(n, device=DEV)[have]
    ref_dx = torch.full_like(dx, 9.0)
    ref_dx[s] = (w[s, pair % topk, None] * dy[pair // topk].float()).to(torch.bfloat16)
    ref_dw = torch.zeros(n, device=DEV)
    ref_dw[pair] = (dy[pair // topk].float() * x[s].float()).sum(1)
    assert torch.equal(dx, ref_dx) and torch.equal(dw.reshape(-1), ref_dw)


# every form at the most experts and at a number that leaves a thread's last ones
# out; experts without rows among them
@pytest.mark.parametrize("E", [300, 512])
@pytest.mark.parametrize("rows_each", [1, 20, 40, 80])
def test_products_of_many_experts(E, rows_each):
    """Small integers: bit for bit, forward and gradients."""
    rng = np.random.default_rng(E + rows_each)
    T, fin, fout = E * rows_each, 72, 40
    idx = rng.integers(0, E - 3, (T, 1)).astype(np.int32)
    idx[idx == 7] = 8
    _, off = layout(idx, E)
    print(f"experts {E}, {T} rows", flush=True)
    op = routed_op(idx, E)
    x, w, dy = ints(rng, (T, fin)), ints(rng, (E, fout, fin)), ints(rng, (T, fout))
    got = op.expert_product(x, w)
    gx, gw, gb = op.expert_product_backward(dy, x, w, bias=True, weight_dtype=torch.float32)
    e = torch.repeat_interleave(torch.arange(E, device=DEV),
                                torch.from_numpy(np.diff(off)).to(DEV))
    step = 4096
    for a in range(0, T, step):
        s = slice(a, min(a + step, T))
        we = w[e[s]].float()
        assert torch.equal(got[s].float(), (we * x[s, None].float()).sum(2))
        assert torch.equal(gx[s].float(), (we * dy[s, :, None].float()).sum(1))
    for i in range(E):
        s = slice(off[i], off[i + 1])
        d = dy[s].float()
        assert torch.equal(gw[i], torch.mm(d.t().contiguous(), x[s].float()))
        assert torch.equal(gb[i], d.sum(0))


@pytest.mark.parametrize("T", [60, 8300])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_of_the_most_experts(T, score):
    """512 experts, top-16, both forms, with bias and mask, against 64 bits."""
    rng = np.random.default_rng(T)
    E, K = 512, 16
    logits = torch.from_numpy(2 * rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
    bias = torch.from_numpy(0.2 * rng.standard_normal(E).astype(np.float32)).to(DEV)
    mask = torch.from_numpy((rng.random(T) < 0.8).astype(np.uint8)).to(DEV)
    _check(_op(T, E, K), logits, K, GateConfig(score, True, 2.5), bias=bias, mask=mask)
