"""The layer operators at sizes where a launch's own limits show."""
import pytest
import torch

from combine_routing_histogram_amd import layer as L
from layer_common import DEV

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
