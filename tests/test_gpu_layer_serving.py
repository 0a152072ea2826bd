"""The operators of a layer in 8 bits together, as a server runs them: the norm with the
residual's addition into bf16 (for the router) and 8-bit rows, the gate, dispatch of
those rows with their scales, both products in 8 bits with the rows between them
quantized, combine, the next layer's norm; the same tokens through the layer for
few tokens; and, in training, the norm's gradient behind the layer's.

Bounds, in the norm of the result.  Each 8-bit rounding is off by at most half a step: of
an element for e4m3, 2^-4, of the row's largest for int8, 2^-8 of it, and rows here
hold elements down to a fifth of that in the root of the mean square: 5 * 2^-8.  A
product's result carries its operand's relative error in the norm, as rounding
errors are independent of the weights they meet (and at most twice it through the
product of two activations, gate and up).  So with d the 8-bit step (2^-4 or 5 * 2^-8):
first operand 2 d, second d, and six bf16 roundings of 2^-8 each.
"""
import numpy as np
import pytest
import torch

from combine_routing_histogram_amd.op import (EpDispatchCombineConfig, EpDispatchCombineOp,
                                              GateConfig)
from layer_common import DEV, normal

pytestmark = pytest.mark.gpu
CFG = GateConfig("softmax", True, 1.0)
EPS, BF = 1e-6, torch.bfloat16
STEP = {"int8_row": 5 * 2.0 ** -8, "fp8_e4m3_b128": 2.0 ** -4}


def _weight(rng, shape, quant):
    """An expert weight in 8 bits, its scales, its values in 64 bits."""
    n, o, i = shape
    w = normal(rng, shape, i ** -0.5, torch.float32)
    if quant == "int8_row":
        s = w.abs().amax(2) / 127
        q = (w / s[..., None]).round().to(torch.int8)
        return q, s, q.double() * s.double()[..., None]
    b = w.reshape(n, o // 128, 128, i // 128, 128)
    s = b.abs().amax((2, 4)) / 448
    q = (b / s[:, :, None, :, None]).to(torch.float8_e4m3fn)
    full = (q.double() * s.double()[:, :, None, :, None]).reshape(shape)
    return q.reshape(shape), s, full


class Server:
    def __init__(self, T, H, I, E, K, quant, seed=0):
        rng = np.random.default_rng(seed)
        self.quant, self.shape = quant, (T, H, I, E, K)
        scale_bytes = 4 if quant == "int8_row" else H // 128 * 4
        self.op = EpDispatchCombineOp(EpDispatchCombineConfig(
            T, H, K, E, 2, raw_row_bytes=H, scale_row_bytes=scale_bytes), DEV)
        self.x, self.r = normal(rng, (T, H)), normal(rng, (T, H))
        self.norm = (1 + normal(rng, (H,), 0.2, torch.float32)).to(BF)
        self.router = normal(rng, (E, H), 2 * H ** -0.5)
        self.w1, self.s1, self.d1 = _weight(rng, (E, 2 * I, H), quant)
        self.w2, self.s2, self.d2 = _weight(rng, (E, H, I), quant)

    def route(self):
        out, total, codes, scales = self.op.add_rms_norm(self.x, self.norm, self.r, eps=EPS,
                                                         quant=self.quant)
        logits = (out.float() @ self.router.float().t()).contiguous()
        return out, total, codes, scales, self.op.gate(logits, CFG)

    def step(self):
        op = self.op
        out, total, codes, scales, (weights, indices) = self.route()
        rows, row_w, row_s, _, _ = op.dispatch(codes.view(torch.uint8), weights, scales, indices)
        h = op.expert_product(rows.view(codes.dtype), self.w1, scales=row_s,
                              weight_scales=self.s1, activation="swiglu")
        hq, hs = op.quantize_rows(h, self.quant, routed=True)
        o = op.expert_product(hq, self.w2, scales=hs, weight_scales=self.s2)
        y, _ = op.combine(o, row_w)
        last, total2, _, _ = op.add_rms_norm(y, self.norm, total, eps=EPS)
        return last, total2, y.clone(), indices.clone()

    def few(self):
        out, total, _, _, (weights, indices) = self.route()
        return self.op.few_token_layer(out, weights, indices, self.w1, self.w2,
                                       w1_scales=self.s1, w2_scales=self.s2, activation="swiglu")

    def exact(self, indices):
        """y in 64 bits over the routing that the program chose."""
        s = self.x.double() + self.r.double()
        n = s / (s.square().mean(1, keepdim=True) + EPS).sqrt() * self.norm.double()
        l = n @ self.router.double().t().contiguous()
        w = torch.softmax(l, 1).gather(1, indices.long())
        w = w / w.sum(1, keepdim=True)
        y = torch.zeros_like(s)
        for e in range(self.shape[3]):
            t, k = torch.nonzero(indices == e, as_tuple=True)
            g, u = (n[t] @ self.d1[e].t().contiguous()).chunk(2, dim=1)
            h = torch.nn.functional.silu(g) * u
            y.index_add_(0, t, w[t, k][:, None] * (h @ self.d2[e].t().contiguous()))
        return y


def _near(got, ref, rel, what):
    d = float((got.double() - ref).norm() / ref.norm())
    assert d <= rel, f"{what}: {d}"


@pytest.mark.parametrize("quant", sorted(STEP))
@pytest.mark.parametrize("T,H,I,E,K", [(3, 256, 128, 8, 2), (48, 512, 256, 16, 4),
                                       (640, 640, 384, 8, 2)])
def test_layer_in_8_bits(T, H, I, E, K, quant):
    m = Server(T, H, I, E, K, quant)
    last, total, y, indices = m.step()
    ref = m.exact(indices)
    bound = 3 * STEP[quant] + 6 * 2.0 ** -8
    _near(y, ref, bound, "layer")
    s = m.x.double() + m.r.double() + ref
    _near(total, s, bound, "stream")
    _near(last, s / (s.square().mean(1, keepdim=True) + EPS).sqrt() * m.norm.double(), 2 * bound,
          "next norm")
    if T <= 64:     # weights in 8 bits, rows in bf16
        _near(m.few(), ref, 6 * 2.0 ** -8, "few")
    assert m.op.device_error() == 0


@pytest.mark.parametrize("quant", sorted(STEP))
def test_layer_in_8_bits_captured(quant):
    """The whole step in a graph, and the layer for few tokens in another of the same op,
    replayed in turn on new inputs with eager steps between."""
    m = Server(40, 256, 128, 16, 4, quant, seed=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.step()
        m.few()
    torch.cuda.current_stream().wait_stream(side)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        whole = m.step()
    with torch.cuda.graph(g2):
        few = m.few()
    for k in range(3):
        rng = np.random.default_rng(k + 5)
        m.x.copy_(normal(rng, tuple(m.x.shape)))
        m.r.copy_(normal(rng, tuple(m.x.shape)))
        want, want_few = [t.clone() for t in m.step()], m.few().clone()
        torch.cuda.synchronize()
        for g, outs, refs in ((g1, whole, want), (g2, [few], [want_few]), (g1, whole, want)):
            g.replay()
            torch.cuda.synchronize()
            for i, (a, b) in enumerate(zip(outs, refs)):
                assert torch.equal(a, b), (k, i)


def test_norm_in_training():
    """Norm, router, gate, experts and combine forward and backward to the residual stream:
    the stream's gradient through the norm and beside it, against autograd in 64 bits.
    Eleven bf16 roundings lie on the way, 2^-8 each."""
    rng = np.random.default_rng(2)
    T, H, I, E, K = 48, 256, 136, 8, 2
    op = EpDispatchCombineOp(EpDispatchCombineConfig(T, H, K, E, 1), DEV)
    x, r, dy, dsum = (normal(rng, (T, H)) for _ in range(4))
    norm = 1 + normal(rng, (H,), 0.2, torch.float32)
    w1, w2 = normal(rng, (E, 2 * I, H), H ** -0.5), normal(rng, (E, H, I), I ** -0.5)
    logits = normal(rng, (T, E), 1.5, torch.float32)
    n, s, _, _ = op.add_rms_norm(x, norm, r, eps=EPS)
    weights, indices = op.gate(logits, CFG)
    rows, row_w, _, _, _ = op.dispatch(n, weights, None, indices)
    z = torch.empty(T * K, 2 * I, dtype=BF, device=DEV)
    h = op.expert_product(rows, w1, activation="swiglu", preact=z)
    o = op.expert_product(h, w2)
    y, _ = op.combine(o, row_w)
    do, _ = op.combine_backward(dy, o, row_w)
    dh, _, _ = op.expert_product_backward(do, h, w2)
    drows, _, _ = op.expert_product_backward(dh, rows, w1, activation="swiglu", preact=z)
    dx, dnorm = op.add_rms_norm_backward(op.dispatch_backward(drows), s, norm, eps=EPS,
                                         grad_sum=dsum)

    xd, wd = (x.double() + r.double()).requires_grad_(True), norm.double().requires_grad_(True)
    nd = xd / (xd.square().mean(1, keepdim=True) + EPS).sqrt() * wd
    p = torch.softmax(logits.double(), 1).gather(1, indices.long())
    p = p / p.sum(1, keepdim=True)
    yd = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for e in range(E):
        t, k = torch.nonzero(indices == e, as_tuple=True)
        g, u = (nd[t] @ w1[e].double().t().contiguous()).chunk(2, dim=1)
        yd = yd.index_add(0, t, p[t, k][:, None] * ((torch.nn.functional.silu(g) * u)
                                                    @ w2[e].double().t().contiguous()))
    gx, gw = torch.autograd.grad((yd * dy.double()).sum() + (xd * dsum.double()).sum(), (xd, wd))
    _near(y, yd.detach(), 11 * 2.0 ** -8, "output")
    _near(dx, gx, 11 * 2.0 ** -8, "stream")
    _near(dnorm, gw, 11 * 2.0 ** -8, "norm weight")
