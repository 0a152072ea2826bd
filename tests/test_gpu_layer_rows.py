"""The norm before the gate, its gradient, and rows in 8 bits, against 64 bits.

Bounds.  A row's sum of squares is added in fp32, at most 32 terms in a lane and
22 steps across lanes and waves, all positive: off by 54 * 2^-24 at most, the
root's inverse by half of that; the sum s, the mean, the root, its inverse and the two
products add a rounding each: together below 2^-18 of y.  out is y rounded to
bf16, 2^-8.  A code is off by half a step: e4m3 2^-4 of the value or, among its
subnormals, 2^-10 scales; int8 half a scale.  The gradient's terms carry the
same errors, its sum over the row of products of either sign 2^-18 of their
absolute values: 2^-17 of q (|g| + |n| mean|g n|).  A weight's gradient adds its
rows in fp32, at most rows/512 in a team and 72 across: 2^-16 of the absolute
values' sum.
"""
import numpy as np
import pytest
import torch

from combine_routing_histogram_amd import layer as L
from combine_routing_histogram_amd.op import EpDispatchCombineConfig, EpDispatchCombineOp
from layer_common import DEV, draw_indices, layout, normal, routed_op
from oracle import oracle

pytestmark = pytest.mark.gpu
U, BF = 2.0 ** -8, torch.bfloat16
FORMATS = {"fp8_e4m3_b128": (128, 448.0), "int8_row": (0, 127.0)}


@pytest.fixture(scope="module")
def op():
    return EpDispatchCombineOp(EpDispatchCombineConfig(1, 8, 1, 1, 1), DEV)


def _wide(rng, shape):
    """Rows as a residual stream has them: a few columns far larger than the others."""
    x = rng.standard_normal(shape, dtype=np.float32)
    return torch.from_numpy(x * np.where(rng.random(shape[1]) < 0.02, 30, 1)).to(DEV).to(BF)


def _within(got, ref, tol, what):
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), \
        f"{what}: off by {float((err - tol).max())} beyond the bound, worst {float(err.max())}"


def _norm(x, r, w, eps):
    s = x.double() if r is None else x.double() + r.double()
    return s, s / (s.square().mean(1, keepdim=True) + eps).sqrt() * w.double()


def _check_codes(codes, scales, y, quant):
    block, limit = FORMATS[quant]
    rows, cols = y.shape
    b = y.reshape(rows, -1, block or cols)
    ref = b.abs().amax(-1) / limit
    assert scales.shape == ref.shape and scales.dtype == torch.float32
    _within(scales, ref, 2.0 ** -17 * ref + 2.0 ** -149, "scales")
    s = scales.double()[..., None]
    got = codes.double().reshape(b.shape) * s
    step = torch.maximum(2.0 ** -4 * b.abs(), 2.0 ** -10 * s) if block else 0.5 * s
    _within(got, b, step * (1 + 2.0 ** -15) + 2.0 ** -15 * b.abs(), "codes")


# one lane's vector to 16 waves of four; odd row counts; a row per team of one wave
SHAPES = [(1, 8), (1, 7168), (3, 512), (5, 520), (61, 2048), (7, 2056), (9, 4104), (130, 7168),
          (3, 8200), (4, 16384), (2, 16392), (2, 32768), (1500, 128)]


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm(op, T, H, residual):
    print(f"norm T={T} H={H} residual={residual}", flush=True)
    rng = np.random.default_rng(T + H)
    x, r = _wide(rng, (T, H)), _wide(rng, (T, H)) if residual else None
    for dtype in (BF, torch.float32):
        w = normal(rng, (H,), dtype=dtype)
        out, total, codes, scales = op.add_rms_norm(x, w, r, eps=1e-5)
        s, y = _norm(x, r, w, 1e-5)
        _within(out, y, (U + 2.0 ** -18) * y.abs(), "out")
        assert codes is None and scales is None
        if residual:
            assert torch.equal(total, (x.float() + r.float()).to(BF))
        else:
            assert total is None


@pytest.mark.parametrize("quant,T,H", [("fp8_e4m3_b128", 1, 128), ("fp8_e4m3_b128", 33, 640),
                                       ("fp8_e4m3_b128", 5, 2176), ("fp8_e4m3_b128", 200, 7168),
                                       ("fp8_e4m3_b128", 3, 16512), ("int8_row", 1, 16),
                                       ("int8_row", 33, 528), ("int8_row", 200, 7168),
                                       ("int8_row", 5, 2064), ("int8_row", 3, 32768)])
def test_norm_in_8_bits(op, quant, T, H):
    print(f"norm {quant} T={T} H={H}", flush=True)
    rng = np.random.default_rng(T + H)
    x, r, w = _wide(rng, (T, H)), _wide(rng, (T, H)), normal(rng, (H,))
    plain, total, _, _ = op.add_rms_norm(x, w, r)
    out, total2, codes, scales = op.add_rms_norm(x, w, r, quant=quant)
    assert torch.equal(plain, out) and torch.equal(total, total2)
    _check_codes(codes, scales, _norm(x, r, w, 1e-6)[1], quant)
    none, _, codes2, scales2 = op.add_rms_norm(x, w, r, quant=quant, output=False)
    assert none is None and torch.equal(codes.view(torch.uint8), codes2.view(torch.uint8))
    assert torch.equal(scales, scales2)


def test_norm_in_place_and_empty(op):
    rng = np.random.default_rng(0)
    x, r, w = normal(rng, (37, 4112)), normal(rng, (37, 4112)), normal(rng, (4112,))
    out, total, _, _ = op.add_rms_norm(x, w, r)
    keep = r.clone()
    out2, same, _, _ = op.add_rms_norm(x, w, keep, sum_out=keep)
    assert same is keep and torch.equal(keep, total) and torch.equal(out2, out)
    none = torch.empty(0, 4112, dtype=BF, device=DEV)
    for t in op.add_rms_norm(none, w, none, quant="int8_row")[:3]:
        assert t.shape == (0, 4112)
    gx, gw = op.add_rms_norm_backward(none, none, w)
    assert gx.shape == (0, 4112) and not gw.any()
    assert op.quantize_rows(none, "int8_row")[1].shape == (0, 1)


def test_in_place_of_what_flows_in(op):
    """The sum over its input, the gradient over grad_out or grad_sum, as the header allows."""
    rng = np.random.default_rng(3)
    T, H = 700, 1288
    x, r, dy, ds = (normal(rng, (T, H)) for _ in range(4))
    w = normal(rng, (H,))
    out, total, _, _ = op.add_rms_norm(x, w, r)
    keep = x.clone()
    out2, _, _, _ = op.add_rms_norm(keep, w, r, sum_out=keep)
    assert torch.equal(out2, out) and torch.equal(keep, total)
    want, dw = op.add_rms_norm_backward(dy, total, w, grad_sum=ds)
    args = L.make_norm_args(T, H, L.EPDC_DT_BF16, 1e-6, total.data_ptr(), 0, w.data_ptr())
    for over in (0, 1):
        g, s = dy.clone(), ds.clone()
        gw = torch.empty(H, device=DEV)
        scratch = torch.empty(L.epdc_rms_norm_scratch_bytes(H), dtype=torch.uint8, device=DEV)
        L.epdc_rms_norm_backward(args, torch.cuda.current_stream().cuda_stream, g.data_ptr(),
                                 s.data_ptr(), (s if over else g).data_ptr(), gw.data_ptr(),
                                 scratch.data_ptr())
        assert torch.equal(s if over else g, want) and torch.equal(gw, dw)


def test_rows_past_four_gigabytes(op):
    """Arrays whose last rows lie beyond 2^32 bytes."""
    T, H = 66000, 32768
    x = torch.zeros(T, H, dtype=BF, device=DEV)
    tail = normal(np.random.default_rng(5), (3, H))
    x[-3:] = tail
    w = normal(np.random.default_rng(6), (H,))
    small = op.add_rms_norm(tail, w, tail, quant="int8_row")
    big = op.add_rms_norm(x, w, x, quant="int8_row")
    for a, b in zip(small, big):
        assert torch.equal(a, b[-3:])
    assert not big[0][:-3].any() and not big[3][:-3].any()
    del big
    small, _ = op.add_rms_norm_backward(tail, tail, w)
    big, _ = op.add_rms_norm_backward(x, x, w)
    assert torch.equal(small, big[-3:])
    del big
    for quant in sorted(FORMATS):
        small, big = op.quantize_rows(tail, quant), op.quantize_rows(x, quant)
        for a, b in zip(small, big):
            assert torch.equal(a.view(torch.uint8), b[-3:].view(torch.uint8))


def test_norm_of_extreme_rows(op):
    """Zeros, the smallest and the largest numbers; a NaN or infinity stays in its row."""
    H = 1040
    x = normal(np.random.default_rng(1), (8, H))
    w = torch.ones(H, dtype=torch.float32, device=DEV)
    x[0] = 0
    x[1] *= 2.0 ** 100         # squares beyond fp32
    x[2] *= 2.0 ** -100        # squares below it: eps rules
    x[3, 5] = float("nan")
    x[4, 5] = float("inf")
    x[5] *= 2.0 ** 61          # the sum of squares just beyond fp32
    for quant in ("none", "int8_row"):
        out, _, codes, scales = op.add_rms_norm(x, w, eps=1e-6, quant=quant)
        y = _norm(x, None, w, 1e-6)[1]
        for i in (0, 1, 2, 5, 6, 7):
            _within(out[i], y[i], (U + 2.0 ** -18) * y[i].abs() + 2.0 ** -133, f"row {i}")
        assert bool(out[3].isnan().all()) and bool(out[4, 5].isnan())
        if quant != "none":
            assert float(scales[0]) == 0 and not codes[0].any()
            assert bool(scales[3].isnan()) and not bool(scales[4].isfinite())
            keep = [1, 5, 6, 7]
            _check_codes(codes[keep], scales[keep], y[keep], quant)
    q = op.add_rms_norm(x[:, :1024].contiguous(), w[:1024].contiguous(), quant="fp8_e4m3_b128")
    y = _norm(x[:, :1024], None, w[:1024], 1e-6)[1]
    keep = [1, 5, 6, 7]
    _check_codes(q[2][keep], q[3][keep], y[keep], "fp8_e4m3_b128")
    assert not q[3][0].any() and bool(q[3][3].isnan().all())
    dy = normal(np.random.default_rng(2), (8, H))
    gx, gw = op.add_rms_norm_backward(dy, x, w, eps=1e-6)
    s = x.double()
    q64 = 1 / (s.square().mean(1, keepdim=True) + 1e-6).sqrt()
    n, g = s * q64, dy.double()
    ref = q64 * (g - n * (g * n).mean(1, keepdim=True))
    tol = 2.0 ** -17 * q64 * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    for i in (0, 1, 2, 5, 6, 7):
        _within(gx[i], ref[i], tol[i] + U * (ref[i].abs() + tol[i]) + 2.0 ** -133, f"gradient {i}")
    assert bool(gx[3].isnan().all())


def _gradient(s, dy, w, eps, ds):
    """(dx, dw) of the formula in 64 bits, and their bounds."""
    s, dy, w = s.double(), dy.double(), w.double()
    q = 1 / (s.square().mean(1, keepdim=True) + eps).sqrt()
    n, g = s * q, dy * w
    dx = q * (g - n * (g * n).mean(1, keepdim=True))
    tol = 2.0 ** -17 * q * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if ds is not None:
        dx = dx + ds.double()
        tol = tol + 2.0 ** -23 * ds.double().abs()
    return dx, tol + U * (dx.abs() + tol), (dy * n).sum(0), 2.0 ** -16 * (dy * n).abs().sum(0)


@pytest.mark.parametrize("T,H", SHAPES + [(2100, 264), (5000, 136)])
def test_norm_backward(op, T, H):
    print(f"norm backward T={T} H={H}", flush=True)
    rng = np.random.default_rng(T * 3 + H)
    s, dy = _wide(rng, (T, H)), normal(rng, (T, H))
    for dtype, ds in ((BF, normal(rng, (T, H))), (torch.float32, None)):
        w = normal(rng, (H,), dtype=dtype)
        gx, gw = op.add_rms_norm_backward(dy, s, w, eps=1e-5, grad_sum=ds)
        dx, tol, dw, wtol = _gradient(s, dy, w, 1e-5, ds)
        _within(gx, dx, tol, "grad_input")
        _within(gw, dw, wtol, "grad_weight")
        again, none = op.add_rms_norm_backward(dy, s, w, eps=1e-5, grad_sum=ds, need_weight=False)
        assert none is None and torch.equal(again, gx)


def test_norm_backward_against_differences(op):
    """dx and dw against central differences of the norm in 64 bits.  The step's own error
    is below 1e-9 of the sums here; the result's bounds are the test's above."""
    rng = np.random.default_rng(4)
    T, H = 3, 24
    s, dy, w = normal(rng, (T, H)), normal(rng, (T, H)), normal(rng, (H,), dtype=torch.float32)
    gx, gw = op.add_rms_norm_backward(dy, s, w, eps=1e-3)
    _, tol, _, wtol = _gradient(s, dy, w, 1e-3, None)

    def value(s, w):
        return (s / (s.square().mean(1, keepdim=True) + 1e-3).sqrt() * w * dy.double()).sum()

    step = 2.0 ** -17
    for i in range(T):
        for j in range(H):
            d = torch.zeros(T, H, dtype=torch.float64, device=DEV)
            d[i, j] = step
            ref = (value(s.double() + d, w.double()) - value(s.double() - d, w.double())) / 2 / step
            assert abs(float(gx[i, j]) - float(ref)) <= float(tol[i, j]) + 1e-8
    for j in range(H):
        d = torch.zeros(H, dtype=torch.float64, device=DEV)
        d[j] = step
        ref = (value(s.double(), w.double() + d) - value(s.double(), w.double() - d)) / 2 / step
        assert abs(float(gw[j]) - float(ref)) <= float(wtol[j]) + 1e-8


def _int8(x):
    """Codes and scales of float32 rows by whole fp32 divisions (numpy)."""
    scale = np.abs(x).max(1, keepdims=True) / np.float32(127)
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.rint(x / scale)
    return np.where(scale > 0, q, 0).astype(np.int8), scale


@pytest.mark.parametrize("T,I", [(1, 16), (1, 1024), (77, 1040), (6, 4096), (5, 4112), (3, 8208),
                                 (2, 32784), (2, 131072), (900, 48)])
def test_quantize_int8_bits(op, T, I):
    print(f"int8 rows T={T} I={I}", flush=True)
    rng = np.random.default_rng(T + I)
    x = rng.standard_normal((T, I), dtype=np.float32) * np.exp(rng.normal(0, 3, (T, 1)))
    x = torch.from_numpy(x.astype(np.float32)).to(BF)
    x[0] = 0 if T > 1 else x[0]
    codes, scales = op.quantize_rows(x.to(DEV), "int8_row")
    want, scale = _int8(x.float().numpy())
    assert np.array_equal(scales.cpu().numpy(), scale)
    assert np.array_equal(codes.cpu().numpy(), want)


def test_quantize_int8_every_quotient(op):
    """Rows whose largest element takes every significand of bf16 beside elements of every
    significand: the quotients nearest to a border between two codes are among them,
    and scales far from 1 with them."""
    m = np.arange(128, 256, dtype=np.float32)
    for power in (0, -100, 60, -126):
        top = m * np.float32(2.0) ** np.float32(power)
        x = np.concatenate([np.broadcast_to(top * np.float32(2.0) ** -k, (128, 128))
                            for k in range(1, 9)], axis=1)
        x = np.concatenate([top[:, None], x[:, :-1]], axis=1).astype(np.float32)
        x[:, 1::2] *= -1
        t = torch.from_numpy(np.ascontiguousarray(x)).to(BF)
        codes, scales = op.quantize_rows(t.to(DEV), "int8_row")
        want, scale = _int8(t.float().numpy())
        assert np.array_equal(scales.cpu().numpy(), scale), power
        assert np.array_equal(codes.cpu().numpy(), want), power


@pytest.mark.parametrize("T,I,spread", [(1, 128, 0), (77, 1152, 3), (3, 131072, 0), (400, 384, 40)])
def test_quantize_e4m3_bits(op, T, I, spread):
    """Codes and scales of the quantizing dispatch, as the oracle has them."""
    print(f"e4m3 rows T={T} I={I}", flush=True)
    rng = np.random.default_rng(T + I)
    size = np.clip(rng.normal(0, spread, (T, I // 128, 1)), -85, 85)   # finite: the oracle's domain
    x = rng.standard_normal((T, I // 128, 128)) * np.exp(size)
    t = torch.from_numpy(x.reshape(T, I).astype(np.float32)).to(BF)
    t[-1, :128] = 0
    codes, scales = op.quantize_rows(t.to(DEV), "fp8_e4m3_b128")
    want, scale = oracle.quant_fp8(t.view(torch.int16).numpy().view(np.uint16))
    assert np.array_equal(scales.cpu().numpy(), np.asarray(scale).reshape(T, -1))
    assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), np.asarray(want).reshape(T, -1))


@pytest.mark.parametrize("quant", sorted(FORMATS))
def test_quantize_received_rows(quant):
    """Only rows that hold a pair are read and written."""
    rng = np.random.default_rng(3)
    idx = draw_indices(rng, 60, 4, 8)
    idx[::2, 1] = -1
    _, off = layout(idx, 8)
    op = routed_op(idx, 8)
    x = normal(rng, (245, 256))
    x[off[-1]:] = float("nan")
    codes, scales = op.quantize_rows(x, quant, routed=True)
    want, wscales = op.quantize_rows(x[:off[-1]].contiguous(), quant)
    assert codes.shape == (240, 256)
    assert torch.equal(codes[:off[-1]].view(torch.uint8), want.view(torch.uint8))
    assert torch.equal(scales[:off[-1]], wscales)
    # through the library, into buffers of the test's own: the rows behind stay
    codes = torch.full((240, 256), 9, dtype=torch.uint8, device=DEV)
    scales = torch.full((240, 256 // (FORMATS[quant][0] or 256)), 5.0, device=DEV)
    expert_off, _ = op.get_offsets()
    L.epdc_quantize_rows(torch.cuda.current_stream().cuda_stream, 240, 256,
                         L.EPDC_DT_INT8 if quant == "int8_row" else L.EPDC_DT_E4M3,
                         x.data_ptr(), expert_off.data_ptr(), 8, codes.data_ptr(),
                         scales.data_ptr())
    assert torch.equal(codes[:off[-1]], want.view(torch.uint8))
    assert bool((codes[off[-1]:] == 9).all()) and bool((scales[off[-1]:] == 5).all())


def test_rows_captured_and_on_another_stream(op):
    """Forward, gradient and both formats in a graph, replayed on new inputs."""
    rng = np.random.default_rng(6)
    T, H = 100, 1280
    x, r, dy, w = (normal(rng, (T, H)) for _ in range(4))
    w = w[0].contiguous()

    def step():
        out, total, codes, scales = op.add_rms_norm(x, w, r, quant="fp8_e4m3_b128")
        gx, gw = op.add_rms_norm_backward(dy, total, w, grad_sum=out)
        q, s = op.quantize_rows(gx, "int8_row")
        return [out, total, codes.view(torch.uint8), scales, gx, gw, q, s]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, step()):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for k in range(3):
        for t in (x, r, dy):
            t.copy_(normal(rng, (T, H)))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), (k, i)
