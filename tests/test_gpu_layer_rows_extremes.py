"""The norm, its gradient and rows in 8 bits where a number on the way leaves fp32's range or
loses its sign, against 64 bits; the bounds are those of test_gpu_layer_rows.py."""
import numpy as np
import pytest
import torch

from layer_common import DEV, normal
from oracle import oracle
from test_gpu_layer_rows import (BF, FORMATS, U, _check_codes, _gradient, _int8,  # noqa: F401
                                 _norm, _within, op)

pytestmark = pytest.mark.gpu


def test_negative_zeros_in_e4m3_rows(op):  # noqa: F811
    """-0.0 beside other numbers keeps its sign in e4m3, as the quantizing dispatch has it, at
    scales of every size; a block of zeros has codes 0."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((9, 512)).astype(np.float32)
    x *= np.float32(2) ** np.array([0, -30, 30, -58, 68, -70, -110, 100, 0], np.float32)[:, None]
    x[:, ::3] = -0.0
    x[:, 1::7] = 0.0
    x[-1, :256] = -0.0
    t = torch.from_numpy(x).to(BF)
    codes, scales = op.quantize_rows(t.to(DEV), "fp8_e4m3_b128")
    want, scale = oracle.quant_fp8(t.view(torch.int16).numpy().view(np.uint16))
    assert np.array_equal(scales.cpu().numpy(), np.asarray(scale).reshape(9, -1))
    got = codes.view(torch.uint8).cpu().numpy()
    assert np.array_equal(got, np.asarray(want).reshape(9, -1))
    zero = np.signbit(x) & (x == 0)
    assert (got[:-1][zero[:-1]] == 0x80).all() and not got[-1, :256].any()
    # the norm's: the sign of s * w
    w = torch.where(torch.arange(512) % 2 == 0, 1.0, -1.0).to(DEV)
    codes = op.add_rms_norm(t[:3].to(DEV), w, quant="fp8_e4m3_b128", eps=1e-20)[2]
    got = codes.view(torch.uint8).cpu().numpy()
    assert (got[:, ::2][zero[:3, ::2]] == 0x80).all() and not got[:, 1::2][zero[:3, 1::2]].any()


def _steady(rng, shape):
    """Numbers of either sign between 0.5 and 1.5."""
    v = rng.uniform(0.5, 1.5, shape) * rng.choice([-1.0, 1.0], shape)
    return torch.from_numpy(v.astype(np.float32)).to(DEV)


# (power of two of the rows, eps): sums of squares beyond fp32 beside an eps of their size, a
# mean that fp32 holds and the eps with it does not, squares at and below the smallest numbers
# beside no eps or one of their size
RANGES = [(61, 3e38), (61, 3.4e38), (62, 0.0), (0, 3.4e38), (120, 3e38), (126, 1e-6), (-50, 0.0),
          (-60, 0.0), (-66, 1e-40), (-72, 0.0), (-75, 0.0), (-75, 1e-45), (-100, 0.0),
          (-124, 0.0), (-20, 1e-30)]


@pytest.mark.parametrize("H", [16, 1040, 4104])
def test_means_outside_fp32(op, H):  # noqa: F811
    """Every row by the whole of mean(s^2) + eps, with its gradient."""
    rng = np.random.default_rng(H)
    base, dy = _steady(rng, (3, H)), normal(rng, (3, H))
    for power, eps in RANGES:
        print(f"H={H} rows of 2^{power} eps={eps}", flush=True)
        x = (base * 2.0 ** power).to(BF)
        w = _steady(rng, (H,))
        eps = float(np.float32(eps))
        y = _norm(x, None, w, eps)[1]
        for quant in ["none"] + sorted(FORMATS):
            if quant == "none" or H % (FORMATS[quant][0] or 16) == 0:
                out, _, codes, scales = op.add_rms_norm(x, w, eps=eps, quant=quant)
                _within(out, y, (U + 2.0 ** -18) * y.abs() + 2.0 ** -133, "out")
                if quant != "none":
                    _check_codes(codes, scales, y, quant)
        gx, gw = op.add_rms_norm_backward(dy, x, w, eps=eps)
        dx, tol, dw, wtol = _gradient(x, dy, w, eps, None)
        held = dx.abs() < 2.0 ** 127          # bf16 has no larger numbers
        tol = torch.where(held, tol, torch.inf)
        _within(torch.where(held, gx.double(), 0), torch.where(held, dx, 0), tol + 2.0 ** -133,
                "grad_input")
        _within(gw, dw, wtol + 2.0 ** -149, "grad_weight")


@pytest.mark.parametrize("H", [16, 520, 2056, 7168, 16392])
def test_gradient_of_large_rows(op, H):  # noqa: F811
    """Rows and gradients whose products are beyond fp32: sum(dy w s), and its terms."""
    rng = np.random.default_rng(H)
    x = _steady(rng, (5, H)) * 2.0 ** torch.tensor([60.0, 100, 120, 126, 0], device=DEV)[:, None]
    dy = _steady(rng, (5, H)) * 2.0 ** torch.tensor([70.0, 40, 20, 0, 0], device=DEV)[:, None]
    x, dy = x.to(BF), dy.to(BF)
    x[3] = 3.38e38 * x[3].sign()
    for w in (_steady(rng, (H,)), _steady(rng, (H,)).to(BF)):
        gx, gw = op.add_rms_norm_backward(dy, x, w)
        dx, tol, dw, wtol = _gradient(x, dy, w, 1e-6, None)
        _within(gx, dx, tol + 2.0 ** -133, "grad_input")
        _within(gw, dw, wtol, "grad_weight")


@pytest.mark.parametrize("H", [16, 1152, 2176, 4224, 8320, 32768])
def test_products_outside_fp32(op, H):  # noqa: F811
    """s * w beyond fp32, or too small for it, where y = s * w / rms(s) is neither; also where
    that is so of some columns or rows alone."""
    rng = np.random.default_rng(H)
    base = _steady(rng, (4, H))
    mixed = torch.where(torch.arange(H, device=DEV) % 3 == 0, 2.0 ** 60, 1.0)
    for power, wide, eps in ((80, 2.0 ** 60, 1e-6), (120, 2.0 ** 30, 1e-6), (-40, 2.0 ** -95, 1e-20),
                             (-50, 2.0 ** -90, 1e-24), (-100, 2.0 ** -40, 0.0), (80, mixed, 1e-6),
                             (-100, 1 / mixed, 0.0)):
        x = (base * 2.0 ** power).to(BF)
        x[1] = base[1].to(BF)
        x[2] = 0
        x[2, 0] = 2.0 ** power
        w = _steady(rng, (H,)) * wide
        y = _norm(x, None, w, eps)[1]
        for quant in ["none"] + sorted(FORMATS):
            if quant != "none" and H % (FORMATS[quant][0] or 16):
                continue
            print(f"H={H} rows of 2^{power} {quant}", flush=True)
            out, _, codes, scales = op.add_rms_norm(x, w, eps=eps, quant=quant)
            _within(out, y, (U + 2.0 ** -18) * y.abs() + 2.0 ** -133, "out")
            if quant != "none":
                _check_codes(codes, scales, y, quant)


def test_gradient_whose_mean_alone_is_in_range(op):  # noqa: F811
    """sum(dy w s) within fp32, that times 1 / rms(s) beyond it, its mean within it again."""
    rng = np.random.default_rng(7)
    H = 16392
    x, w = (_steady(rng, (2, H)) * 2.0 ** -8).to(BF), _steady(rng, (H,))
    dy = (_steady(rng, (2, H)).abs() * 2.0 ** 115 * (x.float() * w).sign()).to(BF)
    gx, gw = op.add_rms_norm_backward(dy, x, w)
    dx, tol, dw, wtol = _gradient(x, dy, w, 1e-6, None)
    _within(gx, dx, tol, "grad_input")
    _within(gw, dw, wtol, "grad_weight")


def test_codes_of_subnormal_rows(op):  # noqa: F811
    """Blocks and rows of bf16's subnormal numbers, whose scales fp32 holds to a few bits: codes
    and scales of whole fp32 divisions, e4m3 as the oracle has them."""
    rng = np.random.default_rng(9)
    bits = rng.integers(0, 1 << np.arange(1, 8).repeat(3)[:, None], (21, 256)).astype(np.uint16)
    bits |= (rng.integers(0, 2, bits.shape) << 15).astype(np.uint16)
    t = torch.from_numpy(bits.view(np.int16)).view(BF)
    codes, scales = op.quantize_rows(t.to(DEV), "fp8_e4m3_b128")
    want, scale = oracle.quant_fp8(bits)
    assert np.array_equal(scales.cpu().numpy(), np.asarray(scale).reshape(21, -1))
    assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), np.asarray(want).reshape(21, -1))
    codes, scales = op.quantize_rows(t.to(DEV), "int8_row")
    want, scale = _int8(t.float().numpy())
    assert np.array_equal(scales.cpu().numpy(), scale)
    assert np.array_equal(codes.cpu().numpy(), want)
