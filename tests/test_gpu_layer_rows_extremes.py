"""Rows in 8 bits and the norm at the ends of their numbers."""
import numpy as np
import pytest
import torch

from layer_common import DEV
from oracle import oracle
from test_gpu_layer_rows import BF, op  # noqa: F401

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
