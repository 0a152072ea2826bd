"""Teams of several waves that take more than one row each: the norm's gradient as training has
it, and the norm and int8 rows past the 2^20 blocks of a launch.  The bounds are those of
test_gpu_layer_rows.py; a weight's gradient adds at most rows/512 rows in a team of 1 or 4 waves
and rows/256 in one of 8 or 16, here at most 40, and 72 across: within its 2^-16.
"""
import numpy as np
import pytest
import torch

from layer_common import DEV, normal
from test_gpu_layer_rows import BF, U, _check_codes, _gradient, _int8, _norm, _wide, _within, op  # noqa: F401

pytestmark = pytest.mark.gpu


# forms of 4 waves with one and two vectors a lane, 8 with two, 16 with two and four; two to 40
# rows a team, the last of them for some teams only
@pytest.mark.parametrize("T,H", [(1100, 520), (1537, 2048), (1100, 2056), (2048, 4096),
                                 (700, 4104), (1025, 7168), (700, 8200), (513, 16384),
                                 (520, 16392), (300, 32768), (10000, 1032)])
def test_gradient(op, T, H):  # noqa: F811
    print(f"norm backward T={T} H={H}", flush=True)
    rng = np.random.default_rng(T + H)
    s, dy = _wide(rng, (T, H)), normal(rng, (T, H))
    for dtype, ds in ((BF, normal(rng, (T, H))), (torch.float32, None)):
        w = normal(rng, (H,), dtype=dtype)
        gx, gw = op.add_rms_norm_backward(dy, s, w, eps=1e-5, grad_sum=ds)
        dx, tol, dw, wtol = _gradient(s, dy, w, 1e-5, ds)
        _within(gx, dx, tol, "grad_input")
        _within(gw, dw, wtol, "grad_weight")
        for _ in range(3):
            again = op.add_rms_norm_backward(dy, s, w, eps=1e-5, grad_sum=ds)
            assert torch.equal(again[0], gx) and torch.equal(again[1], gw)


def test_gradient_of_rows_of_every_range(op):  # noqa: F811
    """Rows that need a second sum between rows that do not, in one team."""
    for T, H in ((1100, 264), (1100, 1032), (700, 4104), (520, 8200), (300, 16392)):
        print(f"norm backward T={T} H={H}", flush=True)
        rng = np.random.default_rng(H)
        s = normal(rng, (T, H)) * 2.0 ** torch.from_numpy(rng.choice([-70, 0, 64, 110], (T, 1))).to(DEV)
        s, dy, w = s.to(BF), normal(rng, (T, H)), normal(rng, (H,))
        gx, gw = op.add_rms_norm_backward(dy, s, w, eps=0.0)
        dx, tol, dw, wtol = _gradient(s, dy, w, 0.0, None)
        _within(gx, dx, tol + 2.0 ** -133, "grad_input")
        _within(gw, dw, wtol, "grad_weight")
        y = _norm(s, None, w, 0.0)[1]
        out = op.add_rms_norm(s, w, eps=0.0)[0]
        _within(out, y, (U + 2.0 ** -18) * y.abs(), "out")


MANY = (1 << 20) + 3000    # rows: 3000 blocks take a second one


def _ends(*tensors):
    """The rows of the blocks that take two."""
    return [None if t is None else torch.cat([t[:3000], t[-3000:]]) for t in tensors]


@pytest.mark.parametrize("quant,H", [("none", 520), ("int8_row", 528), ("fp8_e4m3_b128", 640),
                                     ("int8_row", 4112)])
def test_norm_past_the_blocks_of_a_launch(op, quant, H):  # noqa: F811
    print(f"norm {quant} T={MANY} H={H}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(H)
    x = torch.empty((MANY, H), dtype=BF, device=DEV).normal_(generator=g)
    w = torch.empty(H, dtype=BF, device=DEV).normal_(generator=g)
    out, total, codes, scales = op.add_rms_norm(x, w, x, quant=quant)
    x, out, total, codes, scales = _ends(x, out, total, codes, scales)
    y = _norm(x, x, w, 1e-6)[1]
    _within(out, y, (U + 2.0 ** -18) * y.abs(), "out")
    assert torch.equal(total, (x.float() * 2).to(BF))
    if quant != "none":
        _check_codes(codes, scales, y, quant)


@pytest.mark.parametrize("I", [1040, 4112])
def test_int8_rows_past_the_blocks_of_a_launch(op, I):  # noqa: F811
    print(f"int8 rows T={MANY} I={I}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(I)
    x = torch.empty((MANY, I), dtype=BF, device=DEV).normal_(generator=g)
    codes, scales = op.quantize_rows(x, "int8_row")
    x, codes, scales = _ends(x, codes, scales)
    want, scale = _int8(x.float().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), scale)
    assert np.array_equal(codes.cpu().numpy(), want)
