"""Outputs that overlap what a call still reads, or each other, are refused on the
host; overlaps of what it does not read are not its business."""
import pytest

from combine_routing_histogram_amd import binding as B
from combine_routing_histogram_amd import build as hip_build
from combine_routing_histogram_amd import layer as L

STEP = 1 << 44     # stand-in addresses, one array each: refused calls never touch them
ROWS, E, IN, OUT = 64, 4, 128, 64
ARR = {n: (i + 1) * STEP for i, n in enumerate(
    ("input", "weight", "scales", "weight_scales", "bias", "expert_off", "residual", "out",
     "preact", "grad_out", "dz", "grad_input", "grad_weight", "grad_bias", "slot_of",
     "grad_output", "weights", "grad_weights"))}


@pytest.fixture(scope="module", autouse=True)
def lib():
    if hip_build.is_stale():
        hip_build.build()
    return L.lib()


def _refused(call):
    with pytest.raises(B.EpdcError) as ei:
        call()
    assert ei.value.status == B.EPDC_ERR_INVALID_ARGS and "overlap" in str(ei.value)


# out and preact against arrays of the call: at the start, at the last bytes, from before
FORWARD = [("out", "input", 0), ("out", "input", ROWS * IN * 2 - 16),
           ("out", "input", -ROWS * OUT * 2 + 16), ("out", "weight", E * OUT * IN * 2 - 16),
           ("out", "bias", E * OUT * 4 - 16), ("out", "residual", 16), ("out", "residual", -16),
           ("out", "expert_off", 16), ("out", "preact", 0), ("preact", "input", 16),
           ("preact", "weight", 0), ("preact", "bias", 0), ("preact", "residual", 0),
           ("preact", "out", 32)]


@pytest.mark.parametrize("what,over,by", FORWARD)
def test_forward(what, over, by):
    a = dict(ARR)
    a[what] = a[over] + by
    p = L.make_product_args(ROWS, E, IN, OUT, input=a["input"], weight=a["weight"],
                            bias=a["bias"], expert_off=a["expert_off"])
    _refused(lambda: L.epdc_expert_product(p, 0, a["residual"], a["out"], a["preact"]))


@pytest.mark.parametrize("over,size", [("scales", ROWS * 4), ("weight_scales", E * 4)])
def test_forward_e4m3_scales(over, size):
    p = L.make_product_args(ROWS, E, IN, OUT, L.EPDC_DT_E4M3, input=ARR["input"],
                            weight=ARR["weight"], scales=ARR["scales"],
                            weight_scales=ARR["weight_scales"], expert_off=ARR["expert_off"])
    _refused(lambda: L.epdc_expert_product(p, 0, 0, ARR[over] + size - 16, 0))


# with SwiGLU and every output
BACKWARD = [("grad_input", "grad_out", 0), ("grad_input", "preact", 16), ("grad_input", "dz", 16),
            ("grad_input", "weight", 0), ("grad_input", "input", 0),
            ("grad_weight", "weight", 0), ("grad_weight", "input", 0),
            ("grad_weight", "dz", 0), ("grad_weight", "grad_input", 16),
            ("grad_bias", "grad_weight", 16), ("grad_bias", "grad_out", 0),
            ("grad_bias", "preact", 0), ("grad_bias", "dz", 0), ("dz", "grad_out", 0),
            ("dz", "preact", 0), ("dz", "input", 0), ("dz", "weight", 0)]


@pytest.mark.parametrize("what,over,by", BACKWARD)
def test_backward(what, over, by):
    a = dict(ARR)
    a[what] = a[over] + by
    p = L.make_product_args(ROWS, E, IN, OUT, activation=L.EPDC_ACT_SWIGLU, input=a["input"],
                            weight=a["weight"], expert_off=a["expert_off"])
    _refused(lambda: L.epdc_expert_backward(p, 0, a["grad_out"], a["preact"], a["dz"],
                                            a["grad_input"], a["grad_weight"], L.EPDC_DT_BF16,
                                            a["grad_bias"]))


@pytest.mark.parametrize("act,by", [(L.EPDC_ACT_SILU, 16), (L.EPDC_ACT_SWIGLU, 16)])
def test_dz_beside_its_factors(act, by):
    """dz in place of preact has to start where it does."""
    a = dict(ARR, dz=ARR["preact"] + by)
    p = L.make_product_args(ROWS, E, IN, OUT, activation=act, input=a["input"],
                            weight=a["weight"], expert_off=a["expert_off"])
    _refused(lambda: L.epdc_expert_backward(p, 0, a["grad_out"], a["preact"], a["dz"],
                                            a["grad_input"], 0, L.EPDC_DT_BF16, 0))


@pytest.mark.parametrize("what,over,by", [
    ("grad_input", "grad_output", 0), ("grad_input", "input", 16), ("grad_input", "weights", 0),
    ("grad_input", "slot_of", 0), ("grad_weights", "grad_output", 0), ("grad_weights", "input", 0),
    ("grad_weights", "weights", 0), ("grad_weights", "slot_of", 0),
    ("grad_weights", "grad_input", 0)])
def test_combine_backward(what, over, by):
    a = dict(ARR)
    a[what] = a[over] + by
    _refused(lambda: L.epdc_combine_backward(0, 32, 2, 64, a["slot_of"], a["grad_output"],
                                             a["input"], a["weights"], a["grad_input"],
                                             a["grad_weights"]))
