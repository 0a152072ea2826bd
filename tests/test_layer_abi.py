"""CPU checks of the layer operators' boundary: libepdc_layer.so exports what
include/epdc_layer.h declares, its enums match the binding, and bad arguments
are refused before anything is launched.
"""
import os
import re
import shutil
import subprocess

import pytest
import torch

from combine_routing_histogram_amd import binding as B
from combine_routing_histogram_amd import build as hip_build
from combine_routing_histogram_amd import layer as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 4096          # an aligned stand-in address: refused calls never touch it


@pytest.fixture(scope="module")
def lib():
    if hip_build.is_stale():
        hip_build.build()
    return L.lib()


def test_exports_and_enums(lib):
    names = L.header_entry_points()
    assert set(names) == set(L._SIGNATURES)
    for n in names:
        assert hasattr(lib, n)
    text = open(L.HEADER).read()
    found = re.findall(r"\b(EPDC_[A-Z0-9_]+)\s*=\s*(-?\d+)", text)
    assert len(found) >= 11
    for name, val in found:
        assert getattr(L, name) == int(val), name


def test_header_is_plain_c(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no gcc")
    src = tmp_path / "use.c"
    src.write_text('#include "epdc_layer.h"\ntypedef void (*any_fn)(void);\n'
                   + "".join(f"any_fn p_{n} = (any_fn)&{n};\n" for n in L.header_entry_points())
                   + "int main(void) { return 0; }\n")
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-fsyntax-only",
                    "-I", os.path.join(ROOT, "include"), str(src)], check=True)


def _refused(call, msg):
    with pytest.raises(B.EpdcError) as ei:
        call()
    assert ei.value.status == B.EPDC_ERR_INVALID_ARGS
    assert msg in str(ei.value)


def _gate(**kw):
    d = dict(num_tokens=4, num_experts=8, topk=2, logits=A)
    d.update(kw)
    return L.make_gate_args(**d)


@pytest.mark.parametrize("kw,msg", [
    (dict(num_tokens=-1), "num_tokens"),
    (dict(num_experts=0), "num_experts"),
    (dict(num_experts=513), "num_experts"),
    (dict(topk=0), "topk"),
    (dict(topk=17, num_experts=64), "topk"),
    (dict(topk=9), "topk"),
    (dict(score=2), "score"),
    (dict(logits_dtype=L.EPDC_DT_E4M3), "logits"),
    (dict(scale=0.0), "scale"),
    (dict(scale=float("nan")), "scale"),
    (dict(scale=float("inf")), "scale"),
    (dict(logits=0), "logits"),
    (dict(logits=A + 8), "aligned"),
    (dict(bias=A + 2), "aligned"),
])
def test_gate_refusals(lib, kw, msg):
    _refused(lambda: L.epdc_gate(_gate(**kw), 0, A, A), msg)
    _refused(lambda: L.epdc_gate_backward(_gate(**kw), 0, A, A, 0, 0, A), msg)


def test_gate_pointer_refusals(lib):
    g = _gate()
    _refused(lambda: L.epdc_gate(g, 0, 0, A), "required")
    _refused(lambda: L.epdc_gate(g, 0, A, 0), "required")
    _refused(lambda: L.epdc_gate(g, 0, A, A, A, 0, 0), "all")
    _refused(lambda: L.epdc_gate(g, 0, A, A, 0, A, A), "all")
    _refused(lambda: L.epdc_gate(g, 0, A, A, A, A, A + 16), "256")
    _refused(lambda: L.epdc_gate_backward(g, 0, A, A, A, 0, A), "both")
    _refused(lambda: L.epdc_gate_backward(g, 0, A, A, 0, 0, 0), "grad_logits")
    _refused(lambda: L.epdc_gate_backward(g, 0, 0, A, 0, 0, A), "indices")
    _refused(lambda: L.epdc_gate_backward(g, 0, A, A, 0, 0, A + 4), "aligned")
    _refused(lambda: L.epdc_gate_scratch_bytes(-1, 8), "max_tokens")
    _refused(lambda: L.epdc_gate_scratch_bytes(8, 513), "num_experts")
    assert lib.epdc_gate(None, None, A, A, None, None, None) == B.EPDC_ERR_INVALID_ARGS
    assert L.epdc_gate_scratch_bytes(0, 1) >= 256
    assert L.epdc_gate_scratch_bytes(1 << 20, 256) == L.epdc_gate_scratch_bytes(1 << 30, 256)
    # nothing to do: no launch, success
    L.epdc_gate(_gate(num_tokens=0, logits=0), 0, 0, 0)
    L.epdc_gate_backward(_gate(num_tokens=0, logits=0), 0, 0, 0, 0, 0, 0)
    assert L.epdc_layer_last_error() == ""


def _prod(**kw):
    d = dict(rows=16, num_experts=4, in_features=128, out_features=64, input=A, weight=A,
             expert_off=A)
    d.update(kw)
    return L.make_product_args(**d)


BAD_PRODUCTS = [
    (dict(rows=-1), "rows"),
    (dict(rows=(1 << 30) + 1), "rows"),
    (dict(num_experts=0), "num_experts"),
    (dict(num_experts=513), "num_experts"),
    (dict(in_features=0), "in_features"),
    (dict(in_features=132), "in_features"),
    (dict(in_features=(1 << 20) + 8), "in_features"),
    (dict(out_features=60), "out_features"),
    (dict(out_features=72, activation=L.EPDC_ACT_SWIGLU), "out_features"),
    (dict(in_features=1 << 20, out_features=1 << 10), "2 GiB"),
    (dict(expected_rows=-1), "expected_rows"),
    (dict(activation=6), "activation"),
    (dict(activation=-1), "activation"),
    (dict(dtype=L.EPDC_DT_FP32), "bf16 or e4m3"),
    (dict(expert_off=0), "expert_off"),
    (dict(input=A + 8), "aligned"),
    (dict(weight=A + 2), "aligned"),
    (dict(bias=A + 2), "aligned"),
]


@pytest.mark.parametrize("kw,msg", BAD_PRODUCTS)
def test_product_refusals(lib, kw, msg):
    _refused(lambda: L.epdc_expert_product(_prod(**kw), 0, 0, A, 0), msg)
    _refused(lambda: L.epdc_expert_backward(_prod(**kw), 0, A, A, A, A, A, 0, 0), msg)


def test_product_pointer_refusals(lib):
    p = _prod()
    f8 = dict(dtype=L.EPDC_DT_E4M3)
    _refused(lambda: L.epdc_expert_product(_prod(input=0), 0, 0, A, 0), "required")
    _refused(lambda: L.epdc_expert_product(_prod(weight=0), 0, 0, A, 0), "required")
    _refused(lambda: L.epdc_expert_product(p, 0, 0, 0, 0), "required")
    _refused(lambda: L.epdc_expert_product(p, 0, A + 8, A, 0), "aligned")
    _refused(lambda: L.epdc_expert_product(p, 0, 0, A + 8, 0), "aligned")
    _refused(lambda: L.epdc_expert_product(p, 0, 0, A, A + 4), "aligned")
    _refused(lambda: L.epdc_expert_product(_prod(scales=A), 0, 0, A, 0), "e4m3")
    _refused(lambda: L.epdc_expert_product(_prod(**f8), 0, 0, A, 0), "e4m3")
    _refused(lambda: L.epdc_expert_product(_prod(scales=A, **f8), 0, 0, A, 0), "e4m3")
    _refused(lambda: L.epdc_expert_product(_prod(in_features=64, **f8), 0, 0, A, 0), "128")
    _refused(lambda: L.epdc_expert_backward(_prod(scales=A, weight_scales=A, **f8), 0, A, A, A, A,
                                            A, 0, 0), "bf16")
    _refused(lambda: L.epdc_expert_backward(p, 0, A, A, A, A, A, L.EPDC_DT_E4M3, 0), "grad_weight")
    _refused(lambda: L.epdc_expert_backward(p, 0, 0, 0, 0, A, A, 0, 0), "grad_out")
    act = _prod(activation=L.EPDC_ACT_SILU)
    _refused(lambda: L.epdc_expert_backward(act, 0, A, 0, A, A, A, 0, 0), "preact")
    _refused(lambda: L.epdc_expert_backward(act, 0, A, A, 0, A, A, 0, 0), "preact")
    _refused(lambda: L.epdc_expert_backward(p, 0, A, 0, 0, A + 8, A, 0, 0), "aligned")
    L.epdc_expert_product(_prod(rows=0, input=0, weight=0), 0, 0, 0, 0)   # nothing to do


def test_combine_backward_refusals(lib):
    f = L.epdc_combine_backward
    _refused(lambda: f(0, -1, 2, 64, A, A, A, 0, A, A), "num_tokens")
    _refused(lambda: f(0, 4, 0, 64, A, A, A, 0, A, A), "topk")
    _refused(lambda: f(0, 4, 17, 64, A, A, A, 0, A, A), "topk")
    _refused(lambda: f(0, 1 << 28, 8, 64, A, A, A, 0, A, A), "2^30")
    _refused(lambda: f(0, 4, 2, 60, A, A, A, 0, A, A), "hidden")
    _refused(lambda: f(0, 4, 2, 64, 0, A, A, 0, A, A), "slot_of")
    _refused(lambda: f(0, 4, 2, 64, A, 0, A, 0, A, A), "grad_output")
    _refused(lambda: f(0, 4, 2, 64, A, A, 0, 0, A, A), "input")
    _refused(lambda: f(0, 4, 2, 64, A, A + 4, A, 0, A, A), "aligned")
    f(0, 0, 2, 64, 0, 0, 0, 0, 0, 0)                                      # nothing to do


def _host_op(tokens=10):
    """An op's host state only: the checks run before anything reaches a device."""
    from combine_routing_histogram_amd.op import EpDispatchCombineConfig, EpDispatchCombineOp
    op = EpDispatchCombineOp.__new__(EpDispatchCombineOp)
    op.config = EpDispatchCombineConfig(16, 256, 4, 8, 2)
    op.device = torch.device("cpu")
    op._dev_index = -1
    op._tokens = tokens
    return op


def test_op_refuses_bad_gate_tensors():
    from combine_routing_histogram_amd.op import GateConfig
    op = _host_op()
    bf = torch.bfloat16
    for logits, kw in [(torch.zeros(4, 7), {}), (torch.zeros(17, 8), {}), (torch.zeros(8), {}),
                       (torch.zeros(4, 8, dtype=torch.float64), {}),
                       (torch.zeros(8, 4).t(), {}),
                       (torch.zeros(4, 8), dict(bias=torch.zeros(7))),
                       (torch.zeros(4, 8), dict(bias=torch.zeros(8, dtype=bf))),
                       (torch.zeros(4, 8), dict(mask=torch.zeros(4))),
                       (torch.zeros(4, 8), dict(mask=torch.zeros(5, dtype=torch.uint8)))]:
        with pytest.raises(ValueError):
            op.gate(logits, **kw)
    idx = torch.zeros(4, 4, dtype=torch.int32)
    for i, kw in [(idx.long(), {}), (idx[:3].contiguous(), {}),
                  (idx, dict(grad_weights=torch.zeros(4, 3))),
                  (idx, dict(counts=torch.zeros(9, dtype=torch.int32))),
                  (idx, dict(grad_losses=torch.zeros(2))),
                  (idx, dict(counts=torch.zeros(8, dtype=torch.int32),
                             grad_losses=torch.zeros(2)))]:
        with pytest.raises(ValueError):
            op.gate_backward(torch.zeros(4, 8), i, **kw)
    for kw in (dict(score="relu"), dict(scale=0.0), dict(scale=float("nan"))):
        with pytest.raises(ValueError):
            GateConfig(**kw)


def test_op_refuses_bad_product_tensors(monkeypatch):
    op = _host_op()
    op._op = 0
    monkeypatch.setattr(B, "epdc_get_offsets", lambda op: (A, A))
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    x, w = torch.zeros(40, 256, dtype=bf), torch.zeros(8, 64, 256, dtype=bf)
    x8, w8 = torch.zeros(40, 256).to(f8), torch.zeros(8, 64, 256).to(f8)
    s8, ws8 = torch.zeros(40, 2), torch.zeros(8, 1, 2)
    g = torch.zeros(40, 64, dtype=bf)
    bad = [(x[:39], w, {}), (x[:, :128].contiguous(), w, {}), (x.float(), w, {}),
           (x, w.float(), {}), (x, w[0], {}), (x, w, dict(first_expert=1)),
           (x, w, dict(first_expert=-1)), (x, w, dict(activation="tanh")),
           (x, w, dict(residual=g[:, :32].contiguous())), (x, w, dict(out=g[:39])),
           (x, torch.zeros(8, 256, 256, dtype=bf), dict(out=x)),
           (x, w, dict(preact=g.float())), (x, w, dict(bias=torch.zeros(8, 63))), (x, w, dict(bias=torch.zeros(8, 64, dtype=bf))),
           (x, w, dict(scales=s8, weight_scales=ws8)), (x8, w8, {}),
           (x8, w, {}), (x8, w8, dict(scales=s8[:39], weight_scales=ws8)),
           (x8, w8, dict(scales=s8, weight_scales=ws8[:, :, :1].contiguous())),
           (x, w.transpose(1, 2), {})]
    for a, b, kw in bad:
        with pytest.raises(ValueError):
            op.expert_product(a, b, **kw)
    for a, kw in [(g[:, :32].contiguous(), {}), (g.float(), {}), (g, dict(activation="swiglu")),
                  (g, dict(activation="silu")), (g, dict(weight_dtype=torch.float16))]:
        with pytest.raises(ValueError):
            op.expert_product_backward(a, x, w, **kw)


def test_product_needs_a_dispatch(lib):
    op = _host_op(tokens=0)
    op._op = 0
    with pytest.raises(B.EpdcError):
        op.expert_product(torch.zeros(0, 256, dtype=torch.bfloat16),
                          torch.zeros(8, 64, 256, dtype=torch.bfloat16))
