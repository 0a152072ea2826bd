"""CPU checks of the boundary of the norm, rows in 8 bits, integer products and the layer
for few tokens: bad arguments are refused before anything is launched."""
import pytest
import torch

from combine_routing_histogram_amd import binding as B
from combine_routing_histogram_amd import build as hip_build
from combine_routing_histogram_amd import layer as L
from test_layer_abi import _host_op, _prod, _refused

STEP = 1 << 44    # stand-in addresses, an array each: refused calls never touch them
A = {n: (i + 1) * STEP for i, n in enumerate(
    ("input", "residual", "weight", "out", "sum", "codes", "scales", "grad_out", "grad_sum",
     "grad_input", "grad_weight", "scratch", "weights", "indices", "w1", "w2", "w1_scales",
     "w2_scales", "bias1", "bias2", "h", "expert_off"))}
BF16, FP32, E4M3, INT8 = L.EPDC_DT_BF16, L.EPDC_DT_FP32, L.EPDC_DT_E4M3, L.EPDC_DT_INT8


@pytest.fixture(scope="module", autouse=True)
def lib():
    if hip_build.is_stale():
        hip_build.build()
    return L.lib()


def _norm(**kw):
    d = dict(rows=16, features=256, input=A["input"], residual=A["residual"], weight=A["weight"])
    d.update(kw)
    return L.make_norm_args(**d)


@pytest.mark.parametrize("kw,msg", [
    (dict(rows=-1), "rows"), (dict(rows=(1 << 30) + 1), "rows"), (dict(features=0), "features"),
    (dict(features=260), "features"), (dict(features=(1 << 15) + 8), "features"),
    (dict(weight_dtype=E4M3), "weight"), (dict(eps=-1e-6), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"),
    (dict(input=0), "required"), (dict(weight=0), "required"),
    (dict(input=A["input"] + 8), "aligned"), (dict(residual=A["residual"] + 4), "aligned"),
    (dict(weight=A["weight"] + 2), "aligned")])
def test_norm_refusals(kw, msg):
    _refused(lambda: L.epdc_rms_norm(_norm(**kw), 0, A["out"], A["sum"], 0, 0, BF16), msg)
    back = dict(kw, residual=kw.get("residual", 0))
    _refused(lambda: L.epdc_rms_norm_backward(_norm(**back), 0, A["grad_out"], 0, A["grad_input"],
                                              0, 0), msg)


def test_norm_output_refusals(lib):
    f = L.epdc_rms_norm
    _refused(lambda: f(_norm(), 0, 0, A["sum"], 0, 0, BF16), "out or codes")
    _refused(lambda: f(_norm(), 0, A["out"], 0, A["codes"], 0, BF16), "belong")
    _refused(lambda: f(_norm(), 0, A["out"], 0, 0, A["scales"], BF16), "belong")
    _refused(lambda: f(_norm(), 0, A["out"], 0, 0, 0, INT8), "required")
    _refused(lambda: f(_norm(), 0, A["out"], 0, A["codes"], 0, E4M3), "required")
    _refused(lambda: f(_norm(), 0, A["out"], 0, A["codes"], A["scales"], FP32), "codes must be")
    _refused(lambda: f(_norm(features=264), 0, A["out"], 0, A["codes"], A["scales"], INT8), "16")
    _refused(lambda: f(_norm(features=272), 0, A["out"], 0, A["codes"], A["scales"], E4M3), "128")
    _refused(lambda: f(_norm(), 0, A["out"] + 8, 0, 0, 0, BF16), "aligned")
    _refused(lambda: f(_norm(), 0, A["out"], A["sum"] + 8, 0, 0, BF16), "aligned")
    _refused(lambda: f(_norm(), 0, 0, 0, A["codes"] + 8, A["scales"], INT8), "aligned")
    _refused(lambda: f(_norm(), 0, 0, 0, A["codes"], A["scales"] + 2, INT8), "aligned")
    f(_norm(rows=0, input=0, residual=0, weight=0), 0, 0, 0, 0, 0, INT8)   # nothing to do
    assert L.epdc_layer_last_error() == ""
    assert lib.epdc_rms_norm(None, None, 64, None, None, None, BF16) == B.EPDC_ERR_INVALID_ARGS
    assert L.epdc_rms_norm_scratch_bytes(4096) >= 4096 * 4
    for features in (0, 12, (1 << 15) + 8):
        _refused(lambda: L.epdc_rms_norm_scratch_bytes(features), "features")


def test_norm_backward_refusals(lib):
    f = L.epdc_rms_norm_backward
    n = _norm(residual=0)
    g = (A["grad_out"], A["grad_sum"], A["grad_input"])
    _refused(lambda: f(_norm(), 0, *g, 0, 0), "no residual")
    _refused(lambda: f(n, 0, *g, A["grad_weight"], 0), "both")
    _refused(lambda: f(n, 0, *g, 0, A["scratch"]), "both")
    _refused(lambda: f(n, 0, 0, 0, A["grad_input"], 0, 0), "required")
    _refused(lambda: f(n, 0, A["grad_out"], 0, 0, 0, 0), "required")
    _refused(lambda: f(n, 0, A["grad_out"] + 8, 0, A["grad_input"], 0, 0), "aligned")
    _refused(lambda: f(n, 0, *g, A["grad_weight"] + 4, A["scratch"]), "aligned")
    assert lib.epdc_rms_norm_backward(None, *[None] * 6) == B.EPDC_ERR_INVALID_ARGS


# rows of 16 x 256 bf16 are 8192 bytes
@pytest.mark.parametrize("what,over,by", [
    ("out", "input", 0), ("out", "input", 8176), ("out", "residual", -8176), ("out", "weight", 0),
    ("out", "sum", 16), ("out", "codes", 0), ("out", "scales", 48), ("sum", "input", 16),
    ("sum", "residual", 16), ("sum", "weight", 0), ("sum", "codes", 4080), ("codes", "input", 0),
    ("codes", "residual", 8176), ("codes", "scales", 0), ("codes", "weight", 496),
    ("scales", "input", 0), ("scales", "weight", 0)])
def test_norm_overlaps(what, over, by):
    a = dict(A)
    a[what] = a[over] + by
    with pytest.raises(B.EpdcError) as e:
        L.epdc_rms_norm(_norm(), 0, a["out"], a["sum"], a["codes"], a["scales"], INT8)
    assert "overlap" in str(e.value)


@pytest.mark.parametrize("what,over,by", [
    ("grad_input", "input", 0), ("grad_input", "weight", 0), ("grad_input", "grad_out", 16),
    ("grad_input", "grad_sum", -16), ("grad_input", "grad_weight", 0),
    ("grad_input", "scratch", 0), ("grad_weight", "input", 0), ("grad_weight", "grad_out", 0),
    ("grad_weight", "grad_sum", 0), ("grad_weight", "weight", 0), ("grad_weight", "scratch", 0),
    ("scratch", "input", 0), ("scratch", "grad_out", 0), ("scratch", "weight", 0)])
def test_norm_backward_overlaps(what, over, by):
    a = dict(A)
    a[what] = a[over] + by
    with pytest.raises(B.EpdcError) as e:
        L.epdc_rms_norm_backward(_norm(residual=0), 0, a["grad_out"], a["grad_sum"],
                                 a["grad_input"], a["grad_weight"], a["scratch"])
    assert "overlap" in str(e.value)


def test_quantize_refusals():
    f = L.epdc_quantize_rows
    x, c, s, off = A["input"], A["codes"], A["scales"], A["expert_off"]
    _refused(lambda: f(0, 4, 128, BF16, x, 0, 0, c, s), "e4m3 or int8")
    _refused(lambda: f(0, -1, 128, INT8, x, 0, 0, c, s), "rows")
    _refused(lambda: f(0, 4, 136, INT8, x, 0, 0, c, s), "16")
    _refused(lambda: f(0, 4, 144, E4M3, x, 0, 0, c, s), "128")
    _refused(lambda: f(0, 4, (1 << 17) + 128, E4M3, x, 0, 0, c, s), "features")
    _refused(lambda: f(0, 4, 128, INT8, x, off, 0, c, s), "num_experts")
    _refused(lambda: f(0, 4, 128, INT8, x, off, 513, c, s), "num_experts")
    for bad in ((0, 0, 0, c, s), (x, 0, 0, 0, s), (x, 0, 0, c, 0)):
        _refused(lambda: f(0, 4, 128, INT8, *bad), "required")
    for bad in ((x + 8, 0, 0, c, s), (x, 0, 0, c + 8, s), (x, 0, 0, c, s + 2),
                (x, off + 2, 1, c, s)):
        _refused(lambda: f(0, 4, 128, INT8, *bad), "aligned")
    for bad in ((x, 0, 0, x + 1008, s), (x, 0, 0, c, c + 508), (x, 0, 0, c, x),
                (x, off, 8, off, s), (x, off, 8, c, off + 32)):
        _refused(lambda: f(0, 4, 128, INT8, *bad), "overlap")
    f(0, 0, 128, INT8, 0, 0, 0, 0, 0)     # nothing to do


def test_integer_product_refusals():
    i8 = dict(dtype=INT8, scales=A["scales"], weight_scales=A["w1_scales"], input=A["input"],
              weight=A["w1"], expert_off=A["expert_off"])
    f = lambda kw: L.epdc_expert_product(_prod(**dict(i8, **kw)), 0, 0, A["out"], 0)
    _refused(lambda: f(dict(scales=0)), "scales")
    _refused(lambda: f(dict(weight_scales=0)), "scales")
    _refused(lambda: f(dict(in_features=136)), "16")
    _refused(lambda: f(dict(in_features=1 << 17)), "in_features")
    _refused(lambda: f(dict(out_features=60)), "out_features")
    _refused(lambda: f(dict(scales=A["scales"] + 2)), "aligned")
    _refused(lambda: f(dict(scales=A["out"] + 16 * 64 * 2 - 4)), "overlap")
    _refused(lambda: f(dict(scales=A["out"] - 60)), "overlap")
    _refused(lambda: f(dict(weight_scales=A["out"] - 4 * 64 * 4 + 4)), "overlap")
    _refused(lambda: L.epdc_expert_backward(_prod(**i8), 0, A["grad_out"], 0, 0, A["grad_input"],
                                            0, 0, 0), "bf16")


def _few(**kw):
    d = dict(num_tokens=8, topk=2, num_experts=4, hidden=256, inner=128, input=A["input"],
             weights=A["weights"], indices=A["indices"], w1=A["w1"], w2=A["w2"])
    d.update(kw)
    return L.make_few_args(**d)


@pytest.mark.parametrize("kw,msg", [
    (dict(num_tokens=-1), "num_tokens"), (dict(num_tokens=65), "num_tokens"),
    (dict(topk=0), "topk"), (dict(topk=17), "topk"), (dict(num_experts=0), "num_experts"),
    (dict(num_experts=513), "num_experts"), (dict(first_expert=-1), "first_expert"),
    (dict(first_expert=513), "first_expert"), (dict(activation=6), "activation"),
    (dict(dtype=FP32), "bf16"), (dict(hidden=260), "multiples of 8"),
    (dict(inner=4), "multiples of 8"), (dict(inner=(1 << 20) + 8), "at most"),
    (dict(dtype=INT8, inner=136), "multiples of 16"),
    (dict(dtype=E4M3, hidden=320), "multiples of 128"),
    (dict(hidden=1 << 18, inner=1 << 13), "2 GiB"),
    (dict(num_tokens=64, topk=16, num_experts=64, hidden=256, inner=1 << 20), "2 GiB"),
    (dict(w1_scales=A["w1_scales"]), "w1_scales"), (dict(dtype=INT8), "w1_scales"),
    (dict(dtype=E4M3, w1_scales=A["w1_scales"]), "w1_scales"),
    (dict(input=0), "required"), (dict(indices=0), "required"), (dict(w1=0), "required"),
    (dict(w2=0), "required"), (dict(input=A["input"] + 8), "aligned"),
    (dict(w2=A["w2"] + 4), "aligned"), (dict(weights=A["weights"] + 2), "aligned"),
    (dict(bias2=A["bias2"] + 2), "aligned")])
def test_few_token_refusals(kw, msg):
    _refused(lambda: L.epdc_few_tokens(_few(**kw), 0, A["h"], A["out"]), msg)


def test_few_token_scratch(lib):
    f = L.epdc_few_tokens_scratch_bytes
    assert f(L.make_few_args(0, 2, 4, 256, 128)) == 0
    assert f(_few()) >= 8 * 2 * 128 * 2
    # blocks that share a tile leave their sums: more than h alone
    assert f(_few(hidden=1024, inner=8192, num_tokens=64)) > 64 * 2 * 8192 * 2
    _refused(lambda: f(_few(topk=0)), "topk")
    assert lib.epdc_few_tokens_scratch_bytes(_few(), None) == B.EPDC_ERR_INVALID_ARGS


def test_few_token_buffers(lib):
    f = lambda h, out, **kw: L.epdc_few_tokens(_few(bias1=A["bias1"], bias2=A["bias2"], **kw), 0,
                                               h, out)
    _refused(lambda: f(0, A["out"]), "required")
    _refused(lambda: f(A["h"], 0), "required")
    _refused(lambda: f(A["h"] + 128, A["out"]), "aligned")
    _refused(lambda: f(A["h"], A["out"] + 8), "aligned")
    for over in ("input", "weights", "indices", "w1", "w2", "bias1", "bias2"):
        _refused(lambda: f(A[over], A["out"]), "overlap")
        _refused(lambda: f(A["h"], A[over] + 16), "overlap")
    _refused(lambda: f(A["h"], A["h"] + 16), "overlap")
    _refused(lambda: f(A["h"], A["input"] - 16), "overlap")
    # the sums behind h are part of the scratch
    kw = dict(hidden=1024, inner=8192, num_tokens=64)
    end = L.epdc_few_tokens_scratch_bytes(_few(**kw))
    _refused(lambda: f(A["h"], A["h"] + end - 16, **kw), "overlap")
    L.epdc_few_tokens(_few(num_tokens=0, input=0, indices=0, w1=0, w2=0), 0, 0, 0)
    assert lib.epdc_few_tokens(None, None, None, None) == B.EPDC_ERR_INVALID_ARGS


@pytest.fixture
def op(monkeypatch):
    """An op of 8 experts, top-4, hidden 256, whose last dispatch had 10 tokens; the library's
    calls leave their arguments in op.calls."""
    op = _host_op()
    op._op, op.calls = 0, []
    op._stream = lambda: 0
    monkeypatch.setattr(B, "epdc_get_offsets", lambda op: (4096, 4096))
    for name in ("epdc_expert_product", "epdc_rms_norm", "epdc_rms_norm_backward",
                 "epdc_quantize_rows", "epdc_few_tokens"):
        monkeypatch.setattr(L, name, lambda *a: op.calls.append(a))
    return op


BF = torch.bfloat16


def test_op_norm(op):
    x, w = torch.zeros(5, 256, dtype=BF), torch.zeros(256)
    out, total, codes, scales = op.add_rms_norm(x, w, x, quant="fp8_e4m3_b128", output=False)
    assert out is None and total.shape == (5, 256) and codes.dtype == torch.float8_e4m3fn
    assert scales.shape == (5, 2)
    assert op.add_rms_norm(x, w, quant="int8_row")[3].shape == (5, 1)
    assert len(op.calls) == 2
    for a, b, kw in [(x.float(), w, {}), (x[0], w, {}), (x, w[:128], {}), (x, w.double(), {}),
                     (x.t(), w, {}), (x, w, dict(residual=x[:4])),
                     (x, w, dict(residual=x.float())), (x, w, dict(quant="mxfp4_b32")),
                     (x, w, dict(output=False)), (x, w, dict(sum_out=x)),
                     (x, w, dict(residual=x, sum_out=x[:4])),
                     (x[:, :200].contiguous(), w[:200], dict(quant="int8_row"))]:
        with pytest.raises(ValueError):
            op.add_rms_norm(a, b, **kw)
    gx, gw = op.add_rms_norm_backward(x, x, w)
    assert gx.shape == (5, 256) and gw.shape == (256,) and gw.dtype == torch.float32
    for g, kw in [(x[:4], {}), (x.float(), {}), (x, dict(grad_sum=x[:4]))]:
        with pytest.raises(ValueError):
            op.add_rms_norm_backward(g, x, w, **kw)
    assert len(op.calls) == 3


def test_op_quantize_and_integer_product(op):
    x = torch.zeros(45, 256, dtype=BF)
    codes, scales = op.quantize_rows(x, "int8_row", routed=True)
    assert codes.shape == (40, 256) and scales.shape == (40, 1) and op.calls[0][5] == 4096
    assert op.quantize_rows(x, "fp8_e4m3_b128")[1].shape == (45, 2) and op.calls[1][5] == 0
    for a, q, kw in [(x, "none", {}), (x.float(), "int8_row", {}), (x[0], "int8_row", {}),
                     (x[:39], "int8_row", dict(routed=True)),
                     (x[:, :144].contiguous(), "fp8_e4m3_b128", {})]:
        with pytest.raises(ValueError):
            op.quantize_rows(a, q, **kw)
    w, sw = torch.zeros(8, 64, 256, dtype=torch.int8), torch.zeros(8, 64)
    op.expert_product(codes, w, scales=scales, weight_scales=sw)
    for a, b, s, t in [(codes, w, None, sw), (codes, w, scales, None), (codes, w, scales[:39], sw),
                       (codes, w, torch.zeros(40, 2), sw), (codes, w, scales, sw[:, :63]),
                       (codes, w, scales, torch.zeros(8, 1, 2)), (x, w, scales, sw),
                       (codes, w.to(BF), scales, sw), (codes, w.to(torch.uint8), scales, sw)]:
        with pytest.raises(ValueError):
            op.expert_product(a, b, scales=s, weight_scales=t)


def test_op_few_tokens(op):
    x, idx = torch.zeros(6, 256, dtype=BF), torch.zeros(6, 4, dtype=torch.int32)
    g, w1, w2 = torch.zeros(6, 4), torch.zeros(8, 128, 256, dtype=BF), torch.zeros(8, 256, 64,
                                                                                  dtype=BF)
    run = lambda **kw: op.few_token_layer(**dict(dict(input=x, weights=g, indices=idx, w1=w1,
                                                      w2=w2, activation="swiglu"), **kw))
    assert run().shape == (6, 256) and run(weights=None, out=x) is x
    many = torch.zeros(65, 256, dtype=BF)
    for kw in [dict(input=x.float()), dict(input=x[0]), dict(input=x[:, :128].contiguous()),
               dict(input=many, weights=None, indices=torch.zeros(65, 4, dtype=torch.int32)),
               dict(indices=idx.long()), dict(indices=idx[:5]), dict(weights=g[:, :3]),
               dict(weights=g.to(BF)), dict(w1=w1.float()), dict(w2=w2.float()),
               dict(activation="none"), dict(activation="tanh"), dict(w2=w2[:, :128].contiguous()),
               dict(w1=w1[:4]), dict(first_expert=1), dict(first_expert=-1),
               dict(w1_scales=torch.zeros(8, 128)), dict(bias1=torch.zeros(8, 64)),
               dict(bias2=torch.zeros(8, 256, dtype=BF)), dict(out=x[:5]),
               dict(w1=w1.to(torch.int8), w2=w2.to(torch.int8)),
               dict(w1=w1.to(torch.int8), w2=w2.to(torch.int8), w1_scales=torch.zeros(8, 128),
                    w2_scales=torch.zeros(8, 64))]:
        with pytest.raises(ValueError):
            run(**kw)
    assert len(op.calls) == 2
    run(w1=w1.to(torch.int8), w2=w2.to(torch.int8), w1_scales=torch.zeros(8, 128),
        w2_scales=torch.zeros(8, 256))
