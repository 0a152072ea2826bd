"""The gate around the split phases, on the host: what is called in which order.

A dispatch or combine that was sent runs on the op's side stream and may still
read the gate's weights and indices, so the next gate has to wait for it.
"""
import pytest
import torch

from combine_routing_histogram_amd import binding as B
from combine_routing_histogram_amd import layer as L
from combine_routing_histogram_amd.op import EpDispatchCombineConfig, EpDispatchCombineOp


class _Stream:
    """Stands for a stream; notes what waits for it."""
    cuda_stream = 0

    def __init__(self, name, log):
        self.name, self.log = name, log

    def wait_stream(self, other):
        self.log.append(f"{self.name} waits for {other.name}")


@pytest.fixture
def traced(monkeypatch):
    """(op with host buffers and stand-in streams, log)."""
    log = []
    op = EpDispatchCombineOp.__new__(EpDispatchCombineOp)
    op.config = EpDispatchCombineConfig(16, 256, 4, 8, 2)
    op.device, op._dev_index = torch.device("cpu"), -1
    op._op, op._tokens = 0, 0
    op._sent_dispatch = op._sent_combine = None
    op._side_stream = _Stream("side", log)
    op._gate_cut = (-1, None)
    op._gate = {"weights": torch.zeros(16, 4), "indices": torch.zeros(16, 4, dtype=torch.int32),
                "counts": torch.zeros(9, dtype=torch.int32), "losses": torch.zeros(2),
                "scratch": torch.zeros(256, dtype=torch.uint8)}
    op._out = op._out_weights = op._out_indices = op._recv_count = torch.zeros(64)
    op._combined = op._combined_weights = torch.zeros(16, 256)
    op._out_scales, op._payload_v, op._views = None, None, {}
    op._stream = lambda: 0
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: _Stream("caller", log))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: None)
    for mod, names in ((B, ("epdc_dispatch_send", "epdc_dispatch_recv", "epdc_combine_send",
                            "epdc_combine_recv", "epdc_reset")), (L, ("epdc_gate",))):
        for name in names:
            monkeypatch.setattr(mod, name, lambda *a, _n=name[5:]: log.append(_n))
    return op, log


LOGITS = torch.zeros(16, 8)


def _send(op):
    w, idx = op.gate(LOGITS)
    op.dispatch_send(torch.zeros(16, 256, dtype=torch.bfloat16), w, None, idx)


@pytest.mark.parametrize("balance", [False, True])
def test_gate_waits_for_a_sent_dispatch(traced, balance):
    op, log = traced
    _send(op)
    op.gate(LOGITS, balance=balance)
    assert log == ["gate", "side waits for caller", "dispatch_send", "caller waits for side",
                   "gate"]
    op.dispatch_recv()


def test_gate_waits_for_a_sent_combine(traced):
    op, log = traced
    op._tokens = 16
    _, idx = op.gate(LOGITS)
    op.combine_send(torch.zeros(64, 256, dtype=torch.bfloat16), None, idx)
    op.gate(LOGITS)
    assert log[-2:] == ["caller waits for side", "gate"]


def test_gate_does_not_wait_after_the_recv(traced):
    op, log = traced
    _send(op)
    op.dispatch_recv()
    del log[:]
    op.gate(LOGITS)
    assert log == ["gate"]


def test_gate_waits_for_a_send_that_a_reset_forgot(traced):
    """reset() drops the phase, not the work on the side stream."""
    op, log = traced
    _send(op)
    op.reset()
    del log[:]
    op.gate(LOGITS)
    assert log == ["caller waits for side", "gate"]


def test_gate_in_a_capture_refuses_a_send_from_outside_it(traced, monkeypatch):
    """A captured wait for work outside the capture would end the capture."""
    op, log = traced
    _send(op)
    del log[:]
    on = ["caller"]

    class _On:
        def __init__(self, stream):
            self.name = stream.name

        def __enter__(self):
            on.append(self.name)

        def __exit__(self, *exc):
            on.pop()
    monkeypatch.setattr(torch.cuda, "stream", _On)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: on[-1] == "caller")
    with pytest.raises(B.EpdcError) as ei:
        op.gate(LOGITS)
    assert ei.value.status == B.EPDC_ERR_BAD_STATE and log == []
    # sent inside the same capture: both streams belong to it
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    op.gate(LOGITS)
    assert log == ["caller waits for side", "gate"]


def test_products_and_gradients_refuse_a_dispatch_not_received(traced, monkeypatch):
    """They read the routing that the sent dispatch is still writing."""
    op, log = traced
    _send(op)
    monkeypatch.setattr(B, "epdc_get_offsets", lambda op: (4096, 4096))
    monkeypatch.setattr(B, "epdc_get_routing", lambda op: (4096, 4096, 4096))
    for mod, name in ((L, "epdc_expert_product"), (L, "epdc_expert_backward"),
                      (L, "epdc_combine_backward"), (B, "epdc_combine")):
        monkeypatch.setattr(mod, name, lambda *a, _n=name[5:]: log.append(_n))
    bf = torch.bfloat16
    x, w, g = torch.zeros(64, 256, dtype=bf), torch.zeros(8, 64, 256, dtype=bf), \
        torch.zeros(64, 64, dtype=bf)
    calls = [lambda: op.expert_product(x, w), lambda: op.expert_product_backward(g, x, w),
             lambda: op.combine_backward(torch.zeros(16, 256, dtype=bf), x),
             lambda: op.dispatch_backward(x)]
    del log[:]
    for call in calls:
        with pytest.raises(B.EpdcError) as ei:
            call()
        assert ei.value.status == B.EPDC_ERR_BAD_STATE and log == []
    op.dispatch_recv()
    del log[:]
    for call in calls:
        call()
    assert log == ["expert_product", "expert_backward", "combine_backward", "combine"]
