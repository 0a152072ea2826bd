"""EpDispatchCombineConfig / EpDispatchCombineOp: the MORI-EP method surface
(MORI "Communication APIs" page, MORI-EP section, methods table) on top of the
C ABI.  PyTorch provides device memory and the current HIP stream; every step
of dispatch and combine runs in the HIP kernels behind libepdc.so.

Receive buffers are allocated once per op at capacity (max_tokens * topk rows)
-- the analogue of MORI's pre-registered buffers -- and dispatch/combine
return views of them without synchronizing the host.  Rows
[rank_off[r], rank_off[r+1]) of every received tensor belong to virtual rank r;
only the first sum(recv_count) rows are written by a dispatch.
"""
from __future__ import annotations

import dataclasses
import enum
import functools
from typing import Optional, Tuple

import torch

from . import binding as B
from . import layer as L

QUANT = {"none": B.EPDC_QUANT_NONE, "fp8_e4m3_b128": B.EPDC_QUANT_FP8_E4M3_B128,
         "mxfp4_b32": B.EPDC_QUANT_MXFP4_B32}


class EpDispatchCombineKernelType(enum.IntEnum):
    """The kernel types of the MORI-EP section ("Communication APIs" page,
    kernel types table), kept with their values so that code written against
    that enum imports unchanged.  On one GPU the destination ranks are
    segments of one HBM buffer, which is the intra-node case; the others move
    data across nodes or through SDMA queues and are not built here."""
    IntraNode = 0
    InterNode = 1
    InterNodeV1 = 2
    InterNodeV1LL = 3
    AsyncLL = 4


@dataclasses.dataclass
class EpDispatchCombineConfig:
    max_tokens: int
    hidden: int
    topk: int
    num_experts: int
    num_ranks: int
    quant: str = "none"            # "none", "fp8_e4m3_b128", "mxfp4_b32"
    raw_row_bytes: int = 0         # > 0: dispatch carries opaque byte rows
    scale_row_bytes: int = 0       # bytes of a carried per-token scale row
    kernel_type: int = EpDispatchCombineKernelType.IntraNode

    def __post_init__(self):
        kt = EpDispatchCombineKernelType(self.kernel_type)   # ValueError for unknown values
        if kt != EpDispatchCombineKernelType.IntraNode:
            raise ValueError(f"kernel_type {kt.name} moves rows between nodes or through SDMA "
                             "queues; on one GPU only IntraNode (rank segments of one HBM "
                             "buffer) exists")
        if self.quant not in QUANT:
            raise ValueError(f"quant must be one of {sorted(QUANT)}")

    def to_c(self) -> B.epdc_config:
        kind = B.EPDC_IN_RAW if self.raw_row_bytes > 0 else B.EPDC_IN_BF16
        return B.make_config(self.max_tokens, self.hidden, self.topk, self.num_experts,
                             self.num_ranks, kind, QUANT[self.quant], self.raw_row_bytes,
                             self.scale_row_bytes)


GATE_SCORES = {"softmax": L.EPDC_GATE_SOFTMAX, "sigmoid": L.EPDC_GATE_SIGMOID}
ACTIVATIONS = {"none": L.EPDC_ACT_NONE, "relu": L.EPDC_ACT_RELU, "gelu": L.EPDC_ACT_GELU,
               "silu": L.EPDC_ACT_SILU, "swiglu": L.EPDC_ACT_SWIGLU, "geglu": L.EPDC_ACT_GEGLU}
GATED = ("swiglu", "geglu")


@dataclasses.dataclass(frozen=True)
class GateConfig:
    """How a gate turns logits into routing weights (epdc_gate)."""
    score: str = "softmax"         # "softmax" or "sigmoid"
    renormalize: bool = True       # divide by the sum of the chosen scores
    scale: float = 1.0             # multiplies the weights

    def __post_init__(self):
        if self.score not in GATE_SCORES:
            raise ValueError(f"score must be one of {sorted(GATE_SCORES)}")
        if not 0.0 < self.scale < float("inf"):
            raise ValueError("scale must be positive and finite")


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _raw_stream(device_index: int) -> int:
    """The current stream of the device as a raw handle."""
    return torch._C._cuda_getCurrentRawStream(device_index)


if not hasattr(torch._C, "_cuda_getCurrentRawStream"):  # older torch
    def _raw_stream(device_index: int) -> int:  # noqa: F811
        return torch.cuda.current_stream(device_index).cuda_stream


def _on_op_device(method):
    """Run a method with the op's device current, whatever the caller's is: its
    kernels and its new tensors belong there."""
    @functools.wraps(method)
    def call(self, *args, **kwargs):
        if self._dev_index < 0 or torch.cuda.current_device() == self._dev_index:
            return method(self, *args, **kwargs)
        with torch.cuda.device(self._dev_index):
            return method(self, *args, **kwargs)
    return call


class EpDispatchCombineOp:
    # phases sent to the side stream and not known to be over; unlike
    # _sent_dispatch and _sent_combine they outlive a reset(), as the work does
    _on_side = frozenset()
    _sent_dispatch = _sent_combine = None
    _routing_sent = False       # the last dispatch was sent and not received

    def __init__(self, config: EpDispatchCombineConfig, device: Optional[torch.device] = None):
        self.config = config
        self.device = torch.device(device) if device is not None else torch.device(
            "cuda", torch.cuda.current_device())
        c = config.to_c()
        self._c = c
        ws_bytes = B.epdc_workspace_bytes(c)
        self.payload_row_bytes, self.scale_row_bytes = B.epdc_row_bytes(c)
        n_cap = config.max_tokens * config.topk
        self.n_cap = n_cap
        dev = self.device
        with torch.cuda.device(dev):
            self.workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
            self._out = torch.empty((n_cap, self.payload_row_bytes), dtype=torch.uint8, device=dev)
            self._out_weights = torch.empty((n_cap, config.topk), dtype=torch.float32, device=dev)
            self._out_indices = torch.empty((n_cap, config.topk), dtype=torch.int32, device=dev)
            self._out_scales = (torch.empty((n_cap, self.scale_row_bytes), dtype=torch.uint8,
                                            device=dev) if self.scale_row_bytes else None)
            self._recv_count = torch.empty(config.num_ranks, dtype=torch.int32, device=dev)
            self._combined = torch.empty((config.max_tokens, config.hidden), dtype=torch.bfloat16,
                                         device=dev)
            self._combined_weights = torch.empty((config.max_tokens, config.topk),
                                                 dtype=torch.float32, device=dev)
            self._combine_in = None
            # zeroed here, before epdc_create waits for the device: a first gate()
            # on another stream or under graph capture finds the scratch ready
            self._gate = self._gate_buffers()
            self._op = B.epdc_create(c, self.workspace.data_ptr(), ws_bytes)
        self._tokens = 0
        self._scales_dtype = None
        self._dev_index = self.device.index if self.device.index is not None else \
            torch.cuda.current_device()
        lib = B.lib()
        self._f_dispatch, self._f_combine = lib.epdc_dispatch, lib.epdc_combine
        self._views = {}
        self._payload_v = self._payload_view(self._out)
        self._combined_cut = (-1, None)   # (T, (output view, weights view))
        self._side_stream = None
        self.u_cap = config.max_tokens * min(config.topk, config.num_ranks)
        self._last_dedup = False
        self._staging = None
        self._units = None          # unit-row buffers, allocated on first use
        self._gate_cut = (-1, None)
        self._unit_carried = (False, False)

    def __del__(self):
        op = getattr(self, "_op", None)
        if op:
            try:
                B.epdc_destroy(op)
            except Exception:
                pass
            self._op = None

    # ---- helpers -------------------------------------------------------------------
    # Host cost matters for small batches (a 128-token step is ~16 us of GPU
    # time): the stream is read as a raw handle, library functions and buffer
    # views are looked up once, and the argument checks use cheap accessors.
    def _stream(self) -> int:
        return _raw_stream(self._dev_index)

    def _need(self, t: torch.Tensor, name: str, dtype=None, shape=None):
        if t.get_device() != self._dev_index:
            raise ValueError(f"{name} is on {t.device}, op is on {self.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")

    def _ws_view(self, ptr: int, count: int) -> torch.Tensor:
        off = ptr - self.workspace.data_ptr()
        return self.workspace[off:off + 4 * count].view(torch.int32)

    def _side(self) -> torch.cuda.Stream:
        # default priority: the send phases run here while the caller's stream computes
        if self._side_stream is None:
            self._side_stream = torch.cuda.Stream(device=self.device)
        return self._side_stream

    def _check_payload(self, input, weights, scales, T: int) -> None:
        cfg = self.config
        if cfg.raw_row_bytes:
            self._need(input, "input")
            if input.numel() * input.element_size() != T * cfg.raw_row_bytes:
                raise ValueError("input must hold raw_row_bytes per token")
        else:
            self._need(input, "input", torch.bfloat16, (T, cfg.hidden))
        if weights is not None:
            self._need(weights, "weights", torch.float32, (T, cfg.topk))
        if scales is not None:
            self._need(scales, "scales")
            if scales.numel() * scales.element_size() != T * cfg.scale_row_bytes:
                raise ValueError("scales must hold scale_row_bytes per token")
            self._scales_dtype = scales.dtype

    def _dispatch_ptrs(self, input, weights, scales):
        quant = self.config.quant != "none"
        return (_ptr(input), _ptr(weights), _ptr(scales), _ptr(self._out),
                _ptr(self._out_weights) if weights is not None else 0,
                _ptr(self._out_scales) if (scales is not None or quant) else 0)

    def _dispatch_views(self, weights, scales):
        return (self.received_payload(),
                self._out_weights if weights is not None else None,
                self.received_scales(scales is not None),
                self._out_indices, self._recv_count)

    # ---- methods table ---------------------------------------------------------------
    def dispatch(self, input: torch.Tensor, weights: Optional[torch.Tensor],
                 scales: Optional[torch.Tensor], indices: torch.Tensor):
        """Route tokens to expert slots.

        Returns (output, weights, scales, indices, recv_count) as views of the
        op's capacity-sized receive buffers (scales is None when there are
        none).  output is bf16 [N_cap, H] for bf16 input, float8_e4m3fn
        [N_cap, H] for FP8, uint8 [N_cap, H/2] (packed E2M1) for MXFP4, or
        uint8 [N_cap, raw_row_bytes] for raw rows.
        """
        T = indices.shape[0]
        self._need(indices, "indices", torch.int32, (T, self.config.topk))
        self._check_payload(input, weights, scales, T)
        i, w, s, o, ow, os_ = self._dispatch_ptrs(input, weights, scales)
        st = self._f_dispatch(self._op, _raw_stream(self._dev_index), T, i or None, w or None,
                              s or None, indices.data_ptr(), o, ow or None, os_ or None,
                              self._out_indices.data_ptr(), self._recv_count.data_ptr())
        if st:
            B._check(st)
        self._tokens = T
        self._last_dedup = self._routing_sent = False
        return self._dispatch_views(weights, scales)

    def dispatch_replay(self, input: torch.Tensor, weights: Optional[torch.Tensor] = None,
                        scales: Optional[torch.Tensor] = None):
        """Dispatch a new payload for the same tokens with the routing of the
        last dispatch (no histogram, scan or ranking).  Returns the views of
        dispatch(); indices and recv_count keep the recorded dispatch's values."""
        T = self._tokens
        units = self._last_dedup
        views = (lambda: self._unit_views(weights is not None, scales is not None)) if units \
            else (lambda: self._dispatch_views(weights, scales))
        if T == 0:
            # nothing to move; the library still refuses a replay with no dispatch recorded
            B.epdc_dispatch_replay(self._op, self._stream(), 0, 0, 0, 0, 0, 0)
            return views()
        self._check_payload(input, weights, scales, T)
        if units:  # a rank-deduplicated dispatch replays into the unit rows
            ub = self._unit_buffers()
            quant = self.config.quant != "none"
            i, w, s = _ptr(input), _ptr(weights), _ptr(scales)
            o = _ptr(ub["out"])
            ow = _ptr(ub["weights"]) if weights is not None else 0
            os_ = _ptr(ub["scales"]) if (scales is not None or quant) else 0
        else:
            i, w, s, o, ow, os_ = self._dispatch_ptrs(input, weights, scales)
        B.epdc_dispatch_replay(self._op, self._stream(), i, w, s, o, ow, os_)
        return views()

    def dispatch_send(self, input: torch.Tensor, weights: Optional[torch.Tensor],
                      scales: Optional[torch.Tensor], indices: torch.Tensor) -> None:
        """First phase of a split dispatch: enqueue the whole dispatch on the
        op's side stream (after the work already on the caller's stream) and
        return at once, so the caller's stream can compute meanwhile."""
        T = int(indices.shape[0])
        self._need(indices, "indices", torch.int32, (T, self.config.topk))
        self._check_payload(input, weights, scales, T)
        side = self._side()
        side.wait_stream(torch.cuda.current_stream(self.device))
        for t in (input, weights, scales, indices):
            if t is not None:
                t.record_stream(side)
        i, w, s, o, ow, os_ = self._dispatch_ptrs(input, weights, scales)
        B.epdc_dispatch_send(self._op, side.cuda_stream, T, i, w, s, _ptr(indices), o, ow, os_,
                             _ptr(self._out_indices), _ptr(self._recv_count))
        self._tokens = T
        self._last_dedup = False
        self._sent_dispatch = (weights is not None, scales is not None)
        self._routing_sent = True
        self._on_side |= {"dispatch"}

    def dispatch_recv(self):
        """Second phase: the caller's stream waits for the sent dispatch;
        returns what dispatch() returns."""
        if self._sent_dispatch is None:
            raise B.EpdcError(B.EPDC_ERR_BAD_STATE, "dispatch_recv without a dispatch_send")
        B.epdc_dispatch_recv(self._op, self._stream())
        has_w, has_s = self._sent_dispatch
        self._sent_dispatch = None
        self._routing_sent = False
        self._on_side -= {"dispatch"}
        return (self.received_payload(), self._out_weights if has_w else None,
                self.received_scales(has_s), self._out_indices, self._recv_count)

    def _payload_view(self, buf: torch.Tensor) -> torch.Tensor:
        cfg = self.config
        if cfg.raw_row_bytes:
            return buf
        if cfg.quant == "none":
            return self._view(buf, torch.bfloat16)
        if cfg.quant == "fp8_e4m3_b128":
            return self._view(buf, torch.float8_e4m3fn)
        return buf

    def _view(self, buf: torch.Tensor, dtype) -> torch.Tensor:
        """buf viewed as dtype; the op's buffers live as long as the op, so
        the views are made once."""
        key = (id(buf), dtype)
        v = self._views.get(key)
        if v is None:
            v = self._views[key] = buf.view(dtype)
        return v

    def _scales_view(self, buf: Optional[torch.Tensor], carried: bool) -> Optional[torch.Tensor]:
        cfg = self.config
        if cfg.quant == "fp8_e4m3_b128":
            return self._view(buf, torch.float32)
        if cfg.quant == "mxfp4_b32":
            return buf
        if not carried or buf is None:
            return None
        return self._view(buf, self._scales_dtype or torch.uint8)

    def received_payload(self) -> torch.Tensor:
        return self._payload_v

    def _combined_views(self, T: int):
        if self._combined_cut[0] != T:  # the views of the last token count are kept
            self._combined_cut = (T, (self._combined[:T], self._combined_weights[:T]))
        return self._combined_cut[1]

    def received_scales(self, carried: bool = True) -> Optional[torch.Tensor]:
        return self._scales_view(self._out_scales, carried)

    def combine(self, input: torch.Tensor, weights: Optional[torch.Tensor] = None,
                indices: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Weighted gather of the expert outputs back to token order.

        input: bf16 [n, H] in the received layout with n >= T*K of the last
        dispatch (e.g. the dispatch output itself); weights: fp32 [n, K] in
        the received layout or None.  Returns (output bf16 [T, H], weights fp32 [T, K]).
        """
        self._check_combine(input, weights)
        st = self._f_combine(self._op, _raw_stream(self._dev_index), input.data_ptr(),
                             None if weights is None else weights.data_ptr(),
                             None if indices is None else indices.data_ptr(),
                             self._combined.data_ptr(), self._combined_weights.data_ptr())
        if st:
            B._check(st)
        return self._combined_views(self._tokens)

    def combine_scatter(self, input: torch.Tensor, weights: Optional[torch.Tensor] = None,
                        indices: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Scatter combine: every received row pushes its weighted fp32 product
        to a per-(token, k) staging row, then each token adds its K staging
        rows in k order; same arguments and (bit-identical) result as combine().
        The fp32 staging rows (max_tokens*topk x hidden) are allocated on
        first use and kept."""
        self._check_combine(input, weights)
        if self._staging is None:
            self._staging = torch.empty((self.n_cap, self.config.hidden), dtype=torch.float32,
                                        device=self.device)
        B.epdc_combine_scatter(self._op, self._stream(), _ptr(input), _ptr(weights),
                               _ptr(indices), _ptr(self._staging), _ptr(self._combined),
                               _ptr(self._combined_weights))
        T = self._tokens
        return self._combined[:T], self._combined_weights[:T]

    def combine_send(self, input: torch.Tensor, weights: Optional[torch.Tensor] = None,
                     indices: Optional[torch.Tensor] = None) -> None:
        """First phase of a split combine, on the op's side stream (see dispatch_send)."""
        self._check_combine(input, weights)
        side = self._side()
        side.wait_stream(torch.cuda.current_stream(self.device))
        for t in (input, weights, indices):
            if t is not None:
                t.record_stream(side)
        B.epdc_combine_send(self._op, side.cuda_stream, _ptr(input), _ptr(weights), _ptr(indices),
                            _ptr(self._combined), _ptr(self._combined_weights))
        self._sent_combine = True
        self._on_side |= {"combine"}

    def combine_recv(self) -> Tuple[torch.Tensor, torch.Tensor]:
        """Second phase: the caller's stream waits for the sent combine;
        returns what combine() returns."""
        if not self._sent_combine:
            raise B.EpdcError(B.EPDC_ERR_BAD_STATE, "combine_recv without a combine_send")
        B.epdc_combine_recv(self._op, self._stream())
        self._sent_combine = None
        self._on_side -= {"combine"}
        T = self._tokens
        return self._combined[:T], self._combined_weights[:T]

    def _check_combine(self, input, weights) -> None:
        cfg = self.config
        self._need(input, "input", torch.bfloat16)
        if input.dim() != 2 or input.shape[1] != cfg.hidden:
            raise ValueError("combine input must be [rows, hidden] bf16")
        rows = self._tokens * cfg.topk          # received rows are a prefix of these
        if input.shape[0] < rows:
            raise ValueError(f"combine input needs at least {rows} rows")
        if weights is not None:
            self._need(weights, "weights", torch.float32)
            if weights.dim() != 2 or weights.shape[0] < rows or weights.shape[1] != cfg.topk:
                raise ValueError(f"combine weights must be [>= {rows}, topk] fp32")

    # ---- rank-deduplicated dispatch and the standard-MoE conversion -------------------
    def _unit_buffers(self) -> dict:
        if self._units is None:
            cfg, dev = self.config, self.device
            u = self.u_cap
            with torch.cuda.device(dev):
                self._units = {
                    "out": torch.empty((u, self.payload_row_bytes), dtype=torch.uint8, device=dev),
                    "weights": torch.empty((u, cfg.topk), dtype=torch.float32, device=dev),
                    "indices": torch.empty((u, cfg.topk), dtype=torch.int32, device=dev),
                    "scales": (torch.empty((u, self.scale_row_bytes), dtype=torch.uint8,
                                           device=dev) if self.scale_row_bytes else None),
                    "recv": torch.empty(cfg.num_ranks, dtype=torch.int32, device=dev),
                    "partial": torch.empty((u, cfg.hidden), dtype=torch.bfloat16, device=dev),
                }
        return self._units

    def received_unit_payload(self) -> torch.Tensor:
        """The unit rows of the last rank-deduplicated dispatch ([U_cap, ...])."""
        return self._payload_view(self._unit_buffers()["out"])

    def received_unit_scales(self, carried: bool = True) -> Optional[torch.Tensor]:
        return self._scales_view(self._unit_buffers()["scales"], carried)

    def _unit_views(self, has_w: bool, has_s: bool):
        ub = self._unit_buffers()
        return (self._payload_view(ub["out"]), ub["weights"] if has_w else None,
                self._scales_view(ub["scales"], has_s), ub["indices"], ub["recv"])

    def dispatch_dedup(self, input: torch.Tensor, weights: Optional[torch.Tensor],
                       scales: Optional[torch.Tensor], indices: torch.Tensor):
        """Dispatch with one received row per (token, destination rank).

        Returns (output, weights, scales, indices, recv_count) like dispatch()
        but over unit rows: views of [U_cap, ...] buffers, U_cap = max_tokens *
        min(topk, num_ranks); rank r owns rows [unit_off[r], unit_off[r+1])
        (get_unit_routing) and recv_count[r] of them."""
        T = int(indices.shape[0])
        self._need(indices, "indices", torch.int32, (T, self.config.topk))
        self._check_payload(input, weights, scales, T)
        ub = self._unit_buffers()
        quant = self.config.quant != "none"
        B.epdc_dispatch_dedup(self._op, self._stream(), T, _ptr(input), _ptr(weights),
                              _ptr(scales), _ptr(indices), _ptr(ub["out"]),
                              _ptr(ub["weights"]) if weights is not None else 0,
                              _ptr(ub["scales"]) if (scales is not None or quant) else 0,
                              _ptr(ub["indices"]), _ptr(ub["recv"]))
        self._tokens = T
        self._last_dedup = True
        self._routing_sent = False
        self._unit_carried = (weights is not None, scales is not None)
        return self._unit_views(*self._unit_carried)

    def get_unit_routing(self):
        """(unit_off [R+1], unit_of [T*K], unit_src [U_cap]) of the last
        rank-deduplicated dispatch (only the first unit_off[R] of unit_src
        are meaningful)."""
        a, b, c = B.epdc_get_unit_routing(self._op)
        cfg = self.config
        return (self._ws_view(a, cfg.num_ranks + 1), self._ws_view(b, self._tokens * cfg.topk),
                self._ws_view(c, self.u_cap))

    def units_to_experts(self, input: Optional[torch.Tensor] = None,
                         weights: Optional[torch.Tensor] = None,
                         scales: Optional[torch.Tensor] = None,
                         indices: Optional[torch.Tensor] = None):
        """Standard-MoE conversion: expand unit rows (by default the op's own,
        with whatever the last dispatch_dedup carried) into the expert-layout
        rows dispatch() would have written; returns dispatch()'s views."""
        if input is None:
            has_w, has_s = self._unit_carried
            ub = self._unit_buffers()
            input, indices = ub["out"], ub["indices"]
            weights = ub["weights"] if has_w else None
            scales = ub["scales"] if (has_s or self.config.quant != "none") else None
        self._check_unit_rows(input, weights, scales, indices)
        B.epdc_units_to_experts(self._op, self._stream(), _ptr(input), _ptr(weights),
                                _ptr(scales), _ptr(indices), _ptr(self._out),
                                _ptr(self._out_weights) if weights is not None else 0,
                                _ptr(self._out_scales) if scales is not None else 0,
                                _ptr(self._out_indices) if indices is not None else 0)
        return (self.received_payload(), self._out_weights if weights is not None else None,
                self.received_scales(scales is not None), self._out_indices, None)

    def _check_unit_rows(self, input, weights, scales, indices) -> None:
        """The conversion reads up to T * min(K, R) unit rows of each given
        array (T of the last dispatch): check rows, row widths and dtypes on
        the host so that no undersized tensor reaches the kernel."""
        cfg = self.config
        rows = self._tokens * min(cfg.topk, cfg.num_ranks)
        for t, name, row_bytes, dtype in ((input, "input", self.payload_row_bytes, None),
                                          (weights, "weights", 4 * cfg.topk, torch.float32),
                                          (scales, "scales", self.scale_row_bytes, None),
                                          (indices, "indices", 4 * cfg.topk, torch.int32)):
            if t is None:
                continue
            self._need(t, name, dtype)
            if t.dim() < 1 or t.shape[0] < rows:
                raise ValueError(f"{name} needs at least {rows} unit rows, got "
                                 f"{tuple(t.shape)}")
            if t.shape[0] and (t.numel() // t.shape[0]) * t.element_size() != row_bytes:
                raise ValueError(f"{name} rows must be {row_bytes} bytes, got "
                                 f"{(t.numel() // t.shape[0]) * t.element_size()}")

    def experts_to_units(self, input: torch.Tensor,
                         weights: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Weighted sum of each unit's expert rows (bf16 [>= T*K, H] in the
        expert layout, fp32 weights [>= T*K, K] or None) into bf16 unit rows
        [U_cap, H] (an op-owned buffer)."""
        self._check_combine(input, weights)
        part = self._unit_buffers()["partial"]
        B.epdc_experts_to_units(self._op, self._stream(), _ptr(input), _ptr(weights), _ptr(part))
        return part

    def combine_units(self, input: Optional[torch.Tensor] = None,
                      weights: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Sum each token's unit rows (by default the last experts_to_units
        result); weights: the unit rows' fp32 [U_cap, K] weights to hand back
        per token, or None.  Returns (output bf16 [T, H], weights fp32 [T, K])."""
        cfg = self.config
        ub = self._unit_buffers()
        if input is None:
            input = ub["partial"]
        self._need(input, "input", torch.bfloat16)
        if input.dim() != 2 or input.shape[1] != cfg.hidden or input.shape[0] < self.u_cap:
            raise ValueError(f"unit rows must be bf16 [>= {self.u_cap}, {cfg.hidden}]")
        if weights is not None:
            self._need(weights, "weights", torch.float32)
            if weights.dim() != 2 or weights.shape[0] < self.u_cap or weights.shape[1] != cfg.topk:
                raise ValueError(f"unit weights must be fp32 [>= {self.u_cap}, {cfg.topk}]")
        B.epdc_combine_units(self._op, self._stream(), _ptr(input), _ptr(weights),
                             _ptr(self._combined), _ptr(self._combined_weights))
        T = self._tokens
        return self._combined[:T], self._combined_weights[:T]

    # ---- the gate ------------------------------------------------------------------------
    def _gate_buffers(self) -> dict:
        cfg, dev = self.config, self.device
        scratch = L.epdc_gate_scratch_bytes(cfg.max_tokens, cfg.num_experts)
        return {
            "weights": torch.empty((cfg.max_tokens, cfg.topk), dtype=torch.float32, device=dev),
            "indices": torch.empty((cfg.max_tokens, cfg.topk), dtype=torch.int32, device=dev),
            "counts": torch.empty(cfg.num_experts + 1, dtype=torch.int32, device=dev),
            "losses": torch.empty(2, dtype=torch.float32, device=dev),
            "scratch": torch.zeros(scratch, dtype=torch.uint8, device=dev),
        }

    def _wait_for_side(self) -> None:
        """The caller's stream waits for sent phases, which may still read the
        gate's weights and indices."""
        if not self._on_side:
            return
        captured = torch.cuda.is_current_stream_capturing()
        if captured:
            with torch.cuda.stream(self._side_stream):
                inside = torch.cuda.is_current_stream_capturing()
            if not inside:   # its end cannot be waited for from within a graph
                raise B.EpdcError(B.EPDC_ERR_BAD_STATE, "gate is being captured while a phase "
                                  "sent before the capture may still read its buffers")
        torch.cuda.current_stream(self.device).wait_stream(self._side_stream)
        if not captured:
            self._on_side = frozenset()

    def _gate_args(self, logits, gate, bias, mask) -> L.epdc_gate_args:
        cfg = self.config
        if logits.dim() != 2 or logits.shape[1] != cfg.num_experts:
            raise ValueError(f"logits must be [tokens, {cfg.num_experts}], got "
                             f"{tuple(logits.shape)}")
        T = logits.shape[0]
        if T > cfg.max_tokens:
            raise ValueError(f"logits have {T} tokens, the op holds {cfg.max_tokens}")
        self._need(logits, "logits")
        if logits.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"logits must be float32 or bfloat16, got {logits.dtype}")
        if bias is not None:
            self._need(bias, "bias", torch.float32, (cfg.num_experts,))
        if mask is not None:
            if mask.dtype not in (torch.uint8, torch.bool):
                raise ValueError(f"mask must be uint8 or bool, got {mask.dtype}")
            self._need(mask, "mask", None, (T,))
        return L.make_gate_args(T, cfg.num_experts, cfg.topk, GATE_SCORES[gate.score],
                                int(gate.renormalize),
                                L.EPDC_DT_FP32 if logits.dtype == torch.float32
                                else L.EPDC_DT_BF16,
                                gate.scale, logits.data_ptr(), _ptr(bias), _ptr(mask))

    @_on_op_device
    def gate(self, logits: torch.Tensor, gate: GateConfig = GateConfig(), *,
             bias: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
             balance: bool = False):
        """Choose each token's experts from the router's logits.

        logits: fp32 or bf16 [T, E], T <= max_tokens; bias: fp32 [E] added to the
        scores for the choice only; mask: uint8 or bool [T], 0 = padding.
        Returns (weights fp32 [T, K], indices int32 [T, K]) as dispatch takes
        them, and with balance also (counts int32 [E + 1], losses fp32 [2]):
        choices per expert followed by the number of tokens that took part, and
        the balance and z losses (epdc_layer.h gives the formulas).  All are
        views of buffers of the op that the next gate() overwrites; a dispatch or
        combine that was sent and may still read them it waits for first."""
        args = self._gate_args(logits, gate, bias, mask)
        self._wait_for_side()
        T = args.num_tokens
        g = self._gate
        if self._gate_cut[0] != T:
            self._gate_cut = (T, (g["weights"][:T], g["indices"][:T]))
        views = self._gate_cut[1]
        if not balance:
            L.epdc_gate(args, self._stream(), _ptr(g["weights"]), _ptr(g["indices"]))
            return views
        L.epdc_gate(args, self._stream(), _ptr(g["weights"]), _ptr(g["indices"]),
                    _ptr(g["counts"]), _ptr(g["losses"]), _ptr(g["scratch"]))
        return views + (g["counts"], g["losses"])

    @_on_op_device
    def gate_backward(self, logits: torch.Tensor, indices: torch.Tensor,
                      gate: GateConfig = GateConfig(), *,
                      grad_weights: Optional[torch.Tensor] = None,
                      mask: Optional[torch.Tensor] = None,
                      counts: Optional[torch.Tensor] = None,
                      grad_losses: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Gradient of gate() with respect to the logits, in their dtype.

        indices, counts: the forward's; grad_weights: fp32 [T, K] or None;
        grad_losses: fp32 [2], with counts, or None."""
        args = self._gate_args(logits, gate, None, mask)
        T, cfg = args.num_tokens, self.config
        self._need(indices, "indices", torch.int32, (T, cfg.topk))
        if grad_weights is not None:
            self._need(grad_weights, "grad_weights", torch.float32, (T, cfg.topk))
        if (counts is None) != (grad_losses is None):
            raise ValueError("counts and grad_losses go together")
        if counts is not None:
            self._need(counts, "counts", torch.int32, (cfg.num_experts + 1,))
            self._need(grad_losses, "grad_losses", torch.float32, (2,))
        grad = torch.empty_like(logits)
        L.epdc_gate_backward(args, self._stream(), _ptr(indices), _ptr(grad_weights),
                             _ptr(counts), _ptr(grad_losses), _ptr(grad))
        return grad

    # ---- the experts' products -------------------------------------------------------------
    def _routed(self) -> int:
        """Rows the last dispatch may have written; raises if there is none, or it
        was sent and not received: its routing is still being written."""
        if self._routing_sent:
            raise B.EpdcError(B.EPDC_ERR_BAD_STATE, "the dispatch that was sent has not been "
                              "received (dispatch_recv)")
        if self._tokens == 0:
            B.epdc_get_offsets(self._op)   # BAD_STATE without a recorded dispatch
        return self._tokens * self.config.topk

    def _product_args(self, rows, input, weight, scales, weight_scales, bias, activation,
                      first_expert) -> L.epdc_product_args:
        cfg = self.config
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
        self._need(weight, "weight")
        if weight.dim() != 3:
            raise ValueError("weight must be [experts, out_features, in_features]")
        n, out_f, in_f = weight.shape
        if n < 1 or first_expert < 0 or first_expert + n > cfg.num_experts:
            raise ValueError(f"experts [{first_expert}, {first_expert + n}) are not within "
                             f"[0, {cfg.num_experts})")
        if weight.dtype == torch.bfloat16:
            dtype = L.EPDC_DT_BF16
        elif weight.dtype == torch.float8_e4m3fn:
            dtype = L.EPDC_DT_E4M3
        else:
            raise ValueError(f"weight must be bfloat16 or float8_e4m3fn, got {weight.dtype}")
        self._need(input, "input", weight.dtype)
        if input.dim() != 2 or input.shape[1] != in_f or input.shape[0] < rows:
            raise ValueError(f"input must be [>= {rows}, {in_f}], got {tuple(input.shape)}")
        if dtype == L.EPDC_DT_E4M3:
            if scales is None or weight_scales is None:
                raise ValueError("e4m3 operands need scales and weight_scales")
            blocks = in_f // 128
            self._need(scales, "scales", torch.float32)
            if scales.dim() != 2 or scales.shape[0] < rows or scales.shape[1] != blocks:
                raise ValueError(f"scales must be [>= {rows}, {blocks}], got "
                                 f"{tuple(scales.shape)}")
            self._need(weight_scales, "weight_scales", torch.float32,
                       (n, (out_f + 127) // 128, blocks))
        elif scales is not None or weight_scales is not None:
            raise ValueError("scales and weight_scales belong to e4m3 operands")
        if bias is not None:
            self._need(bias, "bias", torch.float32, (n, out_f))
        off, _ = B.epdc_get_offsets(self._op)
        expected = max(1, rows * n // cfg.num_experts)   # 0 would stand for all rows
        return L.make_product_args(rows, n, in_f, out_f, dtype, ACTIVATIONS[activation],
                                   expected, input.data_ptr(), _ptr(scales),
                                   weight.data_ptr(), _ptr(weight_scales), _ptr(bias),
                                   off + 4 * first_expert)

    def _need_rows(self, t, name, rows, cols) -> None:
        self._need(t, name, torch.bfloat16)
        if t.dim() != 2 or t.shape[0] < rows or t.shape[1] != cols:
            raise ValueError(f"{name} must be [>= {rows}, {cols}], got {tuple(t.shape)}")

    @_on_op_device
    def expert_product(self, input: torch.Tensor, weight: torch.Tensor, *,
                       scales: Optional[torch.Tensor] = None,
                       weight_scales: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, activation: str = "none",
                       residual: Optional[torch.Tensor] = None, first_expert: int = 0,
                       out: Optional[torch.Tensor] = None,
                       preact: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The experts' matrix product over the rows of the last dispatch:
        out[s] = act(input[s] @ weight[e].T + bias[e]) + residual[s] for every
        row s of expert first_expert + e.

        input: bf16 [>= T*K, in], or float8_e4m3fn with scales fp32 [>= T*K,
        in/128], as dispatch gives them; weight: [n, out, in] in the same type,
        e4m3 with weight_scales fp32 [n, ceil(out/128), in/128]; bias: fp32
        [n, out].  activation: "none", "relu", "gelu", "silu", or "swiglu" /
        "geglu", whose weight holds out/2 gate rows and then out/2 up rows.
        residual: bf16 rows of the result.  preact: bf16 [>= T*K, out], filled
        with the value before the activation for expert_product_backward.

        Returns out, bf16 [>= T*K, out or out/2] (allocated with T*K rows if
        None).  Only the rows of these experts are written."""
        rows = self._routed()
        args = self._product_args(rows, input, weight, scales, weight_scales, bias, activation,
                                  first_expert)
        cols = args.out_features // 2 if activation in GATED else args.out_features
        if residual is not None:
            self._need_rows(residual, "residual", rows, cols)
        if preact is not None:
            self._need_rows(preact, "preact", rows, args.out_features)
        if out is None:
            out = torch.empty((rows, cols), dtype=torch.bfloat16, device=self.device)
        else:
            self._need_rows(out, "out", rows, cols)
            if out.data_ptr() in (input.data_ptr(), _ptr(preact) or -1):
                raise ValueError("out must be a tensor of its own (or residual)")
        L.epdc_expert_product(args, self._stream(), _ptr(residual), out.data_ptr(), _ptr(preact))
        return out

    @_on_op_device
    def expert_product_backward(self, grad_output: torch.Tensor, input: torch.Tensor,
                                weight: torch.Tensor, *, activation: str = "none",
                                preact: Optional[torch.Tensor] = None, bias: bool = False,
                                first_expert: int = 0, need_input: bool = True,
                                need_weight: bool = True,
                                weight_dtype: torch.dtype = torch.bfloat16,
                                grad_input: Optional[torch.Tensor] = None):
        """Gradients of a bf16 expert_product.

        grad_output: bf16 rows like its result; preact: what the forward filled
        (with an activation).  Returns (grad_input bf16 [T*K, in], grad_weight
        [n, out, in] in weight_dtype (bfloat16 or float32), grad_bias fp32 [n,
        out]); None for what is not asked for.  Experts without rows get zero
        weight and bias gradients.  The residual's gradient is grad_output.

        grad_input: a bf16 buffer [>= T*K, in] of which only the rows of these
        experts are written, so that ranks can share one.  Without it a call over
        some of the experts returns zeros in all other rows; a call over all of
        them leaves the rows behind the last expert's, which hold no pair, unset."""
        rows = self._routed()
        if weight.dtype != torch.bfloat16:
            raise ValueError("the gradients take bf16 operands")
        if weight_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("weight_dtype must be bfloat16 or float32")
        args = self._product_args(rows, input, weight, None, None, None, activation, first_expert)
        n, out_f, in_f = weight.shape
        if grad_input is not None:
            if not need_input:
                raise ValueError("grad_input is given but not asked for")
            self._need_rows(grad_input, "grad_input", rows, in_f)
        self._need_rows(grad_output, "grad_output", rows,
                        out_f // 2 if activation in GATED else out_f)
        dz = None
        if activation == "none":
            preact = None
        else:
            if preact is None:
                raise ValueError("an activation's gradient needs preact")
            self._need_rows(preact, "preact", rows, out_f)
            if need_input or need_weight:
                dz = torch.empty((rows, out_f), dtype=torch.bfloat16, device=self.device)
        new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=self.device)
        if need_input and grad_input is None:
            grad_input = new((rows, in_f), torch.bfloat16)
            if n < self.config.num_experts:
                grad_input.zero_()
        grad_weight = new((n, out_f, in_f), weight_dtype) if need_weight else None
        grad_bias = new((n, out_f), torch.float32) if bias else None
        L.epdc_expert_backward(args, self._stream(), grad_output.data_ptr(), _ptr(preact),
                               _ptr(dz), _ptr(grad_input), _ptr(grad_weight),
                               L.EPDC_DT_FP32 if weight_dtype == torch.float32
                               else L.EPDC_DT_BF16, _ptr(grad_bias))
        return grad_input, grad_weight, grad_bias

    # ---- gradients of combine and dispatch ---------------------------------------------------
    @_on_op_device
    def combine_backward(self, grad_output: torch.Tensor, input: torch.Tensor,
                         weights: Optional[torch.Tensor] = None):
        """Gradients of combine(input, weights) under the routing of the last
        dispatch: (grad_input bf16 [T*K, H] in the received layout, grad_weights
        fp32 [T, K] in token order, the gradient of dispatch's weights).  Only
        rows that hold a pair are written; a pair without a slot gets 0."""
        self._routed()
        self._check_combine(input, weights)
        cfg, T = self.config, self._tokens
        self._need(grad_output, "grad_output", torch.bfloat16, (T, cfg.hidden))
        _, _, slot_of = B.epdc_get_routing(self._op)
        grad_input = torch.empty((T * cfg.topk, cfg.hidden), dtype=torch.bfloat16,
                                 device=self.device)
        grad_weights = torch.empty((T, cfg.topk), dtype=torch.float32, device=self.device)
        L.epdc_combine_backward(self._stream(), T, cfg.topk, cfg.hidden, slot_of,
                                grad_output.data_ptr(), input.data_ptr(), _ptr(weights),
                                grad_input.data_ptr(), grad_weights.data_ptr())
        return grad_input, grad_weights

    @_on_op_device
    def dispatch_backward(self, grad_output: torch.Tensor) -> torch.Tensor:
        """Gradient of dispatch's bf16 input: bf16 [T, H], the fp32 sum of each
        token's rows of grad_output (bf16 [>= T*K, H], received layout)."""
        self._routed()
        self._check_combine(grad_output, None)
        grad = torch.empty((self._tokens, self.config.hidden), dtype=torch.bfloat16,
                           device=self.device)
        B.epdc_combine(self._op, self._stream(), grad_output.data_ptr(), 0, 0, grad.data_ptr(), 0)
        return grad

    def reset(self) -> None:
        B.epdc_reset(self._op)
        self._tokens = 0
        self._last_dedup = self._routing_sent = False
        self._sent_dispatch = self._sent_combine = None

    def get_dispatch_src_token_pos(self) -> torch.Tensor:
        """Per received row, the pair index t*K + k it came from (the first
        sum(recv_count) entries are meaningful)."""
        ptr, n = B.epdc_get_dispatch_src_token_pos(self._op)
        return self._ws_view(ptr, n)

    def get_routing(self):
        """(expert_off [E+1], rank_off [R+1], slot_of [T*K]) of the last dispatch."""
        a, b, c = B.epdc_get_routing(self._op)
        cfg = self.config
        return (self._ws_view(a, cfg.num_experts + 1), self._ws_view(b, cfg.num_ranks + 1),
                self._ws_view(c, self._tokens * cfg.topk))

    def get_offsets(self):
        """(expert_off [E+1], rank_off [R+1]) of the last dispatch."""
        a, b = B.epdc_get_offsets(self._op)
        cfg = self.config
        return self._ws_view(a, cfg.num_experts + 1), self._ws_view(b, cfg.num_ranks + 1)

    def set_debug(self, check_indices: bool = True) -> None:
        """With check_indices, combine checks a given `indices` against the
        recorded routing and raises bit 4 of the device error flag on a mismatch."""
        B.epdc_set_debug(self._op, B.EPDC_DEBUG_CHECK_INDICES if check_indices else 0)

    def set_combine_hint(self, recent_input: bool) -> None:
        """Say whether combine's input rows were written just before it (the
        expert output, or the dispatch output itself); only how the combine
        launches and stores depends on it (epdc_set_combine_hint), never its
        result."""
        B.epdc_set_combine_hint(self._op, B.EPDC_COMBINE_INPUT_RECENT if recent_input
                                else B.EPDC_COMBINE_INPUT_COLD)

    def get_registered_combine_input_buffer(self, dtype=torch.bfloat16) -> torch.Tensor:
        """A capacity-sized [N_cap, H] buffer owned by the op, for expert outputs."""
        if dtype != torch.bfloat16:
            raise ValueError("combine input is bf16")
        if self._combine_in is None:
            self._combine_in = torch.empty((self.n_cap, self.config.hidden), dtype=torch.bfloat16,
                                           device=self.device)
        return self._combine_in

    def device_error(self) -> int:
        """Synchronize and return/clear the sticky bad-expert-id flag."""
        return B.epdc_get_device_error(self._op, self._stream())

    # ---- timing ------------------------------------------------------------------------
    def profile_begin(self, max_launches: int) -> None:
        B.epdc_profile_begin(self._op, max_launches)

    def profile_end(self):
        """{kernel name: (total ms, launches)} for the launches since profile_begin."""
        ms, n = B.epdc_profile_end(self._op)
        return {B.epdc_kernel_name(k): (ms[k], n[k]) for k in range(B.EPDC_NUM_KERNELS) if n[k]}
