"""ctypes binding of libepdc_layer.so (include/epdc_layer.h): the gate, the
experts' matrix products and the gradients.  One Python function per C entry
point with the same name; arguments are plain integers (device addresses,
sizes, a hipStream_t as an integer) and the two argument structures.  A
non-SUCCESS status raises; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import List

from .binding import EPDC_SUCCESS, EpdcError

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB_PATH = os.path.join(PKG, "libepdc_layer.so")
HEADER = os.path.join(ROOT, "include", "epdc_layer.h")

EPDC_DT_BF16 = 0
EPDC_DT_FP32 = 1
EPDC_DT_E4M3 = 2
EPDC_GATE_SOFTMAX = 0
EPDC_GATE_SIGMOID = 1
EPDC_ACT_NONE = 0
EPDC_ACT_RELU = 1
EPDC_ACT_GELU = 2
EPDC_ACT_SILU = 3
EPDC_ACT_SWIGLU = 4
EPDC_ACT_GEGLU = 5

P = ctypes.c_void_p
I32 = ctypes.c_int32
SZ = ctypes.c_size_t


class epdc_gate_args(ctypes.Structure):
    _fields_ = [(n, I32) for n in ("num_tokens", "num_experts", "topk", "score", "renormalize",
                                   "logits_dtype")] + \
               [("scale", ctypes.c_float), ("logits", P), ("bias", P), ("mask", P)]


class epdc_product_args(ctypes.Structure):
    _fields_ = [(n, I32) for n in ("rows", "num_experts", "in_features", "out_features", "dtype",
                                   "activation", "expected_rows")] + \
               [(n, P) for n in ("input", "scales", "weight", "weight_scales", "bias",
                                 "expert_off")]


PGATE = ctypes.POINTER(epdc_gate_args)
PPROD = ctypes.POINTER(epdc_product_args)

_SIGNATURES = {
    "epdc_gate_scratch_bytes": (I32, [I32, I32, ctypes.POINTER(SZ)]),
    "epdc_gate": (I32, [PGATE, P, P, P, P, P, P]),
    "epdc_gate_backward": (I32, [PGATE, P, P, P, P, P, P]),
    "epdc_expert_product": (I32, [PPROD, P, P, P, P]),
    "epdc_expert_backward": (I32, [PPROD, P, P, P, P, P, P, I32, P]),
    "epdc_combine_backward": (I32, [P, I32, I32, I32, P, P, P, P, P, P]),
    "epdc_layer_last_error": (ctypes.c_char_p, []),
}

_lib = None


def lib():
    """Load libepdc_layer.so; raises if it has not been built (no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; build it with "
                           "`python -m combine_routing_histogram_amd.build`")
    l = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        f = getattr(l, name)
        f.restype = res
        f.argtypes = args
    _lib = l
    return l


def header_entry_points() -> List[str]:
    """Names of the functions include/epdc_layer.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[a-z_]+\s*\**\s*(epdc_[a-z_]+)\s*\(", text,
                                 flags=re.M)))


def _check(status: int) -> None:
    if status != EPDC_SUCCESS:
        raise EpdcError(status, lib().epdc_layer_last_error().decode())


def make_gate_args(num_tokens: int, num_experts: int, topk: int, score: int = EPDC_GATE_SOFTMAX,
                   renormalize: int = 1, logits_dtype: int = EPDC_DT_FP32, scale: float = 1.0,
                   logits: int = 0, bias: int = 0, mask: int = 0) -> epdc_gate_args:
    return epdc_gate_args(num_tokens, num_experts, topk, score, renormalize, logits_dtype, scale,
                          logits or None, bias or None, mask or None)


def make_product_args(rows: int, num_experts: int, in_features: int, out_features: int,
                      dtype: int = EPDC_DT_BF16, activation: int = EPDC_ACT_NONE,
                      expected_rows: int = 0, input: int = 0, scales: int = 0, weight: int = 0,
                      weight_scales: int = 0, bias: int = 0,
                      expert_off: int = 0) -> epdc_product_args:
    return epdc_product_args(rows, num_experts, in_features, out_features, dtype, activation,
                             expected_rows, input or None, scales or None, weight or None,
                             weight_scales or None, bias or None, expert_off or None)


# ---- one wrapper per entry point --------------------------------------------------

def epdc_gate_scratch_bytes(max_tokens: int, num_experts: int) -> int:
    n = SZ(0)
    _check(lib().epdc_gate_scratch_bytes(max_tokens, num_experts, ctypes.byref(n)))
    return n.value


def epdc_gate(args: epdc_gate_args, stream: int, weights: int, indices: int, counts: int = 0,
              losses: int = 0, scratch: int = 0) -> None:
    _check(lib().epdc_gate(ctypes.byref(args), stream or None, weights or None, indices or None,
                           counts or None, losses or None, scratch or None))


def epdc_gate_backward(args: epdc_gate_args, stream: int, indices: int, grad_weights: int,
                       counts: int, grad_losses: int, grad_logits: int) -> None:
    _check(lib().epdc_gate_backward(ctypes.byref(args), stream or None, indices or None,
                                    grad_weights or None, counts or None, grad_losses or None,
                                    grad_logits or None))


def epdc_expert_product(args: epdc_product_args, stream: int, residual: int, out: int,
                        preact: int) -> None:
    _check(lib().epdc_expert_product(ctypes.byref(args), stream or None, residual or None,
                                     out or None, preact or None))


def epdc_expert_backward(args: epdc_product_args, stream: int, grad_out: int, preact: int, dz: int,
                         grad_input: int, grad_weight: int, grad_weight_dtype: int,
                         grad_bias: int) -> None:
    _check(lib().epdc_expert_backward(ctypes.byref(args), stream or None, grad_out or None,
                                      preact or None, dz or None, grad_input or None,
                                      grad_weight or None, grad_weight_dtype, grad_bias or None))


def epdc_combine_backward(stream: int, num_tokens: int, topk: int, hidden: int, slot_of: int,
                          grad_output: int, input: int, weights: int, grad_input: int,
                          grad_weights: int) -> None:
    _check(lib().epdc_combine_backward(stream or None, num_tokens, topk, hidden, slot_of or None,
                                       grad_output or None, input or None, weights or None,
                                       grad_input or None, grad_weights or None))


def epdc_layer_last_error() -> str:
    return lib().epdc_layer_last_error().decode()
