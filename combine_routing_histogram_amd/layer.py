"""ctypes binding of libepdc_layer.so (include/epdc_layer.h): the gate, the
experts' matrix products, the norm, rows in 8 bits, the layer for few tokens and
the gradients.  One Python function per C entry point with the same name;
arguments are plain integers (device addresses, sizes, a hipStream_t as an
integer) and the argument structures.  A
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
EPDC_DT_INT8 = 3
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


class epdc_norm_args(ctypes.Structure):
    _fields_ = [(n, I32) for n in ("rows", "features", "weight_dtype")] + \
               [("eps", ctypes.c_float)] + [(n, P) for n in ("input", "residual", "weight")]


class epdc_few_args(ctypes.Structure):
    _fields_ = [(n, I32) for n in ("num_tokens", "topk", "num_experts", "first_expert", "hidden",
                                   "inner", "dtype", "activation")] + \
               [(n, P) for n in ("input", "weights", "indices", "w1", "w2", "w1_scales",
                                 "w2_scales", "bias1", "bias2")]


PGATE = ctypes.POINTER(epdc_gate_args)
PPROD = ctypes.POINTER(epdc_product_args)
PNORM = ctypes.POINTER(epdc_norm_args)
PFEW = ctypes.POINTER(epdc_few_args)

_SIGNATURES = {
    "epdc_gate_scratch_bytes": (I32, [I32, I32, ctypes.POINTER(SZ)]),
    "epdc_gate": (I32, [PGATE, P, P, P, P, P, P]),
    "epdc_gate_backward": (I32, [PGATE, P, P, P, P, P, P]),
    "epdc_expert_product": (I32, [PPROD, P, P, P, P]),
    "epdc_expert_backward": (I32, [PPROD, P, P, P, P, P, P, I32, P]),
    "epdc_combine_backward": (I32, [P, I32, I32, I32, P, P, P, P, P, P]),
    "epdc_rms_norm": (I32, [PNORM, P, P, P, P, P, I32]),
    "epdc_rms_norm_scratch_bytes": (I32, [I32, ctypes.POINTER(SZ)]),
    "epdc_rms_norm_backward": (I32, [PNORM, P, P, P, P, P, P]),
    "epdc_quantize_rows": (I32, [P, I32, I32, I32, P, P, I32, P, P]),
    "epdc_few_tokens_scratch_bytes": (I32, [PFEW, ctypes.POINTER(SZ)]),
    "epdc_few_tokens": (I32, [PFEW, P, P, P]),
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


def make_norm_args(rows: int, features: int, weight_dtype: int = EPDC_DT_BF16, eps: float = 1e-6,
                   input: int = 0, residual: int = 0, weight: int = 0) -> epdc_norm_args:
    return epdc_norm_args(rows, features, weight_dtype, eps, input or None, residual or None,
                          weight or None)


def make_few_args(num_tokens: int, topk: int, num_experts: int, hidden: int, inner: int,
                  dtype: int = EPDC_DT_BF16, activation: int = EPDC_ACT_NONE,
                  first_expert: int = 0, input: int = 0, weights: int = 0, indices: int = 0,
                  w1: int = 0, w2: int = 0, w1_scales: int = 0, w2_scales: int = 0,
                  bias1: int = 0, bias2: int = 0) -> epdc_few_args:
    return epdc_few_args(num_tokens, topk, num_experts, first_expert, hidden, inner, dtype,
                         activation, input or None, weights or None, indices or None, w1 or None,
                         w2 or None, w1_scales or None, w2_scales or None, bias1 or None,
                         bias2 or None)


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


def epdc_rms_norm(args: epdc_norm_args, stream: int, out: int, sum: int, codes: int, scales: int,
                  codes_dtype: int) -> None:
    _check(lib().epdc_rms_norm(ctypes.byref(args), stream or None, out or None, sum or None,
                               codes or None, scales or None, codes_dtype))


def epdc_rms_norm_scratch_bytes(features: int) -> int:
    n = SZ(0)
    _check(lib().epdc_rms_norm_scratch_bytes(features, ctypes.byref(n)))
    return n.value


def epdc_rms_norm_backward(args: epdc_norm_args, stream: int, grad_out: int, grad_sum: int,
                           grad_input: int, grad_weight: int, scratch: int) -> None:
    _check(lib().epdc_rms_norm_backward(ctypes.byref(args), stream or None, grad_out or None,
                                        grad_sum or None, grad_input or None, grad_weight or None,
                                        scratch or None))


def epdc_quantize_rows(stream: int, rows: int, features: int, codes_dtype: int, input: int,
                       expert_off: int, num_experts: int, codes: int, scales: int) -> None:
    _check(lib().epdc_quantize_rows(stream or None, rows, features, codes_dtype, input or None,
                                    expert_off or None, num_experts, codes or None,
                                    scales or None))


def epdc_few_tokens_scratch_bytes(args: epdc_few_args) -> int:
    n = SZ(0)
    _check(lib().epdc_few_tokens_scratch_bytes(ctypes.byref(args), ctypes.byref(n)))
    return n.value


def epdc_few_tokens(args: epdc_few_args, stream: int, scratch: int, out: int) -> None:
    _check(lib().epdc_few_tokens(ctypes.byref(args), stream or None, scratch or None,
                                 out or None))


def epdc_layer_last_error() -> str:
    return lib().epdc_layer_last_error().decode()
