"""MI355X (gfx950) MoE expert-parallel dispatch/combine hot path.

``binding`` is the ctypes layer over libepdc.so (include/epdc.h) and ``layer``
over libepdc_layer.so (include/epdc_layer.h: the gate, the experts' products
and the gradients); ``op`` holds EpDispatchCombineConfig / EpDispatchCombineOp
on top of both; ``workloads`` draws seeded synthetic inputs.  Submodules are imported on use so that the
input generator works without the HIP library.
"""
__all__ = ["binding", "layer", "op", "workloads", "build"]
