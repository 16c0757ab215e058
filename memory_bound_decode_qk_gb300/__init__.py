"""GB300-native fused decode-seam operators.

The per-head QK-RMSNorm + RoPE attention prologue, residual-add RMSNorm,
RMSNorm and SiLU / tanh-GELU gated activations, each with an optional
static-scale FP8 E4M3 output; and the operators of a paged KV cache: its write
fused with the QKV split, attention over its pages, rotary positions with
several axes, and the moves of its pages.  Every op is a hand-written sm_103a CUDA kernel
behind the C ABI declared in ``include/edge_ops.h``; ``edge_ops`` is the thin
ctypes binding over it, and ``synth`` draws the seeded inputs.
"""

__all__ = ["edge_ops", "synth"]


def __getattr__(name):
    if name in ("edge_ops", "synth"):
        import importlib

        return importlib.import_module(f"{__name__}.{name}")
    raise AttributeError(name)
