"""Quantized mixture-of-experts FFN layer for one GB300 (sm_103a), and the
sequence-side operators of the same decoder.

The compute path is the CUDA library behind include/moe.h and
include/moe_model.h (built in-tree by ``build.build_cuda``); ``moe`` is its
thin ctypes binding, ``attention`` (per-head norm + rotation, quantised paged
cache, attention over it) and ``sampling`` are those of moe_model.h, and
``synth`` the seeded input generator.  There is no CPU fallback: using ``moe`` without the
CUDA library, or without a GPU, raises.
"""
from . import synth  # noqa: F401

__all__ = ["synth", "moe", "stack", "attention", "sampling"]


def __getattr__(name):
    if name in ("moe", "stack", "attention", "sampling"):
        import importlib
        return importlib.import_module(__name__ + "." + name)
    raise AttributeError(name)
